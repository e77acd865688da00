"""Plain 64-bit forms of the paged 4-bit cache's operators, in numpy: what the
GPU tests compare with.  Written from the record layout and the formulas in
include/dsa_select.h; rounding goes by searching the nearest number of the
type, not by bit tricks."""
import numpy as np

REC = 144
DIM = 128

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def _e4m3_table():
    v = np.empty(256)
    for b in range(256):
        e, m = (b >> 3) & 15, b & 7
        x = (1 + m / 8) * 2.0 ** (e - 7) if e else m / 8 * 2.0 ** -6
        v[b] = -x if b & 128 else x
    v[0x7F] = v[0xFF] = np.nan
    return v


E4M3 = _e4m3_table()


def nearest(x, numbers):
    """Index of the nearest of the ascending `numbers` to x >= 0, the even
    index where two are equally near; past the last one, the last."""
    x = np.asarray(x, dtype=np.float64)
    hi = np.clip(np.searchsorted(numbers, x), 1, len(numbers) - 1)
    lo = hi - 1
    with np.errstate(invalid="ignore"):
        dl, dh = x - numbers[lo], numbers[hi] - x
    up = (dh < dl) | ((dh == dl) & (hi % 2 == 0)) | (x >= numbers[-1])
    return np.where(up, hi, lo)


def quantise(x):
    """codes uint8 [..., 128] and scale bytes uint8 [..., 8] of rows x [..., 128]."""
    y = np.asarray(x, dtype=np.float64).reshape(*x.shape[:-1], 8, 16)
    top = np.abs(y).max(-1)
    nan = np.isnan(y).any(-1)
    scale = nearest(np.where(nan, 0.0, top) / 6.0, E4M3[:0x7F]).astype(np.uint8)
    s = E4M3[scale][..., None]
    with np.errstate(invalid="ignore", divide="ignore"):
        m = np.where(s > 0, np.abs(y) / np.where(s > 0, s, 1.0), 0.0)
    code = nearest(np.where(np.isnan(m), 0.0, m), E2M1) + 8 * np.signbit(y)
    code = np.where((s > 0) & ~nan[..., None], code, 0).astype(np.uint8)
    return code.reshape(x.shape), np.where(nan, 0x7F, scale).astype(np.uint8)


def pack(k, v):
    """Records uint8 [..., 144] of key and value rows [..., 128]."""
    kc, ks = quantise(k)
    vc, vs = quantise(v)
    return np.concatenate([kc[..., 0::2] | (kc[..., 1::2] << 4), vc[..., 0::2] | (vc[..., 1::2] << 4), ks, vs], -1)


def expand(rec):
    """Keys and values (float64 [..., 128]) of records [..., 144]."""
    out = []
    for which in (0, 1):
        b = rec[..., 64 * which:64 * which + 64]
        code = np.stack([b & 15, b >> 4], -1).reshape(*b.shape[:-1], DIM)
        val = np.where(code >= 8, -1.0, 1.0) * E2M1[code & 7]
        out.append(val * np.repeat(E4M3[rec[..., 128 + 8 * which:136 + 8 * which]], 16, -1))
    return out


def attention(cache, page_size, q, idx, token_req, tables, scale, k_shift=0, v_shift=0, distinct=False):
    """(o, lse, vmax, amax) in float64: cache [pages, page_size, kv_heads, 144],
    q [T, H, 128], idx [T, Kc], tables [R, P]; vmax [T, H]: the largest |v| a
    row attends to, amax: the largest scale * sum_d |q_d k_d|.  distinct: a
    position listed twice counts once."""
    pages, _, KV, _ = cache.shape
    T, H, _ = q.shape
    n = H // KV
    R, P = tables.shape
    o = np.zeros((T, H, DIM))
    lse = np.full((T, H), -np.inf)
    vmax, amax = np.zeros((T, H)), np.zeros((T, H))
    for t in range(T):
        r = int(token_req[t])
        if not 0 <= r < R:
            continue
        pos = idx[t][idx[t] >= 0]
        if distinct:
            pos = np.unique(pos)
        pos = pos[pos // page_size < P]
        page = tables[r][pos // page_size]
        ok = (page >= 0) & (page < pages)
        pos, page = pos[ok], page[ok]
        if not len(pos):
            continue
        for kv in range(KV):
            k, v = expand(cache[page, pos % page_size, kv])
            x = (q[t, kv * n:(kv + 1) * n].astype(np.float64) @ k.T) * (scale * 2.0 ** k_shift)
            m = x.max(-1, keepdims=True)
            w = np.exp(x - m)
            z = w.sum(-1, keepdims=True)
            o[t, kv * n:(kv + 1) * n] = (w @ v) / z * 2.0 ** v_shift
            lse[t, kv * n:(kv + 1) * n] = (m + np.log(z))[:, 0]
            vmax[t, kv * n:(kv + 1) * n] = np.abs(v).max() * 2.0 ** v_shift
            a = np.abs(q[t, kv * n:(kv + 1) * n].astype(np.float64)) @ np.abs(k).T
            amax[t, kv * n:(kv + 1) * n] = a.max(-1) * abs(scale) * 2.0 ** k_shift
    return o, lse, vmax, amax


def plan(page_size, pages, lens, fresh, tables, held, free, count, T):
    """One step: a dict of the updated and written arrays (copies)."""
    tables, held, free = tables.copy(), held.copy(), free.copy()
    R, P = tables.shape
    token_req, ends, slots = np.full(T, -1), np.zeros(T, int), np.full(T, -1)
    first = np.zeros(R + 1, int)
    need = [-(-int(n) // page_size) for n in lens]
    a = sum(max(n - int(h), 0) for n, h in zip(need, held))
    p = sum(max(int(h) - n, 0) for n, h in zip(need, held))
    code = 0
    if a > count or count - a + p > len(free):
        code = 1
    if fresh.astype(np.int64).sum() > T:
        code = 3
    if any(n > P for n in need):
        code = 2
    if (lens < 0).any() or (fresh < 0).any() or (fresh > lens).any() or (held < 0).any() or (held > P).any() \
            or not 0 <= count <= len(free):
        code = 4
    total = 0
    short = max(a - count, 0) if code == 1 else 0
    if code == 0:
        top = count
        for r in range(R):
            for j in range(held[r], need[r]):
                top -= 1
                tables[r, j] = free[top]
        given = [(r, j) for r in range(R) for j in range(need[r], held[r])]
        for i in range(R):
            first[i] = total
            for x in range(lens[i] - fresh[i], lens[i]):
                page = tables[i, x // page_size]
                token_req[total], ends[total] = i, x + 1
                slots[total] = page * page_size + x % page_size if 0 <= page < pages else -1
                total += 1
        first[R] = total
        for r, j in reversed(given):
            free[top] = tables[r, j]
            top += 1
            tables[r, j] = -1
        held[:] = need
        count = top
    return dict(tables=tables, held=held, free=free, count=np.array([count]), first=first, token_req=token_req,
                ends=ends, slots=slots, status=np.array([code, short, total, count]))
