"""Plain 64-bit forms of the paged 16-bit cache's operators, in torch, on the
tensors' own device: what the tests compare with.  Written from the formulas in
include/dsa_select.h."""
import math

import torch

DIM = 128
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}  # half a step, relative


def rotate(x, pos, inv_freq, neighbours, gain=1.0):
    """Rows x [T, heads, 128] turned by their positions, in f64."""
    y = x.double().clone()
    n = len(inv_freq)
    if n:
        angle = pos.double()[:, None] * inv_freq.double()[None, :]
        c, s = gain * torch.cos(angle)[:, None], gain * torch.sin(angle)[:, None]
        i = torch.arange(n, device=x.device)
        a, b = (2 * i, 2 * i + 1) if neighbours else (i, i + n)
        y[..., a], y[..., b] = (x.double()[..., a] * c - x.double()[..., b] * s,
                                x.double()[..., b] * c + x.double()[..., a] * s)
    return y


class Step:
    """A step of requests with `lens` positions, the last `new` of them its
    tokens, over a pool whose pages are in no order."""

    def __init__(self, lens, new, *, H, Hk, page, dtype, seed=0, pad=0, spare=3, device="cuda:0", width=None, lo=0):
        g = torch.Generator().manual_seed(seed)
        self.lens_list, self.new_list, self.H, self.Hk, self.page, self.dtype = list(lens), list(new), H, Hk, page, dtype
        need = [-(-n // page) for n in lens]
        self.pages = sum(need) + spare + lo
        order = (torch.randperm(sum(need) + spare, generator=g) + lo).int()
        self.P = max(need + [0]) + 1 if width is None else width
        tables = torch.full((len(need), self.P), -1, dtype=torch.int32)
        at = 0
        for r, n in enumerate(need):
            tables[r, :n] = order[at:at + n][:self.P]
            at += n
        first = [0]
        for n in new:
            first.append(first[-1] + n)
        self.first_list, self.T = first, first[-1] + pad
        i32 = dict(dtype=torch.int32, device=device)
        self.tables, self.first, self.lens = tables.to(device), torch.tensor(first, **i32), torch.tensor(lens, **i32)
        self.device, self.gen = device, g

    def normal(self, *shape, dtype=None):
        return torch.randn(*shape, generator=self.gen).to(dtype or self.dtype).to(self.device)

    def rows(self):
        """q [T, H, 128] and a full cache."""
        q = self.normal(self.T, self.H, DIM)
        k, v = (self.normal(self.pages, self.page, self.Hk, DIM) for _ in range(2))
        return q, k, v

    def tokens(self):
        """(request, position, token) of every token."""
        for r, (n, f) in enumerate(zip(self.lens_list, self.new_list)):
            for i in range(f):
                yield r, n - f + i, self.first_list[r] + i


def attention(step, q, k, v, scale, idx=None):
    """o [T, H, 128], lse [T, H] in f64, and what bounds their errors: the
    weighted mean of |v| [T, H, 128], the largest sum of |q k| [T, H] and the
    positions attended to [T, H]; rows of no token are NaN."""
    T, H, Hk, page, dev = step.T, step.H, step.Hk, step.page, step.device
    n = H // Hk
    out = {"o": torch.full((T, H, DIM), math.nan, dtype=torch.float64, device=dev),
           "lse": torch.full((T, H), math.nan, dtype=torch.float64, device=dev),
           "vabs": torch.zeros(T, H, DIM, dtype=torch.float64, device=dev),
           "amax": torch.zeros(T, H, dtype=torch.float64, device=dev),
           "count": torch.zeros(T, H, dtype=torch.float64, device=dev)}
    for r, (length, fresh) in enumerate(zip(step.lens_list, step.new_list)):
        a, b = step.first_list[r], step.first_list[r + 1]
        if a == b:
            continue
        L = min(max(length, 0), step.P * page)
        ids = step.tables[r].repeat_interleave(page)[:L].long()
        pos = torch.arange(length - fresh, length, device=dev)
        j = torch.arange(L, device=dev)
        real = (ids >= 0) & (ids < step.pages)
        seen = (j[None, :] <= pos[:, None]) & real[None, :]
        if length < fresh:
            seen[:] = False
        slot = torch.where(real, ids, 0) * page + j % page
        for g in range(Hk):
            mine = seen
            if idx is not None:
                listed = idx[a:b, g].long()
                mine = seen & ((j // page)[None, None, :] == listed[:, :, None]).any(1)
            kk, vv = k.reshape(-1, Hk, DIM)[slot, g].double(), v.reshape(-1, Hk, DIM)[slot, g].double()
            qq = q[a:b, g * n:(g + 1) * n].double()
            some = mine.any(0)  # positions no row attends to are out of it altogether
            kk, vv = torch.where(some[:, None], kk, 0), torch.where(some[:, None], vv, 0)
            x = torch.einsum("thd,jd->thj", qq, kk) * scale
            x = torch.where(mine[:, None, :], x, -math.inf)
            lse = torch.logsumexp(x, -1)
            w = torch.where(mine[:, None, :], torch.exp(x - torch.where(lse == -math.inf, 0.0, lse)[..., None]), 0.0)
            if torch.isfinite(vv).all() and torch.isfinite(w).all():
                o, va = torch.einsum("thj,jd->thd", w, vv), torch.einsum("thj,jd->thd", w, vv.abs())
            else:  # a row by itself: what it does not attend to has no part in it
                o, va = torch.zeros_like(qq), torch.zeros_like(qq)
                for t in range(b - a):
                    o[t] = w[t][:, mine[t]] @ vv[mine[t]]
                    va[t] = w[t][:, mine[t]] @ vv[mine[t]].abs()
            sl = (slice(a, b), slice(g * n, (g + 1) * n))
            out["o"][sl], out["lse"][sl], out["vabs"][sl] = o, lse, va
            ab = torch.einsum("thd,jd->thj", qq.abs(), kk.abs()) * abs(scale)
            if L:
                out["amax"][sl] = torch.where(mine[:, None, :], ab, 0.0).amax(-1)
            out["count"][sl] = mine.sum(-1)[:, None].double()
    return out


def check_attention(step, o, lse, want, dtype, v_largest, before_o=None, before_lse=None):
    """o and lse within what the arithmetic allows.

    A score is a sum of 128 exact products in f32 (2^-23 of the sum of their
    sizes each, at most 128 of them: delta = 2^-16 amax), its exponent is off by
    2^-22 of it, and the base-2 exponential by 2^-22; lse sums f32 weights.  A
    weight is then off by 2 delta + 2^-20 (1 + |exponent|), and rounded to the
    type, half a step; o is rounded once more.  What f16 does not hold of small
    weights is 2^-30 of the row's largest each."""
    half = HALF[dtype]
    live = torch.zeros(step.T, dtype=torch.bool, device=o.device)
    live[:step.first_list[-1]] = True
    delta = 2.0 ** -16 * want["amax"]
    got_o, got_lse = o.double(), lse.double()
    empty = want["lse"] == -math.inf
    assert torch.equal(got_lse[live] == -math.inf, empty[live])
    fine = torch.isfinite(want["lse"]) & live[:, None]
    allow = delta + 2.0 ** -21 * (8 + want["lse"].abs())
    bad = fine & ~((got_lse - want["lse"]).abs() <= allow)
    assert not bad.any(), f"lse: {int(bad.sum())} rows off, first {bad.nonzero()[0].tolist()}"
    assert torch.equal(torch.isnan(got_lse[live]), torch.isnan(want["lse"][live]))
    assert (got_o[empty & live[:, None]] == 0).all()
    allow = half * want["o"].abs() + (half + 2 * delta + 2.0 ** -18 * (8 + want["amax"]))[..., None] * want["vabs"] * 1.01
    allow = allow + (want["count"] * 2.0 ** -30 * v_largest + 1e-30)[..., None]
    rows = live[:, None, None] & ~empty[..., None]
    whole = torch.isfinite(want["o"]) & rows
    bad = whole & ~((got_o - want["o"]).abs() <= allow)
    assert not bad.any(), f"o: {int(bad.sum())} elements off, first {bad.nonzero()[0].tolist()}"
    rest = rows & ~whole  # a NaN or an infinity that is attended to
    assert not torch.isfinite(got_o[rest.expand_as(got_o)]).any()
    if before_o is not None:
        assert torch.equal(o[~live].view(torch.int16), before_o[~live].view(torch.int16))
        assert torch.equal(lse[~live], before_lse[~live])


def select(step, means, q, n_out, lead, trail, shift=0):
    """idx [T, Hk, n_out] int32: scores in f64, NaN and pages without an id last, ties to the lower page."""
    Hk, page, n = step.Hk, step.page, step.H // step.Hk
    idx = torch.full((step.T, Hk, n_out), -1, dtype=torch.int32)
    for r, (length, fresh) in enumerate(zip(step.lens_list, step.new_list)):
        ids = step.tables[r].long()
        real = ((ids >= 0) & (ids < step.pages)).cpu()
        rows = means[torch.where((ids >= 0) & (ids < step.pages), ids, 0)].double() if step.pages else None
        a, b = step.first_list[r], step.first_list[r + 1]
        if a == b or length < fresh:
            continue
        qs = q[a:b].double().view(b - a, Hk, n, DIM).sum(2)
        score = torch.einsum("thd,jhd->thj", qs, rows).cpu()
        for i in range(b - a):
            own = min((length - fresh + i) // page, step.P - 1)
            pinned = [j for j in range(own + 1) if j < lead or j > own - trail]
            free = [j for j in range(own + 1) if lead <= j <= own - trail]
            for g in range(Hk):
                s = score[i, g].tolist()
                free_g = sorted(free, key=lambda j: (0, -s[j], j) if real[j] and s[j] == s[j] else (1, 0.0, j))
                take = sorted(pinned + free_g[:n_out - len(pinned)])[:n_out]
                idx[a + i, g, :len(take)] = torch.tensor(take, dtype=torch.int32)
    return idx
