"""The paged 4-bit cache on the GPU against its plain 64-bit forms
(tests/cache_ref.py): plans, stored records and read rows exactly, the
attention within a bound derived from its arithmetic.

Bound.  The expanded keys, values and (scaled by a power of two) queries are
exact in f16, so a score's error is that of summing 128 products in fp32:
delta = 128 * 2^-23 * scale * sum |q k| <= 2^-16 amax, and 2^-22 of the
exponent (its scaling and the base-2 exponential).  lse sums unrounded fp32
weights: |error| <= delta + 2^-22 (8 + |lse|).  For o each weight is off by
2 delta (itself and the normaliser), is rounded to f16 (2^-11, or 2^-25 below
the normal range, against a largest weight of at least 1), and o is rounded
once to its type: |error| <= half |o| + vmax (2 delta + 2^-11 + n 2^-25 +
2^-19), half = 2^-8 (bf16) or 2^-11 (f16).
"""
import numpy as np
import pytest

from tests import cache_ref as ref

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
HALF = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}


def _mods():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    import sparse_attention_indexer_live_gb300 as dsa
    return torch, dsa


def _type(torch, name):
    return {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}[name]


# ---------------------------------------------------------------------------
# plan

def _run_plan(torch, dsa, page, pages, lens, fresh, tables, held, free, count, T):
    cfg = dsa.cache_cfg(pages=pages, page_size=page)
    d = {n: torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).to(DEV)
         for n, x in dict(lens=lens, fresh=fresh, tables=tables, held=held, free=free).items()}
    d["count"] = torch.tensor([count], dtype=torch.int32, device=DEV)
    R = len(lens)
    out = {n: torch.full((k,), -77, dtype=torch.int32, device=DEV)
           for n, k in dict(first=R + 1, token_req=T, ends=T, slots=T, status=4).items()}
    dsa.dsa_cache_plan(cfg, d["lens"], d["fresh"], d["tables"], d["held"], d["free"], d["count"], out["first"],
                       out["token_req"], out["ends"], out["slots"], out["status"])
    torch.cuda.synchronize()
    out.update({n: d[n] for n in ("tables", "held", "free", "count")})
    return {n: x.cpu().numpy() for n, x in out.items()}


def _same_plan(got, want):
    for n, x in want.items():
        assert np.array_equal(got[n], x), f"{n}: got {got[n]} want {x}"


@pytest.mark.parametrize("R,page,P,T,seed", [(1, 64, 4, 5, 0), (48, 64, 260, 96, 1), (7, 1, 9, 40, 2),
                                             (513, 16, 40, 3000, 3), (2000, 128, 8, 9001, 4),
                                             (8192, 4096, 3, 20000, 5)])
def test_plan_steps(R, page, P, T, seed):
    torch, dsa = _mods()
    rng = np.random.default_rng(seed)
    pages = R * P // 2 + 3
    tables, held = np.full((R, P), -1), np.zeros(R, int)
    free, count = rng.permutation(pages), pages
    lens = np.zeros(R, int)
    for step in range(6):
        fresh = rng.integers(0, 2 * T // (R + 1) + 2, R)
        fresh = np.where(np.cumsum(fresh) <= T, fresh, 0)
        move = rng.integers(-2 * page, 2 * page + 1, R) + fresh
        new = np.clip(lens + move, fresh, P * page)
        new[rng.random(R) < 0.2] = 0
        fresh = np.minimum(fresh, new)
        want = ref.plan(page, pages, new, fresh, tables, held, free, count, T)
        got = _run_plan(torch, dsa, page, pages, new, fresh, tables, held, free, count, T)
        _same_plan(got, want)
        tables, held, free, count = want["tables"], want["held"], want["free"], int(want["count"][0])
        if want["status"][0] == 0:
            lens = new


@pytest.mark.parametrize("what,code", [("pages", 1), ("width", 2), ("tokens", 3), ("fresh", 4), ("negative", 4),
                                       ("held", 4), ("count", 4), ("room", 1)])
def test_plan_refuses_and_changes_nothing(what, code):
    torch, dsa = _mods()
    page, pages, R, P, T = 8, 10, 3, 4, 12
    tables = np.array([[3, -1, -1, -1], [5, 6, -1, -1], [-1, -1, -1, -1]])
    held, free, count = np.array([1, 2, 0]), np.array([9, 8, 7, 4, 2, 1, 0, -5, -5, -5]), 7
    lens, fresh = np.array([10, 17, 3]), np.array([2, 1, 3])
    if what == "pages":
        count = 2
    elif what == "width":
        lens[0] = 33
    elif what == "tokens":
        fresh = np.array([5, 6, 3])
    elif what == "fresh":
        fresh[2] = 4
    elif what == "negative":
        lens[1] = fresh[1] = -1
    elif what == "held":
        held[2] = 5
    elif what == "count":
        count = 11
    elif what == "room":  # the stack cannot take a page back
        lens, fresh, count = np.array([0, 17, 0]), np.array([0, 1, 0]), 10
        held = np.array([1, 3, 0])
    want = ref.plan(page, pages, lens, fresh, tables, held, free, count, T)
    assert want["status"][0] == code and np.array_equal(want["tables"], tables)
    _same_plan(_run_plan(torch, dsa, page, pages, lens, fresh, tables, held, free, count, T), want)


def test_plan_empty_and_bad_pages():
    torch, dsa = _mods()
    z = np.zeros(0, int)
    got = _run_plan(torch, dsa, 16, 4, z, z, np.zeros((0, 3)), z, np.array([1, 2, 3]), 3, 5)
    assert got["first"].tolist() == [0] and got["token_req"].tolist() == [-1] * 5
    assert got["ends"].tolist() == [0] * 5 and got["slots"].tolist() == [-1] * 5
    assert got["status"].tolist() == [0, 0, 0, 3]
    # page ids outside the cache give no slot
    tables, held = np.array([[7, -2, 1]]), np.array([3])
    got = _run_plan(torch, dsa, 2, 4, np.array([6]), np.array([6]), tables, held, np.array([0]), 1, 6)
    assert got["slots"].tolist() == [-1, -1, -1, -1, 2, 3] and got["ends"].tolist() == [1, 2, 3, 4, 5, 6]


# ---------------------------------------------------------------------------
# rows

@pytest.mark.parametrize("T,KV,dtype,layout", [(1, 1, "bf16", "packed"), (37, 3, "f16", "packed"),
                                               (300, 2, "f32", "packed"), (65, 2, "bf16", "half"),
                                               (65, 2, "f32", "half"), (33, 1, "f16", "odd"),
                                               (0, 2, "bf16", "packed")])
def test_write_and_read(T, KV, dtype, layout):
    torch, dsa = _mods()
    page, pages = 8, T // 8 + 3
    g = torch.Generator().manual_seed(T + KV)
    dt = _type(torch, dtype)
    spread = torch.exp(2 * torch.randn(T, 2, KV, 128, generator=g))
    both = (torch.randn(T, 2, KV, 128, generator=g) * spread).to(dt)
    if T > 10:
        both[2, 0, 0, 3], both[3, 1, 0, 17], both[4, 0, 0, 40] = float("nan"), float("inf"), -float("inf")
        both[5] = 0
        both[6, 0, 0, :16] = 2.0 ** -13
    if layout == "half":    # keys and values in one projection's output
        dev = both.to(DEV)
        k, v = dev[:, 0], dev[:, 1]
    elif layout == "odd":   # a token stride and a start that are no multiple of 16 bytes
        buf = torch.zeros(T * 131 + 3, dtype=dt, device=DEV)
        k = buf[1:1 + T * 131].view(T, 1, 131)[:, :, :128]
        k.copy_(both[:, 0])
        v = both[:, 1].to(DEV)
    else:
        k, v = both[:, 0].contiguous().to(DEV), both[:, 1].contiguous().to(DEV)
    slots = torch.randperm(pages * page, generator=g)[:T].int()
    skip = torch.zeros(T, dtype=torch.bool)
    if T > 10:
        slots[7], slots[8], slots[9] = -1, pages * page, -(2 ** 31)
        skip[7:10] = True
    cfg = dsa.cache_cfg(pages=pages, page_size=page, kv_heads=KV)
    cache = torch.full((dsa.dsa_cache_bytes(cfg),), 0xA5, dtype=torch.uint8, device=DEV)
    dsa.dsa_cache_write(cfg, k, v, slots.to(DEV), cache)
    ko = torch.full((T, KV, 128), 9.0, dtype=dt, device=DEV)
    vo = torch.full((T, KV, 128), 9.0, dtype=dt, device=DEV)
    dsa.dsa_cache_read(cfg, cache, slots.to(DEV), ko, vo)
    torch.cuda.synchronize()
    kn, vn = both[:, 0].double().numpy(), both[:, 1].double().numpy()
    want = np.full((pages * page, KV, ref.REC), 0xA5, dtype=np.uint8)
    rec = ref.pack(kn, vn)
    live = ~skip.numpy()
    want[slots.numpy()[live]] = rec[live]
    assert np.array_equal(cache.cpu().numpy().reshape(want.shape), want)
    kr, vr = ref.expand(rec)
    kr[~live], vr[~live] = 0, 0
    assert np.array_equal(ko.double().cpu().numpy(), kr, equal_nan=True)
    assert np.array_equal(vo.double().cpu().numpy(), vr, equal_nan=True)


@pytest.mark.parametrize("k_shift,v_shift", [(3, -9), (-32, 32)])
def test_shifts(k_shift, v_shift):
    torch, dsa = _mods()
    g = torch.Generator().manual_seed(5)
    x = torch.randn(2, 20, 1, 128, generator=g)
    k, v = x[0] * 2.0 ** k_shift, x[1] * 2.0 ** v_shift
    cfg = dsa.cache_cfg(pages=5, page_size=4, kv_heads=1, k_shift=k_shift, v_shift=v_shift)
    cache = torch.zeros(dsa.dsa_cache_bytes(cfg), dtype=torch.uint8, device=DEV)
    slots = torch.arange(20, dtype=torch.int32, device=DEV)
    dsa.dsa_cache_write(cfg, k.to(DEV), v.to(DEV), slots, cache)
    ko, vo = torch.empty(2, 20, 1, 128, device=DEV).unbind(0)
    dsa.dsa_cache_read(cfg, cache, slots, ko, vo)
    rec = ref.pack(x[0].double().numpy(), x[1].double().numpy())
    assert np.array_equal(cache.cpu().numpy().reshape(rec.shape), rec)
    kr, vr = ref.expand(rec)
    assert np.array_equal(ko.double().cpu().numpy(), kr * 2.0 ** k_shift)
    assert np.array_equal(vo.double().cpu().numpy(), vr * 2.0 ** v_shift)


# ---------------------------------------------------------------------------
# attention

class _Case:
    """A cache of random records, queries, lists and tables on host and device."""

    def __init__(self, T, H, KV, Kc, *, page=16, R=None, ctx=200, dtype="bf16", seed=0, k_shift=0, v_shift=0,
                 tables=None, q=None, sort=True):
        self.torch, self.dsa = _mods()
        torch = self.torch
        rng = np.random.default_rng(seed)
        self.page, self.KV, self.dtype = page, KV, dtype
        R = max(1, T // 2) if R is None else R
        P = -(-ctx // page)
        self.pages = R * P + 2
        order = rng.permutation(self.pages)[:R * P]
        self.tables = order.reshape(R, P).astype(np.int32) if tables is None else tables
        kv = rng.standard_normal((2, self.pages, page, KV, 128))
        self.cache = ref.pack(kv[0], kv[1])
        self.req = rng.integers(0, R, T).astype(np.int32)
        self.idx = np.full((T, Kc), -1, np.int32)
        for t in range(T):
            n = min(Kc, ctx)
            pick = rng.permutation(ctx)[:n]
            self.idx[t, :n] = np.sort(pick) if sort else pick
        q = rng.standard_normal((T, H, 128)) if q is None else q
        self.q = torch.from_numpy(np.asarray(q, dtype=np.float32)).to(_type(torch, dtype))
        self.cfg = self.dsa.cache_cfg(pages=self.pages, page_size=page, kv_heads=KV, k_shift=k_shift, v_shift=v_shift)
        self.scale = 128 ** -0.5 * 2.0 ** -k_shift
        self.T, self.H = T, H

    def device(self):
        t = self.torch
        d = lambda x: t.from_numpy(np.ascontiguousarray(x)).to(DEV)  # noqa: E731
        self.d = dict(cache=d(self.cache.reshape(-1)), q=self.q.to(DEV), idx=d(self.idx), req=d(self.req),
                      tables=d(self.tables))
        dt = _type(t, self.dtype)
        # a guard row after the last token
        self.o = t.full((self.T + 1, self.H, 128), 7.0, dtype=dt, device=DEV)
        self.lse = t.full((self.T + 1, self.H), 7.0, dtype=t.float32, device=DEV)
        return self

    def launch(self, form="decode", ws=None):
        d, dsa = self.d, self.dsa
        if form == "decode":
            dsa.dsa_cache_attention(self.cfg, d["cache"], d["q"], d["idx"], d["req"], d["tables"], self.scale,
                                    self.o[:self.T], self.lse[:self.T])
        else:
            if ws is None:
                ws = self.torch.empty(dsa.dsa_cache_attention_prompt_workspace(self.cfg, d["q"], d["idx"]),
                                      dtype=self.torch.uint8, device=DEV)
            dsa.dsa_cache_attention_prompt(self.cfg, d["cache"], d["q"], d["idx"], d["tables"][0], self.scale, ws,
                                           self.o[:self.T], self.lse[:self.T])
        return self

    def check(self, form="decode"):
        self.torch.cuda.synchronize()
        assert self.dsa.dsa_cache_attention_status() == self.dsa.DSA_OK
        o = self.o.double().cpu().numpy()
        lse = self.lse.double().cpu().numpy()
        assert (o[self.T:] == 7.0).all() and (lse[self.T:] == 7.0).all(), "rows behind the last token"
        req = self.req if form == "decode" else np.zeros(self.T, int)
        tables = self.tables if form == "decode" else self.tables[:1]
        c = self.cfg
        with np.errstate(invalid="ignore"):
            wo, wl, vmax, amax = ref.attention(self.cache, self.page, self.q.double().numpy(), self.idx, req, tables,
                                               self.scale, c.k_shift, c.v_shift, distinct=form != "decode")
        o, lse = o[:self.T], lse[:self.T]
        empty = np.isneginf(wl)
        assert (lse[empty] == -np.inf).all() and (o[empty] == 0).all(), "rows without a position"
        n = self.idx.shape[1]
        with np.errstate(invalid="ignore"):
            delta = 2.0 ** -16 * amax
            lerr = np.where(empty, 0, np.abs(lse - wl))
            lmax = np.where(empty, 1, delta + 2.0 ** -22 * (8 + np.abs(wl)))
            omax = HALF[self.dtype] * np.abs(wo) + (vmax * (2 * delta + 2.0 ** -11 + n * 2.0 ** -25 + 2.0 ** -19))[..., None]
            oerr = np.abs(o - wo)
            nan = np.isnan(wo)
        assert np.array_equal(nan, np.isnan(o)) and np.array_equal(np.isnan(wl), np.isnan(lse))
        assert (lerr <= lmax)[~np.isnan(wl)].all(), f"lse: {np.nanmax(lerr / lmax)} of its bound"
        assert (oerr <= omax)[~nan].all(), f"o: {np.nanmax(oerr / np.maximum(omax, 1e-30))} of its bound"
        return o, lse


SHAPES = [  # T, H, kv_heads, select, page, context, type
    (1, 8, 1, 1, 16, 40, "bf16"), (1, 8, 1, 300, 16, 400, "bf16"), (1, 1, 1, 17, 16, 100, "f16"),
    (3, 16, 1, 100, 8, 333, "f16"), (5, 5, 1, 33, 64, 200, "bf16"), (4, 12, 1, 64, 32, 90, "f16"),
    (6, 32, 4, 129, 16, 500, "bf16"), (2, 64, 1, 257, 16, 300, "f16"), (3, 128, 1, 140, 16, 300, "bf16"),
    (2, 96, 2, 70, 1, 150, "f16"), (9, 7, 7, 50, 4, 90, "bf16"), (40, 8, 1, 300, 64, 1000, "bf16"),
    (33, 20, 1, 31, 128, 200, "bf16"), (1, 8, 1, 5000, 64, 6000, "f16"), (2, 34, 2, 700, 16, 1000, "bf16"),
    (200, 8, 2, 40, 16, 64, "f16"), (1, 128, 1, 2048, 64, 3000, "f16"), (300, 16, 1, 64, 64, 300, "bf16"),
    (6, 8, 1, 3000, 64, 4000, "bf16"), (20, 16, 1, 2100, 16, 2500, "f16"),
    # more than 16 heads a key/value head and many tokens: tiles of 128 rows, whole and split over 2 and 4 CTAs
    (70, 17, 1, 1, 16, 40, "bf16"), (34, 24, 1, 129, 16, 300, "f16"), (40, 64, 1, 130, 8, 500, "bf16"),
    (160, 32, 1, 65, 64, 300, "f16"), (20, 128, 1, 2050, 64, 3000, "bf16"), (34, 96, 2, 1100, 16, 1500, "f16"),
    (9, 128, 1, 1030, 32, 1200, "bf16"),
    # rows split over 2, 4 and 8 CTAs that share SMs
    (150, 7, 1, 1100, 64, 1300, "bf16"), (80, 8, 1, 1100, 64, 1300, "f16"), (45, 16, 1, 2050, 64, 2300, "bf16"),
    (22, 8, 2, 2049, 16, 2300, "bf16"), (100, 16, 1, 2050, 64, 2300, "f16"), (50, 12, 1, 900, 32, 1000, "bf16"),
    (30, 10, 2, 800, 16, 900, "f16"), (7, 13, 1, 650, 16, 700, "bf16"),
    # tiles, whole: short lists of many tokens
    (100, 64, 1, 300, 16, 400, "bf16"), (90, 17, 1, 200, 64, 300, "f16"), (130, 100, 1, 5, 16, 60, "bf16"),
    (70, 128, 1, 33, 8, 90, "f16"), (75, 120, 2, 129, 16, 200, "bf16"),
]


@pytest.mark.parametrize("T,H,KV,Kc,page,ctx,dtype", SHAPES)
def test_attention(T, H, KV, Kc, page, ctx, dtype):
    _Case(T, H, KV, Kc, page=page, ctx=ctx, dtype=dtype, seed=T + H + Kc).device().launch().check()


@pytest.mark.parametrize("H,KV,T", [(8, 1, 14), (16, 2, 14), (64, 1, 14), (64, 1, 40), (128, 1, 14), (128, 1, 70)])
def test_attention_edge_rows(H, KV, T):
    c = _Case(T, H, KV, 150, page=16, ctx=200, R=5, sort=False, seed=H)
    c.idx[0] = -1                                   # nothing
    c.idx[1, :] = -1
    c.idx[1, 149] = 199                             # one position, in the last entry
    c.idx[2, ::2] = -1                              # holes
    c.idx[3] = -(2 ** 31)
    c.idx[4, :] = 7                                 # one position 150 times
    c.idx[5, 3:140] = 2 ** 31 - 1                   # past the table
    c.req[6], c.req[7], c.req[8] = -1, 5, 2 ** 31 - 1   # of no request
    c.req[9] = 4
    c.tables[4, 3], c.tables[4, 5], c.tables[4, 6] = -1, c.pages, -(2 ** 31)  # bad pages
    c.idx[10, 128:] = -1                            # a tile's worth
    c.idx[11, 1:] = -1
    c.idx[12, :130] = -1                            # the tail only
    c.device().launch().check()


@pytest.mark.parametrize("H,T", [(8, 6), (64, 6), (128, 12), (128, 70)])
def test_attention_ignores_what_is_not_selected(H, T):
    # NaN scales in places no row lists
    c = _Case(T, H, 1, 60, page=8, ctx=80, R=2, seed=3)
    c.idx[:, 40:] = -1
    c.idx[:, :40] = np.where(c.idx[:, :40] % 8 == 7, -1, c.idx[:, :40])
    listed = np.zeros((c.pages, 8), bool)
    for t in range(T):
        p = c.idx[t][c.idx[t] >= 0]
        listed[c.tables[c.req[t]][p // 8], p % 8] = True
    assert not listed.all()
    c.cache[~listed] = 0xFF
    o, _ = c.device().launch().check()
    assert np.isfinite(o).all()
    # a NaN record makes the rows that list it NaN, no others
    p = int(c.idx[2][c.idx[2] >= 0][5])
    c.cache[c.tables[c.req[2], p // 8], p % 8, 0, 128:] = 0x7F
    o, _ = c.device().launch().check()
    assert np.isnan(o[2]).all() and np.isfinite(o).any()


@pytest.mark.parametrize("H,T", [(8, 7), (24, 7), (128, 12), (128, 70)])
def test_attention_query_magnitudes(H, T):
    rng = np.random.default_rng(8)
    q = rng.standard_normal((T, H, 128))
    q[0] *= 1e30
    q[1] *= 1e-30
    q[2] = 0
    q[3, :, 1:] *= 1e-6      # one large element
    q[4, 0] = np.inf
    q[5, H - 1, 3] = np.nan
    q[6] *= 2.0 ** -120
    c = _Case(T, H, 1, 90, ctx=120, q=q, seed=9)
    # scores of 1e30 leave one position; infinite and NaN queries give NaN rows
    c.device().launch()
    c.torch.cuda.synchronize()
    got_o, got_l = c.o.double().cpu().numpy(), c.lse.double().cpu().numpy()
    assert np.isnan(got_l[4, 0]) and np.isnan(got_o[4, 0]).all() and np.isnan(got_l[5, H - 1])
    assert np.isfinite(got_o[4, 1:]).all() and np.isfinite(got_o[5, :H - 1]).all()
    with np.errstate(invalid="ignore"):
        wo, wl, vmax, _ = ref.attention(c.cache, c.page, c.q.double().numpy(), c.idx, c.req, c.tables, c.scale)
    assert np.abs(got_o[0] - wo[0]).max() <= 2.0 ** -7 * vmax[0].max()
    assert (np.abs(got_l[0] - wl[0]) <= 2.0 ** -16 * np.abs(wl[0])).all()
    for x in (c.q, c.idx, c.req):
        x[[0, 4, 5]] = x[[1, 1, 1]]
    c.device().launch().check()


def test_attention_scores_that_rise():
    # keys that grow with the position: the running maximum moves in every tile
    for T, H in ((2, 8), (2, 128), (20, 128)):
        c = _Case(T, H, 1, 3000, page=64, ctx=4000, R=2, dtype="f16", seed=1)
        pos = np.zeros((c.pages, 64))
        for r in range(2):
            for j in range(c.tables.shape[1]):
                pos[c.tables[r, j]] = j * 64 + np.arange(64)
        k = 0.55 * pos[..., None, None] / 4000 + 0.02 * np.random.default_rng(2).standard_normal((c.pages, 64, 1, 128))
        v = np.random.default_rng(3).standard_normal((c.pages, 64, 1, 128))
        c.cache = ref.pack(k, v)
        c.q = c.q * 0.05 + 0.5
        c.scale = 1.0
        c.device().launch().check()


def test_attention_shifts():
    for T, H in ((4, 8), (4, 64), (20, 64)):
        _Case(T, H, 1, 100, ctx=150, k_shift=5, v_shift=-7, seed=4).device().launch().check()
        # no scale: every weight is the same; a negative one
        for scale in (0.0, -0.05):
            c = _Case(T, H, 1, 100, ctx=150, seed=4)
            c.scale = scale
            c.device().launch().check()


def test_attention_past_32_bits():
    # records behind 2^32 bytes and past 2^31 elements
    torch, dsa = _mods()
    page, pages = 4096, 8000
    cfg = dsa.cache_cfg(pages=pages, page_size=page)
    cache = torch.empty(dsa.dsa_cache_bytes(cfg), dtype=torch.uint8, device=DEV)
    rng = np.random.default_rng(6)
    kv = rng.standard_normal((2, 64, 1, 128)).astype(np.float32)
    slots = np.sort(rng.choice(100 * page, 64, replace=False)) + (pages - 100) * page
    assert slots.min() * 144 > 2 ** 32
    dsa.dsa_cache_write(cfg, torch.from_numpy(kv[0]).to(DEV), torch.from_numpy(kv[1]).to(DEV),
                        torch.from_numpy(slots.astype(np.int32)).to(DEV), cache)
    tables = torch.arange(pages, dtype=torch.int32, device=DEV)[None, :].contiguous()
    rec = ref.pack(kv[0].astype(np.float64), kv[1].astype(np.float64))
    for H in (8, 128):
        T = 2 if H == 8 else 10
        q = torch.randn(T, H, 128, generator=torch.Generator().manual_seed(1)).bfloat16()
        idx = torch.from_numpy(np.tile(slots.astype(np.int32), (T, 1))).to(DEV)
        o = torch.empty(T, H, 128, dtype=torch.bfloat16, device=DEV)
        lse = torch.empty(T, H, device=DEV)
        dsa.dsa_cache_attention(cfg, cache, q.to(DEV), idx, torch.zeros(T, dtype=torch.int32, device=DEV), tables,
                                128 ** -0.5, o, lse)
        small = rec.reshape(1, 64, 1, 144)
        wo, wl, vmax, amax = ref.attention(small, 64, q.double().numpy(), np.tile(np.arange(64), (T, 1)), [0] * T,
                                           np.zeros((1, 1), int), 128 ** -0.5)
        assert (np.abs(lse.double().cpu().numpy() - wl) <= 2.0 ** -16 * amax + 2.0 ** -22 * (8 + np.abs(wl))).all()
        assert (np.abs(o.double().cpu().numpy() - wo) <= 2.0 ** -8 * np.abs(wo) + 2.0 ** -10 * vmax[..., None]).all()


def test_attention_repeats_bit_for_bit():
    for H, T in ((8, 1), (8, 100), (128, 2), (128, 20)):
        c = _Case(T, H, 1, 900, page=64, ctx=1500, seed=5).device().launch()
        o, lse = c.o.clone(), c.lse.clone()
        for _ in range(3):
            c.launch()
            assert c.torch.equal(c.o, o) and c.torch.equal(c.lse, lse)


def test_attention_empty_shapes():
    torch, dsa = _mods()
    c = _Case(3, 8, 1, 0, ctx=20).device().launch().check()   # lists of no entry
    _Case(0, 8, 1, 5, ctx=20, R=1).device().launch().check()  # no token
    # no request and no page
    cfg = dsa.cache_cfg(pages=0, page_size=16)
    i32 = dict(dtype=torch.int32, device=DEV)
    o = torch.full((2, 8, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((2, 8), 7.0, device=DEV)
    dsa.dsa_cache_attention(cfg, torch.empty(0, dtype=torch.uint8, device=DEV), torch.ones_like(o),
                            torch.zeros((2, 4), **i32), torch.zeros(2, **i32), torch.empty((0, 3), **i32), 1.0, o, lse)
    assert (o == 0).all() and torch.isneginf(lse).all()


def test_attention_in_a_graph_and_on_a_stream():
    c = _Case(5, 8, 1, 200, page=16, ctx=400, R=3, seed=11).device()
    torch = c.torch
    c.launch()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        c.launch()
    torch.cuda.current_stream().wait_stream(s)
    c.check()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.launch()
    rng = np.random.default_rng(12)
    for _ in range(2):
        c.idx = np.stack([np.sort(rng.permutation(400)[:200]) for _ in range(5)]).astype(np.int32)
        c.idx[3, 50:] = -1
        c.req = rng.integers(0, 3, 5).astype(np.int32)
        c.d["idx"].copy_(torch.from_numpy(c.idx))
        c.d["req"].copy_(torch.from_numpy(c.req))
        c.o.fill_(7.0)
        c.lse.fill_(7.0)
        g.replay()
        c.check()


def test_calls_on_two_streams_at_once():
    """Nothing is shared between calls: decode and prompt calls that overlap in
    time, each with its own outputs (and workspace), give what they give alone."""
    torch, dsa = _mods()
    a = _Case(64, 8, 1, 600, page=16, ctx=900, R=1, seed=41).device()
    b = _Case(40, 64, 1, 500, page=32, ctx=800, R=3, seed=42).device()
    c = _Case(64, 16, 1, 500, page=32, ctx=800, R=1, seed=43).device()
    ws = torch.empty(dsa.dsa_cache_attention_prompt_workspace(c.cfg, c.d["q"], c.d["idx"]), dtype=torch.uint8,
                     device=DEV)
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, x, form in zip(streams, (a, b, c), ("decode", "decode", "prompt")):
            with torch.cuda.stream(s):
                x.launch(form, ws)
    a.check()
    b.check()
    c.check("prompt")


def test_explicit_stream():
    torch, dsa = _mods()
    c = _Case(5, 8, 1, 60, ctx=100, seed=44).device()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    d = c.d
    with torch.cuda.stream(s):
        torch.cuda._sleep(2000000)  # what the call must queue behind
        late = d["q"].clone()
        d["q"].zero_()
        d["q"].copy_(late)
    dsa.dsa_cache_attention(c.cfg, d["cache"], d["q"], d["idx"], d["req"], d["tables"], c.scale, c.o[:5], c.lse[:5],
                            stream=s)
    torch.cuda.current_stream().wait_stream(s)
    c.check()


# ---------------------------------------------------------------------------
# the prompt form

PROMPTS = [  # T, H, kv_heads, select, page, context, type
    (1, 8, 1, 1, 16, 30, "bf16"), (1, 16, 1, 200, 16, 300, "f16"), (37, 8, 1, 64, 64, 500, "bf16"),
    (29, 16, 1, 100, 8, 333, "f16"), (40, 8, 1, 300, 16, 6000, "bf16"), (17, 32, 2, 130, 32, 400, "bf16"),
    (50, 16, 2, 257, 64, 700, "f16"), (130, 8, 1, 33, 128, 4000, "f16"),
    # few groups: their tiles over 8, 4 and 2 CTAs
    (20, 8, 1, 2100, 64, 5000, "bf16"), (100, 16, 1, 1100, 64, 3000, "f16"), (300, 16, 2, 520, 64, 2000, "bf16"),
]


@pytest.mark.parametrize("T,H,KV,Kc,page,ctx,dtype", PROMPTS)
def test_prompt(T, H, KV, Kc, page, ctx, dtype):
    _Case(T, H, KV, Kc, page=page, ctx=ctx, dtype=dtype, R=1, seed=T + H).device().launch("prompt").check("prompt")


@pytest.mark.parametrize("H", [8, 16])
def test_prompt_edge_rows(H):
    c = _Case(35, H, 1, 150, page=16, ctx=200, R=1, seed=H)
    c.idx[0] = -1
    c.idx[1, 1:] = -1
    c.idx[2, 100:] = -1
    c.idx[16:24] = -1                             # a group (of 16 heads) without a position
    c.idx[30, 140:150] = np.arange(10) * 100000 + 200   # past the table
    c.tables[0, 3], c.tables[0, 5] = -1, c.pages  # bad pages
    c.device().launch("prompt").check("prompt")


def test_prompt_rising_and_odd_queries():
    c = _Case(18, 8, 1, 700, page=64, ctx=2000, R=1, dtype="f16", seed=1)
    pos = np.zeros((c.pages, 64))
    for j in range(c.tables.shape[1]):
        pos[c.tables[0, j]] = j * 64 + np.arange(64)
    k = 0.55 * pos[..., None, None] / 2000 + 0.02 * np.random.default_rng(2).standard_normal((c.pages, 64, 1, 128))
    c.cache = ref.pack(k, np.random.default_rng(3).standard_normal((c.pages, 64, 1, 128)))
    c.q = c.q * 0.05 + 0.5
    c.scale = 1.0
    c.device().launch("prompt").check("prompt")
    q = np.random.default_rng(4).standard_normal((20, 8, 128))
    q[3] *= 1e-30
    q[4] = 0
    q[5] *= 1e-6
    _Case(20, 8, 1, 90, ctx=120, q=q, R=1, k_shift=4, v_shift=3, seed=9).device().launch("prompt").check("prompt")
    c = _Case(20, 8, 1, 90, ctx=120, R=1, seed=9)
    c.scale = -0.05
    c.device().launch("prompt").check("prompt")


def test_prompt_nan_stays_in_its_rows():
    c = _Case(20, 8, 1, 40, page=16, ctx=300, R=1, seed=2)
    seen = np.unique(c.idx)
    rest = np.setdiff1d(np.arange(300), seen)
    c.cache[c.tables[0][rest // 16], rest % 16] = 0xFF       # no row lists these
    o, _ = c.device().launch("prompt").check("prompt")
    assert np.isfinite(o).all()
    # a record of NaN: the rows that list it are NaN, no others of the group
    p = int(c.idx[3][7])
    c.cache[c.tables[0, p // 16], p % 16, 0, 128:] = 0x7F
    o, _ = c.device().launch("prompt").check("prompt")
    assert np.isfinite(o).any() and np.isnan(o).any()
    # one whose values alone are NaN, or a single group of them
    for lo, hi in ((136, 144), (140, 141)):
        p = int(c.idx[12][20])
        c.cache[c.tables[0, p // 16], p % 16, 0, lo:hi] = 0x7F
        c.device().launch("prompt")
        c.torch.cuda.synchronize()
        bad = np.isnan(c.o[:20].float().cpu().numpy()).any((1, 2))
        first = int(c.idx[3][7])
        assert np.array_equal(bad, (c.idx == p).any(1) | (c.idx == first).any(1))


def test_prompt_graphs_sharing_a_workspace():
    a = _Case(33, 8, 1, 120, page=16, ctx=600, R=1, seed=21).device()
    b = _Case(20, 16, 1, 90, page=32, ctx=500, R=1, seed=22).device()
    torch = a.torch
    ws = torch.empty(max(a.dsa.dsa_cache_attention_prompt_workspace(x.cfg, x.d["q"], x.d["idx"]) for x in (a, b)),
                     dtype=torch.uint8, device=DEV)
    a.launch("prompt", ws)
    b.launch("prompt", ws)
    graphs = []
    for x in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            x.launch("prompt", ws)
        graphs.append(g)
    for g in (0, 1, 0, 1, 1, 0):
        x = (a, b)[g]
        x.o.fill_(7.0)
        x.lse.fill_(7.0)
        graphs[g].replay()
        x.check("prompt")


# ---------------------------------------------------------------------------
# the operators together, as a server runs them

def test_a_decode_step_with_the_selection():
    """Prompts stored, then decode steps: plan, store, select on logits, join
    with a window, attend; drafts taken back; a request finished."""
    torch, dsa = _mods()
    R, page, P, KV, H, K, window = 4, 16, 16, 2, 16, 24, 8
    c = dsa.PagedCache(requests=R, pages=40, pages_per_request=P, page_size=page, kv_heads=KV)
    rng = np.random.default_rng(31)
    rows = {}  # (request, position) -> (k, v) as stored
    dev = lambda x: torch.from_numpy(np.asarray(x, dtype=np.int32)).to(DEV)  # noqa: E731

    def step(lens, fresh, tokens):
        c.step(dev(lens), dev(fresh), tokens)
        c.ok()
        kv = torch.from_numpy(rng.standard_normal((2, tokens, KV, 128)).astype(np.float32)).bfloat16().to(DEV)
        c.store(kv[0], kv[1])
        req, ends = c.token_req.cpu().numpy(), c.ends.cpu().numpy()
        rec = ref.pack(kv[0].double().cpu().numpy(), kv[1].double().cpu().numpy())
        for i, (r, e) in enumerate(zip(req, ends)):
            if r >= 0:
                rows[(int(r), int(e) - 1)] = rec[i]
        return req, ends

    lens = np.array([100, 37, 0, 150])
    step(lens, lens, 300)
    for it in range(3):
        step_lens = lens + 2
        T = 2 * R + 3  # a padded batch
        req, ends = step(step_lens, np.full(R, 2), T)
        W = P * page
        logits = torch.from_numpy(rng.standard_normal((T, W)).astype(np.float32)).to(DEV)
        plan = dsa.dsa_select_init(rows=T, width=W, block_size=4, block_topk=10, row_topk=K)
        cand = torch.empty((T, 11), dtype=torch.int32, device=DEV)
        topk = torch.empty((T, K), dtype=torch.int32, device=DEV)
        idx = torch.empty((T, K + window), dtype=torch.int32, device=DEV)
        dsa.dsa_select_topk(plan, logits, None, c.ends, cand, topk)
        dsa.dsa_combine_window(plan, None, c.ends, topk, window, idx)
        q = torch.from_numpy(rng.standard_normal((T, H, 128)).astype(np.float32)).bfloat16().to(DEV)
        o, lse = c.attend(q, idx, 128 ** -0.5)
        torch.cuda.synchronize()
        # against the rows kept on the host
        lists = idx.cpu().numpy()
        for t in range(T):
            sel = lists[t][lists[t] >= 0]
            if req[t] < 0:
                assert len(sel) == 0 and (o[t] == 0).all()
                continue
            assert ends[t] - 1 in sel
            mine = np.stack([rows[(int(req[t]), int(p))] for p in sel])[None]
            wo, wl, vmax, amax = ref.attention(mine, len(sel), q[t:t + 1].double().cpu().numpy(),
                                               np.arange(len(sel))[None], [0], np.zeros((1, 1), int), 128 ** -0.5)
            delta = 2.0 ** -16 * amax
            assert (np.abs(lse[t].double().cpu().numpy() - wl[0]) <= delta[0] + 2.0 ** -22 * (8 + np.abs(wl[0]))).all()
            lim = 2.0 ** -8 * np.abs(wo[0]) + (vmax * (2 * delta + 2.0 ** -11 + 2.0 ** -18))[0][:, None]
            assert (np.abs(o[t].double().cpu().numpy() - wo[0]) <= lim).all()
        # request it keeps its draft, the others reject theirs; then request 3 finishes
        lens = lens + 1
        lens[it] += 1
        if it == 1:
            lens[3] = 0
        c.step(dev(lens), dev(np.zeros(R)), T)
        c.ok()
        assert c.status[3].item() == 40 - sum(-(-int(n) // page) for n in lens)
    # a request's rows, fetched by the slots of its whole length
    n = int(lens[0])
    c.step(dev(lens), dev([n, 0, 0, 0]), n)
    k, v = c.fetch(c.slots)
    want = [ref.expand(rows[(0, p)]) for p in range(n)]
    assert np.array_equal(k.double().cpu().numpy(), np.stack([w[0] for w in want]))
    assert np.array_equal(v.double().cpu().numpy(), np.stack([w[1] for w in want]))
    # the chunk form over the same rows
    q = torch.randn(n, H, 128, device=DEV, generator=torch.Generator(DEV).manual_seed(2)).bfloat16()
    lists = torch.arange(n, device=DEV, dtype=torch.int32).repeat(n, 1)
    lists = torch.where(lists <= torch.arange(n, device=DEV)[:, None], lists, -1).int().contiguous()
    o1, l1 = c.attend(q, lists, 128 ** -0.5)
    o2, l2 = c.attend(q, lists, 128 ** -0.5, request=0)
    assert (l1 - l2).abs().max() < 1e-4 and (o1.float() - o2.float()).abs().max() < 0.05
    with pytest.raises(RuntimeError, match="pages short"):
        c.step(dev([256, 256, 256, 0]), dev(np.zeros(R)), 0)
        c.ok()


def test_captured_steps_of_several_sizes():
    """A graph of a step stays good when larger steps follow: plan, store and
    attend captured for 3 tokens, then run again after a step of 400."""
    torch, dsa = _mods()
    R, page = 3, 16
    c = dsa.PagedCache(requests=R, pages=64, pages_per_request=32, page_size=page)
    lens = torch.tensor([5, 9, 2], dtype=torch.int32, device=DEV)
    fresh = lens.clone()
    gen = torch.Generator(DEV).manual_seed(41)
    c.step(lens, fresh, 16)
    c.ok()
    c.store(*torch.randn(2, 16, 1, 128, device=DEV, generator=gen).bfloat16().unbind(0))
    kv = torch.randn(2, R, 1, 128, device=DEV, generator=gen).bfloat16()
    q = torch.randn(R, 8, 128, device=DEV, generator=gen).bfloat16()
    idx = torch.arange(16, device=DEV, dtype=torch.int32).repeat(R, 1)

    def decode():
        lens.add_(1)
        c.step(lens, fresh, R)
        c.store(kv[0], kv[1])
        return c.attend(q, torch.where(idx < c.ends[:, None], idx, -1), 0.1)

    fresh.fill_(1)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        decode()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o, lse = decode()
    maps = (c.token_req, c.ends, c.slots)
    # a step of another size, which outgrows the first one's memory, and rows
    # of the same sizes as its maps to fall into memory that was given up
    c.step(lens, torch.zeros_like(lens), 400)
    c.ok()
    others = [torch.full((n,), 12345, dtype=torch.int32, device=DEV) for n in (3, 9, 64, 192, 400) for _ in range(8)]
    for _ in range(2):
        g.replay()
        torch.cuda.synchronize()
        assert maps[0].tolist() == [0, 1, 2] and maps[1].tolist() == lens.tolist()
        assert all((x == 12345).all() for x in others)
        # the same answer from a fresh call on the same state
        c.step(lens, fresh, R)
        c.ok()
        assert torch.equal(c.slots, maps[2])
        want = c.attend(q, torch.where(idx < c.ends[:, None], idx, -1), 0.1)
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
        c.step(lens, torch.zeros_like(lens), 400)


@pytest.mark.parametrize("H,KV,R", [(8, 1, 5), (16, 2, 40), (64, 1, 70)])
def test_calls_follow_one_another(H, KV, R):
    """Steps whose calls depend on one another, enqueued without a pause, give
    what they give when each call has ended before the next begins."""
    torch, dsa = _mods()
    page, P, K, steps = 16, 8, 48, 12
    gen = torch.Generator(DEV).manual_seed(51)
    kv = torch.randn(steps, 2, 2 * R, KV, 128, device=DEV, generator=gen).bfloat16()
    q = torch.randn(steps, 2 * R, H, 128, device=DEV, generator=gen).bfloat16()
    grow = torch.randint(0, 3, (steps, R), device=DEV, generator=gen, dtype=torch.int32)
    pick = torch.randint(0, 1 << 20, (steps, 2 * R, K), device=DEV, generator=gen, dtype=torch.int32)

    def run(pause):
        wait = torch.cuda.synchronize if pause else lambda: None
        c = dsa.PagedCache(requests=R, pages=R * P, pages_per_request=P, page_size=page, kv_heads=KV)
        lens = torch.zeros(R, dtype=torch.int32, device=DEV)
        got = []
        for i in range(steps):
            lens.add_(grow[i])
            wait()
            c.step(lens, grow[i], 2 * R)
            wait()
            c.store(kv[i, 0], kv[i, 1])
            wait()
            idx = torch.where(c.ends[:, None] > 0, pick[i] % c.ends.clamp(min=1)[:, None], -1)
            wait()
            got += c.attend(q[i], idx, 0.1)
            wait()
            got += c.fetch(c.slots)
            wait()
            got += c.attend(q[i], idx, 0.1)  # straight after another call
            wait()
            got += [c.slots.clone(), c.status.clone(), c.free_pages.clone()]
            if H // KV in (8, 16):
                n = 2 * R
                rows = torch.arange(K, device=DEV, dtype=torch.int32).repeat(n, 1)
                got += c.attend(q[i], torch.where(rows < lens[0], rows, -1), 0.1, request=0)
                wait()
        torch.cuda.synchronize()
        return got

    want = run(True)
    for _ in range(3):
        for a, b in zip(run(False), want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("form", ["decode", "prompt"])
def test_captured_between_copies_and_streams(form):
    """A graph in which copies and clears come right before the calls and one
    call runs on a second stream: the same results as without a graph."""
    torch, dsa = _mods()
    R, page, T, H = 2, 16, 8, 16
    gen = torch.Generator(DEV).manual_seed(61)
    c = dsa.PagedCache(requests=R, pages=32, pages_per_request=16, page_size=page)
    lens0 = torch.tensor([90, 33], dtype=torch.int32, device=DEV)
    c.step(lens0, lens0, 123)
    c.ok()
    c.store(*torch.randn(2, 123, 1, 128, device=DEV, generator=gen).bfloat16().unbind(0))
    src = [torch.randn(2, T, 1, 128, device=DEV, generator=gen).bfloat16() for _ in range(3)]
    qs = [torch.randn(T, H, 128, device=DEV, generator=gen).half() for _ in range(3)]
    lists = torch.arange(80, device=DEV, dtype=torch.int32).repeat(T, 1)
    lens_in, fresh_in = lens0 + torch.tensor([6, 2], dtype=torch.int32, device=DEV), torch.tensor(
        [6, 2], dtype=torch.int32, device=DEV)
    lens, fresh, idx = torch.empty_like(lens_in), torch.empty_like(fresh_in), torch.empty_like(lists)
    kv_in, kv = src[0].clone(), torch.empty_like(src[0])
    q_in, q = qs[0].clone(), torch.empty_like(qs[0])
    rows = torch.empty(2, T, 1, 128, dtype=torch.bfloat16, device=DEV)
    side = torch.cuda.Stream()
    c.step(lens_in, fresh_in, T)  # makes the maps

    def step():
        main = torch.cuda.current_stream()
        lens.copy_(lens_in)
        fresh.copy_(fresh_in)
        c.step(lens, fresh, T)
        kv.copy_(kv_in)
        c.store(kv[0], kv[1])
        side.wait_stream(main)
        with torch.cuda.stream(side):
            rows.zero_()
            dsa.dsa_cache_read(c.cfg, c.data, c.slots, rows[0], rows[1])
        q.copy_(q_in)
        idx.copy_(lists)
        o, lse = c.attend(q, idx, 0.1, request=0 if form == "prompt" else None)
        main.wait_stream(side)
        again = c.attend(q, idx, 0.1, request=0 if form == "prompt" else None)
        return o, lse, rows.clone(), *again

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step()
    for x, y in zip(src, qs):
        kv_in.copy_(x)
        q_in.copy_(y)
        g.replay()
        g.replay()
        torch.cuda.synchronize()
        have = [t.clone() for t in got]
        want = step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(have, want))
        assert torch.equal(have[0], have[3]) and torch.equal(have[1], have[4])
    assert dsa.dsa_cache_attention_status() == dsa.DSA_OK
