"""The paged 16-bit cache on the GPU against its plain 64-bit forms
(tests/kv_ref.py, which derives the tolerances)."""
import math

import pytest

torch = pytest.importorskip("torch")

from tests import kv_ref as ref  # noqa: E402

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]

DEV = "cuda:0"
BF16, F16 = torch.bfloat16, torch.float16
I32 = dict(dtype=torch.int32, device=DEV)


def _dsa():
    import sparse_attention_indexer_live_gb300 as dsa
    return dsa


def _cfg(step):
    return _dsa().kv_cfg(pages=step.pages, page_size=step.page, kv_heads=step.Hk, dtype=step.dtype)


# ---------------------------------------------------------------------------
# append

def _append(step, H, rot, neighbours, gain=1.0, theta=1e4, q=True, means=True, inplace=False, far=0, drop=()):
    """One call on a step's tokens against f64; everything it should leave alone is as it was."""
    dsa = _dsa()
    Hk, page, T, dt = step.Hk, step.page, step.T, step.dtype
    qkv = step.normal(T, H + 2 * Hk, 128)
    if inplace:
        qq, kk, vv = qkv[:, :H].contiguous(), qkv[:, H:H + Hk].contiguous(), qkv[:, H + Hk:]
    else:
        qq, kk, vv = qkv[:, :H], qkv[:, H:H + Hk], qkv[:, H + Hk:]
    k0, v0 = (step.normal(step.pages, page, Hk, 128) for _ in range(2))
    m0 = step.normal(step.pages, Hk, 128)
    ends, slots = torch.zeros(T, **I32), torch.full((T,), -1, **I32)
    table = step.tables.cpu().tolist()
    for r, p, t in step.tokens():
        ends[t] = p + 1 + far
        slots[t] = -1 if t in drop else table[r][p // page] * page + p % page
    inv = theta ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=DEV) / max(rot, 1))
    k, v, m, q0 = k0.clone(), v0.clone(), m0.clone(), qq.clone()
    out = qq if inplace else torch.full((T, H, 128), 7.0, dtype=dt, device=DEV)
    out0 = out.clone()
    dsa.dsa_kv_append(_cfg(step), qq if q else None, kk, vv, ends, slots, dsa.rotary_turns(inv), neighbours, gain,
                      out if q else None, k, v, m if means else None)
    torch.cuda.synchronize()
    pos, half = ends.long() - 1, ref.HALF[dt]
    live = ends > 0

    def near(got, rows, what):
        # a rounding, and in f32 the angle (2^-24 of a turn's radians), its sine (2^-22) and three operations
        want = ref.rotate(rows, pos.clamp(min=0), inv, neighbours, gain)
        size = rows.double().abs().amax(-1, keepdim=True) * abs(gain)
        bad = live[:, None, None] & ~((got.double() - want).abs() <= half * want.abs() + 2.0 ** -20 * size + 1e-30)
        assert not bad.any(), f"{what}: {int(bad.sum())} off, first {bad.nonzero()[0].tolist()}"

    if q:
        near(out, q0, "q")
        assert torch.equal(out[~live], out0[~live])
    held = (slots >= 0).nonzero().flatten()
    at = slots[held].long()
    flat = k.view(-1, Hk, 128)
    rows = torch.zeros(T, Hk, 128, dtype=dt, device=DEV)
    rows[held] = flat[at]
    live = live & (slots >= 0)
    near(rows, kk, "k")
    assert torch.equal(v.view(-1, Hk, 128)[at], vv[held])
    for x, x0 in ((k, k0), (v, v0)):
        y = x.clone().view(-1, Hk, 128)
        y[at] = x0.view(-1, Hk, 128)[at]
        assert torch.equal(y.view_as(x0), x0)
    filled = (at[at % page == page - 1] // page).tolist() if means else []
    for j in range(step.pages):
        if j in filled:
            want = k[j].double().mean(0)
            # f32 sums of `page` rows: 2^-24 of the running sum each
            assert ((m[j].double() - want).abs() <= half * want.abs() + 2.0 ** -17 * k[j].double().abs().mean(0)).all(), j
        else:
            assert torch.equal(m[j], m0[j]), j
    return len(filled)


@pytest.mark.parametrize("lens,new,H,Hk,page,rot,neighbours,dtype", [
    ([1], [1], 1, 1, 16, 128, False, BF16),
    ([64], [1], 8, 1, 64, 128, False, BF16),
    ([130, 33, 64, 700], [2, 2, 2, 2], 32, 8, 64, 128, False, BF16),
    ([300, 1, 129], [300, 1, 77], 12, 4, 32, 64, True, F16),
    ([700], [700], 5, 1, 16, 96, False, F16),
    ([700, 256], [333, 256], 24, 2, 128, 32, True, BF16),
    ([90, 0, 17], [50, 0, 17], 128, 1, 16, 16, False, F16),
    ([500], [250], 6, 3, 32, 0, False, BF16),
    ([3000], [2500], 32, 8, 64, 128, False, BF16)])
def test_append(lens, new, H, Hk, page, rot, neighbours, dtype):
    step = ref.Step(lens, new, H=H, Hk=Hk, page=page, dtype=dtype, seed=len(lens) + H, pad=3)
    filled = _append(step, H, rot, neighbours)
    assert filled == sum(n // page - (n - f) // page for n, f in zip(lens, new))


@pytest.mark.parametrize("kw", [dict(q=False), dict(means=False), dict(inplace=True), dict(gain=-0.3), dict(theta=1e6),
                                dict(drop=(0, 3, 64, 65))])
def test_append_forms(kw):
    step = ref.Step([200, 70], [130, 5], H=16, Hk=2, page=32, dtype=BF16, seed=5, pad=1)
    _append(step, 16, 128, False, **kw)


def test_append_far_positions():
    # angles of positions near 2^31: the fastest pair has turned 3 * 10^8 times
    step = ref.Step([40], [40], H=4, Hk=2, page=16, dtype=F16, seed=6)
    _append(step, 4, 128, False, theta=5e5, far=2 ** 31 - 64)


# ---------------------------------------------------------------------------
# attention

def _strided(x):
    """x [T, H, 128] as part of wider rows."""
    T, H, D = x.shape
    wide = torch.full((T, H + 3, D), math.nan, dtype=x.dtype, device=x.device)
    wide[:, 1:H + 1] = x
    return wide[:, 1:H + 1]


def _attend(step, q, k, v, scale=0.09, idx=None, want=None, ws=None, stride=False):
    dsa, cfg = _dsa(), _cfg(step)
    o = torch.full((step.T, step.H, 128), 5.0, dtype=step.dtype, device=DEV)
    lse = torch.full((step.T, step.H), 5.0, device=DEV)
    o0, l0 = o.clone(), lse.clone()
    qq = _strided(q) if stride else q
    n = (dsa.dsa_kv_attention_workspace(cfg, q, step.tables) if idx is None
         else dsa.dsa_kv_block_attention_workspace(cfg, q, idx, step.tables))
    ws = torch.full((n,), 255, dtype=torch.uint8, device=DEV) if ws is None else ws
    if idx is None:
        dsa.dsa_kv_attention(cfg, k, v, qq, step.first, step.lens, step.tables, scale, ws, o, lse)
    else:
        dsa.dsa_kv_block_attention(cfg, k, v, qq, idx, step.first, step.lens, step.tables, scale, ws, o, lse)
    torch.cuda.synchronize()
    assert dsa.dsa_kv_status() == dsa.DSA_OK
    if want is None:
        want = ref.attention(step, q, k, v, scale, idx)
    big = v.float().abs()
    ref.check_attention(step, o, lse, want, step.dtype, float(big[torch.isfinite(big)].max()), o0, l0)
    return o, lse


SHAPES = [
    ([1], [1], 1, 1, 16, BF16),
    ([300], [1], 8, 1, 64, BF16),
    ([5000], [1], 8, 1, 64, F16),
    ([20000, 3, 128, 129, 127], [1] * 5, 32, 8, 64, BF16),
    ([700] * 40, [2] * 40, 16, 2, 32, BF16),
    ([900, 0, 333, 64], [3, 0, 3, 1], 24, 2, 16, F16),
    ([256], [256], 4, 4, 64, BF16),          # a head each
    ([1000], [1000], 8, 1, 128, F16),
    ([1500], [700], 40, 8, 64, BF16),        # 5 heads a group
    ([2000, 40, 513], [513, 3, 1], 12, 1, 32, BF16),
    ([400, 350], [130, 350], 128, 1, 16, F16),   # one token a tile
    ([800], [200], 100, 1, 64, BF16),
    ([640] * 3, [129, 17, 1], 130, 2, 64, BF16),
    ([16384], [5], 64, 1, 128, BF16),
    ([2500], [2048], 32, 8, 64, F16),
]


@pytest.mark.parametrize("lens,new,H,Hk,page,dtype", SHAPES)
def test_attention(lens, new, H, Hk, page, dtype):
    step = ref.Step(lens, new, H=H, Hk=Hk, page=page, dtype=dtype, seed=H + page, pad=2)
    _attend(step, *step.rows(), stride=H % 3 == 0)


def _lists(step, n_out, share=0.7):
    """Ascending page lists: each token's own page most times, others at random, runs of neighbours sharing theirs."""
    idx = torch.full((step.T, step.Hk, n_out), -1, dtype=torch.int32)
    for r, (length, fresh) in enumerate(zip(step.lens_list, step.new_list)):
        for g in range(step.Hk):
            base = torch.rand(max(1, -(-length // step.page)), generator=step.gen)
            for i in range(fresh):
                own = (length - fresh + i) // step.page
                x = torch.where(torch.rand(own + 1, generator=step.gen) < share, base[:own + 1],
                                torch.rand(own + 1, generator=step.gen))
                if i % 7:
                    x[own] = 2.0
                m = min(own + 1, n_out if i % 5 else n_out // 2)
                idx[step.first_list[r] + i, g, :m] = x.topk(m).indices.sort().values.int()
    return idx.to(step.device)


@pytest.mark.parametrize("select", [1, 5, 16])
@pytest.mark.parametrize("lens,new,H,Hk,page,dtype", SHAPES)
def test_block_attention(lens, new, H, Hk, page, dtype, select):
    step = ref.Step(lens, new, H=H, Hk=Hk, page=page, dtype=dtype, seed=H + page + select, pad=2)
    _attend(step, *step.rows(), idx=_lists(step, select), stride=H % 3 == 1)


@pytest.mark.parametrize("scale", [-0.2, 0.0, 1e-40, 30.0])
@pytest.mark.parametrize("sparse", [False, True])
def test_scales(scale, sparse):
    step = ref.Step([700, 90], [150, 1], H=16, Hk=2, page=32, dtype=BF16, seed=11)
    q, k, v = step.rows()
    _attend(step, q, k, v, scale=scale, idx=_lists(step, 6) if sparse else None)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("sparse", [False, True])
def test_scores_that_rise(dtype, sparse):
    # every page outweighs those before it, by steps small and large
    step = ref.Step([3000, 2900], [1, 300], H=8, Hk=1, page=64, dtype=dtype, seed=12)
    q, k, v = step.rows()
    q.fill_(1.0)
    for r, n in enumerate(step.lens_list):
        for j in range(-(-n // 64)):
            k[step.tables[r, j].long()] = (j * (0.02 if r else 0.4)) / 2
    _attend(step, q, k, v, scale=1.0, idx=_lists(step, 20) if sparse else None)


@pytest.mark.parametrize("sparse", [False, True])
@pytest.mark.parametrize("H,Hk,new", [(8, 1, 1), (8, 2, 300), (1, 1, 200), (32, 1, 7)])
def test_what_is_not_attended_to_has_no_effect(H, Hk, new, sparse):
    """NaN and infinities in stale rows, in pages of no list and in later positions."""
    step = ref.Step([777, 450], [new, 1], H=H, Hk=Hk, page=32, dtype=BF16, seed=13)
    q, k, v = step.rows()
    idx = _lists(step, 4) if sparse else None
    ids = step.tables.cpu()
    for r, n in enumerate(step.lens_list):
        last = ids[r, (n - 1) // 32]
        for x, bad in ((k, math.nan), (v, math.inf)):
            x[last, n - (n - 1) // 32 * 32:] = bad
    used = ids[ids >= 0]
    spare = [j for j in range(step.pages) if j not in used.tolist()]
    k[spare], v[spare] = math.nan, math.nan
    want = ref.attention(step, q, k, v, 0.1, idx)
    assert torch.isfinite(want["o"][:step.first_list[-1]]).all()
    _attend(step, q, k, v, 0.1, idx, want)
    # a later position's NaN reaches those at and after it only
    if new > 1:
        at = 777 - new // 2
        page = ids[0, at // 32]
        v[page, at % 32, 0, 5] = math.nan
        v[page, at % 32, 0, 77] = -math.inf
        want = ref.attention(step, q, k, v, 0.1, idx)
        assert sparse or torch.isnan(want["o"][:, 0, 5]).any() and torch.isfinite(want["o"][0, 0]).all()
        _attend(step, q, k, v, 0.1, idx, want)
        v[page, at % 32, 0] = 1.0
        k[page, at % 32, 0, 3] = math.nan
        _attend(step, q, k, v, 0.1, idx)


def test_pages_without_an_id():
    step = ref.Step([900, 500], [40, 1], H=8, Hk=1, page=64, dtype=F16, seed=14)
    q, k, v = step.rows()
    step.tables[0, 2] = -1
    step.tables[0, 7] = step.pages
    step.tables[1, :] = 2 ** 31 - 1
    _attend(step, q, k, v)
    _attend(step, q, k, v, idx=_lists(step, 6))


@pytest.mark.parametrize("sparse", [False, True])
def test_lengths_past_the_table_and_below_the_step(sparse):
    step = ref.Step([900, 500, 64], [40, 10, 3], H=8, Hk=1, page=64, dtype=F16, seed=15, width=9)
    q, k, v = step.rows()
    idx = _lists(step, 6) if sparse else None
    step.lens[2], step.lens_list[2] = 2, 2
    _attend(step, q, k, v, idx=idx)
    step.lens[1], step.lens_list[1] = 2 ** 31 - 1, 2 ** 31 - 1
    step.lens[2], step.lens_list[2] = -5, -5
    _attend(step, q, k, v, idx=idx)


def test_lists_beyond_a_token():
    """Pages after a token's own, past the table and of no entry."""
    step = ref.Step([900, 500], [40, 1], H=8, Hk=1, page=64, dtype=BF16, seed=16)
    q, k, v = step.rows()
    idx = _lists(step, 6)
    idx[0, 0] = torch.tensor([3, 13, 14, 15, 100, 2 ** 31 - 1], **I32)
    idx[1, 0] = torch.tensor([14, 15, 16, 17, -1, -1], **I32)
    idx[2, 0] = -1
    idx[40, 0] = -1
    o, lse = _attend(step, q, k, v, idx=idx)
    assert (o[1] == 0).all() and (lse[40] == -math.inf).all()


def test_empty_pool_and_tables():
    dsa = _dsa()
    cfg = dsa.kv_cfg(pages=0, page_size=64, kv_heads=2)
    for P in (0, 3):
        q = torch.randn(5, 8, 128, device=DEV).to(BF16)
        none = torch.empty(0, 64, 2, 128, dtype=BF16, device=DEV)
        first, lens = torch.tensor([0, 2, 5], **I32), torch.tensor([2, 90], **I32)
        tables = torch.zeros(2, P, **I32)
        o, lse = torch.full_like(q, 3.0), torch.zeros(5, 8, device=DEV)
        ws = torch.empty(dsa.dsa_kv_attention_workspace(cfg, q, tables), dtype=torch.uint8, device=DEV)
        dsa.dsa_kv_attention(cfg, none, none, q, first, lens, tables, 0.1, ws, o, lse)
        assert (o == 0).all() and (lse == -math.inf).all()
        idx = torch.zeros(5, 2, 3, **I32)
        o, lse = torch.full_like(q, 3.0), torch.zeros(5, 8, device=DEV)
        ws = torch.empty(dsa.dsa_kv_block_attention_workspace(cfg, q, idx, tables), dtype=torch.uint8, device=DEV)
        dsa.dsa_kv_block_attention(cfg, none, none, q, idx, first, lens, tables, 0.1, ws, o, lse)
        assert (o == 0).all() and (lse == -math.inf).all()


def test_past_32_bits():
    """Pages whose rows lie beyond 2^32 elements."""
    step = ref.Step([1000, 300], [150, 1], H=32, Hk=8, page=64, dtype=BF16, seed=17, lo=66000)
    small = ref.Step([1000, 300], [150, 1], H=32, Hk=8, page=64, dtype=BF16, seed=17)
    q, ks, vs = small.rows()
    k, v = (torch.zeros(step.pages, 64, 8, 128, dtype=BF16, device=DEV) for _ in range(2))
    assert k.numel() > 2 ** 32
    k[66000:], v[66000:] = ks, vs
    assert torch.equal(step.tables.clamp(min=65999) - 66000, small.tables)
    for idx in (None, _lists(small, 5)):
        want = ref.attention(small, q, ks, vs, 0.1, idx)
        _attend(step, q, k, v, 0.1, idx, want)


# ---------------------------------------------------------------------------
# selection

def _select(step, means, q, n, lead, trail):
    dsa, cfg = _dsa(), _cfg(step)
    idx = torch.full((step.T, step.Hk, n), -9, **I32)
    ws = torch.full((dsa.dsa_kv_select_workspace(cfg, q, step.tables),), 255, dtype=torch.uint8, device=DEV)
    dsa.dsa_kv_select(cfg, means, q, step.first, step.lens, step.tables, lead, trail, ws, idx)
    want = ref.select(step, means, q, n, lead, trail)
    live = step.first_list[-1]
    assert (idx[live:] == -9).all()
    bad = (idx[:live].cpu() != want[:live]).any(-1).nonzero()
    assert not len(bad), f"{len(bad)} rows, first {bad[0].tolist()}: {idx[tuple(bad[0])].tolist()} {want[tuple(bad[0])].tolist()}"
    return idx


@pytest.mark.parametrize("lens,new,H,Hk,page,dtype,n,lead,trail", [
    ([1], [1], 1, 1, 16, BF16, 1, 0, 1),
    ([3000], [1], 8, 1, 16, BF16, 8, 1, 2),
    ([40000, 100, 9000, 17], [1, 1, 1, 1], 32, 8, 16, BF16, 16, 1, 1),
    ([5000] * 30, [3] * 30, 10, 2, 32, F16, 7, 2, 2),
    ([9000], [300], 12, 4, 16, F16, 20, 0, 1),
    ([4000, 50, 6000], [129, 0, 64], 128, 1, 16, BF16, 33, 3, 30),
    ([3000, 2000, 2000], [70, 1, 200], 24, 8, 32, BF16, 256, 1, 1),
    ([6000], [65], 8, 8, 16, F16, 256, 0, 1),
    ([2000], [40], 4, 2, 16, BF16, 3, 1, 2),     # only the pinned ones
    ([70000], [2], 5, 1, 16, BF16, 12, 1, 1)])
def test_select(lens, new, H, Hk, page, dtype, n, lead, trail):
    step = ref.Step(lens, new, H=H, Hk=Hk, page=page, dtype=dtype, seed=H + n, pad=2)
    means = step.normal(step.pages, Hk, 128)
    _select(step, means, step.normal(step.T, H, 128), n, lead, trail)


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_select_ties_and_neighbours_in_rank(dtype):
    step = ref.Step([30000, 2000], [40, 30], H=8, Hk=2, page=16, dtype=dtype, seed=21)
    q = step.normal(step.T, 8, 128)
    # few different means: hundreds of equal scores
    kinds = step.normal(5, 2, 128)
    means = kinds[torch.arange(step.pages, device=DEV) % 5].contiguous()
    _select(step, means, q, 16, 1, 1)
    _select(step, torch.zeros_like(means), q, 16, 1, 1)
    # a row each, but for one element's last bit
    means = kinds[:1].repeat(step.pages, 1, 1).contiguous()
    bits = means.view(torch.int16)
    bits[torch.arange(step.pages), 0, torch.randint(128, (step.pages,), generator=step.gen)] += 1
    bits[torch.arange(step.pages), 1, torch.randint(128, (step.pages,), generator=step.gen)] -= 1
    _select(step, means, q, 16, 1, 1)
    _select(step, means, q, 200, 1, 1)


@pytest.mark.parametrize("dtype,q_size,m_size", [(BF16, 1e30, 1e-30), (BF16, 1e-30, 1e8), (F16, 6e4, 6e4), (F16, 1e-6, 1e-6),
                                                 (BF16, 1e-36, 1e-20), (F16, 6e4, 1e-7)])
def test_select_magnitudes(dtype, q_size, m_size):
    step = ref.Step([9000, 700], [20, 3], H=16, Hk=2, page=16, dtype=dtype, seed=22)
    top = 6e4 if dtype == F16 else 3e38
    q = (step.normal(step.T, 16, 128, dtype=torch.float64) * q_size).clamp(-top, top).to(dtype)
    means = (step.normal(step.pages, 2, 128, dtype=torch.float64) * m_size).clamp(-top, top).to(dtype)
    _select(step, means, q, 12, 1, 2)


def test_select_nan_and_infinities():
    step = ref.Step([9000, 700, 20000], [20, 3, 1], H=16, Hk=2, page=16, dtype=BF16, seed=23)
    q, means = step.normal(step.T, 16, 128), step.normal(step.pages, 2, 128)
    ids = step.tables[0].long()
    means[ids[5], 0, 7] = math.nan
    means[ids[9], 0, 1] = math.inf
    means[ids[11], 1, 1] = -math.inf
    means[ids[12], 1, 1], means[ids[12], 1, 2] = math.inf, -math.inf
    _select(step, means, q, 12, 1, 2)
    q[3] = math.nan
    q[4, 0, 0] = math.inf
    _select(step, means, q, 12, 1, 2)
    means[:] = math.nan
    _select(step, means, q, 12, 1, 2)


def test_select_pages_without_an_id():
    step = ref.Step([900, 500], [40, 1], H=8, Hk=1, page=16, dtype=F16, seed=24)
    q, means = step.normal(step.T, 8, 128), step.normal(step.pages, 1, 128)
    step.tables[0, 2:30] = -1
    step.tables[0, 33] = step.pages
    step.tables[1, :] = 2 ** 31 - 1
    _select(step, means, q, 24, 1, 1)
    _select(step, means, q, 50, 0, 1)


def test_select_in_parts_of_a_step():
    # a row of scores so wide that a step's tokens are taken 64 at a time
    step = ref.Step([1500, 2000], [130, 77], H=8, Hk=8, page=16, dtype=BF16, seed=25, width=40000)
    means = step.normal(step.pages, 8, 128)
    _select(step, means, step.normal(step.T, 8, 128), 9, 1, 1)


def test_select_past_the_table_and_below_the_step():
    step = ref.Step([900, 500, 64], [40, 10, 3], H=8, Hk=1, page=16, dtype=F16, seed=26, width=30)
    q, means = step.normal(step.T, 8, 128), step.normal(step.pages, 1, 128)
    step.lens[2], step.lens_list[2] = 2, 2
    step.lens[1], step.lens_list[1] = 2 ** 31 - 1, 2 ** 31 - 1
    _select(step, means, q, 8, 1, 1)


# ---------------------------------------------------------------------------
# together

@pytest.mark.parametrize("page,dtype,neighbours", [(16, BF16, False), (64, F16, True)])
def test_steps_of_a_cache(page, dtype, neighbours):
    """Prompts, decode steps, drafts taken back: append, attend, select and attend to the selection, against f64 on
    the rows themselves."""
    dsa = _dsa()
    H, Hk, R = 16, 2, 3
    inv = 1e4 ** (-torch.arange(0, 128, 2, dtype=torch.float64) / 128)
    c = dsa.PagedKV(requests=R, pages=3 * 40, pages_per_request=40, page_size=page, kv_heads=Hk, dtype=dtype,
                    inv_freq=inv, neighbours=neighbours)
    g = torch.Generator().manual_seed(3)
    rows = [torch.zeros(0, 2, Hk, 128, dtype=dtype) for _ in range(R)]  # what each request holds
    lens = [0] * R
    for keep, new in (([0, 0, 0], [37, 5, 150]), ([37, 5, 150], [1, 1, 1]), ([38, 6, 151], [3, 100, 3]),
                      ([38, 6, 151], [2, 0, 1]), ([40, 6, 152], [60, 90, 1])):
        lens = [a + b for a, b in zip(keep, new)]
        T = sum(new)
        c.step(torch.tensor(lens, **I32), torch.tensor(new, **I32), T + 2)
        c.ok()
        qkv = torch.randn(T + 2, H + 2 * Hk, 128, generator=g).to(dtype)
        d = qkv.to(DEV)
        q = c.append(d[:, :H], d[:, H:H + Hk], d[:, H + Hk:])
        at = 0
        for r in range(R):
            rows[r] = torch.cat([rows[r][:keep[r]], qkv[at:at + new[r], H:].view(new[r], 2, Hk, 128)])
            at += new[r]
        # the cache as the formulas have it, in pages of its own
        step = ref.Step(lens, new, H=H, Hk=Hk, page=page, dtype=dtype, pad=2, width=40)
        step.tables, step.pages = c.tables, c.cfg.pages
        k64 = torch.zeros(step.pages * page, Hk, 128, dtype=torch.float64, device=DEV)
        v64 = torch.zeros_like(k64)
        for r in range(R):
            p = torch.arange(lens[r], device=DEV)
            slot = c.tables[r].long().repeat_interleave(page)[:lens[r]] * page + p % page
            k64[slot] = ref.rotate(rows[r][:, 0].to(DEV), p, inv.to(DEV), neighbours)
            v64[slot] = rows[r][:, 1].to(DEV).double()
        assert torch.equal(c.v.view(-1, Hk, 128).double()[v64.abs().sum((1, 2)) > 0], v64[v64.abs().sum((1, 2)) > 0])
        stored = k64.abs().sum((1, 2)) > 0
        near = (c.k.view(-1, Hk, 128).double() - k64).abs()
        assert (near[stored] <= ref.HALF[dtype] * k64.abs()[stored] + 2.0 ** -18).all()
        o, lse = c.attend(q, 0.09)
        want = ref.attention(step, q, c.k, c.v, 0.09)
        ref.check_attention(step, o, lse, want, dtype, 6.0)
        assert (o[T:] == 0).all() and (lse[T:] == -math.inf).all()
        # full pages' means are those of the rows
        for r in range(R):
            for j in range(lens[r] // page):
                m = c.k[c.tables[r, j].long()].double().mean(0)
                assert ((c.means[c.tables[r, j].long()].double() - m).abs() <= ref.HALF[dtype] * m.abs() + 2.0 ** -15).all()
        idx = c.select(q, 4)
        assert torch.equal(idx[:T].cpu(), ref.select(step, c.means, q, 4, 1, 1)[:T])
        assert (idx[T:] == -1).all()
        o, lse = c.attend_pages(q, idx, 0.09)
        ref.check_attention(step, o, lse, ref.attention(step, q, c.k, c.v, 0.09, idx), dtype, 6.0)


# ---------------------------------------------------------------------------
# streams, graphs, workspaces

def _state(step, n=5):
    """Everything a step's four calls take, with outputs."""
    dsa, cfg = _dsa(), _cfg(step)
    s = dict(cfg=cfg, q=step.normal(step.T, step.H, 128), kn=step.normal(step.T, step.Hk, 128),
             vn=step.normal(step.T, step.Hk, 128), means=step.normal(step.pages, step.Hk, 128))
    s["k"], s["v"] = (step.normal(step.pages, step.page, step.Hk, 128) for _ in range(2))
    s["ends"], s["slots"] = torch.zeros(step.T, **I32), torch.full((step.T,), -1, **I32)
    for r, p, t in step.tokens():
        s["ends"][t] = p + 1
        s["slots"][t] = int(step.tables[r, p // step.page]) * step.page + p % step.page
    s["turns"] = dsa.rotary_turns(1e4 ** (-torch.arange(0, 128, 2, dtype=torch.float64) / 128), DEV)
    s["idx"] = torch.full((step.T, step.Hk, n), -1, **I32)
    sizes = [dsa.dsa_kv_attention_workspace(cfg, s["q"], step.tables),
             dsa.dsa_kv_select_workspace(cfg, s["q"], step.tables),
             dsa.dsa_kv_block_attention_workspace(cfg, s["q"], s["idx"], step.tables)]
    s["ws"] = torch.full((max(sizes),), 255, dtype=torch.uint8, device=DEV)
    for x in ("qr", "o", "ob"):
        s[x] = torch.zeros(step.T, step.H, 128, dtype=step.dtype, device=DEV)
    for x in ("lse", "lseb"):
        s[x] = torch.zeros(step.T, step.H, device=DEV)
    return s


def _all(step, s, stream=None):
    """The four calls one after another, one workspace for all."""
    dsa, c = _dsa(), s["cfg"]
    dsa.dsa_kv_append(c, s["q"], s["kn"], s["vn"], s["ends"], s["slots"], s["turns"], False, 1.0, s["qr"], s["k"], s["v"],
                      s["means"], stream=stream)
    dsa.dsa_kv_attention(c, s["k"], s["v"], s["qr"], step.first, step.lens, step.tables, 0.1, s["ws"], s["o"], s["lse"],
                         stream=stream)
    dsa.dsa_kv_select(c, s["means"], s["qr"], step.first, step.lens, step.tables, 1, 1, s["ws"], s["idx"], stream=stream)
    dsa.dsa_kv_block_attention(c, s["k"], s["v"], s["qr"], s["idx"], step.first, step.lens, step.tables, 0.1, s["ws"],
                               s["ob"], s["lseb"], stream=stream)


OUT = ("qr", "k", "v", "means", "o", "lse", "idx", "ob", "lseb")


def _copy(s):
    torch.cuda.synchronize()
    return {x: s[x].clone() for x in OUT}


def _same(a, b):
    for x in OUT:
        assert torch.equal(a[x].view(torch.int16 if a[x].element_size() == 2 else torch.int32),
                           b[x].view(torch.int16 if b[x].element_size() == 2 else torch.int32)), x


MIXED = dict(lens=[900, 30, 3000, 64], new=[1, 2, 400, 64])


def test_results_repeat_without_a_pause():
    step = ref.Step(**MIXED, H=16, Hk=2, page=32, dtype=BF16, seed=31, pad=1)
    s = _state(step)
    _all(step, s)
    want = _copy(s)
    for x in OUT:
        if x not in ("k", "v", "means"):
            s[x][:step.first_list[-1]] = 0
    for _ in range(20):
        _all(step, s)
    s2 = _copy(s)
    _same(s2, want)
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    _all(step, s, stream=other)
    _same(_copy(s), want)


def test_graphs_share_a_workspace_and_follow_new_lengths():
    step = ref.Step(**MIXED, H=16, Hk=2, page=32, dtype=BF16, seed=32, pad=1)
    s = _state(step)
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            _all(step, s)
        graphs.append(g)
    for lens, new in ((MIXED["lens"], MIXED["new"]), ([700, 1000, 64, 0], [300, 100, 1, 0]), ([1, 1, 1, 467], [1, 1, 1, 460])):
        st = ref.Step(lens, new, H=16, Hk=2, page=32, dtype=BF16, seed=33, width=step.P, pad=step.T - sum(new),
                      spare=step.pages - sum(-(-n // 32) for n in lens))
        step.tables.copy_(st.tables)
        step.first.copy_(st.first)
        step.lens.copy_(st.lens)
        s["ends"].zero_()
        s["slots"].fill_(-1)
        for r, p, t in st.tokens():
            s["ends"][t] = p + 1
            s["slots"][t] = int(st.tables[r, p // 32]) * 32 + p % 32
        _all(st, s)
        want = _copy(s)
        for g in graphs:
            for x in ("qr", "o", "lse", "ob", "lseb"):
                s[x][:sum(new)] = 0
            s["ws"].random_(0, 255)
            g.replay()
            _same(_copy(s), want)


def test_two_streams_at_once():
    steps = [ref.Step(**MIXED, H=16, Hk=2, page=32, dtype=BF16, seed=34 + i, pad=1) for i in range(2)]
    states = [_state(x) for x in steps]
    wants = []
    for x, s in zip(steps, states):
        _all(x, s)
        wants.append(_copy(s))
    streams = [torch.cuda.Stream() for _ in steps]
    torch.cuda.synchronize()
    for _ in range(10):
        for x, s, st in zip(steps, states, streams):
            _all(x, s, stream=st)
    torch.cuda.synchronize()
    for s, want in zip(states, wants):
        _same(_copy(s), want)
