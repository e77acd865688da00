"""The 16-bit cache's attentions beside what a row does not attend to: requests
whose length is below the step's own tokens, pages without an id under queries
that are not finite, finite keys whose scores pass f32's range.  Against the
plain 64-bit forms (tests/kv_ref.py, which derives the tolerances)."""
import math

import pytest

torch = pytest.importorskip("torch")

from tests import kv_ref as ref  # noqa: E402
from tests.test_gpu_kv import BF16, F16, _attend, _dsa, _lists, _select  # noqa: E402

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]


def _shorten(step, r, n):
    """Request r's length, of which its pages in hand are more."""
    step.lens[r], step.lens_list[r] = n, n


@pytest.mark.parametrize("sparse", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("H,new", [(8, [3, 5, 40]), (8, [40, 70, 3]), (1, [200, 1, 150]), (128, [2, 3, 2])])
def test_rows_without_a_position(H, new, dtype, sparse):
    """A NaN or an infinity in the pages of a request whose tokens attend to nothing."""
    step = ref.Step([300, 300, 400], new, H=H, Hk=1, page=16, dtype=dtype, seed=H + new[0], pad=1)
    q, k, v = step.rows()
    idx = _lists(step, 5) if sparse else None
    if sparse:  # they list pages all the same, the first ones among them
        idx[:step.first_list[2], :, :3] = torch.arange(3, dtype=torch.int32, device=idx.device)
        idx[:step.first_list[2], :, 3:] = -1
    _shorten(step, 0, new[0] - 1)
    _shorten(step, 1, -7)
    for kk, vv in ((math.nan, 1.0), (math.inf, 1.0), (-math.inf, 1.0), (1.0, math.nan), (1.0, -math.inf)):
        for r in (0, 1):
            ids = step.tables[r, :3].long()
            k[ids, 1::2], v[ids, 1::2] = kk, vv
        o, lse = _attend(step, q, k, v, 0.1, idx)
        few = step.first_list[2]
        assert (o[:few] == 0).all() and (lse[:few] == -math.inf).all()


def _odd_queries(step, q):
    """Rows whose scores against zeros are NaN: a NaN, infinities of either sign."""
    q[0::4, 0, 3] = math.nan
    q[1::4, :, 0] = math.inf
    q[2::4, :, 1] = -math.inf
    return q


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("H,new", [(8, 5), (8, 70), (1, 300)])
def test_queries_that_are_not_finite_over_pages_without_an_id(H, new, dtype):
    """Pages without an id are not attended to: no score of theirs reaches a row."""
    step = ref.Step([500, 700], [new, new], H=H, Hk=1, page=64, dtype=dtype, seed=H + new, pad=1)
    q, k, v = step.rows()
    _odd_queries(step, q)
    k[..., :2] = 1.0  # an infinite query has scores of its own sign
    step.tables[0, :] = -1
    step.tables[1, 1:3] = -1
    step.tables[1, 7] = step.pages
    o, lse = _attend(step, q, k, v)
    assert (o[:new] == 0).all() and (lse[:new] == -math.inf).all()
    # (a NaN query over pages that are there has no other result)
    live = slice(step.first_list[1], step.first_list[2])
    t = torch.arange(2 * new, device=o.device)[live]
    assert torch.isnan(lse[live][t % 4 == 0, 0]).all() and (lse[live][t % 4 == 2] == -math.inf).all()
    idx = _lists(step, 6)
    o, lse = _attend(step, q, k, v, idx=idx)
    assert (o[:new] == 0).all() and (lse[:new] == -math.inf).all()


@pytest.mark.parametrize("sparse", [False, True])
@pytest.mark.parametrize("lens,new,H,page", [
    ([5, 77], [1, 3], 8, 16),              # a tile of rows each
    ([300, 1030], [200, 1030], 8, 64),     # two
    ([40000, 20], [1, 20], 8, 64),         # shared by many CTAs
    ([20000, 50], [100, 50], 32, 128)])
def test_finite_keys_whose_scores_are_not(lens, new, H, page, sparse):
    """bf16 keys so large that their scores pass f32's range, where no row attends to them: the last page's stale rows,
    pages of no list, and the chunk's later positions."""
    step = ref.Step(lens, new, H=H, Hk=1, page=page, dtype=BF16, seed=lens[0], pad=1)
    q, k, v = step.rows()
    idx = _lists(step, 4) if sparse else None
    ids = step.tables.cpu()
    sign = torch.where(torch.arange(128) % 3 == 0, -3e38, 3e38).to(BF16).to(k.device)
    for r, n in enumerate(lens):
        last = (n - 1) // page
        k[ids[r, last], n - last * page:] = sign if r else 3e38
    _attend(step, q, k, v, 0.1, idx)
    # a late position; the rows that attend to it have no score but 0
    at = lens[0] - 1 - new[0] // 3
    k[ids[0, at // page], at % page] = sign
    q[new[0] - 1 - new[0] // 3:new[0]] = 0
    _attend(step, q, k, v, 0.1, idx)
    _attend(step, q, k, v, -30.0, idx)


@pytest.mark.parametrize("P", [0, 3])
def test_a_pool_of_no_pages_and_odd_queries(P):
    """Nothing is attended to, whatever the first token's queries hold."""
    dsa, dev = _dsa(), "cuda:0"
    i32 = dict(dtype=torch.int32, device=dev)
    cfg = dsa.kv_cfg(pages=0, page_size=64, kv_heads=2)
    none = torch.empty(0, 64, 2, 128, dtype=BF16, device=dev)
    first, lens, tables = torch.tensor([0, 2, 70], **i32), torch.tensor([2, 150], **i32), torch.zeros(2, P, **i32)
    idx = torch.zeros(70, 2, 3, **i32)
    for bad in (math.nan, math.inf):
        q = torch.randn(70, 8, 128, device=dev).to(BF16)
        q[0] = bad
        q[40, 5, 7] = -bad
        for lists in (None, idx):
            o, lse = torch.full_like(q, 3.0), torch.zeros(70, 8, device=dev)
            if lists is None:
                ws = torch.empty(dsa.dsa_kv_attention_workspace(cfg, q, tables), dtype=torch.uint8, device=dev)
                dsa.dsa_kv_attention(cfg, none, none, q, first, lens, tables, 0.1, ws, o, lse)
            else:
                ws = torch.empty(dsa.dsa_kv_block_attention_workspace(cfg, q, idx, tables), dtype=torch.uint8, device=dev)
                dsa.dsa_kv_block_attention(cfg, none, none, q, idx, first, lens, tables, 0.1, ws, o, lse)
            assert (o == 0).all() and (lse == -math.inf).all()


def test_no_pages_for_rows_without_a_position():
    """The selection's side of it: none of a request's tokens has a page where its length is below them."""
    step = ref.Step([300, 300, 400], [40, 5, 40], H=8, Hk=2, page=16, dtype=BF16, seed=3, pad=1)
    q, means = step.normal(step.T, 8, 128), step.normal(step.pages, 2, 128)
    for n in (39, 1, 0, -1, -2 ** 31):
        _shorten(step, 0, n)
        idx = _select(step, means, q, 6, 1, 1)
        assert (idx[:40] == -1).all() and (idx[40:85] >= 0).any(-1).all()
