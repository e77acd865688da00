"""The paged 16-bit cache on the GPU where its work is split or laid out otherwise:
many requests, few heads a group, lists over more units than SMs, values that are
not finite beside long shares, a draft's tokens at the limits of the selection's
small form, and first calls inside a capture.  Against the plain 64-bit forms
(tests/kv_ref.py, which derives the tolerances)."""
import math
import os
import subprocess
import sys
import textwrap

import pytest

torch = pytest.importorskip("torch")

from tests import kv_ref as ref  # noqa: E402
from tests.test_gpu_kv import (BF16, F16, _all, _append, _attend, _copy, _dsa, _lists, _same, _select,  # noqa: E402
                               _state)

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("requests", [128, 129, 700])
@pytest.mark.parametrize("sparse", [False, True])
def test_many_requests(requests, sparse):
    """More than a warp sums up, with empty ones between, one of them long."""
    new = [(0, 1, 3, 1, 0, 2)[r % 6] for r in range(requests)]
    lens = [max(f, 37 * r % 190) for r, f in enumerate(new)]
    lens[requests // 2 + 1] = 9000
    step = ref.Step(lens, new, H=8, Hk=2, page=16, dtype=BF16, seed=requests, pad=3)
    q, k, v = step.rows()
    _attend(step, q, k, v, idx=_lists(step, 5) if sparse else None)
    if sparse:
        _select(step, step.normal(step.pages, 2, 128), q, 6, 1, 1)


@pytest.mark.parametrize("select", [3, 12])
@pytest.mark.parametrize("lens,new,H,Hk,page,dtype", [
    ([300], [300], 1, 1, 16, BF16),          # 32 tokens a tile
    ([300, 200], [200, 1], 2, 1, 16, F16),
    ([700], [260], 2, 2, 32, BF16),          # 64 and a head each
    ([400], [300], 9, 3, 16, F16),
    ([500], [128], 8, 8, 128, BF16),         # 128
    ([4000], [2600], 32, 4, 64, BF16),       # lists dealt out whole, the rest shared out
    ([30000], [3], 16, 1, 32, F16)])
def test_lists_of_every_layout(lens, new, H, Hk, page, dtype, select):
    step = ref.Step(lens, new, H=H, Hk=Hk, page=page, dtype=dtype, seed=H + page + select, pad=1)
    _attend(step, *step.rows(), idx=_lists(step, select, share=0.9 if select == 3 else 0.2))


@pytest.mark.parametrize("select", [1000, 4096])
def test_the_longest_lists(select):
    step = ref.Step([70000, 200], [3, 20], H=8, Hk=1, page=16, dtype=BF16, seed=select)
    _attend(step, *step.rows(), idx=_lists(step, select))


@pytest.mark.parametrize("sparse", [False, True])
@pytest.mark.parametrize("n,new", [(60000, 1), (20000, 40)])
def test_not_finite_beside_long_shares(n, new, sparse):
    """Stale rows, pages of no list and a late position, of a unit that many CTAs share."""
    step = ref.Step([n, 100], [new, 1], H=8, Hk=1, page=64, dtype=BF16, seed=n, spare=2)
    q, k, v = step.rows()
    idx = _lists(step, 40) if sparse else None
    ids = step.tables.cpu()
    last = ids[0, (n - 1) // 64]
    k[last, (n - 1) % 64 + 1:], v[last, (n - 1) % 64 + 1:] = math.inf, math.nan
    if sparse:
        listed = set(idx[:new].flatten().tolist())
        for j in range(0, n // 64, 3):
            if j not in listed:
                k[ids[0, j]], v[ids[0, j]] = math.nan, -math.inf
    _attend(step, q, k, v, 0.1, idx)
    at = n - 1 - new // 2  # those before it do not see it
    v[ids[0, at // 64], at % 64, 0, 100] = math.nan
    k[ids[0, at // 64], at % 64, 0, 1] = 3.0
    _attend(step, q, k, v, 0.1, idx)
    # a sum that is not finite: a key's infinity, of either sign by row
    v[ids[0, at // 64], at % 64, 0, 100] = 1.0
    k[ids[0, at // 64], at % 64, 0, 1] = -math.inf
    _attend(step, q, k, v, 0.1, idx)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("new", [2, 7, 8, 9])
def test_select_for_drafts(new, dtype):
    step = ref.Step([5000, 40, 3000], [new, 0, new], H=12, Hk=2, page=16, dtype=dtype, seed=new, pad=1)
    q, means = step.normal(step.T, 12, 128), step.normal(step.pages, 2, 128)
    _select(step, means, q, 14, 1, 2)
    # tokens and pages that are not finite have no part in others
    ids = step.tables.cpu()
    q[new - 1, 3, 17] = math.nan
    q[new, 0, 2] = math.inf
    means[ids[0, 11], 0, 5] = math.nan
    means[ids[2, 90], 1, 100] = -math.inf
    _select(step, means, q, 14, 1, 2)
    # one dim far above the others: their squares' bound is eight times what it is
    means[:, 0, 64] = 500.0
    _select(step, means, q, 14, 1, 2)


@pytest.mark.parametrize("lens,new,page,dtype", [([3000, 100], [2000, 70], 16, BF16), ([700] * 9, [65] * 9, 128, F16),
                                                 ([40] * 40, [13] * 40, 32, BF16)])
def test_append_of_long_steps(lens, new, page, dtype):
    step = ref.Step(lens, new, H=8, Hk=2, page=page, dtype=dtype, seed=page, pad=2)
    _append(step, 8, 128, page == 16)


@pytest.mark.parametrize("new", [1, 40])
def test_memory_on_16_byte_boundaries(new):
    """Everything a multiple of 16 bytes, and of no more, from an address of many."""
    dsa = _dsa()
    step = ref.Step([900, 2500], [new, 1], H=8, Hk=2, page=16, dtype=BF16, seed=41)

    def odd(x):
        y = torch.zeros(x.numel() + 16 // x.element_size(), dtype=x.dtype, device=x.device)[16 // x.element_size():]
        assert y.data_ptr() % 32 == 16
        return y.copy_(x.reshape(-1)).view(x.shape)
    s, t = _state(step), _state(step)
    for x in ("q", "kn", "vn", "k", "v", "means"):
        t[x] = odd(s[x])
    for x in ("qr", "o", "ob", "ws"):
        t[x] = odd(t[x])
    _all(step, s)
    _all(step, t)
    _same(_copy(s), _copy(t))
    assert dsa.dsa_kv_status() == dsa.DSA_OK


def test_first_calls_inside_a_capture():
    script = textwrap.dedent(f"""
        import sys, torch
        sys.path.insert(0, {ROOT!r})
        import sparse_attention_indexer_live_gb300 as dsa
        d, n = "cuda:0", 700
        c = dsa.PagedKV(requests=2, pages=80, pages_per_request=40, page_size=32, kv_heads=2, inv_freq=[0.5, 0.25] * 8)
        lens, fresh = (torch.tensor(x, dtype=torch.int32, device=d) for x in ([n, 3], [n, 3]))
        gen = torch.Generator(device=d).manual_seed(1)
        x = torch.randn(n + 3, 12, 128, device=d, generator=gen).bfloat16()

        def run():
            c.step(lens, fresh, n + 3)
            q = c.append(x[:, :8], x[:, 8:10], x[:, 10:])
            return c.attend(q, 0.1) + c.attend_pages(q, c.select(q, 5), 0.1)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = run()
        g.replay()
        torch.cuda.synchronize()
        got = [y.clone() for y in got]
        c.held.zero_()
        want = run()
        print(all(torch.equal(a, b) for a, b in zip(got, want)), dsa.dsa_kv_status(), torch.isfinite(want[1]).all().item())
    """)
    res = subprocess.run([sys.executable, "-c", script], capture_output=True, text=True, timeout=300)
    assert res.returncode == 0, res.stderr[-2000:]
    assert res.stdout.split() == ["True", "0", "True"]
