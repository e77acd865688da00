"""The paged 4-bit cache where its forms, types and plans could differ from their
definition, against the plain forms of tests/cache_ref.py."""
import os
import subprocess
import sys
import textwrap

import numpy as np
import pytest

from tests import cache_ref as ref
from tests.test_gpu_cache import DEV, HALF, _Case, _mods, _run_plan, _same_plan, _type

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("form,T,H,KV,Kc,ctx", [
    ("decode", 6, 8, 1, 60, 200), ("decode", 5, 16, 2, 300, 700), ("decode", 2, 8, 1, 2100, 2500),
    # tiles of a token's heads: whole, and split over CTAs
    ("decode", 70, 128, 1, 60, 200), ("decode", 100, 64, 1, 300, 900), ("decode", 10, 128, 1, 1100, 1500),
    # tiles of neighbours: whole, and split
    ("prompt", 40, 8, 1, 60, 400), ("prompt", 20, 16, 2, 1100, 3000)])
def test_nan_value_scales_reach_their_dims(form, T, H, KV, Kc, ctx):
    """A NaN among a record's value scales makes that scale's 16 dims of the rows
    that attend to it NaN: no other dim, no other row and no lse."""
    c = _Case(T, H, KV, Kc, page=16, ctx=ctx, R=1, seed=T + H)
    c.idx[1, 5:] = -1
    clean = c.cache.copy()
    p, q, r = int(c.idx[0][Kc // 2]), int(c.idx[T - 1 if T > 2 else 0][Kc - 1]), int(c.idx[T // 2][0])
    c.cache[c.tables[0, p // 16], p % 16, 0, 139] = 0x7F
    for g in (0, 4, 7):
        c.cache[c.tables[0, q // 16], q % 16, KV - 1, 136 + g] = 0xFF
    for step in range(2):
        if step == 1:  # beside a NaN key, whose rows are NaN as a whole
            c.cache[c.tables[0, r // 16], r % 16, 0, 130] = 0x7F
        c.device().launch(form)
        c.torch.cuda.synchronize()
        o, lse = c.o[:T].double().cpu().numpy(), c.lse[:T].double().cpu().numpy()
        args = (c.page, c.q.double().numpy(), c.idx, c.req, c.tables, c.scale)
        with np.errstate(invalid="ignore"):
            nan_o, nan_l = (np.isnan(x) for x in ref.attention(c.cache, *args)[:2])
        assert nan_o.any() and nan_l.any() == (step == 1) and (step == 1 or not nan_o.all())
        assert np.array_equal(np.isnan(o), nan_o) and np.array_equal(np.isnan(lse), nan_l)
        wo, wl, vmax, amax = ref.attention(clean, *args)
        delta = 2.0 ** -16 * amax
        assert (np.abs(lse - wl) <= delta + 2.0 ** -22 * (8 + np.abs(wl)))[~nan_l].all()
        bound = HALF["bf16"] * np.abs(wo) + (vmax * (2 * delta + 2.0 ** -11 + Kc * 2.0 ** -25 + 2.0 ** -19))[..., None]
        assert (np.abs(o - wo) <= bound)[~nan_o].all()


@pytest.mark.parametrize("H,KV,P", [(8, 1, 4), (32, 2, 4), (8, 1, 9000), (16, 1, 0)])
def test_prompt_lists_of_no_entry(H, KV, P):
    torch, dsa = _mods()
    cfg = dsa.cache_cfg(pages=4, page_size=16, kv_heads=KV)
    cache = torch.full((dsa.dsa_cache_bytes(cfg),), 0xFF, dtype=torch.uint8, device=DEV)
    q = torch.ones(21, H, 128, dtype=torch.bfloat16, device=DEV)
    idx = torch.empty((21, 0), dtype=torch.int32, device=DEV)
    o, lse = torch.full_like(q, 7.0), torch.full((21, H), 7.0, device=DEV)
    ws = torch.empty(dsa.dsa_cache_attention_prompt_workspace(cfg, q, idx), dtype=torch.uint8, device=DEV)
    dsa.dsa_cache_attention_prompt(cfg, cache, q, idx, torch.zeros(P, dtype=torch.int32, device=DEV), 0.1, ws, o, lse)
    assert (o == 0).all() and torch.isneginf(lse).all()
    assert dsa.dsa_cache_attention_status() == dsa.DSA_OK


def test_union_of_lists_of_no_entry():
    """The bf16 attention's lists of no entry, which share the union launch."""
    torch, dsa = _mods()
    q = torch.ones(21, 8, 128, dtype=torch.bfloat16, device=DEV)
    k = torch.ones(70, 128, dtype=torch.bfloat16, device=DEV)
    idx = torch.empty((21, 0), dtype=torch.int32, device=DEV)
    cfg = dsa.attention_cfg(q, k, idx)
    ws = torch.empty(dsa.dsa_sparse_attention_workspace(cfg), dtype=torch.uint8, device=DEV)
    o, lse = torch.full((21, 8, 128), 7.0, device=DEV), torch.full((21, 8), 7.0, device=DEV)
    dsa.dsa_sparse_attention(cfg, q, k, k, idx, 0.1, ws, o, lse)
    assert (o == 0).all() and torch.isneginf(lse).all()
    assert dsa.dsa_sparse_attention_status() == dsa.DSA_OK


def test_status_waits_for_every_stream():
    c = _Case(20, 128, 1, 130, ctx=200, seed=3).device()
    torch, dsa = c.torch, c.dsa
    s = torch.cuda.Stream()
    c.launch()
    assert dsa.dsa_cache_attention_status() == dsa.DSA_OK
    with torch.cuda.stream(s):
        torch.cuda._sleep(200000000)  # 0.1 s
        c.launch()
    assert dsa.dsa_cache_attention_status() == dsa.DSA_OK
    assert s.query(), "the status came before the launch it is asked about had ended"
    c.check()


@pytest.mark.parametrize("H,KV,T,dtype", [(512, 64, 4, "f16"), (1024, 64, 4, "bf16"), (2560, 20, 4, "f16")])
def test_long_lists_of_small_weights(H, KV, T, dtype):
    """2^20 entries, of which the first outweighs each of the others by 2^25.5 and
    all of them together by 45: what they bring is in o as it is in lse.  The
    bound is the other tests', its term for weights below f16's normal range
    against a largest weight of 2^7 at least, n 2^-32, and what so long a list
    adds: a thread sums n / 64 weights at most one after another (2^-24 of the sum
    each), a product n / 16 times 16 of them (2^-23 of what o has by then)."""
    torch, dsa = _mods()
    n, page = 1 << 20, 64
    k, v = np.zeros((64, 128)), np.full((64, 128), 6.0)
    k[0], v[0] = 6.0, 0.0  # exact in 4 bits
    cfg = dsa.cache_cfg(pages=1, page_size=page, kv_heads=KV)
    cache = torch.from_numpy(np.repeat(ref.pack(k, v)[:, None], KV, 1).reshape(-1)).to(DEV)
    q = torch.ones(T, H, 128, dtype=_type(torch, dtype), device=DEV)
    idx = (torch.arange(n, device=DEV) % 63 + 1).int()
    idx[0] = 0
    o, lse = torch.empty_like(q), torch.empty(T, H, device=DEV)
    score = 25.5 * np.log(2.0)
    dsa.dsa_cache_attention(cfg, cache, q, idx.repeat(T, 1), torch.zeros(T, dtype=torch.int32, device=DEV),
                            torch.zeros((1, 1), dtype=torch.int32, device=DEV), score / 768, o, lse)
    rest = (n - 1) * np.exp(-score)
    wo, wl = 6.0 * rest / (1 + rest), score + np.log1p(rest)
    delta = 2.0 ** -16 * score
    total = n / 64 * 2.0 ** -24
    assert np.abs(lse.double().cpu().numpy() - wl).max() <= delta + total + 2.0 ** -22 * (8 + wl)
    err = np.abs(o.double().cpu().numpy() - wo).max()
    assert err <= (HALF[dtype] + total + n / 16 * 2.0 ** -23) * wo + 6.0 * (
        2 * delta + 2.0 ** -11 + n * 2.0 ** -32 + 2.0 ** -19), err


@pytest.mark.parametrize("fresh", [32, 33, 300000])
def test_plans_whose_sums_pass_32_bits(fresh):
    """8,192 requests and 262,144 tokens: filled exactly, passed by 8,192, and with
    counts whose sum is past 2^31."""
    torch, dsa = _mods()
    R, T, page, P = 8192, 1 << 18, 4096, 80
    rng = np.random.default_rng(fresh)
    lens = np.minimum(fresh + rng.integers(0, 20000, R), P * page)
    held = np.minimum(rng.integers(0, 4, R), P)
    tables = np.where(np.arange(P)[None, :] < held[:, None], np.arange(R * P).reshape(R, P) % 70000, -1)
    free = rng.permutation(70000)
    args = (page, 70000, lens, np.full(R, fresh), tables, held, free, 60000, T)
    want = ref.plan(*args)
    assert want["status"][0] == (0 if fresh == 32 else 3)
    _same_plan(_run_plan(torch, dsa, *args), want)


@pytest.mark.parametrize("dtype,k_shift,v_shift", [("bf16", 3, -9), ("bf16", -32, 32), ("f16", 2, -3), ("f16", -5, 4)])
def test_shifts_of_16_bit_rows(dtype, k_shift, v_shift):
    torch, dsa = _mods()
    dt = _type(torch, dtype)
    shift = torch.tensor([2.0 ** k_shift, 2.0 ** v_shift], dtype=torch.float64).view(2, 1, 1, 1)
    g = torch.Generator().manual_seed(7)
    rows = (torch.randn(2, 40, 2, 128, generator=g).to(dt).double() * shift).to(dt)
    x = (rows.double() / shift).numpy()
    cfg = dsa.cache_cfg(pages=10, page_size=4, kv_heads=2, k_shift=k_shift, v_shift=v_shift)
    cache = torch.zeros(dsa.dsa_cache_bytes(cfg), dtype=torch.uint8, device=DEV)
    slots = torch.arange(40, dtype=torch.int32, device=DEV)
    dsa.dsa_cache_write(cfg, *rows.to(DEV).unbind(0), slots, cache)
    rec = ref.pack(x[0], x[1])
    assert np.array_equal(cache.cpu().numpy().reshape(rec.shape), rec)
    out = torch.empty(2, 40, 2, 128, dtype=dt, device=DEV)
    dsa.dsa_cache_read(cfg, cache, slots, *out.unbind(0))
    want = torch.from_numpy(np.stack(ref.expand(rec))) * shift
    assert torch.equal(out.cpu(), want.to(dt))


def test_first_calls_inside_a_capture():
    """A process whose first use of every kernel is in a capture: the graph gives
    what the calls give without one."""
    _mods()
    script = textwrap.dedent(f"""
        import sys
        sys.path.insert(0, {ROOT!r})
        import torch
        import sparse_attention_indexer_live_gb300 as dsa
        d = dict(dtype=torch.int32, device="cuda:0")
        gen = torch.Generator("cuda:0").manual_seed(1)
        R, T = 4, 9000  # a plan of several CTAs
        lens = torch.tensor([4000, 3000, 1500, 500], **d)
        rows = torch.randn(2, T, 1, 128, device="cuda:0", generator=gen).half()
        lists = torch.arange(2048, **d).repeat(32, 1).contiguous()
        qs = [torch.randn(n, h, 128, device="cuda:0", generator=gen).half() for n, h in ((1, 8), (16, 16), (20, 128), (32, 8))]
        def run():
            c = dsa.PagedCache(requests=R, pages=200, pages_per_request=100)
            c.step(lens, lens, T)
            c.store(rows[0], rows[1])
            out = [c.attend(q, lists[:len(q)], 0.1) for q in qs] + [c.attend(qs[3], lists, 0.1, request=0)]
            return [x for pair in out for x in pair] + list(c.fetch(c.slots)) + [c.status, c.data]
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = run()
        g.replay()
        torch.cuda.synchronize()
        want = run()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert want[-2].tolist() == [0, 0, T, 200 - 63 - 47 - 24 - 8], want[-2].tolist()
        print("same")
    """)
    res = subprocess.run([sys.executable, "-c", script], capture_output=True, text=True, timeout=300)
    assert res.returncode == 0 and res.stdout.split()[-1] == "same", res.stderr[-2000:]
