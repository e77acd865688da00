"""Waits of the cache's tile attention that run out, without a GPU fault: a test
build of the library shortens its bounded waits to 20 M cycles and makes the
barrier of the queries expect one arrival more than there are.  Every role of the
kernel then winds down and frees its tensor memory, the status call reports
DSA_ERR_TIMEOUT once, and the context stays usable."""
import os
import subprocess
import sys
import textwrap
from concurrent.futures import ThreadPoolExecutor

import pytest

torch = pytest.importorskip("torch")

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def starved_lib(tmp_path_factory):
    import importlib
    B = importlib.import_module("sparse_attention_indexer_live_gb300.build")
    tmp = tmp_path_factory.mktemp("starved")
    objs = [str(tmp / (os.path.basename(s) + ".o")) for s in B.SOURCES]

    def compile_one(a):
        subprocess.run([B.nvcc_path(), *B.ARCH, "-O3", "-std=c++17", "-Xcompiler", "-fPIC", "-c",
                        "-DDSA_CACHE_TEST_WAIT_CYCLES=20000000ll", "-I", B.INCLUDE, "-o", a[1], a[0]], check=True)
    with ThreadPoolExecutor(8) as ex:
        list(ex.map(compile_one, zip(B.SOURCES, objs)))
    so = str(tmp / "libdsa_timeout.so")
    subprocess.run([B.nvcc_path(), *B.ARCH, "-shared", "-o", so, *objs], check=True)
    return so


@pytest.mark.parametrize("form,T,H,Kc,ctx", [
    ("decode", 70, 128, 600, 900), ("decode", 10, 128, 1100, 1500),   # a token a tile: whole, split
    ("prompt", 2000, 8, 300, 900), ("prompt", 20, 8, 2100, 4000)])    # neighbours: whole, split
def test_waits_that_run_out(starved_lib, form, T, H, Kc, ctx):
    script = textwrap.dedent(f"""
        import sys, torch
        sys.path.insert(0, {ROOT!r})
        from sparse_attention_indexer_live_gb300 import binding
        binding.load({starved_lib!r})
        import sparse_attention_indexer_live_gb300 as dsa
        d = "cuda:0"
        c = dsa.PagedCache(requests=1, pages=({ctx} + 63) // 64, pages_per_request=({ctx} + 63) // 64)
        lens = torch.tensor([{ctx}], dtype=torch.int32, device=d)
        c.step(lens, lens, {ctx})
        c.store(*torch.randn(2, {ctx}, 1, 128, device=d).bfloat16().unbind(0))
        c.step(lens, torch.full_like(lens, min({T}, {ctx})), {T})
        c.token_req.zero_()
        q = torch.randn({T}, {H}, 128, device=d).bfloat16()
        idx = torch.arange({Kc}, dtype=torch.int32, device=d).repeat({T}, 1) % {ctx}
        if {form!r} == "prompt":
            idx = idx.sort(1).values.contiguous()
        got = [dsa.dsa_cache_attention_status()]
        for _ in range(2):
            c.attend(q, idx, 0.1, request=0 if {form!r} == "prompt" else None)
            got += [dsa.dsa_cache_attention_status(), dsa.dsa_cache_attention_status()]
        # the other form of the kernels has no such wait
        o, lse = c.attend(q[:1, :8].contiguous(), idx[:1].contiguous(), 0.1)
        print(*got, dsa.dsa_cache_attention_status(), torch.isfinite(lse).all().item())
    """)
    res = subprocess.run([sys.executable, "-c", script], capture_output=True, text=True, timeout=300)
    assert res.returncode == 0, res.stderr[-2000:]
    import sparse_attention_indexer_live_gb300 as dsa
    ok, late = str(dsa.DSA_OK), str(dsa.DSA_ERR_TIMEOUT)
    assert res.stdout.split() == [ok, late, ok, late, ok, ok, "True"]
