"""Waits of the 16-bit cache's kernels that run out, without a GPU fault: a test
build of the library shortens their bounded waits to 20 M cycles and makes the
barriers of the weights (attention) and of the mean keys (selection) expect one
arrival more than there are.  Every role of the kernels then winds down and frees
its tensor memory, the status call reports DSA_ERR_TIMEOUT once, and the context
stays usable."""
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
    tmp = tmp_path_factory.mktemp("starved_kv")
    objs = [str(tmp / (os.path.basename(s) + ".o")) for s in B.SOURCES]

    def compile_one(a):
        subprocess.run([B.nvcc_path(), *B.ARCH, "-O3", "-std=c++17", "-Xcompiler", "-fPIC", "-c",
                        "-DDSA_KV_TEST_WAIT_CYCLES=20000000ll", "-I", B.INCLUDE, "-o", a[1], a[0]], check=True)
    with ThreadPoolExecutor(16) as ex:
        list(ex.map(compile_one, zip(B.SOURCES, objs)))
    so = str(tmp / "libdsa_timeout_kv.so")
    subprocess.run([B.nvcc_path(), *B.ARCH, "-shared", "-o", so, *objs], check=True)
    return so


@pytest.mark.parametrize("form,T,ctx", [
    ("attend", 1, 300), ("attend", 1, 20000), ("attend", 300, 20000),     # a tile of rows: whole, cut; two
    ("pages", 1, 300), ("pages", 300, 20000), ("pages", 8000, 20000),     # whole, shared out, dealt and shared out
    ("select", 40, 20000)])
def test_waits_that_run_out(starved_lib, form, T, ctx):
    script = textwrap.dedent(f"""
        import sys, torch
        sys.path.insert(0, {ROOT!r})
        from sparse_attention_indexer_live_gb300 import binding
        binding.load({starved_lib!r})
        import sparse_attention_indexer_live_gb300 as dsa
        d, n, form = "cuda:0", ({ctx} + 63) // 64, {form!r}
        c = dsa.PagedKV(requests=1, pages=n, pages_per_request=n, kv_heads=2, inv_freq=[1.0] * 32)
        lens = torch.tensor([{ctx}], dtype=torch.int32, device=d)
        c.step(lens, lens, {ctx})
        x = torch.randn({ctx}, 8, 128, device=d).bfloat16()
        c.append(x, x[:, :2], x[:, 2:4])
        c.step(lens, torch.full_like(lens, {T}), {T})
        q = torch.randn({T}, 8, 128, device=d).bfloat16()
        idx = torch.arange(4, dtype=torch.int32, device=d).expand({T}, 2, 4).contiguous()
        call = dict(attend=lambda: c.attend(q, 0.1), pages=lambda: c.attend_pages(q, idx, 0.1),
                    select=lambda: c.select(q, 8))[form]
        got = [dsa.dsa_kv_status()]
        for _ in range(2):
            call()
            got += [dsa.dsa_kv_status(), dsa.dsa_kv_status()]
        # what has no such wait: an append, and the selection for few tokens
        c.append(x[:{T}], x[:{T}, :2], x[:{T}, 2:4])
        c.step(lens, torch.ones_like(lens), 1)
        y = c.select(q[:1], 4)
        print(*got, dsa.dsa_kv_status(), (y[0, :, 0] == 0).all().item())
    """)
    res = subprocess.run([sys.executable, "-c", script], capture_output=True, text=True, timeout=300)
    assert res.returncode == 0, res.stderr[-2000:]
    import sparse_attention_indexer_live_gb300 as dsa
    ok, late = str(dsa.DSA_OK), str(dsa.DSA_ERR_TIMEOUT)
    assert res.stdout.split() == [ok, late, ok, late, ok, ok, "True"]
