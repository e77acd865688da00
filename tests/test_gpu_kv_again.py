"""Rows of the 16-bit cache's attentions that are computed a second time take as
long as they are: no wait for them runs out.  A test build of the library shortens
the kernels' bounded waits to 2 M cycles (1 ms), which the rows of these calls pass
many times over."""
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
def hasty_lib(tmp_path_factory):
    import importlib
    B = importlib.import_module("sparse_attention_indexer_live_gb300.build")
    tmp = tmp_path_factory.mktemp("hasty_kv")
    objs = [str(tmp / (os.path.basename(s) + ".o")) for s in B.SOURCES]

    def compile_one(a):
        subprocess.run([B.nvcc_path(), *B.ARCH, "-O3", "-std=c++17", "-Xcompiler", "-fPIC", "-c", "-DDSA_KV_TEST_FED",
                        "-DDSA_KV_TEST_WAIT_CYCLES=2000000ll", "-I", B.INCLUDE, "-o", a[1], a[0]], check=True)
    with ThreadPoolExecutor(16) as ex:
        list(ex.map(compile_one, zip(B.SOURCES, objs)))
    so = str(tmp / "libdsa_hasty_kv.so")
    subprocess.run([B.nvcc_path(), *B.ARCH, "-shared", "-o", so, *objs], check=True)
    return so


@pytest.mark.parametrize("sparse", [False, True])
def test_long_rows_computed_again(hasty_lib, sparse):
    """The chunk's last tokens share tiles with stale rows that hold NaN, on units that others follow."""
    script = textwrap.dedent(f"""
        import sys, math, torch
        sys.path.insert(0, {ROOT!r})
        from sparse_attention_indexer_live_gb300 import binding
        binding.load({hasty_lib!r})
        import sparse_attention_indexer_live_gb300 as dsa
        from tests import kv_ref as ref
        from tests.test_gpu_kv import BF16, _attend
        n, T, sparse = 60010, 600, {sparse}
        step = ref.Step([n], [T], H=32, Hk=8, page=64, dtype=BF16, seed=5)
        q, k, v = step.rows()
        idx = None
        if sparse:
            last = (n - 1) // 64
            idx = (torch.arange(192, device=q.device) * 4 + last - 4 * 191).int().expand(T, 8, 192).contiguous()
        _attend(step, q, k, v, 0.1, idx)
        print(dsa.dsa_kv_status())
        page = step.tables[0, (n - 1) // 64].long()
        v[page, (n - 1) % 64 + 1:] = math.nan
        o, lse = _attend(step, q, k, v, 0.1, idx)
        print(dsa.dsa_kv_status(), torch.isfinite(o).all().item())
    """)
    res = subprocess.run([sys.executable, "-c", script], capture_output=True, text=True, timeout=300)
    assert res.returncode == 0, res.stderr[-2000:]
    import sparse_attention_indexer_live_gb300 as dsa
    assert res.stdout.split() == [str(dsa.DSA_OK)] * 2 + ["True"]
