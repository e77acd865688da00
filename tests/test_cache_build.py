"""The module of ordinary cache calls is a convenience: where it does not build or
load, the library is built all the same and the calls go through ctypes."""
import contextlib
import os
import subprocess
import sys
import types

import pytest

torch = pytest.importorskip("torch")

import sparse_attention_indexer_live_gb300 as dsa  # noqa: E402
from sparse_attention_indexer_live_gb300 import cache as C  # noqa: E402
from tests.test_cache_args import dev, i32  # noqa: E402

B = __import__("importlib").import_module("sparse_attention_indexer_live_gb300.build")


@pytest.mark.parametrize("why", ["compiler", "no compiler"])
def test_build_without_the_calls_module(tmp_path, monkeypatch, why):
    dsa.build()
    target = tmp_path / "cache_calls.so"
    target.write_bytes(b"an older build")
    os.utime(target, (1, 1))
    monkeypatch.setattr(B, "calls_path", lambda: str(target))
    if why == "compiler":
        source = tmp_path / "cache_calls.cpp"
        source.write_text("#error not on this machine\n")
        monkeypatch.setattr(B, "CALLS_SOURCE", str(source))
    else:
        run = B.subprocess.run
        monkeypatch.setattr(B.subprocess, "run", lambda cmd, **kw: run([str(tmp_path / "none") if c == "g++" else c
                                                                       for c in cmd], **kw))
    with pytest.warns(RuntimeWarning, match="cache_calls"):
        assert B.build() == B.LIB_PATH
    assert not target.exists(), "a module of older sources stays behind"


@pytest.mark.parametrize("file", [None, "not built", b"not a module"])
def test_calls_without_the_module(tmp_path, monkeypatch, file):
    path = None if file is None else str(tmp_path / "cache_calls.so")
    if isinstance(file, bytes):
        (tmp_path / "cache_calls.so").write_bytes(file)
    seen = []
    monkeypatch.setattr(C, "_calls", None)
    monkeypatch.setattr(C, "calls_path", lambda: path)
    monkeypatch.setattr(C.binding, "load", lambda: types.SimpleNamespace(
        dsa_cache_read=lambda *a: seen.append(a) or 0))
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d: types.SimpleNamespace(cuda_stream=77))
    monkeypatch.setattr(torch.cuda, "device", lambda d: contextlib.nullcontext())
    cfg = dsa.cache_cfg(pages=2, page_size=4)
    cache, rows = dev(torch.zeros(2 * 4 * 144, dtype=torch.uint8)), dev(torch.zeros(3, 1, 128))
    with pytest.warns(RuntimeWarning, match="cache_calls"):
        C.dsa_cache_read(cfg, cache, i32(3), rows, rows)
    C.dsa_cache_read(cfg, cache, i32(3), rows, rows)  # and is not looked for again
    assert len(seen) == 2 and seen[0][1:3] == (3, 2) and seen[0][-1] == 77


def test_import_star_without_torch():
    """A Python without torch (-S: without its site packages) gets every name but the cache's."""
    root = os.path.dirname(B.PKG)
    code = (f"import sys; sys.path.insert(0, {root!r})\nfrom importlib.util import find_spec\n"
            "print(find_spec('torch') is None)\nfrom sparse_attention_indexer_live_gb300 import *\n"
            "print(DSA_OK, dsa_select_topk.__name__, 'PagedCache' in globals())")
    out = subprocess.run([sys.executable, "-S", "-c", code], capture_output=True, text=True, check=True).stdout.split()
    if out[0] != "True":
        pytest.skip("torch is part of this Python")
    assert out[1:] == ["0", "dsa_select_topk", "False"]
    assert set(C.__dict__) >= {n for n in dsa.__all__ if "cache" in n.lower()} and "PagedCache" in dsa.__all__
