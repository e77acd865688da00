"""What the cache's calls launch on devices of other sizes: the library's own host
code against a fake runtime (tests/fake_cuda.cpp), whose device has a stated
number of SMs and a largest cluster and refuses larger ones."""
import ctypes
import importlib
import os
import subprocess
from concurrent.futures import ThreadPoolExecutor

import pytest

import sparse_attention_indexer_live_gb300 as dsa

B = importlib.import_module("sparse_attention_indexer_live_gb300.build")
VP, I = ctypes.c_void_p, ctypes.c_int32


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    tmp = tmp_path_factory.mktemp("fake")
    nvcc = B.nvcc_path()
    srcs = [s for s in B.SOURCES if "cache" in os.path.basename(s) or "attention" in os.path.basename(s)]
    srcs.append(os.path.join(os.path.dirname(os.path.abspath(__file__)), "fake_cuda.cpp"))
    objs = [str(tmp / (os.path.basename(s) + ".o")) for s in srcs]

    def compile_one(a):  # the host's half: no machine code for the device's
        subprocess.run([nvcc, "-gencode", "arch=compute_103a,code=compute_103a", "-O1", "-std=c++17", "-Xcompiler",
                        "-fPIC", "-I", B.INCLUDE, "-c", "-o", a[1], a[0]], check=True, capture_output=True)
    with ThreadPoolExecutor(8) as ex:
        list(ex.map(compile_one, zip(srcs, objs)))
    so = str(tmp / "libfake.so")
    # -Bsymbolic: its own runtime, not the one that torch may have loaded
    subprocess.run(["g++", "-shared", "-Wl,-Bsymbolic", "-o", so, *objs], check=True)
    L = ctypes.CDLL(so)
    L.dsa_cache_attention.argtypes = [VP] + [I] * 6 + [VP] * 5 + [ctypes.c_float, VP, VP, VP]
    L.dsa_cache_attention_prompt.argtypes = [VP] + [I] * 5 + [VP] * 4 + [ctypes.c_float, VP, ctypes.c_size_t, VP, VP, VP]
    L.dsa_cache_plan.argtypes = [VP] + [I] * 4 + [VP] * 12
    return L


DEVICES = [(0, 152, 16), (1, 152, 8), (2, 76, 8), (3, 18, 4), (4, 16, 2), (5, 1, 1)]
ATTENTION = [  # tokens, heads, kv_heads, select
    (1, 8, 1, 2048), (1, 16, 1, 5000), (4, 8, 2, 1024), (30, 8, 1, 800), (96, 8, 1, 2176), (150, 8, 1, 1100),
    (512, 32, 4, 1001), (1, 64, 1, 2048), (10, 128, 1, 2048), (17, 64, 1, 2048), (64, 64, 1, 2048), (200, 24, 1, 256)]


def launched(lib, rc):
    n, g, c = I(), I(), I()
    lib.fake_seen(ctypes.byref(n), ctypes.byref(g), ctypes.byref(c))
    assert rc == 0
    return n.value, g.value, c.value


@pytest.mark.parametrize("dev,sms,largest", DEVICES)
def test_clusters_that_the_device_has_room_for(lib, dev, sms, largest):
    p = VP(4096)
    for T, H, KV, Kc in ATTENTION:
        cfg = dsa.cache_cfg(pages=100, page_size=64, kv_heads=KV)
        for dtype in (0, 1):
            lib.fake_device(dev, sms, largest)
            n, g, c = launched(lib, lib.dsa_cache_attention(ctypes.byref(cfg), T, H, Kc, 4, 50, dtype, *[p] * 5, 0.1, p,
                                                            p, None))
            assert n == 1 and c <= largest and g % c == 0
    for T, H, KV, Kc in ((20, 8, 1, 2100), (100, 16, 1, 1100), (300, 16, 2, 520), (2048, 8, 1, 2048)):
        cfg = dsa.cache_cfg(pages=100, page_size=64, kv_heads=KV)
        lib.fake_device(dev, sms, largest)
        n, g, c = launched(lib, lib.dsa_cache_attention_prompt(ctypes.byref(cfg), T, H, Kc, 50, 0, *[p] * 4, 0.1, p,
                                                               1 << 30, p, p, None))
        assert n == 2 and c <= largest and g % c == 0
    cfg = dsa.cache_cfg(pages=100, page_size=64)
    for R, T in ((1, 1), (48, 96), (512, 66016), (8192, 20000), (8192, 1 << 18), (4, 1 << 20), (3000, 5000)):
        lib.fake_device(dev, sms, largest)
        n, g, c = launched(lib, lib.dsa_cache_plan(ctypes.byref(cfg), R, 100, T, 100, *[p] * 11, None))
        assert n == 1 and c <= largest and g == c  # one cluster


def test_what_152_sms_get(lib):
    """The splits that were measured."""
    p = VP(4096)

    def split(T, H, KV, Kc):
        cfg = dsa.cache_cfg(pages=100, page_size=64, kv_heads=KV)
        lib.fake_device(0, 152, 16)
        return launched(lib, lib.dsa_cache_attention(ctypes.byref(cfg), T, H, Kc, 4, 50, 0, *[p] * 5, 0.1, p, p, None))[1:]
    assert split(1, 8, 1, 2048) == (16, 16)
    assert split(96, 8, 1, 2176) == (384, 4)
    assert split(64, 64, 1, 2048) == (128, 2)       # tiles
    assert split(512, 32, 4, 1001) == (2048, 1)
    assert split(1, 8, 1, 256) == (1, 1)
