"""Refusals of the paged 4-bit cache's calls: the C ABI's own checks and the
binding's, none of which needs a GPU (a tensor subclass that reports a CUDA
device stands in for device tensors; every check fires before a launch)."""
import ctypes
import os
import subprocess

import pytest

torch = pytest.importorskip("torch")

import sparse_attention_indexer_live_gb300 as dsa  # noqa: E402
from sparse_attention_indexer_live_gb300 import cache as C  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
VP = ctypes.c_void_p


class _OnCuda(torch.Tensor):
    """A host tensor that reports cuda:0 (for the checks only; never launched)."""

    @property
    def is_cuda(self):
        return True

    @property
    def device(self):
        return torch.device("cuda", 0)

    def get_device(self):
        return 0


class _OnOther(_OnCuda):
    def get_device(self):
        return 1


def dev(t, cls=_OnCuda):
    return torch.Tensor._make_subclass(cls, t)


def i32(*shape):
    return dev(torch.zeros(*shape, dtype=torch.int32))


@pytest.fixture(scope="module")
def lib():
    dsa.build()
    return dsa.load()


def cfg(**kw):
    return dsa.cache_cfg(**{**dict(pages=10, page_size=16, kv_heads=2), **kw})


def test_bytes(lib):
    assert dsa.dsa_cache_bytes(cfg()) == 10 * 16 * 2 * 144 == 10 * 16 * 2 * C.RECORD_BYTES
    assert dsa.dsa_cache_bytes(cfg(pages=0)) == 0
    assert dsa.dsa_cache_bytes(cfg(pages=2 ** 19 - 1, page_size=4096, kv_heads=64)) == (2 ** 19 - 1) * 4096 * 64 * 144


@pytest.mark.parametrize("kw,status", [
    (dict(pages=-1), 1), (dict(page_size=0), 1), (dict(page_size=-8), 1), (dict(page_size=24), 1),
    (dict(page_size=8192), 1), (dict(pages=2 ** 27), 1), (dict(kv_heads=0), 1), (dict(kv_heads=65), 2),
    (dict(k_shift=33), 1), (dict(v_shift=-33), 1)])
def test_cfg_limits(lib, kw, status):
    with pytest.raises(dsa.DsaSelectError) as e:
        dsa.dsa_cache_bytes(cfg(**kw))
    assert e.value.status == status
    c = cfg(**kw)
    r = ctypes.byref(c)
    p = VP(256)
    assert lib.dsa_cache_plan(r, 0, 0, 0, 0, *[p] * 11, None) == status
    assert lib.dsa_cache_write(r, 0, 0, p, p, 256, 256, p, p, None) == status
    assert lib.dsa_cache_read(r, 0, 0, p, p, p, p, None) == status
    assert lib.dsa_cache_attention(r, 0, 130, 0, 0, 0, 0, *[p] * 5, 1.0, p, p, None) == status


def test_null_cfg(lib):
    p = VP(256)
    n = ctypes.c_size_t()
    assert lib.dsa_cache_bytes(None, ctypes.byref(n)) == 1
    assert lib.dsa_cache_bytes(ctypes.byref(cfg()), None) == 1
    assert lib.dsa_cache_plan(None, 0, 0, 0, 0, *[p] * 11, None) == 1
    assert lib.dsa_cache_attention_prompt_workspace(ctypes.byref(cfg()), 1, 16, 1, None) == 1


def test_abi_refusals(lib):
    r = ctypes.byref(cfg())
    p, odd = VP(4096), VP(4100)
    plan = lambda R=2, P=3, T=4, F=5, **kw: lib.dsa_cache_plan(  # noqa: E731
        r, R, P, T, F, *[kw.get(n, p) for n in ("lens", "fresh", "tables", "held", "free", "count", "first", "req",
                                                "ends", "slots", "status")], None)
    for kw in (dict(R=-1), dict(P=-1), dict(T=-1), dict(F=-1), dict(count=None), dict(first=None),
               dict(status=None), dict(lens=None), dict(tables=None), dict(slots=None), dict(free=None)):
        assert plan(**kw) == 1, kw
    assert plan(R=8193) == 2
    # rows
    w = lambda T=1, t=0, k=p, v=p, ks=256, vs=256, s=p, c=p: lib.dsa_cache_write(r, T, t, k, v, ks, vs, s, c, None)  # noqa: E731
    for kw in (dict(T=-1), dict(t=3), dict(t=-1), dict(k=None), dict(v=None), dict(s=None), dict(c=None),
               dict(c=odd), dict(ks=255), dict(vs=0), dict(k=VP(4097)), dict(t=2, v=VP(4098))):
        assert w(**kw) == 1, kw
    assert w(T=0, k=None, v=None) == 0
    rd = lambda T=1, t=0, c=p, s=p, k=p, v=p: lib.dsa_cache_read(r, T, t, c, s, k, v, None)  # noqa: E731
    for kw in (dict(T=-1), dict(t=3), dict(c=None), dict(s=None), dict(k=None), dict(v=odd), dict(c=odd)):
        assert rd(**kw) == 1, kw
    assert rd(T=0, k=None, v=None) == 0
    # attention
    a = lambda T=1, H=16, K=4, R=1, P=1, t=0, cache=p, q=p, idx=p, req=p, tab=p, o=p, lse=p: lib.dsa_cache_attention(  # noqa: E731
        r, T, H, K, R, P, t, cache, q, idx, req, tab, 1.0, o, lse, None)
    for kw in (dict(T=-1), dict(H=0), dict(H=15), dict(K=-1), dict(R=-1), dict(P=-1), dict(t=2), dict(cache=odd),
               dict(q=None), dict(q=odd), dict(o=odd), dict(o=None), dict(lse=None), dict(req=None), dict(idx=None),
               dict(tab=None), dict(cache=None)):
        assert a(**kw) == 1, kw
    assert a(H=258) == 2 and a(T=2 ** 27, H=16) == 2
    assert a(T=0, q=None, o=None) == 0
    n = ctypes.c_size_t()
    ws = lambda T=5, H=16, K=64: lib.dsa_cache_attention_prompt_workspace(r, T, H, K, ctypes.byref(n))  # noqa: E731
    assert ws() == 0 and n.value == 16 + 2 * 16 * 64 * 4   # one group of 16 tokens x 8 heads a key/value head
    assert ws(H=32) == 0 and n.value == 16 + 2 * 8 * 64 * 4
    assert ws(H=8) == 2 and ws(H=64) == 2 and ws(K=3073) == 2 and ws(T=-1) == 1
    pr = lambda size=1 << 20, w=p, t=0, tab=p: lib.dsa_cache_attention_prompt(  # noqa: E731
        r, 5, 16, 64, 3, t, p, p, p, tab, 1.0, w, size, p, p, None)
    assert pr(size=16) == 1 and pr(w=None) == 1 and pr(w=odd) == 1 and pr(t=2) == 1 and pr(tab=None) == 1


@pytest.mark.parametrize("scale,k_shift", [(float("nan"), 0), (float("inf"), 0), (-float("inf"), 3), (1e30, 32)])
def test_scale_has_to_be_finite(lib, scale, k_shift):
    c = cfg(k_shift=k_shift)
    r, p = ctypes.byref(c), VP(256)
    assert lib.dsa_cache_attention(r, 0, 8, 4, 1, 1, 0, *[p] * 5, scale, p, p, None) == 1
    assert lib.dsa_cache_attention_prompt(r, 0, 16, 4, 1, 0, *[p] * 4, scale, p, 1 << 20, p, p, None) == 1
    assert lib.dsa_cache_attention(r, 0, 8, 4, 1, 1, 0, *[p] * 5, -0.1, p, p, None) == 0


def test_binding_plan():
    R, P, T = 3, 4, 5
    good = dict(lens=i32(R), fresh=i32(R), tables=i32(R, P), held=i32(R), free=i32(7), count=i32(1), first=i32(R + 1),
                req=i32(T), ends=i32(T), slots=i32(T), status=i32(4))

    def call(**kw):
        a = {**good, **kw}
        C.dsa_cache_plan(cfg(), *a.values())
    for kw in (dict(fresh=i32(2)), dict(held=i32(2)), dict(tables=i32(2, P)), dict(tables=i32(R * P)),
               dict(count=i32(0)), dict(first=i32(R)), dict(ends=i32(T - 1)), dict(slots=i32(T - 1)),
               dict(status=i32(3)), dict(lens=torch.zeros(R, dtype=torch.int32)),
               dict(held=dev(torch.zeros(R, dtype=torch.int32), _OnOther)),
               dict(tables=dev(torch.zeros(R, 2 * P, dtype=torch.int32)[:, ::2]))):
        with pytest.raises(ValueError):
            call(**kw)
    for kw in (dict(lens=dev(torch.zeros(R, dtype=torch.int64))), dict(slots=None), dict(count=3)):
        with pytest.raises(TypeError):
            call(**kw)
    with pytest.raises(TypeError):
        C.dsa_cache_plan(None, *good.values())


def test_binding_rows():
    c = cfg()
    cache = dev(torch.zeros(dsa.dsa_cache_bytes(c), dtype=torch.uint8))
    k = dev(torch.zeros(3, 2, 128))
    s = i32(3)
    bad_value = [
        (k, dev(torch.zeros(2, 2, 128)), s, cache), (dev(torch.zeros(3, 1, 128)), k, s, cache),
        (dev(torch.zeros(3, 2, 64)), k, s, cache), (dev(torch.zeros(3, 256)), k, s, cache),
        (k, k, i32(4), cache), (k, k, s, cache[:-1]), (torch.zeros(3, 2, 128), k, s, cache),
        (dev(torch.zeros(3, 128, 2).transpose(1, 2)), k, s, cache),        # dims not packed
        (dev(torch.zeros(2, 3, 128).transpose(0, 1)), k, s, cache),        # heads not packed
        (dev(torch.zeros(1, 2, 128).expand(3, 2, 128)), k, s, cache),      # tokens overlap
        (dev(torch.zeros(3, 2, 128), _OnOther), k, s, cache)]
    for a in bad_value:
        with pytest.raises(ValueError):
            C.dsa_cache_write(c, *a)
    for a in [(k, dev(torch.zeros(3, 2, 128).half()), s, cache), (k.double(), k, s, cache), (None, k, s, cache),
              (k, k, dev(torch.zeros(3, dtype=torch.int64)), cache), (k, k, s, dev(torch.zeros(9999).half()))]:
        with pytest.raises(TypeError):
            C.dsa_cache_write(c, *a)
    for a in [(cache, s, k, dev(torch.zeros(2, 2, 128))), (cache[:-1], s, k, k), (cache, i32(4), k, k),
              (cache, s, dev(torch.zeros(3, 2, 256)[..., ::2]), k)]:
        with pytest.raises(ValueError):
            C.dsa_cache_read(c, *a)
    with pytest.raises(TypeError):
        C.dsa_cache_read(c, cache, s, k, dev(torch.zeros(3, 2, 128).half()))
    # strides the write takes: tokens apart, one token of any stride
    assert C._strided_rows("k", dev(torch.zeros(3, 2, 2, 128)[:, 1]), 3, 2, 0) == 512
    assert C._strided_rows("k", dev(torch.zeros(1, 2, 128).expand(1, 2, 128)), 1, 2, 0) == 256


def test_binding_attention():
    c = cfg()
    cache = dev(torch.zeros(dsa.dsa_cache_bytes(c), dtype=torch.uint8))
    T, H, K = 3, 8, 5
    good = dict(cache=cache, q=dev(torch.zeros(T, H, 128).half()), idx=i32(T, K), req=i32(T), tables=i32(2, 3),
                scale=1.0, o=dev(torch.zeros(T, H, 128).half()), lse=dev(torch.zeros(T, H)))

    def call(**kw):
        C.dsa_cache_attention(c, *{**good, **kw}.values())
    for kw in (dict(cache=cache[:-1]), dict(q=dev(torch.zeros(T, H, 64).half())), dict(idx=i32(T + 1, K)),
               dict(idx=i32(T * K)), dict(req=i32(T - 1)), dict(tables=i32(6)), dict(lse=dev(torch.zeros(T, H - 1))),
               dict(o=dev(torch.zeros(T, H - 1, 128).half())), dict(q=torch.zeros(T, H, 128).half()),
               dict(q=dev(torch.zeros(H, T, 128).half().transpose(0, 1))),
               dict(req=dev(torch.zeros(T, dtype=torch.int32), _OnOther))):
        with pytest.raises(ValueError):
            call(**kw)
    for kw in (dict(q=dev(torch.zeros(T, H, 128))), dict(o=dev(torch.zeros(T, H, 128).bfloat16())),
               dict(lse=dev(torch.zeros(T, H).half())), dict(idx=dev(torch.zeros(T, K, dtype=torch.int64)))):
        with pytest.raises(TypeError):
            call(**kw)
    ws = dev(torch.zeros(1 << 16, dtype=torch.uint8))
    good = dict(cache=cache, q=dev(torch.zeros(T, 16, 128).half()), idx=i32(T, K), table=i32(3), scale=1.0,
                workspace=ws, o=dev(torch.zeros(T, 16, 128).half()), lse=dev(torch.zeros(T, 16)))
    for kw, exc in ((dict(table=dev(torch.zeros(3))), TypeError), (dict(workspace=dev(torch.zeros(9))), TypeError),
                    (dict(workspace=torch.zeros(9, dtype=torch.uint8)), ValueError), (dict(idx=i32(2, K)), ValueError)):
        with pytest.raises(exc):
            C.dsa_cache_attention_prompt(c, *{**good, **kw}.values())


def test_struct_layout(tmp_path):
    fields = [f for f, _ in C.dsa_cache_cfg._fields_]
    prog = tmp_path / "layout.c"
    prog.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "dsa_select.h"\nint main(void) {\n'
                    'printf("%zu %d\\n", sizeof(dsa_cache_cfg), DSA_CACHE_RECORD_BYTES);\n'
                    + "".join(f'printf("%zu\\n", offsetof(dsa_cache_cfg, {f}));\n' for f in fields) + "return 0; }\n")
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), "-o", str(exe), str(prog)], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()
    assert [int(x) for x in out] == [ctypes.sizeof(C.dsa_cache_cfg), C.RECORD_BYTES] + [
        getattr(C.dsa_cache_cfg, f).offset for f in fields]


def test_status_is_of_a_device(monkeypatch):
    entered = []

    class device:
        def __init__(self, d):
            self.d = d

        def __enter__(self):
            entered.append(self.d)

        def __exit__(self, *a):
            entered.append("left")
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(C.binding, "load", lambda: type("L", (), dict(
        dsa_cache_attention_status=staticmethod(lambda: entered.append("asked") or 4))))
    assert C.dsa_cache_attention_status(1) == 4 and C.dsa_cache_attention_status() == 4
    assert entered == [1, "asked", "left", "asked"]


def test_a_step_of_negative_size(monkeypatch):
    planned = []
    monkeypatch.setattr(C, "dsa_cache_plan", lambda *a: planned.append(a))
    c = C.PagedCache.__new__(C.PagedCache)
    c._maps = [torch.empty((3, 64), dtype=torch.int32)]
    c.slots = c._maps[0][2, :5]
    with pytest.raises(ValueError, match="tokens"):
        c.step(None, None, -1)
    assert not planned and c.slots.numel() == 5


def test_sizes_are_asked_with_a_cache_cfg(lib):
    q, idx = torch.zeros(5, 16, 128), torch.zeros(5, 64, dtype=torch.int32)
    assert C.dsa_cache_attention_prompt_workspace(cfg(), q, idx) == 16 + 2 * 16 * 64 * 4
    for other in (None, dsa.dsa_attention_cfg(1, 8, 10, 128, 128, 4), (ctypes.c_int32 * 5)(1, 16, 1, 0, 0)):
        with pytest.raises(TypeError):
            C.dsa_cache_bytes(other)
        with pytest.raises(TypeError):
            C.dsa_cache_attention_prompt_workspace(other, q, idx)
    with pytest.raises(TypeError):
        C.dsa_cache_attention_prompt_workspace(cfg(), q, None)
    wide = torch.zeros(1, dtype=torch.int32).expand(5, 2 ** 32 + 4)  # not 4 entries a list
    for a in ((q[0], idx), (q, idx[0]), (q, wide)):
        with pytest.raises(ValueError):
            C.dsa_cache_attention_prompt_workspace(cfg(), *a)


@pytest.mark.parametrize("name", ["pages", "page_size", "kv_heads", "k_shift", "v_shift"])
def test_cfg_numbers_past_32_bits(name):
    for n in (2 ** 32 + 1, 2 ** 31, -2 ** 31 - 1):
        with pytest.raises(ValueError, match=name):
            cfg(**{name: n})
    assert getattr(cfg(**{name: 2 ** 31 - 1}), name) == 2 ** 31 - 1  # the library's to refuse
