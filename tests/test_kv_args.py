"""Refusals of the paged 16-bit cache's calls: the C ABI's own checks and the
binding's, none of which needs a GPU (a tensor subclass that reports a CUDA
device stands in for device tensors; every check fires before a launch)."""
import ctypes
import math
import os
import subprocess

import pytest

torch = pytest.importorskip("torch")

import sparse_attention_indexer_live_gb300 as dsa  # noqa: E402
from sparse_attention_indexer_live_gb300 import kv as K  # noqa: E402
from tests.test_cache_args import _OnOther, dev, i32  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BAD, UNSUPPORTED = dsa.DSA_ERR_INVALID_ARG, dsa.DSA_ERR_UNSUPPORTED
T, H, HK, P, R, N = 4, 8, 2, 3, 2, 2
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def lib():
    dsa.build()
    return dsa.load()


def cfg(**kw):
    return dsa.kv_cfg(**{**dict(pages=10, page_size=16, kv_heads=HK), **kw})


def rows(*shape, dtype=BF16):
    return dev(torch.zeros(*shape, dtype=dtype))


def _size(lib, name, c, *args):
    n = ctypes.c_size_t(7)
    return getattr(lib, name)(ctypes.byref(c), *args, ctypes.byref(n)), n.value


@pytest.mark.parametrize("change,status", [
    (dict(pages=-1), BAD), (dict(page_size=0), BAD), (dict(page_size=48), BAD), (dict(page_size=8192), BAD),
    (dict(page_size=8), UNSUPPORTED), (dict(page_size=256), UNSUPPORTED), (dict(kv_heads=0), BAD),
    (dict(kv_heads=65), UNSUPPORTED), (dict(pages=1 << 27), BAD)])
def test_cfg_limits(lib, change, status):
    assert _size(lib, "dsa_kv_attention_workspace", cfg(**change), 4, 64 * 65, 2, 3)[0] == status
    assert _size(lib, "dsa_kv_select_workspace", cfg(**change), 4, 64 * 65, 2, 3)[0] == status
    assert _size(lib, "dsa_kv_block_attention_workspace", cfg(**change), 4, 64 * 65, 2, 3, 5)[0] == status
    assert lib.dsa_kv_append(ctypes.byref(cfg(**change)), 4, 8, 0, 0, 1.0, None, 0, None, 0, None, 0, None, None, None,
                             None, None, None, None, None) == status


def test_raw_cfg(lib):
    for dtype in (2, -1):
        c = K.dsa_kv_cfg(10, 16, 2, dtype)
        assert _size(lib, "dsa_kv_attention_workspace", c, 4, 8, 2, 3)[0] == BAD
    assert lib.dsa_kv_attention_workspace(None, 1, 1, 1, 1, ctypes.byref(ctypes.c_size_t())) == BAD
    assert lib.dsa_kv_attention_workspace(ctypes.byref(cfg()), 4, 8, 2, 3, None) == BAD


@pytest.mark.parametrize("sizes,status", [
    ((-1, 8, 2, 3), BAD), ((4, 0, 2, 3), BAD), ((4, 7, 2, 3), BAD), ((4, 8, -1, 3), BAD), ((4, 8, 2, -1), BAD),
    ((4, 258, 2, 3), UNSUPPORTED), ((4, 8, 8193, 3), UNSUPPORTED), ((1 << 29, 8, 2, 3), UNSUPPORTED),
    ((0, 8, 0, 0), dsa.DSA_OK), ((4, 256, 8192, 0), dsa.DSA_OK)])
def test_step_limits(lib, sizes, status):
    for name, more in (("dsa_kv_attention_workspace", ()), ("dsa_kv_select_workspace", ()),
                       ("dsa_kv_block_attention_workspace", (3,))):
        assert _size(lib, name, cfg(), *sizes, *more)[0] == status, name
    c = ctypes.byref(cfg())
    if status != dsa.DSA_OK:
        assert lib.dsa_kv_attention(c, *sizes, None, None, None, 0, None, None, None, 1.0, None, 0, None, None, None) == status
        assert lib.dsa_kv_select(c, *sizes, 2, 0, 1, None, None, 0, None, None, None, None, 0, None, None) == status
        assert lib.dsa_kv_block_attention(c, *sizes, 2, None, None, None, 0, None, None, None, None, 1.0, None, 0, None,
                                          None, None) == status


def test_nothing_to_do(lib):
    c = ctypes.byref(cfg())
    for sizes in ((0, 8, 2, 3), (4, 8, 0, 3)):
        assert lib.dsa_kv_attention(c, *sizes, None, None, None, 0, None, None, None, 1.0, None, 0, None, None,
                                    None) == dsa.DSA_OK
        assert lib.dsa_kv_select(c, *sizes, 2, 0, 1, None, None, 0, None, None, None, None, 0, None, None) == dsa.DSA_OK
        assert lib.dsa_kv_block_attention(c, *sizes, 2, None, None, None, 0, None, None, None, None, 1.0, None, 0, None,
                                          None, None) == dsa.DSA_OK
    assert lib.dsa_kv_append(c, 0, 8, 0, 0, 1.0, None, 0, None, 0, None, 0, None, None, None, None, None, None, None,
                             None) == dsa.DSA_OK


X = 1 << 20  # stands for a 16-byte aligned address that is never read


def _attention(lib, **kw):
    a = {**dict(T=T, H=H, R=R, P=P, k=X, v=X, q=X, stride=H * 128, first=X, lens=X, tables=X, scale=1.0, ws=X,
                size=1 << 40, o=X, lse=X), **kw}
    return lib.dsa_kv_attention(ctypes.byref(cfg()), a["T"], a["H"], a["R"], a["P"], a["k"], a["v"], a["q"], a["stride"],
                                a["first"], a["lens"], a["tables"], a["scale"], a["ws"], a["size"], a["o"], a["lse"], None)


@pytest.mark.parametrize("kw", [dict(scale=math.inf), dict(scale=math.nan), dict(scale=3e38), dict(k=None), dict(v=None),
                                dict(q=None), dict(first=None), dict(lens=None), dict(tables=None), dict(ws=None),
                                dict(o=None), dict(lse=None), dict(k=X + 8), dict(v=X + 2), dict(q=X + 4), dict(o=X + 8),
                                dict(ws=X + 8), dict(first=X + 2), dict(lens=X + 1), dict(tables=X + 2), dict(lse=X + 2),
                                dict(stride=H * 128 - 8), dict(stride=H * 128 + 4), dict(size=0)])
def test_attention_refusals(lib, kw):
    assert _attention(lib, **kw) == BAD


def _select(lib, **kw):
    a = {**dict(T=T, H=H, R=R, P=P, n=N, lead=0, trail=1, means=X, q=X, stride=H * 128, first=X, lens=X, tables=X, ws=X,
                size=1 << 40, idx=X), **kw}
    return lib.dsa_kv_select(ctypes.byref(cfg()), a["T"], a["H"], a["R"], a["P"], a["n"], a["lead"], a["trail"],
                             a["means"], a["q"], a["stride"], a["first"], a["lens"], a["tables"], a["ws"], a["size"],
                             a["idx"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(n=0), BAD), (dict(lead=-1), BAD), (dict(trail=0), BAD), (dict(lead=2), BAD), (dict(trail=3), BAD),
    (dict(lead=2 ** 31 - 1), BAD), (dict(n=257), UNSUPPORTED), (dict(means=None), BAD), (dict(q=None), BAD),
    (dict(first=None), BAD), (dict(lens=None), BAD), (dict(tables=None), BAD), (dict(ws=None), BAD), (dict(idx=None), BAD),
    (dict(means=X + 8), BAD), (dict(q=X + 8), BAD), (dict(ws=X + 4), BAD), (dict(idx=X + 2), BAD), (dict(size=0), BAD),
    (dict(stride=H * 128 + 4), BAD), (dict(stride=128), BAD)])
def test_select_refusals(lib, kw, status):
    assert _select(lib, **kw) == status


def _blocks(lib, **kw):
    a = {**dict(T=T, H=H, R=R, P=P, n=N, k=X, v=X, q=X, stride=H * 128, idx=X, first=X, lens=X, tables=X, scale=1.0,
                ws=X, size=1 << 40, o=X, lse=X), **kw}
    return lib.dsa_kv_block_attention(ctypes.byref(cfg()), a["T"], a["H"], a["R"], a["P"], a["n"], a["k"], a["v"], a["q"],
                                      a["stride"], a["idx"], a["first"], a["lens"], a["tables"], a["scale"], a["ws"],
                                      a["size"], a["o"], a["lse"], None)


@pytest.mark.parametrize("kw,status", [(dict(n=0), BAD), (dict(n=4097), UNSUPPORTED), (dict(idx=None), BAD),
                                       (dict(idx=X + 2), BAD), (dict(scale=math.nan), BAD), (dict(size=0), BAD),
                                       (dict(o=X + 8), BAD), (dict(q=None), BAD)])
def test_block_refusals(lib, kw, status):
    assert _blocks(lib, **kw) == status


def _append(lib, **kw):
    a = {**dict(T=T, H=H, rot=128, nb=0, gain=1.0, q=X, qs=H * 128, k=X, ks=HK * 128, v=X, vs=HK * 128, ends=X, slots=X,
                turns=X, out=X, kc=X, vc=X, means=X), **kw}
    return lib.dsa_kv_append(ctypes.byref(cfg()), a["T"], a["H"], a["rot"], a["nb"], a["gain"], a["q"], a["qs"], a["k"],
                             a["ks"], a["v"], a["vs"], a["ends"], a["slots"], a["turns"], a["out"], a["kc"], a["vc"],
                             a["means"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), BAD), (dict(H=-1), BAD), (dict(rot=8), BAD), (dict(rot=144), BAD), (dict(rot=-16), BAD),
    (dict(gain=math.inf), BAD), (dict(gain=math.nan), BAD), (dict(H=8193), UNSUPPORTED), (dict(q=None), BAD),
    (dict(out=None), BAD), (dict(k=None), BAD), (dict(v=None), BAD), (dict(ends=None), BAD), (dict(slots=None), BAD),
    (dict(turns=None), BAD), (dict(kc=None), BAD), (dict(vc=None), BAD), (dict(q=X + 8), BAD), (dict(k=X + 2), BAD),
    (dict(v=X + 8), BAD), (dict(out=X + 8), BAD), (dict(kc=X + 8), BAD), (dict(vc=X + 4), BAD), (dict(means=X + 8), BAD),
    (dict(turns=X + 4), BAD), (dict(ends=X + 2), BAD), (dict(slots=X + 1), BAD), (dict(qs=H * 128 - 8), BAD),
    (dict(ks=128), BAD), (dict(vs=HK * 128 + 4), BAD)])
def test_append_refusals(lib, kw, status):
    assert _append(lib, **kw) == status


def test_binding_cfg():
    with pytest.raises(TypeError):
        cfg(dtype=torch.float32)
    with pytest.raises(ValueError):
        cfg(pages=1 << 32)
    with pytest.raises(TypeError):
        dsa.dsa_kv_attention_workspace(dsa.cache_cfg(pages=1), rows(T, H, 128), i32(R, P))


def test_rotary_turns():
    t = dsa.rotary_turns([2 * math.pi * 0.25, -2 * math.pi * 0.25, math.pi, 0.0])
    assert t.dtype == torch.int64 and t.tolist() == [1 << 62, -(1 << 62), -(1 << 63), 0]
    f = 1e4 ** (-torch.arange(0, 128, 2, dtype=torch.float64) / 128)
    turns = dsa.rotary_turns(f)
    for x, y in zip(f.tolist(), turns.tolist()):
        assert abs(y / 2 ** 64 - x / (2 * math.pi)) <= 2.0 ** -53 * x + 2.0 ** -64
    assert dsa.rotary_turns([]).numel() == 0


def _calls():
    c = cfg()
    pool, means = rows(10, 16, HK, 128), rows(10, HK, 128)
    step = dict(first=i32(R + 1), lens=i32(R), tables=i32(R, P))
    ws = dev(torch.zeros(1 << 16, dtype=torch.uint8))
    out = dict(workspace=ws, o=rows(T, H, 128), lse=rows(T, H, dtype=torch.float32))
    return {
        "append": (dsa.dsa_kv_append, dict(cfg=c, q=rows(T, H, 128), k=rows(T, HK, 128), v=rows(T, HK, 128), ends=i32(T),
                                           slots=i32(T), turns=dev(torch.zeros(64, dtype=torch.int64)), neighbours=False,
                                           gain=1.0, q_out=rows(T, H, 128), k_cache=pool, v_cache=pool, means=means)),
        "attention": (dsa.dsa_kv_attention, dict(cfg=c, k_cache=pool, v_cache=pool, q=rows(T, H, 128), **step, scale=1.0,
                                                 **out)),
        "select": (dsa.dsa_kv_select, dict(cfg=c, means=means, q=rows(T, H, 128), **step, lead=0, trail=1, workspace=ws,
                                           idx=i32(T, HK, N))),
        "blocks": (dsa.dsa_kv_block_attention, dict(cfg=c, k_cache=pool, v_cache=pool, q=rows(T, H, 128),
                                                    idx=i32(T, HK, N), **step, scale=1.0, **out))}


def _other(t):
    return dev(torch.zeros(t.shape, dtype=t.dtype), _OnOther)


@pytest.mark.parametrize("name", ["append", "attention", "select", "blocks"])
def test_binding_refuses_each_tensor(lib, name):
    fn, good = _calls()[name]
    for arg, t in good.items():
        if not isinstance(t, torch.Tensor):
            continue
        wrong = torch.float64 if t.dtype is not torch.float64 else torch.float32
        with pytest.raises(TypeError):
            fn(**{**good, arg: [1, 2]})
        with pytest.raises(TypeError):
            fn(**{**good, arg: dev(torch.zeros(t.shape, dtype=wrong))})
        with pytest.raises(ValueError):
            fn(**{**good, arg: torch.zeros(t.shape, dtype=t.dtype)})
        with pytest.raises(ValueError):
            fn(**{**good, arg: _other(t)})
        if arg not in ("workspace", "turns") and (name, arg) != ("attention", "q"):  # any size, or a smaller step
            with pytest.raises(ValueError):
                fn(**{**good, arg: dev(torch.zeros(t.shape, dtype=t.dtype)[:-1])})
        if t.dtype is BF16:
            with pytest.raises(ValueError):  # off its 16 bytes
                fn(**{**good, arg: dev(torch.zeros(t.numel() + 4, dtype=BF16)[4:].view(t.shape))})
            with pytest.raises(ValueError):  # dims apart
                fn(**{**good, arg: dev(torch.zeros(*t.shape, 2, dtype=BF16)[..., 0])})
    with pytest.raises(TypeError):
        fn(**{**good, "cfg": dsa.cache_cfg(pages=10)})


def test_binding_shapes(lib):
    calls = _calls()
    for name, kw in (("append", dict(k=rows(T, H, 128))), ("append", dict(q=rows(T, H, 64))),
                     ("append", dict(q=rows(T + 1, H, 128))), ("attention", dict(tables=i32(R + 1, P))),
                     ("attention", dict(tables=i32(R))), ("attention", dict(q=rows(T, H * 128))),
                     ("select", dict(idx=i32(T, HK + 1, N))), ("select", dict(idx=i32(T, N))),
                     ("select", dict(lead=1 << 32)), ("blocks", dict(idx=i32(T + 1, HK, N))),
                     ("append", dict(v=dev(torch.zeros(T, HK * 128 + 4, dtype=BF16)[:, :HK * 128].view(T, HK, 128)))),
                     ("append", dict(q=dev(torch.zeros(1, H, 128, dtype=BF16).expand(T, H, 128))))):
        fn, good = calls[name]
        with pytest.raises(ValueError):
            fn(**{**good, **kw})
    for name, kw in (("append", dict(neighbours="no")), ("select", dict(trail=1.0))):
        fn, good = calls[name]
        with pytest.raises(TypeError):
            fn(**{**good, **kw})
    for name, args in (("dsa_kv_attention_workspace", (rows(T, H), i32(R, P))),
                       ("dsa_kv_select_workspace", (rows(T, H, 128), i32(R))),
                       ("dsa_kv_block_attention_workspace", (rows(T, H, 128), i32(T, N), i32(R, P)))):
        with pytest.raises(ValueError):
            getattr(dsa, name)(cfg(), *args)


def test_struct_layout(tmp_path):
    fields = [f for f, _ in K.dsa_kv_cfg._fields_]
    prog = tmp_path / "layout.c"
    prog.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "dsa_select.h"\nint main(void) {\n'
                    'printf("%zu\\n", sizeof(dsa_kv_cfg));\n'
                    + "".join(f'printf("%zu\\n", offsetof(dsa_kv_cfg, {f}));\n' for f in fields) + "return 0; }\n")
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), "-o", str(exe), str(prog)], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()
    assert [int(x) for x in out] == [ctypes.sizeof(K.dsa_kv_cfg)] + [getattr(K.dsa_kv_cfg, f).offset for f in fields]
