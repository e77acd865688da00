"""The module that makes the cache's ordinary calls (csrc/cache_calls.cpp), on
the CPU: bound to stubs in place of the library, with host tensors in place of
the device's.  What it passes on, and every change to a call that has to leave it
to cache.py (None)."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

import sparse_attention_indexer_live_gb300 as dsa  # noqa: E402
from sparse_attention_indexer_live_gb300 import cache as C  # noqa: E402

I, L, F, P, Z = ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_void_p, ctypes.c_size_t
PAGES, PAGE, KV = 10, 16, 2
R, W, T, H, KC, CAP = 3, 4, 5, 8, 7, 10


class Stubs:
    """C functions that note their arguments and return `status`."""

    def __init__(self):
        self.seen, self.status, self.keep = None, 0, []

    def function(self, *types):
        def note(*args):
            self.seen = args
            return self.status
        self.keep.append(ctypes.CFUNCTYPE(I, *types)(note))
        return self.keep[-1]


@pytest.fixture(scope="module")
def calls():
    dsa.build()
    s = Stubs()
    lib = dsa.load()
    m = C._load_calls([lib.dsa_cache_bytes, s.function(P, *[I] * 4, *[P] * 12),
                       s.function(P, I, I, P, P, L, L, P, P, P), s.function(P, I, I, P, P, P, P, P),
                       s.function(P, *[I] * 6, *[P] * 5, F, P, P, P),
                       s.function(P, *[I] * 5, *[P] * 4, F, P, Z, P, P, P)], host=True)
    return m, s


def ints(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


def good(name):
    cfg = dsa.cache_cfg(pages=PAGES, page_size=PAGE, kv_heads=KV)
    data = torch.zeros(PAGES * PAGE * KV * 144, dtype=torch.uint8)
    rows = lambda: torch.zeros(T, KV, 128, dtype=torch.bfloat16)  # noqa: E731
    q = lambda: torch.zeros(T, H, 128, dtype=torch.float16)  # noqa: E731
    return {
        "plan": dict(cfg=cfg, lens=ints(R), fresh=ints(R), tables=ints(R, W), held=ints(R), free=ints(CAP),
                     count=ints(1), first=ints(R + 1), req=ints(T), ends=ints(T), slots=ints(T), status=ints(4)),
        "write": dict(cfg=cfg, k=rows(), v=rows(), slots=ints(T), cache=data),
        "read": dict(cfg=cfg, cache=data, slots=ints(T), k=rows(), v=rows()),
        "attention": dict(cfg=cfg, cache=data, q=q(), idx=ints(T, KC), req=ints(T), tables=ints(R, W), scale=0.25,
                          o=q(), lse=torch.zeros(T, H)),
        "prompt": dict(cfg=cfg, cache=data, q=q(), idx=ints(T, KC), table=ints(W), scale=0.25,
                       workspace=torch.zeros(64, dtype=torch.uint8), o=q(), lse=torch.zeros(T, H)),
    }[name]


NAMES = ("plan", "write", "read", "attention", "prompt")


def pointers(a, *names):
    return [a[n].data_ptr() for n in names]


def expected(name, a):
    c = ctypes.addressof(a["cfg"])
    if name == "plan":
        return [c, R, W, T, CAP, *pointers(a, "lens", "fresh", "tables", "held", "free", "count", "first", "req", "ends",
                                           "slots", "status"), None]
    if name == "write":
        return [c, T, 0, *pointers(a, "k", "v"), KV * 128, KV * 128, *pointers(a, "slots", "cache"), None]
    if name == "read":
        return [c, T, 0, *pointers(a, "cache", "slots", "k", "v"), None]
    if name == "attention":
        return [c, T, H, KC, R, W, 1, *pointers(a, "cache", "q", "idx", "req", "tables"), 0.25, *pointers(a, "o", "lse"),
                None]
    return [c, T, H, KC, W, 1, *pointers(a, "cache", "q", "idx", "table"), 0.25, a["workspace"].data_ptr(), 64,
            *pointers(a, "o", "lse"), None]


@pytest.mark.parametrize("name", NAMES)
def test_what_is_passed_on(calls, name):
    m, s = calls
    a = good(name)
    for status in (0, 3):
        s.seen, s.status = None, status
        assert getattr(m, name)(*a.values()) == status
        assert list(s.seen) == expected(name, a)


# least elements of each tensor (those that a shape fixes: None)
LEAST = {
    "plan": dict(fresh=R, held=R, count=1, first=R + 1, ends=T, slots=T, status=4),
    "write": dict(cache=PAGES * PAGE * KV * 144),
    "read": dict(cache=PAGES * PAGE * KV * 144, k=T * KV * 128, v=T * KV * 128),
    "attention": dict(cache=PAGES * PAGE * KV * 144, req=T, o=T * H * 128, lse=T * H),
    "prompt": dict(cache=PAGES * PAGE * KV * 144, o=T * H * 128, lse=T * H),
}


@pytest.mark.parametrize("name", NAMES)
def test_what_is_left_to_the_binding(calls, name):
    m, s = calls
    call = getattr(m, name)
    s.status = 0

    def left(a):
        s.seen = None
        assert call(*a.values()) is None and s.seen is None
    a = good(name)
    left(dict(list(a.items())[:-1]))  # too few arguments
    for n, x in a.items():
        left({**a, n: None})
        left({**a, n: object()})
        if not isinstance(x, torch.Tensor):
            continue
        left({**a, n: x.numpy() if x.dtype != torch.bfloat16 else x.tolist()})
        other = {torch.int32: torch.int64, torch.uint8: torch.int8, torch.float32: torch.float64}.get(x.dtype, torch.float64)
        left({**a, n: x.to(other)})
        left({**a, n: x.to("meta")})
        left({**a, n: x.to_sparse()})
        if x.numel() > 1 and n not in ("k", "v"):
            left({**a, n: torch.stack([x, x], -1)[..., 0]})  # not contiguous
    for n, least in LEAST[name].items():
        flat = a[n].reshape(-1)
        left({**a, n: flat[:-1]})
        assert flat.numel() == least
        if not (name, n) in (("read", "k"), ("read", "v")):
            s.seen = None
            assert call(*{**a, n: torch.cat([flat, flat])}.values()) == 0  # more is fine
    bad = dsa.cache_cfg(pages=PAGES, page_size=24, kv_heads=KV)
    if name != "plan":  # a plan's cfg is left to the library
        left({**a, "cfg": bad})
        left({**a, "cfg": dsa.cache_cfg(pages=2 ** 30, page_size=1, kv_heads=64)})
    if "scale" in a:
        left({**a, "scale": 1})
        left({**a, "scale": "1"})


def test_shapes(calls):
    m, s = calls
    s.status = 0

    def left(name, **kw):
        s.seen = None
        assert getattr(m, name)(*{**good(name), **kw}.values()) is None and s.seen is None
    left("plan", tables=ints(R * W))
    left("plan", tables=ints(R + 1, W))
    left("plan", lens=ints(R + 1))
    left("plan", req=ints(T + 1))
    half = dict(dtype=torch.float16)
    for name in ("attention", "prompt"):
        left(name, q=torch.zeros(T, H * 128, **half))
        left(name, q=torch.zeros(T, H, 64, **half))
        left(name, q=torch.zeros(T, H, 128))  # f32
        left(name, q=torch.zeros(T, H, 128, dtype=torch.bfloat16))  # not o's type
        left(name, idx=ints(T + 1, KC))
        left(name, idx=ints(T * KC))
    left("attention", tables=ints(R * W))
    bf16 = dict(dtype=torch.bfloat16)
    for n in ("k", "v"):
        for x in (torch.zeros(T + 1, KV, 128, **bf16), torch.zeros(T, KV + 1, 128, **bf16),
                  torch.zeros(T, KV, 64, **bf16), torch.zeros(T, KV * 128, **bf16), torch.zeros(T, KV, 128, **half),
                  torch.zeros(T, 128, KV, **bf16).transpose(1, 2), torch.zeros(KV, T, 128, **bf16).transpose(0, 1),
                  torch.zeros(1, KV, 128, **bf16).expand(T, KV, 128), torch.zeros(T, KV, 256, **bf16)[..., ::2]):
            left("write", **{n: x})


def test_strides_types_and_empty_calls(calls):
    m, s = calls
    s.status = 0
    a = good("write")
    a["k"] = torch.zeros(T, 3, KV, 128, dtype=torch.bfloat16)[:, 1]
    assert m.write(*a.values()) == 0 and s.seen[5:7] == (3 * KV * 128, KV * 128) and s.seen[3] == a["k"].data_ptr()
    one = torch.zeros(1, KV, 128, dtype=torch.float32)
    assert m.write(a["cfg"], one, one.expand(1, KV, 128), ints(1), a["cache"]) == 0
    assert s.seen[1:3] == (1, 2) and s.seen[5:7] == (KV * 128, KV * 128)
    none = torch.zeros(0, KV, 128, dtype=torch.float16)
    assert m.write(a["cfg"], none, none, ints(0), a["cache"]) == 0 and s.seen[1:3] == (0, 1)
    a = good("plan")
    a.update(lens=ints(0), fresh=ints(0), tables=ints(0, W), held=ints(0), first=ints(1))
    assert m.plan(*a.values()) == 0 and s.seen[1:5] == (0, W, T, CAP)
    # a subclass that takes torch functions over is a tensor like others; one
    # whose operations run in Python is not
    a = good("plan")
    assert m.plan(*{**a, "lens": torch.nn.Parameter(a["lens"], requires_grad=False)}.values()) == 0


def test_binding_uses_it(calls, monkeypatch):
    m, s = calls
    monkeypatch.setattr(C, "_calls", m)
    for name in NAMES:
        a = good(name)
        f = getattr(C, {"prompt": "dsa_cache_attention_prompt"}.get(name, "dsa_cache_" + name))
        s.seen, s.status = None, 0
        f(*a.values())
        assert list(s.seen) == expected(name, a)
        s.status = 3
        with pytest.raises(dsa.DsaSelectError) as e:
            f(*a.values())
        assert e.value.status == 3
        with pytest.raises((TypeError, ValueError)):  # the binding's own checks: not CUDA tensors
            f(*{**a, "cfg": dsa.cache_cfg(pages=PAGES, page_size=24, kv_heads=KV)}.values(), **(
                dict(stream=object()) if name == "plan" else {}))
