"""The module that makes the 16-bit cache's ordinary calls (csrc/cache_calls.cpp),
on the CPU: bound to stubs in place of the library, with host tensors in place of
the device's.  What it passes on, and every change to a call that has to leave it
to kv.py (None)."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

import sparse_attention_indexer_live_gb300 as dsa  # noqa: E402
from sparse_attention_indexer_live_gb300 import kv as K  # noqa: E402

I, L, F, P, Z = ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_void_p, ctypes.c_size_t
PAGES, PAGE, KV = 10, 16, 2
R, W, T, H, SEL, ROT = 3, 4, 5, 8, 3, 64
NAMES = ("append", "attention", "select", "blocks")
CALLS = {"append": "dsa_kv_append", "attention": "dsa_kv_attention", "select": "dsa_kv_select",
         "blocks": "dsa_kv_block_attention"}


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
    m = K._bound([s.function(P, *[I] * 4, F, P, L, P, L, P, L, *[P] * 8),
                  s.function(P, *[I] * 4, P, P, P, L, P, P, P, F, P, Z, P, P, P),
                  s.function(P, *[I] * 7, P, P, L, *[P] * 4, Z, P, P),
                  s.function(P, *[I] * 5, P, P, P, L, *[P] * 4, F, P, Z, P, P, P)], host=True)
    yield m, s
    K._bound()  # the library's again, and a device's tensors


def ints(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


def good(name, dtype=torch.bfloat16):
    cfg = dsa.kv_cfg(pages=PAGES, page_size=PAGE, kv_heads=KV, dtype=dtype)
    x = dict(dtype=dtype)
    pool = lambda: torch.zeros(PAGES, PAGE, KV, 128, **x)  # noqa: E731
    step = lambda: dict(first=ints(R + 1), lens=ints(R), tables=ints(R, W))  # noqa: E731
    ws = lambda: torch.zeros(64, dtype=torch.uint8)  # noqa: E731
    q, out = torch.zeros(T, H, 128, **x), dict(o=torch.zeros(T, H, 128, **x), lse=torch.zeros(T, H))
    if name == "append":
        return dict(cfg=cfg, q=q, k=torch.zeros(T, KV, 128, **x), v=torch.zeros(T, KV, 128, **x), ends=ints(T), slots=ints(T),
                    turns=torch.zeros(ROT // 2, dtype=torch.int64), neighbours=True, gain=0.5, q_out=torch.zeros(T, H, 128, **x),
                    k_cache=pool(), v_cache=pool(), means=torch.zeros(PAGES, KV, 128, **x))
    if name == "attention":
        return dict(cfg=cfg, k_cache=pool(), v_cache=pool(), q=q, **step(), scale=0.25, workspace=ws(), **out)
    if name == "select":
        return dict(cfg=cfg, means=torch.zeros(PAGES, KV, 128, **x), q=q, **step(), lead=1, trail=2, workspace=ws(),
                    idx=ints(T, KV, SEL))
    return dict(cfg=cfg, k_cache=pool(), v_cache=pool(), q=q, idx=ints(T, KV, SEL), **step(), scale=0.25, workspace=ws(), **out)


def pointers(a, *names):
    return [None if a[n] is None else a[n].data_ptr() for n in names]


def expected(name, a):
    c = ctypes.addressof(a["cfg"])
    if name == "append":
        row = [a["q"].data_ptr(), H * 128] if a["q"] is not None else [None, 0]
        return [c, T, row[1] // 128, ROT, int(a["neighbours"]), 0.5, *row, a["k"].data_ptr(), KV * 128, a["v"].data_ptr(),
                KV * 128, *pointers(a, "ends", "slots", "turns"), a["q_out"].data_ptr() if a["q"] is not None else None,
                *pointers(a, "k_cache", "v_cache", "means"), None]
    lists = [SEL] if name != "attention" else []
    if name == "select":
        return [c, T, H, R, W, SEL, 1, 2, *pointers(a, "means", "q"), H * 128, *pointers(a, "first", "lens", "tables", "workspace"),
                64, a["idx"].data_ptr(), None]
    idx = pointers(a, "idx") if name == "blocks" else []
    return [c, T, H, R, W, *lists, *pointers(a, "k_cache", "v_cache", "q"), H * 128, *idx,
            *pointers(a, "first", "lens", "tables"), 0.25, a["workspace"].data_ptr(), 64, *pointers(a, "o", "lse"), None]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("name", NAMES)
def test_what_is_passed_on(calls, name, dtype):
    m, s = calls
    a = good(name, dtype)
    for status in (0, 3):
        s.seen, s.status = None, status
        assert getattr(m, "kv_" + name)(*a.values()) == status
        assert list(s.seen) == expected(name, a)
    if name == "append":
        s.status = 0
        for change in (dict(q=None), dict(q=None, q_out=None), dict(means=None), dict(neighbours=False)):
            b = {**a, **change}
            s.seen = None
            assert m.kv_append(*b.values()) == 0
            assert list(s.seen) == expected(name, b)


POOL = PAGES * PAGE * KV * 128
# least elements of each tensor
LEAST = {
    "append": dict(ends=T, q_out=T * H * 128, k_cache=POOL, v_cache=POOL, means=PAGES * KV * 128),
    "attention": dict(first=R + 1, k_cache=POOL, v_cache=POOL, o=T * H * 128, lse=T * H),
    "select": dict(first=R + 1, means=PAGES * KV * 128),
    "blocks": dict(first=R + 1, k_cache=POOL, v_cache=POOL, o=T * H * 128, lse=T * H),
}
NONE_IS_FINE = ("q", "means")  # of an append


@pytest.mark.parametrize("name", NAMES)
def test_what_is_left_to_the_binding(calls, name):
    m, s = calls
    call = getattr(m, "kv_" + name)
    s.status = 0

    def left(a):
        s.seen = None
        assert call(*a.values()) is None and s.seen is None
    a = good(name)
    left(dict(list(a.items())[:-1]))  # too few arguments
    for n, x in a.items():
        left({**a, n: object()})
        if not (name == "append" and n in NONE_IS_FINE):
            left({**a, n: None})
        if not isinstance(x, torch.Tensor):
            continue
        left({**a, n: x.tolist()})
        other = {torch.int32: torch.int64, torch.int64: torch.int32, torch.uint8: torch.int8,
                 torch.float32: torch.float64}.get(x.dtype, torch.float16)
        left({**a, n: x.to(other)})
        left({**a, n: x.to("meta")})
        left({**a, n: x.to_sparse()})
        left({**a, n: torch.stack([x, x], -1)[..., 0]})  # not packed
        if n not in ("ends", "slots", "turns", "first", "lens", "tables", "idx", "lse"):
            odd = torch.zeros(x.numel() + 1, dtype=x.dtype)[1:].view(x.shape)
            left({**a, n: odd})  # not 16-byte aligned
    for n, least in LEAST[name].items():
        flat = a[n].reshape(-1)
        assert flat.numel() == least
        left({**a, n: flat[:-1]})
        s.seen = None
        assert call(*{**a, n: torch.cat([flat, flat])}.values()) == 0  # more is fine
    # (a size of page that the library refuses is left to it)
    for bad in (dict(page_size=0), dict(page_size=8192), dict(kv_heads=0), dict(kv_heads=65), dict(pages=-1)):
        left({**a, "cfg": dsa.kv_cfg(**{**dict(pages=PAGES, page_size=PAGE, kv_heads=KV), **bad})})
    left({**a, "cfg": dsa.cache_cfg(pages=PAGES, page_size=PAGE, kv_heads=KV)})
    wrong = dsa.kv_cfg(pages=PAGES, page_size=PAGE, kv_heads=KV)
    wrong.dtype = 2
    left({**a, "cfg": wrong})
    for n in ("scale", "gain"):
        if n in a:
            left({**a, n: 1})
            left({**a, n: "1"})
    for n in ("lead", "trail"):
        if n in a:
            left({**a, n: True})
            left({**a, n: 1.0})
            left({**a, n: 1 << 31})
    if name == "append":
        left({**a, "neighbours": 1})


def test_shapes(calls):
    m, s = calls
    s.status = 0
    x = dict(dtype=torch.bfloat16)

    def left(name, **kw):
        s.seen = None
        assert getattr(m, "kv_" + name)(*{**good(name), **kw}.values()) is None and s.seen is None
    for name in NAMES[1:]:
        left(name, q=torch.zeros(T, H * 128, **x))
        left(name, q=torch.zeros(T, H, 64, **x))
        left(name, q=torch.zeros(H, T, 128, **x).transpose(0, 1))
        left(name, q=torch.zeros(1, H, 128, **x).expand(T, H, 128))
        left(name, q=torch.zeros(T, H * 128 + 4, **x)[:, :H * 128].view(T, H, 128))  # 8 bytes from row to row
        left(name, tables=ints(R * W))
        left(name, tables=ints(R + 1, W))
        left(name, lens=ints(R + 1))
    for name in ("select", "blocks"):
        left(name, idx=ints(T + 1, KV, SEL))
        left(name, idx=ints(T, KV + 1, SEL))
        left(name, idx=ints(T * KV, SEL))
    for n in ("k", "v"):
        for y in (torch.zeros(T + 1, KV, 128, **x), torch.zeros(T, KV + 1, 128, **x), torch.zeros(T, KV, 64, **x),
                  torch.zeros(T, 128, KV, **x).transpose(1, 2), torch.zeros(T, KV, 128)):
            left("append", **{n: y})
    left("append", q=torch.zeros(T + 1, H, 128, **x))


def test_strides_and_empty_calls(calls):
    m, s = calls
    s.status = 0
    x = dict(dtype=torch.bfloat16)
    fused = torch.zeros(T, H + 2 * KV, 128, **x)
    a = good("append")
    a.update(q=fused[:, :H], k=fused[:, H:H + KV], v=fused[:, H + KV:])
    assert m.kv_append(*a.values()) == 0
    assert s.seen[6:12] == (a["q"].data_ptr(), (H + 2 * KV) * 128, a["k"].data_ptr(), (H + 2 * KV) * 128, a["v"].data_ptr(),
                            (H + 2 * KV) * 128)
    for name, at in (("attention", 8), ("select", 10), ("blocks", 9)):
        a = good(name)
        a["q"] = fused[:, :H]
        assert getattr(m, "kv_" + name)(*a.values()) == 0 and s.seen[at] == (H + 2 * KV) * 128
    none = dict(lens=ints(0), first=ints(1), tables=ints(0, W))
    for name in NAMES[1:]:
        a = {**good(name), **none}
        assert getattr(m, "kv_" + name)(*a.values()) == 0 and s.seen[3] == 0
    a = good("append")
    a.update(q=None, k=torch.zeros(0, KV, 128, **x), v=torch.zeros(0, KV, 128, **x), ends=ints(0), slots=ints(0))
    assert m.kv_append(*a.values()) == 0 and s.seen[1] == 0


def test_binding_uses_it(calls, monkeypatch):
    m, s = calls
    monkeypatch.setattr(K, "_calls", m)
    for name in NAMES:
        a = good(name)
        f = getattr(K, CALLS[name])
        s.seen, s.status = None, 0
        f(*a.values())
        assert list(s.seen) == expected(name, a)
        s.status = 3
        with pytest.raises(dsa.DsaSelectError) as e:
            f(*a.values())
        assert e.value.status == 3
        with pytest.raises((TypeError, ValueError)):  # the binding's own checks: not CUDA tensors
            f(*{**a, "cfg": dsa.kv_cfg(pages=PAGES, page_size=0, kv_heads=KV)}.values())
