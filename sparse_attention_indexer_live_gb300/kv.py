"""The paged 16-bit key/value cache: the binding of the dsa_kv_* calls
(include/dsa_select.h has the layout, the arguments and the limits) and
`PagedKV`, which owns a cache with its block tables and takes steps on it.

As in cache.py, every argument is checked here before a pointer reaches the C
ABI: TypeError for a wrong type, ValueError for a wrong device, layout or size.
The work runs on the current stream of the tensors' own device unless a stream
of that device is given.  Ordinary calls are checked and made by the module built
from csrc/cache_calls.cpp, as cache.py's are (an append takes the host 4.9 us so, 15.3
through ctypes).
"""
from __future__ import annotations

import contextlib
import ctypes
import math
import warnings

import torch

from . import binding
from .cache import _I32, _count, _device_of, _load_calls, _made, _need, cache_cfg, dsa_cache_plan, refusal

_DIM = 128
_TYPES = {torch.bfloat16: 0, torch.float16: 1}
_DTYPE = {code: t for t, code in _TYPES.items()}


class dsa_kv_cfg(ctypes.Structure):
    _fields_ = [("pages", ctypes.c_int32), ("page_size", ctypes.c_int32), ("kv_heads", ctypes.c_int32),
                ("dtype", ctypes.c_int32)]


def kv_cfg(*, pages, page_size=64, kv_heads=1, dtype=torch.bfloat16) -> dsa_kv_cfg:
    """A cache's shape: `pages` pages of `page_size` (16, 32, 64 or 128)
    positions of `kv_heads` key/value heads, in bf16 or f16."""
    if dtype not in _TYPES:
        raise TypeError(f"dtype: {dtype}, expected torch.bfloat16 or torch.float16")
    for name, n in dict(pages=pages, page_size=page_size, kv_heads=kv_heads).items():
        if not -1 << 31 <= n < 1 << 31:  # the structure would keep its low 32 bits
            raise ValueError(f"{name}: {n} is more than 32 bits hold")
    return dsa_kv_cfg(pages, page_size, kv_heads, _TYPES[dtype])


def rotary_turns(inv_freq, device=None):
    """The `turns` of dsa_kv_append for frequencies inv_freq [rotary / 2] in
    radians a position (taken in f64): int64 fractions of 2^64 of a turn."""
    f = inv_freq if isinstance(inv_freq, torch.Tensor) else torch.tensor(inv_freq, dtype=torch.float64)
    device = f.device if device is None else device
    whole = 1 << 64
    turns = [round(math.fmod(x / (2 * math.pi), 1.0) * whole) % whole for x in f.double().tolist()]
    return torch.tensor([t - whole if t >= whole >> 1 else t for t in turns], dtype=torch.int64, device=device)


# ---------------------------------------------------------------------------
# argument checks

def _cfg(cfg):
    if type(cfg) is not dsa_kv_cfg:
        raise TypeError(f"cfg: expected a dsa_kv_cfg, got {type(cfg).__name__}")
    if cfg.dtype not in _DTYPE:
        raise ValueError(f"cfg: dtype {cfg.dtype}")
    return _DTYPE[cfg.dtype]


def _flag(name, x):
    if not isinstance(x, (bool, int)):
        raise TypeError(f"{name}: expected a truth value, got {type(x).__name__}")
    return int(bool(x))


def _number(name, x):
    if not isinstance(x, int) or isinstance(x, bool):
        raise TypeError(f"{name}: expected an int, got {type(x).__name__}")
    if not -1 << 31 <= x < 1 << 31:
        raise ValueError(f"{name}: {x} is more than 32 bits hold")
    return x


def _rows(name, t, dtype, heads, dev):
    """t [tokens, heads, 128] (any number of heads, if None) whose heads and
    dims are packed: (tokens, heads, elements from token to token)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor, got {type(t).__name__}")
    if t.dtype is not dtype:
        raise TypeError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name}: must be a CUDA tensor (got device {t.device})")
    if dev is not None and t.get_device() != dev:
        raise ValueError(f"{name}: on cuda:{t.get_device()}, the other tensors are on cuda:{dev}")
    if t.dim() != 3 or t.shape[2] != _DIM or (heads is not None and t.shape[1] != heads):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected [tokens, {heads or 'heads'}, {_DIM}]")
    T, H, _ = t.shape
    st = t.stride()
    if T and H and (st[2] != 1 or (H > 1 and st[1] != _DIM)):
        raise ValueError(f"{name}: strides {st}, a token's heads and dims must be packed")
    if T <= 1:
        return T, H, H * _DIM
    if st[0] < H * _DIM:
        raise ValueError(f"{name}: strides {st}, tokens overlap")
    if st[0] % 8:
        raise ValueError(f"{name}: strides {st}, a token's must be a multiple of 8")
    return T, H, st[0]


def _aligned(name, t):
    if t.data_ptr() % 16:
        raise ValueError(f"{name}: must be 16-byte aligned")


def _pool(cfg, name, t, dtype, dev, positions):
    _need(name, t, dtype, cfg.pages * positions * cfg.kv_heads * _DIM, dev)
    _aligned(name, t)


def _table(tables, R, dev):
    _need("tables", tables, _I32, 0, dev)
    if tables.dim() != 2 or (R is not None and tables.shape[0] != R):
        raise ValueError(f"tables: shape {tuple(tables.shape)}, expected [{'requests' if R is None else R}, pages per request]")
    return _count("tables", tables.shape[1])


_calls = None  # the module of ordinary calls, once the library is loaded; False where there is none


def _bound(functions=None, host=False):
    """The module of ordinary calls, bound to the library's functions (or those
    given, with tensors of the host in place of a device's)."""
    m = _load_calls()
    if functions is None:
        L = binding.load()
        functions = [getattr(L, "dsa_kv_" + n) for n in ("append", "attention", "select", "block_attention")]
    m.bind_kv(dsa_kv_cfg, host, *(ctypes.cast(f, ctypes.c_void_p).value for f in functions))
    return m


def _call(name, dev, stream, *args):
    """The library's `name`(*args, stream) with `dev` current."""
    global _calls
    if stream is None:
        s = torch.cuda.current_stream(dev).cuda_stream
    else:
        if stream.device.index != dev:
            raise ValueError(f"stream: of cuda:{stream.device.index}, the tensors are on cuda:{dev}")
        s = stream.cuda_stream
    fn = getattr(binding.load(), name)
    if _calls is None:
        try:
            _calls = _bound()
        except (OSError, ImportError) as e:
            _calls = False
            warnings.warn(f"cache_calls is not used, the cache's calls take a few us more each: {e}", RuntimeWarning,
                          stacklevel=3)
    with torch.cuda.device(dev):
        binding._check(fn(*args, s), name)


def _bytes(name, cfg, *args):
    n = ctypes.c_size_t(0)
    binding._check(getattr(binding.load(), name)(ctypes.byref(cfg), *args, ctypes.byref(n)), name)
    return int(n.value)


def _step_sizes(cfg, q, tables):
    """(tokens, heads, requests, table width) for a workspace's size."""
    _cfg(cfg)
    for name, t, dims in (("q", q, 3), ("tables", tables, 2)):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name}: expected a torch.Tensor, got {type(t).__name__}")
        if t.dim() != dims:
            raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {dims} dims")
    return (_count("q", q.shape[0]), _count("q", q.shape[1]), _count("tables", tables.shape[0]),
            _count("tables", tables.shape[1]))


def _step(cfg, q, first, lens, tables, workspace):
    """What the calls of a step share: (type, device, tokens, heads, stride, requests, table width)."""
    dtype = _cfg(cfg)
    T, H, stride = _rows("q", q, dtype, None, None)
    dev = q.get_device()
    _aligned("q", q)
    _need("lens", lens, _I32, 0, dev)
    R = lens.numel()
    _need("first", first, _I32, R + 1, dev)
    P = _table(tables, R, dev)
    _need("workspace", workspace, torch.uint8, 0, dev)
    _aligned("workspace", workspace)
    return dtype, dev, _count("q", T), _count("q", H), stride, _count("lens", R), P


def _lists(cfg, idx, T, dev):
    """select of idx [tokens, kv_heads, select]."""
    _need("idx", idx, _I32, 0, dev)
    if idx.dim() != 3 or idx.shape[0] != T or idx.shape[1] != cfg.kv_heads:
        raise ValueError(f"idx: shape {tuple(idx.shape)}, expected [{T}, {cfg.kv_heads}, select]")
    return _count("idx", idx.shape[2])


# ---------------------------------------------------------------------------
# the calls

def dsa_kv_append(cfg: dsa_kv_cfg, q, k, v, ends, slots, turns, neighbours: bool, gain: float, q_out, k_cache, v_cache,
                  means, stream=None):
    """Rotate and store a step's rows: q [T, H, 128] (or None) to q_out, k and
    v [T, kv_heads, 128] to the slots [T] int32 of k_cache and v_cache; ends
    [T] int32 the positions + 1, turns [rotary / 2] int64 (rotary_turns).
    means (or None): the mean keys of the pages that this fills."""
    if stream is None and _calls and _made(
            _calls.kv_append(cfg, q, k, v, ends, slots, turns, neighbours, gain, q_out, k_cache, v_cache, means),
            "dsa_kv_append"):
        return
    dtype = _cfg(cfg)
    dev = _device_of("slots", slots, _I32)
    T = _count("slots", slots.numel())
    _need("ends", ends, _I32, T, dev)
    Tk, _, ks = _rows("k", k, dtype, cfg.kv_heads, dev)
    Tv, _, vs = _rows("v", v, dtype, cfg.kv_heads, dev)
    Tq, H, qs = (T, 0, 0) if q is None else _rows("q", q, dtype, None, dev)
    for name, n in (("k", Tk), ("v", Tv), ("q", Tq)):
        if n != T:
            raise ValueError(f"{name}: {n} tokens, slots has {T}")
    for name, t in (("k", k), ("v", v), ("q", q)):
        if t is not None:
            _aligned(name, t)
    if q is not None:
        _need("q_out", q_out, dtype, T * H * _DIM, dev)
        _aligned("q_out", q_out)
    _need("turns", turns, torch.int64, 0, dev)
    _pool(cfg, "k_cache", k_cache, dtype, dev, cfg.page_size)
    _pool(cfg, "v_cache", v_cache, dtype, dev, cfg.page_size)
    if means is not None:
        _pool(cfg, "means", means, dtype, dev, 1)
    _call("dsa_kv_append", dev, stream, ctypes.byref(cfg), T, _count("q", H), _count("turns", 2 * turns.numel()),
          _flag("neighbours", neighbours), gain, None if q is None else q.data_ptr(), qs, k.data_ptr(), ks, v.data_ptr(),
          vs, ends.data_ptr(), slots.data_ptr(), turns.data_ptr(), None if q is None else q_out.data_ptr(),
          k_cache.data_ptr(), v_cache.data_ptr(), None if means is None else means.data_ptr())


def dsa_kv_attention_workspace(cfg: dsa_kv_cfg, q, tables) -> int:
    """Workspace bytes of dsa_kv_attention for q [T, H, 128] and tables [R, P]."""
    return _bytes("dsa_kv_attention_workspace", cfg, *_step_sizes(cfg, q, tables))


def dsa_kv_attention(cfg: dsa_kv_cfg, k_cache, v_cache, q, first, lens, tables, scale: float, workspace, o, lse,
                     stream=None):
    """Causal attention of a step's tokens q [T, H, 128], request after
    request: first [R + 1], lens [R], tables [R, P] int32 (a plan's); writes o
    [T, H, 128] and lse [T, H] f32."""
    if stream is None and _calls and _made(
            _calls.kv_attention(cfg, k_cache, v_cache, q, first, lens, tables, scale, workspace, o, lse),
            "dsa_kv_attention"):
        return
    dtype, dev, T, H, stride, R, P = _step(cfg, q, first, lens, tables, workspace)
    _pool(cfg, "k_cache", k_cache, dtype, dev, cfg.page_size)
    _pool(cfg, "v_cache", v_cache, dtype, dev, cfg.page_size)
    _need("o", o, dtype, T * H * _DIM, dev)
    _aligned("o", o)
    _need("lse", lse, torch.float32, T * H, dev)
    _call("dsa_kv_attention", dev, stream, ctypes.byref(cfg), T, H, R, P, k_cache.data_ptr(), v_cache.data_ptr(),
          q.data_ptr(), stride, first.data_ptr(), lens.data_ptr(), tables.data_ptr(), scale, workspace.data_ptr(),
          workspace.numel(), o.data_ptr(), lse.data_ptr())


def dsa_kv_select_workspace(cfg: dsa_kv_cfg, q, tables) -> int:
    """Workspace bytes of dsa_kv_select for q [T, H, 128] and tables [R, P]."""
    return _bytes("dsa_kv_select_workspace", cfg, *_step_sizes(cfg, q, tables))


def dsa_kv_select(cfg: dsa_kv_cfg, means, q, first, lens, tables, lead: int, trail: int, workspace, idx, stream=None):
    """The pages that each token's queries score highest by the mean keys,
    the first `lead` and the last `trail` taken always: idx [T, kv_heads,
    select] int32, ascending page numbers of the request, then -1."""
    if stream is None and _calls and _made(
            _calls.kv_select(cfg, means, q, first, lens, tables, lead, trail, workspace, idx), "dsa_kv_select"):
        return
    dtype, dev, T, H, stride, R, P = _step(cfg, q, first, lens, tables, workspace)
    _pool(cfg, "means", means, dtype, dev, 1)
    n = _lists(cfg, idx, T, dev)
    _call("dsa_kv_select", dev, stream, ctypes.byref(cfg), T, H, R, P, n, _number("lead", lead), _number("trail", trail),
          means.data_ptr(), q.data_ptr(), stride, first.data_ptr(), lens.data_ptr(), tables.data_ptr(),
          workspace.data_ptr(), workspace.numel(), idx.data_ptr())


def dsa_kv_block_attention_workspace(cfg: dsa_kv_cfg, q, idx, tables) -> int:
    """Workspace bytes of dsa_kv_block_attention for q [T, H, 128], idx [T, kv_heads, select] and tables [R, P]."""
    sizes = _step_sizes(cfg, q, tables)
    if not isinstance(idx, torch.Tensor):
        raise TypeError(f"idx: expected a torch.Tensor, got {type(idx).__name__}")
    if idx.dim() != 3:
        raise ValueError(f"idx: shape {tuple(idx.shape)}, expected 3 dims")
    return _bytes("dsa_kv_block_attention_workspace", cfg, *sizes, _count("idx", idx.shape[2]))


def dsa_kv_block_attention(cfg: dsa_kv_cfg, k_cache, v_cache, q, idx, first, lens, tables, scale: float, workspace, o,
                           lse, stream=None):
    """dsa_kv_attention to the pages idx [T, kv_heads, select] int32 (strictly
    ascending, then -1; a selection of dsa_kv_select's) lists."""
    if stream is None and _calls and _made(
            _calls.kv_blocks(cfg, k_cache, v_cache, q, idx, first, lens, tables, scale, workspace, o, lse),
            "dsa_kv_block_attention"):
        return
    dtype, dev, T, H, stride, R, P = _step(cfg, q, first, lens, tables, workspace)
    _pool(cfg, "k_cache", k_cache, dtype, dev, cfg.page_size)
    _pool(cfg, "v_cache", v_cache, dtype, dev, cfg.page_size)
    n = _lists(cfg, idx, T, dev)
    _need("o", o, dtype, T * H * _DIM, dev)
    _aligned("o", o)
    _need("lse", lse, torch.float32, T * H, dev)
    _call("dsa_kv_block_attention", dev, stream, ctypes.byref(cfg), T, H, R, P, n, k_cache.data_ptr(), v_cache.data_ptr(),
          q.data_ptr(), stride, idx.data_ptr(), first.data_ptr(), lens.data_ptr(), tables.data_ptr(), scale,
          workspace.data_ptr(), workspace.numel(), o.data_ptr(), lse.data_ptr())


def dsa_kv_status(device=None) -> int:
    """DSA_OK, or DSA_ERR_TIMEOUT once after an attention kernel over the cache
    gave up a wait on `device` (the current one, if None), which is synchronised."""
    with torch.cuda.device(device) if device is not None else contextlib.nullcontext():
        return int(binding.load().dsa_kv_status())


# ---------------------------------------------------------------------------
# a cache with its tables

class PagedKV:
    """A 16-bit cache of one layer with the pages of up to `requests` requests.

    step(lens, fresh, tokens) plans a step (dsa_cache_plan); append(q, k, v)
    then stores the step's rows, rotated by inv_freq where that is given, and
    returns the rotated queries; attend(q, scale) attends to everything before
    each token, attend_pages(q, idx, scale) to the pages that select(q, ...)
    chose.  Nothing here waits for the device but ok(), which reads the step's
    status.
    """

    def __init__(self, *, requests, pages, pages_per_request, page_size=64, kv_heads=1, dtype=torch.bfloat16,
                 inv_freq=(), neighbours=False, gain=1.0, device=0):
        self.cfg = kv_cfg(pages=pages, page_size=page_size, kv_heads=kv_heads, dtype=dtype)
        self._plan = cache_cfg(pages=pages, page_size=page_size)
        dev = torch.device("cuda", device)
        i32 = dict(dtype=_I32, device=dev)
        # zeros: what a page holds past a request's end is cheap to ignore unless it is a NaN
        self.k, self.v = torch.zeros((2, pages, page_size, kv_heads, _DIM), dtype=dtype, device=dev).unbind(0)
        self.means = torch.zeros((pages, kv_heads, _DIM), dtype=dtype, device=dev)
        self.turns = rotary_turns(inv_freq, dev)
        self.neighbours, self.gain = neighbours, gain
        self.tables = torch.full((requests, pages_per_request), -1, **i32)
        self.held = torch.zeros(requests, **i32)
        self.free_pages = torch.arange(pages - 1, -1, -1, **i32)
        self.free_count = torch.full((1,), pages, **i32)
        self.first = torch.zeros(requests + 1, **i32)
        self.lens = torch.zeros(requests, **i32)
        self.status = torch.zeros(4, **i32)
        self._maps = [torch.empty((3, 0), **i32)]
        self.token_req, self.ends, self.slots = self._maps[0].unbind(0)

    def step(self, lens, fresh, tokens: int):
        """Plan a step of at most `tokens` tokens: lens [requests] int32 after
        it, the last fresh[r] of them new.  A graph that captured steps of one
        size stays good when other sizes follow."""
        if tokens < 0:
            raise ValueError(f"tokens: {tokens}")
        if tokens != self.slots.numel():
            if tokens > self._maps[-1].shape[1]:
                room = max(tokens, 2 * self._maps[-1].shape[1])
                self._maps.append(torch.empty((3, (room + 63) // 64 * 64), dtype=_I32, device=self.tables.device))
            self.token_req, self.ends, self.slots = self._maps[-1][:, :tokens].unbind(0)
        dsa_cache_plan(self._plan, lens, fresh, self.tables, self.held, self.free_pages, self.free_count, self.first,
                       self.token_req, self.ends, self.slots, self.status)
        self.lens.copy_(lens)

    def ok(self):
        """Wait for the last step's status; RuntimeError when it could not be taken."""
        refusal(self.status)

    def append(self, q, k, v):
        """Store the step's rows k and v [tokens, kv_heads, 128]; the rotated q
        [tokens, heads, 128], zeros in rows past the step's last token."""
        out = torch.zeros(q.shape, dtype=q.dtype, device=q.device)
        dsa_kv_append(self.cfg, q, k, v, self.ends, self.slots, self.turns, self.neighbours, self.gain, out, self.k,
                      self.v, self.means)
        return out

    def _out(self, q):
        return (torch.zeros(q.shape, dtype=q.dtype, device=q.device),
                torch.full(q.shape[:2], -math.inf, dtype=torch.float32, device=q.device))

    def _space(self, n):
        return torch.empty(n, dtype=torch.uint8, device=self.tables.device)

    def attend(self, q, scale: float):
        """(o, lse) of the step's tokens q [tokens, heads, 128] over everything
        before them; zeros and -inf for rows past the step's last token."""
        o, lse = self._out(q)
        ws = self._space(dsa_kv_attention_workspace(self.cfg, q, self.tables))
        dsa_kv_attention(self.cfg, self.k, self.v, q, self.first, self.lens, self.tables, scale, ws, o, lse)
        return o, lse

    def select(self, q, pages: int, *, lead=1, trail=1):
        """idx [tokens, kv_heads, pages]: the pages each token's queries score highest."""
        idx = torch.full((q.shape[0], self.cfg.kv_heads, pages), -1, dtype=_I32, device=q.device)
        ws = self._space(dsa_kv_select_workspace(self.cfg, q, self.tables))
        dsa_kv_select(self.cfg, self.means, q, self.first, self.lens, self.tables, lead, trail, ws, idx)
        return idx

    def attend_pages(self, q, idx, scale: float):
        """attend() to the pages of idx [tokens, kv_heads, pages]."""
        o, lse = self._out(q)
        ws = self._space(dsa_kv_block_attention_workspace(self.cfg, q, idx, self.tables))
        dsa_kv_block_attention(self.cfg, self.k, self.v, q, idx, self.first, self.lens, self.tables, scale, ws, o, lse)
        return o, lse
