"""The paged 4-bit key/value cache and the sparse attention over it: the
binding of the dsa_cache_* calls (include/dsa_select.h has the record layout,
the arguments and the limits) and `PagedCache`, which owns a cache with its
block tables and takes steps on it.

As in binding.py, every argument is checked here before a pointer reaches the
C ABI: TypeError for a wrong type, ValueError for a wrong device, layout or
size.  The work runs on the current stream of the tensors' own device unless a
stream of that device is given.

A decode step's kernels take a few microseconds, and so do a dozen tensors looked
at from Python.  Once the library is loaded an ordinary call -- nothing wrong with
it, the tensors on the current device, no stream given -- is checked and made by
the module built from csrc/cache_calls.cpp (two plans 17 -> 5.7 us, an attention
call 7.9 -> 2.8, a read 5.8 -> 2.6); what that returns None for is checked and
made, or refused with the reason, here.  Where the module was not built, every
call is.
"""
from __future__ import annotations

import contextlib
import ctypes
import importlib.machinery
import importlib.util
import os
import warnings

import torch

from . import binding
from .build import calls_path

RECORD_BYTES = 144
PLAN_OK, PLAN_NO_PAGES, PLAN_TABLE_WIDTH, PLAN_TOKENS, PLAN_BAD_LENGTHS = range(5)

_DIM = 128
_ROW_TYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
_I32 = torch.int32


class dsa_cache_cfg(ctypes.Structure):
    _fields_ = [("pages", ctypes.c_int32), ("page_size", ctypes.c_int32), ("kv_heads", ctypes.c_int32),
                ("k_shift", ctypes.c_int32), ("v_shift", ctypes.c_int32)]


def cache_cfg(*, pages, page_size=64, kv_heads=1, k_shift=0, v_shift=0) -> dsa_cache_cfg:
    """A cache's shape: `pages` pages of `page_size` (a power of two) positions
    of `kv_heads` key/value heads; keys are stored divided by 2^k_shift, values
    by 2^v_shift."""
    values = dict(pages=pages, page_size=page_size, kv_heads=kv_heads, k_shift=k_shift, v_shift=v_shift)
    for name, n in values.items():
        if not -1 << 31 <= n < 1 << 31:  # the structure would keep its low 32 bits
            raise ValueError(f"{name}: {n} is more than 32 bits hold")
    return dsa_cache_cfg(**values)


def dsa_cache_bytes(cfg: dsa_cache_cfg) -> int:
    """Bytes of the cache `cfg` describes."""
    _cfg(cfg)
    n = ctypes.c_size_t(0)
    binding._check(binding.load().dsa_cache_bytes(ctypes.byref(cfg), ctypes.byref(n)), "dsa_cache_bytes")
    return int(n.value)


# ---------------------------------------------------------------------------
# argument checks

def _refuse(name, t, dtype, numel, dev):
    """Raise for `t`, which is not a contiguous CUDA tensor of `dtype` on
    device `dev` (any, if None) with at least `numel` elements."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor, got {type(t).__name__}")
    if t.dtype is not dtype:
        raise TypeError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name}: must be a CUDA tensor (got device {t.device})")
    if dev is not None and t.get_device() != dev:
        raise ValueError(f"{name}: on cuda:{t.get_device()}, the other tensors are on cuda:{dev}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    if t.numel() < numel:
        raise ValueError(f"{name}: {t.numel()} elements, at least {numel} needed")
    raise ValueError(f"{name}: not usable")


def _need(name, t, dtype, numel, dev):
    """Check `t` (see _refuse; `dev` >= 0)."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == dev and t.is_contiguous()
            and t.numel() >= numel):
        _refuse(name, t, dtype, numel, dev)


def _device_of(name, t, dtype):
    """The device of `t`, a contiguous CUDA tensor of `dtype`."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.is_cuda and t.is_contiguous()):
        _refuse(name, t, dtype, 0, None)
    return t.get_device()


def _cfg(cfg):
    if type(cfg) is not dsa_cache_cfg:
        raise TypeError(f"cfg: expected a dsa_cache_cfg, got {type(cfg).__name__}")


def _cache(cfg, cache, dev):
    _cfg(cfg)
    need = cfg.pages * cfg.page_size * cfg.kv_heads * RECORD_BYTES  # limits: the C ABI's
    _need("cache", cache, torch.uint8, need, dev)


def _row_type(name, t, types):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor, got {type(t).__name__}")
    code = _ROW_TYPES.get(t.dtype, 99)
    if code >= types:
        want = ", ".join(str(d) for d, c in _ROW_TYPES.items() if c < types)
        raise TypeError(f"{name}: dtype {t.dtype}, expected one of {want}")
    return code


_calls = None  # the module of ordinary calls, once the library is loaded; False where there is none


def _load_calls(functions=None, host=False):
    """The module of ordinary calls, bound to the library's functions (or those
    given, with tensors of the host in place of a device's)."""
    path = calls_path()
    if path is None or not os.path.exists(path):
        raise OSError(f"{path} has not been built: run build()")
    loader = importlib.machinery.ExtensionFileLoader("cache_calls", path)
    m = importlib.util.module_from_spec(importlib.util.spec_from_file_location("cache_calls", path, loader=loader))
    loader.exec_module(m)
    if functions is None:
        L = binding.load()
        functions = [getattr(L, "dsa_cache_" + n) for n in ("bytes", "plan", "write", "read", "attention",
                                                            "attention_prompt")]
    m.bind(dsa_cache_cfg, host, *(ctypes.cast(f, ctypes.c_void_p).value for f in functions))
    return m


def _made(rc, name):
    """Whether the module of ordinary calls made the call (rc: None or a status)."""
    if rc:
        raise binding.DsaSelectError(rc, name)
    return rc is not None


def _count(name, n):
    if n >= 1 << 31:
        raise ValueError(f"{name}: {n} is more than 32 bits hold")
    return n


def _call(name, dev, stream, *args):
    """The library's `name`(*args, stream) with `dev` current: the C ABI launches on the current device."""
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
            _calls = _load_calls()
        except (OSError, ImportError) as e:
            _calls = False
            warnings.warn(f"cache_calls is not used, the cache's calls take a few us more each: {e}", RuntimeWarning,
                          stacklevel=3)
    with torch.cuda.device(dev):
        binding._check(fn(*args, s), name)


# ---------------------------------------------------------------------------
# the calls

def dsa_cache_plan(cfg: dsa_cache_cfg, lens, fresh, tables, held, free_pages, free_count, first, token_req, ends,
                   slots, status, stream=None):
    """One step's pages, block tables and slots from request lengths: lens and
    fresh [R] int32; tables [R, P], held [R], free_pages and free_count [1]
    updated; first [R + 1], token_req, ends and slots [T] and status [4]
    written.  status[0] is one of the PLAN_* codes; a step that cannot be taken
    changes no state."""
    if stream is None and _calls and _made(
            _calls.plan(cfg, lens, fresh, tables, held, free_pages, free_count, first, token_req, ends, slots, status),
            "dsa_cache_plan"):
        return
    _cfg(cfg)
    dev = _device_of("lens", lens, _I32)
    R = lens.numel()
    _need("token_req", token_req, _I32, 0, dev)
    T = token_req.numel()
    for name, x, n in (("fresh", fresh, R), ("tables", tables, 0), ("held", held, R), ("free_pages", free_pages, 0),
                       ("free_count", free_count, 1), ("first", first, R + 1), ("ends", ends, T), ("slots", slots, T),
                       ("status", status, 4)):
        _need(name, x, _I32, n, dev)
    if tables.dim() != 2 or tables.shape[0] != R:
        raise ValueError(f"tables: shape {tuple(tables.shape)}, expected [{R}, pages per request]")
    _call("dsa_cache_plan", dev, stream, ctypes.byref(cfg), _count("lens", R), _count("tables", tables.shape[1]),
          _count("token_req", T), _count("free_pages", free_pages.numel()),
          lens.data_ptr(), fresh.data_ptr(), tables.data_ptr(), held.data_ptr(), free_pages.data_ptr(),
          free_count.data_ptr(), first.data_ptr(), token_req.data_ptr(), ends.data_ptr(), slots.data_ptr(),
          status.data_ptr())


def _strided_rows(name, t, T, H, dev):
    """[T, H, 128] rows whose heads and dims are packed; returns the token stride."""
    if t.get_device() != dev:
        if not t.is_cuda:
            raise ValueError(f"{name}: must be a CUDA tensor (got device {t.device})")
        raise ValueError(f"{name}: on cuda:{t.get_device()}, the other tensors are on cuda:{dev}")
    if t.shape != (T, H, _DIM):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected [{T}, {H}, {_DIM}]")
    st = t.stride()
    if T and (st[2] != 1 or (H > 1 and st[1] != _DIM)):
        raise ValueError(f"{name}: strides {st}, a token's heads and dims must be packed")
    if T <= 1:
        return H * _DIM
    if st[0] < H * _DIM:
        raise ValueError(f"{name}: strides {st}, tokens overlap")
    return st[0]


def dsa_cache_write(cfg: dsa_cache_cfg, k, v, slots, cache, stream=None):
    """Store k and v [T, kv_heads, 128] (bf16, f16 or f32; any token stride) in
    4 bits at the records slots [T] int32 names; -1 stores nothing."""
    if stream is None and _calls and _made(_calls.write(cfg, k, v, slots, cache), "dsa_cache_write"):
        return
    code = _row_type("k", k, 3)
    if not isinstance(v, torch.Tensor) or v.dtype is not k.dtype:
        raise TypeError(f"v: expected a tensor of {k.dtype} like k")
    dev = _device_of("slots", slots, _I32)
    _cache(cfg, cache, dev)
    T = _count("slots", slots.numel())
    ks = _strided_rows("k", k, T, cfg.kv_heads, dev)
    vs = _strided_rows("v", v, T, cfg.kv_heads, dev)
    _call("dsa_cache_write", dev, stream, ctypes.byref(cfg), T, code, k.data_ptr(), v.data_ptr(), ks, vs,
          slots.data_ptr(), cache.data_ptr())


def dsa_cache_read(cfg: dsa_cache_cfg, cache, slots, k, v, stream=None):
    """Read the records slots [T] int32 names into k and v [T, kv_heads, 128]
    (bf16, f16 or f32); zeros for a slot outside the cache."""
    if stream is None and _calls and _made(_calls.read(cfg, cache, slots, k, v), "dsa_cache_read"):
        return
    code = _row_type("k", k, 3)
    dev = _device_of("slots", slots, _I32)
    _cache(cfg, cache, dev)
    T = _count("slots", slots.numel())
    n = T * cfg.kv_heads * _DIM
    _need("k", k, k.dtype, n, dev)
    _need("v", v, k.dtype, n, dev)
    _call("dsa_cache_read", dev, stream, ctypes.byref(cfg), T, code, cache.data_ptr(), slots.data_ptr(),
          k.data_ptr(), v.data_ptr())


def _attention_args(cfg, cache, q, idx, o, lse):
    """(type code, tokens, heads, select, device) of an attention call's tensors."""
    code = _row_type("q", q, 2)
    dev = _device_of("q", q, q.dtype)
    if q.dim() != 3 or q.shape[2] != _DIM:
        raise ValueError(f"q: shape {tuple(q.shape)}, expected [tokens, heads, {_DIM}]")
    T, H, _ = q.shape
    _cache(cfg, cache, dev)
    _need("idx", idx, _I32, 0, dev)
    if idx.dim() != 2 or idx.shape[0] != T:
        raise ValueError(f"idx: shape {tuple(idx.shape)}, expected [{T}, select]")
    _need("o", o, q.dtype, T * H * _DIM, dev)
    _need("lse", lse, torch.float32, T * H, dev)
    return code, _count("q", T), _count("q", H), _count("idx", idx.shape[1]), dev


def dsa_cache_attention(cfg: dsa_cache_cfg, cache, q, idx, token_req, tables, scale: float, o, lse, stream=None):
    """Sparse attention over the cache: q [T, H, 128] (bf16 or f16), idx
    [T, Kc] int32 positions (below 0: unused) of request token_req[t], whose
    pages are tables[request]; writes o [T, H, 128] (q's type) and lse [T, H]
    f32."""
    if stream is None and _calls and _made(
            _calls.attention(cfg, cache, q, idx, token_req, tables, scale, o, lse), "dsa_cache_attention"):
        return
    code, T, H, Kc, dev = _attention_args(cfg, cache, q, idx, o, lse)
    _need("token_req", token_req, _I32, T, dev)
    _need("tables", tables, _I32, 0, dev)
    if tables.dim() != 2:
        raise ValueError(f"tables: shape {tuple(tables.shape)}, expected [requests, pages per request]")
    R, P = (_count("tables", n) for n in tables.shape)
    _call("dsa_cache_attention", dev, stream, ctypes.byref(cfg), T, H, Kc, R, P, code, cache.data_ptr(),
          q.data_ptr(), idx.data_ptr(), token_req.data_ptr(), tables.data_ptr(), scale, o.data_ptr(), lse.data_ptr())


def dsa_cache_attention_prompt_workspace(cfg: dsa_cache_cfg, q, idx) -> int:
    """Workspace bytes of dsa_cache_attention_prompt for q [T, H, 128] and idx [T, Kc]."""
    _cfg(cfg)
    for name, t, dims in (("q", q, 3), ("idx", idx, 2)):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name}: expected a torch.Tensor, got {type(t).__name__}")
        if t.dim() != dims:
            raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {dims} dims")
    n = ctypes.c_size_t(0)
    binding._check(binding.load().dsa_cache_attention_prompt_workspace(
        ctypes.byref(cfg), _count("q", q.shape[0]), _count("q", q.shape[1]), _count("idx", idx.shape[1]),
        ctypes.byref(n)), "dsa_cache_attention_prompt_workspace")
    return int(n.value)


def dsa_cache_attention_prompt(cfg: dsa_cache_cfg, cache, q, idx, table, scale: float, workspace, o, lse,
                               stream=None):
    """dsa_cache_attention for the tokens of one request's prompt chunk, 128 /
    (H / kv_heads) neighbours at a time over the union of their selections:
    idx rows strictly ascending, then -1; table [P] int32 the request's pages."""
    if stream is None and _calls and _made(
            _calls.prompt(cfg, cache, q, idx, table, scale, workspace, o, lse), "dsa_cache_attention_prompt"):
        return
    code, T, H, Kc, dev = _attention_args(cfg, cache, q, idx, o, lse)
    _need("table", table, _I32, 0, dev)
    _need("workspace", workspace, torch.uint8, 0, dev)
    _call("dsa_cache_attention_prompt", dev, stream, ctypes.byref(cfg), T, H, Kc, _count("table", table.numel()), code,
          cache.data_ptr(), q.data_ptr(), idx.data_ptr(), table.data_ptr(), scale, workspace.data_ptr(),
          workspace.numel(), o.data_ptr(), lse.data_ptr())


def dsa_cache_attention_status(device=None) -> int:
    """DSA_OK, or DSA_ERR_TIMEOUT once after an attention kernel over the cache
    gave up a wait on `device` (the current one, if None), which is synchronised."""
    with torch.cuda.device(device) if device is not None else contextlib.nullcontext():
        return int(binding.load().dsa_cache_attention_status())


# ---------------------------------------------------------------------------
# a cache with its tables

def refusal(status):
    """Wait for a plan's status [4]; RuntimeError with the reason when the step could not be taken."""
    code, short, _, _ = status.tolist()
    if code != PLAN_OK:
        why = {PLAN_NO_PAGES: f"{short} pages short", PLAN_TABLE_WIDTH: "a request needs more pages than its table has",
               PLAN_TOKENS: "more tokens than the step has room for"}.get(code, "lengths or counts out of range")
        raise RuntimeError(f"cache step not taken: {why}")


class PagedCache:
    """A cache of one layer with the pages of up to `requests` requests.

    step(lens, fresh, tokens) plans a step (dsa_cache_plan); store(k, v) then
    writes the step's rows, and attend(q, idx, scale) attends to selected
    positions -- idx from dsa_select_topk on the step's `ends` (row_repeat 1),
    or joined with a window by dsa_combine_window.  Nothing here waits for the
    device but ok(), which reads the step's status.
    """

    def __init__(self, *, requests, pages, pages_per_request, page_size=64, kv_heads=1, k_shift=0, v_shift=0,
                 device=0):
        self.cfg = cache_cfg(pages=pages, page_size=page_size, kv_heads=kv_heads, k_shift=k_shift, v_shift=v_shift)
        i32 = dict(dtype=_I32, device=torch.device("cuda", device))
        self.data = torch.zeros(dsa_cache_bytes(self.cfg), dtype=torch.uint8, device=i32["device"])
        self.tables = torch.full((requests, pages_per_request), -1, **i32)
        self.held = torch.zeros(requests, **i32)
        self.free_pages = torch.arange(pages - 1, -1, -1, **i32)
        self.free_count = torch.full((1,), pages, **i32)
        self.first = torch.zeros(requests + 1, **i32)
        self.status = torch.zeros(4, **i32)
        self._maps = [torch.empty((3, 0), **i32)]
        self.token_req, self.ends, self.slots = self._maps[0].unbind(0)

    def step(self, lens, fresh, tokens: int):
        """Plan a step of at most `tokens` tokens: lens [requests] int32 after
        it, the last fresh[r] of them new.  Sets token_req, ends and slots
        [tokens], first and status.  A graph that captured steps of one size
        stays good when other sizes follow: steps share one memory, and what
        they have outgrown is kept."""
        if tokens < 0:
            raise ValueError(f"tokens: {tokens}")
        if tokens != self.slots.numel():
            if tokens > self._maps[-1].shape[1]:
                room = max(tokens, 2 * self._maps[-1].shape[1])
                self._maps.append(torch.empty((3, (room + 63) // 64 * 64), dtype=_I32, device=self.tables.device))
            self.token_req, self.ends, self.slots = self._maps[-1][:, :tokens].unbind(0)
        dsa_cache_plan(self.cfg, lens, fresh, self.tables, self.held, self.free_pages, self.free_count, self.first,
                       self.token_req, self.ends, self.slots, self.status)

    def ok(self):
        """Wait for the last step's status; RuntimeError when it could not be taken."""
        refusal(self.status)

    def store(self, k, v):
        """Write the step's rows, k and v [tokens, kv_heads, 128]."""
        dsa_cache_write(self.cfg, k, v, self.slots, self.data)

    def fetch(self, slots, dtype=torch.bfloat16):
        """The rows of `slots` [n]: (k, v), each [n, kv_heads, 128]."""
        k, v = torch.empty((2, slots.numel(), self.cfg.kv_heads, _DIM), dtype=dtype,
                           device=self.data.device).unbind(0)
        dsa_cache_read(self.cfg, self.data, slots, k, v)
        return k, v

    def attend(self, q, idx, scale: float, *, request=None):
        """(o, lse) of the step's tokens q [tokens, heads, 128] over idx
        [tokens, Kc]; request: every token is of that request's prompt
        chunk (dsa_cache_attention_prompt)."""
        o = torch.empty_like(q)
        lse = torch.empty(q.shape[:2], dtype=torch.float32, device=q.device)
        if request is None:
            dsa_cache_attention(self.cfg, self.data, q, idx, self.token_req, self.tables, scale, o, lse)
        else:
            n = dsa_cache_attention_prompt_workspace(self.cfg, q, idx)
            ws = torch.empty(n, dtype=torch.uint8, device=q.device)
            dsa_cache_attention_prompt(self.cfg, self.data, q, idx, self.tables[request], scale, ws, o, lse)
        return o, lse
