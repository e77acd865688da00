"""The paged 4-bit key/value cache and the sparse attention over it: the
binding of the dsa_cache_* calls (include/dsa_select.h has the record layout,
the arguments and the limits) and `PagedCache`, which owns a cache with its
block tables and takes steps on it.

As in binding.py, every argument is checked here before a pointer reaches the
C ABI: TypeError for a wrong type, ValueError for a wrong device, layout or
size.  The work runs on the current stream of the tensors' own device unless a
stream of that device is given.
"""
from __future__ import annotations

import ctypes

import torch

from . import binding

RECORD_BYTES = 144
PLAN_OK, PLAN_NO_PAGES, PLAN_TABLE_WIDTH, PLAN_TOKENS, PLAN_BAD_LENGTHS = range(5)

_DIM = 128
_ROW_TYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
_I32, _U8, _F32 = torch.int32, torch.uint8, torch.float32
_Tensor = torch.Tensor


class dsa_cache_cfg(ctypes.Structure):
    _fields_ = [("pages", ctypes.c_int32), ("page_size", ctypes.c_int32), ("kv_heads", ctypes.c_int32),
                ("k_shift", ctypes.c_int32), ("v_shift", ctypes.c_int32)]


def cache_cfg(*, pages, page_size=64, kv_heads=1, k_shift=0, v_shift=0) -> dsa_cache_cfg:
    """A cache's shape: `pages` pages of `page_size` (a power of two) positions
    of `kv_heads` key/value heads; keys are stored divided by 2^k_shift, values
    by 2^v_shift."""
    return dsa_cache_cfg(pages=pages, page_size=page_size, kv_heads=kv_heads, k_shift=k_shift, v_shift=v_shift)


def dsa_cache_bytes(cfg: dsa_cache_cfg) -> int:
    """Bytes of the cache `cfg` describes."""
    n = ctypes.c_size_t(0)
    binding._check(binding.load().dsa_cache_bytes(ctypes.byref(cfg), ctypes.byref(n)), "dsa_cache_bytes")
    return int(n.value)


# ---------------------------------------------------------------------------
# argument checks
#
# A decode step's kernels take a few microseconds, and so do checks made one
# call a tensor: the functions below test what they need in line and leave the
# reason to _refuse.

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
    if not (isinstance(t, _Tensor) and t.dtype is dtype and t.get_device() == dev and t.is_contiguous()
            and t.numel() >= numel):
        _refuse(name, t, dtype, numel, dev)


def _device_of(name, t, dtype):
    """The device of `t`, a contiguous CUDA tensor of `dtype`."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.is_cuda and t.is_contiguous()):
        _refuse(name, t, dtype, 0, None)
    return t.get_device()


def _cache(cfg, cache, dev):
    if type(cfg) is not dsa_cache_cfg:
        raise TypeError(f"cfg: expected a dsa_cache_cfg, got {type(cfg).__name__}")
    need = cfg.pages * cfg.page_size * cfg.kv_heads * RECORD_BYTES  # limits: the C ABI's
    _need("cache", cache, _U8, need, dev)


def _row_type(name, t, types):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor, got {type(t).__name__}")
    code = _ROW_TYPES.get(t.dtype, 99)
    if code >= types:
        want = ", ".join(str(d) for d, c in _ROW_TYPES.items() if c < types)
        raise TypeError(f"{name}: dtype {t.dtype}, expected one of {want}")
    return code


_raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice
_functions = {}


def _fn(name):
    f = _functions.get(name)
    if f is None:
        f = _functions[name] = getattr(binding.load(), name)
    return f


def _call(name, dev, stream, *args):
    """The library's `name`(*args, stream) with `dev` current: the C ABI launches on the current device."""
    if stream is None:
        s = _raw_stream(dev)
    else:
        if stream.device.index != dev:
            raise ValueError(f"stream: of cuda:{stream.device.index}, the tensors are on cuda:{dev}")
        s = stream.cuda_stream
    fn = _functions.get(name) or _fn(name)
    if _current_device() == dev:
        rc = fn(*args, s)
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, s)
    if rc:
        raise binding.DsaSelectError(rc, name)


# ---------------------------------------------------------------------------
# the calls

def dsa_cache_plan(cfg: dsa_cache_cfg, lens, fresh, tables, held, free_pages, free_count, first, token_req, ends,
                   slots, status, stream=None):
    """One step's pages, block tables and slots from request lengths: lens and
    fresh [R] int32; tables [R, P], held [R], free_pages and free_count [1]
    updated; first [R + 1], token_req, ends and slots [T] and status [4]
    written.  status[0] is one of the PLAN_* codes; a step that cannot be taken
    changes no state."""
    if type(cfg) is not dsa_cache_cfg:
        raise TypeError(f"cfg: expected a dsa_cache_cfg, got {type(cfg).__name__}")
    dev = _device_of("lens", lens, _I32)
    R = lens.numel()
    try:
        T = token_req.numel()
        fine = (
            fresh.dtype is _I32 and fresh.get_device() == dev and fresh.is_contiguous() and fresh.numel() >= R
            and tables.dtype is _I32 and tables.get_device() == dev and tables.is_contiguous()
            and held.dtype is _I32 and held.get_device() == dev and held.is_contiguous() and held.numel() >= R
            and free_pages.dtype is _I32 and free_pages.get_device() == dev and free_pages.is_contiguous()
            and free_count.dtype is _I32 and free_count.get_device() == dev and free_count.numel() >= 1
            and first.dtype is _I32 and first.get_device() == dev and first.is_contiguous() and first.numel() > R
            and token_req.dtype is _I32 and token_req.get_device() == dev and token_req.is_contiguous()
            and ends.dtype is _I32 and ends.get_device() == dev and ends.is_contiguous() and ends.numel() >= T
            and slots.dtype is _I32 and slots.get_device() == dev and slots.is_contiguous() and slots.numel() >= T
            and status.dtype is _I32 and status.get_device() == dev and status.is_contiguous()
            and status.numel() >= 4)
    except AttributeError:
        fine = False
    if not fine:  # one by one, for the reason
        _need("token_req", token_req, _I32, 0, dev)
        for name, x, n in (("fresh", fresh, R), ("tables", tables, 0), ("held", held, R),
                           ("free_pages", free_pages, 0), ("free_count", free_count, 1), ("first", first, R + 1),
                           ("ends", ends, token_req.numel()), ("slots", slots, token_req.numel()),
                           ("status", status, 4)):
            _need(name, x, _I32, n, dev)
        raise ValueError("a tensor changed while it was checked")
    if tables.dim() != 2 or tables.shape[0] != R:
        raise ValueError(f"tables: shape {tuple(tables.shape)}, expected [{R}, pages per request]")
    _call("dsa_cache_plan", dev, stream, ctypes.byref(cfg), R, tables.shape[1], T, free_pages.numel(),
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
    code = _row_type("k", k, 3)
    if not isinstance(v, _Tensor) or v.dtype is not k.dtype:
        raise TypeError(f"v: expected a tensor of {k.dtype} like k")
    dev = _device_of("slots", slots, _I32)
    _cache(cfg, cache, dev)
    T, heads = slots.numel(), cfg.kv_heads
    shape = (T, heads, _DIM)
    if (k.get_device() == dev and v.get_device() == dev and k.shape == shape and v.shape == shape
            and k.is_contiguous() and v.is_contiguous()):
        ks = vs = heads * _DIM
    else:
        ks, vs = _strided_rows("k", k, T, heads, dev), _strided_rows("v", v, T, heads, dev)
    _call("dsa_cache_write", dev, stream, ctypes.byref(cfg), T, code, k.data_ptr(), v.data_ptr(), ks, vs,
          slots.data_ptr(), cache.data_ptr())


def dsa_cache_read(cfg: dsa_cache_cfg, cache, slots, k, v, stream=None):
    """Read the records slots [T] int32 names into k and v [T, kv_heads, 128]
    (bf16, f16 or f32); zeros for a slot outside the cache."""
    code = _row_type("k", k, 3)
    dev = _device_of("slots", slots, _I32)
    _cache(cfg, cache, dev)
    T = slots.numel()
    n = T * cfg.kv_heads * _DIM
    _need("k", k, k.dtype, n, dev)
    _need("v", v, k.dtype, n, dev)
    _call("dsa_cache_read", dev, stream, ctypes.byref(cfg), T, code, cache.data_ptr(), slots.data_ptr(),
          k.data_ptr(), v.data_ptr())


def _attention_args(cfg, cache, q, idx, o, lse):
    """(type code, tokens, heads, select, device) of an attention call's tensors."""
    if type(cfg) is not dsa_cache_cfg:
        raise TypeError(f"cfg: expected a dsa_cache_cfg, got {type(cfg).__name__}")
    dtype = q.dtype if isinstance(q, _Tensor) else None
    code, dev = _ROW_TYPES.get(dtype, 99), -1
    try:
        T, H, D = q.shape
        rows, Kc = idx.shape
        dev = q.get_device()
        if (code < 2 and dev >= 0 and D == _DIM and rows == T and q.is_contiguous()
                and cache.dtype is _U8 and cache.get_device() == dev and cache.is_contiguous()
                and cache.numel() >= cfg.pages * cfg.page_size * cfg.kv_heads * RECORD_BYTES
                and idx.dtype is _I32 and idx.get_device() == dev and idx.is_contiguous()
                and o.dtype is dtype and o.get_device() == dev and o.is_contiguous() and o.numel() >= T * H * _DIM
                and lse.dtype is _F32 and lse.get_device() == dev and lse.is_contiguous() and lse.numel() >= T * H):
            return code, T, H, Kc, dev
    except (AttributeError, ValueError):
        pass
    # one by one, for the reason
    _row_type("q", q, 2)
    dev = _device_of("q", q, dtype)
    if q.dim() != 3 or q.shape[2] != _DIM:
        raise ValueError(f"q: shape {tuple(q.shape)}, expected [tokens, heads, {_DIM}]")
    T, H, _ = q.shape
    _cache(cfg, cache, dev)
    _need("idx", idx, _I32, 0, dev)
    if idx.dim() != 2 or idx.shape[0] != T:
        raise ValueError(f"idx: shape {tuple(idx.shape)}, expected [{T}, select]")
    _need("o", o, dtype, T * H * _DIM, dev)
    _need("lse", lse, _F32, T * H, dev)
    raise ValueError("a tensor changed while it was checked")


def dsa_cache_attention(cfg: dsa_cache_cfg, cache, q, idx, token_req, tables, scale: float, o, lse, stream=None):
    """Sparse attention over the cache: q [T, H, 128] (bf16 or f16), idx
    [T, Kc] int32 positions (below 0: unused) of request token_req[t], whose
    pages are tables[request]; writes o [T, H, 128] (q's type) and lse [T, H]
    f32."""
    code, T, H, Kc, dev = _attention_args(cfg, cache, q, idx, o, lse)
    _need("token_req", token_req, _I32, T, dev)
    _need("tables", tables, _I32, 0, dev)
    shape = tables.shape
    if len(shape) != 2:
        raise ValueError(f"tables: shape {tuple(shape)}, expected [requests, pages per request]")
    R, P = shape
    _call("dsa_cache_attention", dev, stream, ctypes.byref(cfg), T, H, Kc, R, P, code, cache.data_ptr(),
          q.data_ptr(), idx.data_ptr(), token_req.data_ptr(), tables.data_ptr(), scale, o.data_ptr(), lse.data_ptr())


def dsa_cache_attention_prompt_workspace(cfg: dsa_cache_cfg, q, idx) -> int:
    """Workspace bytes of dsa_cache_attention_prompt for q [T, H, 128] and idx [T, Kc]."""
    n = ctypes.c_size_t(0)
    binding._check(binding.load().dsa_cache_attention_prompt_workspace(
        ctypes.byref(cfg), q.shape[0], q.shape[1], idx.shape[1], ctypes.byref(n)),
        "dsa_cache_attention_prompt_workspace")
    return int(n.value)


def dsa_cache_attention_prompt(cfg: dsa_cache_cfg, cache, q, idx, table, scale: float, workspace, o, lse,
                               stream=None):
    """dsa_cache_attention for the tokens of one request's prompt chunk, 128 /
    (H / kv_heads) neighbours at a time over the union of their selections:
    idx rows strictly ascending, then -1; table [P] int32 the request's pages."""
    code, T, H, Kc, dev = _attention_args(cfg, cache, q, idx, o, lse)
    _need("table", table, _I32, 0, dev)
    _need("workspace", workspace, _U8, 0, dev)
    _call("dsa_cache_attention_prompt", dev, stream, ctypes.byref(cfg), T, H, Kc, table.numel(), code,
          cache.data_ptr(), q.data_ptr(), idx.data_ptr(), table.data_ptr(), scale, workspace.data_ptr(),
          workspace.numel(), o.data_ptr(), lse.data_ptr())


def dsa_cache_attention_status() -> int:
    """DSA_OK, or DSA_ERR_TIMEOUT once after an attention kernel over the cache
    gave up a wait (synchronises the device)."""
    return int(binding.load().dsa_cache_attention_status())


# ---------------------------------------------------------------------------
# a cache with its tables

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
        if tokens != self.slots.numel():
            if tokens > self._maps[-1].shape[1]:
                room = max(tokens, 2 * self._maps[-1].shape[1])
                self._maps.append(torch.empty((3, (room + 63) // 64 * 64), dtype=_I32, device=self.tables.device))
            self.token_req, self.ends, self.slots = self._maps[-1][:, :tokens].unbind(0)
        dsa_cache_plan(self.cfg, lens, fresh, self.tables, self.held, self.free_pages, self.free_count, self.first,
                       self.token_req, self.ends, self.slots, self.status)

    def ok(self):
        """Wait for the last step's status; RuntimeError when it could not be taken."""
        code, short, _, _ = self.status.tolist()
        if code != PLAN_OK:
            why = {PLAN_NO_PAGES: f"{short} pages short", PLAN_TABLE_WIDTH: "a request needs more pages than its table has",
                   PLAN_TOKENS: "more tokens than the step has room for"}.get(code, "lengths or counts out of range")
            raise RuntimeError(f"cache step not taken: {why}")

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
