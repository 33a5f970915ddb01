"""trellis_quantized_gb300 -- Python binding of libexl3 (the EXL3 trellis linear on GB300).

A thin ctypes layer over the C ABI declared in include/exl3.h: every function
here has the name of the C entry point it wraps and only marshals torch
tensors into device pointers, sizes and the current CUDA stream.  All
arithmetic runs in the library's CUDA kernels; there is no CPU path.  If
libexl3.so cannot be built or loaded, importing a function raises.

Tensors: fp16 data is passed as torch.float16 (or any 2-byte dtype holding
binary16 bits), trellis words as a 2-byte integer tensor (torch.int16 or
torch.uint16) shaped [k/16, n/16, 16K], all contiguous on the same CUDA
device.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import threading

import torch

from . import _build

EXL3_OK = 0
EXL3_ERR_ARG = 1
EXL3_ERR_SHAPE = 2
EXL3_ERR_BITS = 3
EXL3_ERR_CODEBOOK = 4
EXL3_ERR_WORKSPACE = 5
EXL3_ERR_CUDA = 6
EXL3_ERR_DEVICE = 7

EXL3_CB_MCG = 1
EXL3_CB_MUL1 = 2
EXL3_CB_3INST = 3
EXL3_OUT_F16 = 0
EXL3_OUT_F32 = 1

EXL3_ROPE_HALF = 0
EXL3_ROPE_PAIRS = 1
EXL3_ROPE_NONE = 0
EXL3_ROPE_LINEAR = 1
EXL3_ROPE_NTK = 2
EXL3_ROPE_BANDS = 3
EXL3_ROPE_YARN = 4

EXL3_SCORE_SOFTMAX = 0
EXL3_SCORE_SIGMOID = 1
EXL3_GROUP_MAX = 0
EXL3_GROUP_TOP2 = 1

_lock = threading.Lock()
_lib = None


class ExpertProj(ctypes.Structure):
    """exl3_expert_proj: one projection kind for all experts (device pointers)."""
    _fields_ = [("trellis", ctypes.c_void_p), ("suh", ctypes.c_void_p), ("svh", ctypes.c_void_p),
                ("k", ctypes.c_int), ("n", ctypes.c_int), ("K", ctypes.c_int), ("codebook", ctypes.c_int),
                ("nslots", ctypes.c_int)]


class ExpertProjMixed(ctypes.Structure):
    """exl3_expert_proj_mixed: one projection kind with a width per expert
    (device trellis/suh/svh, host widths K[E])."""
    _fields_ = [("trellis", ctypes.c_void_p), ("suh", ctypes.c_void_p), ("svh", ctypes.c_void_p),
                ("K", ctypes.POINTER(ctypes.c_int32)), ("k", ctypes.c_int), ("n", ctypes.c_int),
                ("codebook", ctypes.c_int), ("nslots", ctypes.c_int)]


class HeadTransform(ctypes.Structure):
    """exl3_head_transform: head norms and rotary positions (device pointers)."""
    _fields_ = [("q_norm", ctypes.c_void_p), ("k_norm", ctypes.c_void_p), ("eps", ctypes.c_float),
                ("inv_freq", ctypes.c_void_p), ("rotary_dim", ctypes.c_int), ("layout", ctypes.c_int),
                ("magnitude", ctypes.c_float)]


class KvCache(ctypes.Structure):
    """exl3_kv_cache: a paged cache of keys and values (device pointers, strides in elements)."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("num_pages", ctypes.c_int),
                ("page_size", ctypes.c_int), ("heads_kv", ctypes.c_int), ("head_dim", ctypes.c_int),
                ("stride_page", ctypes.c_int64), ("stride_token", ctypes.c_int64), ("stride_head", ctypes.c_int64)]


class PagedBatch(ctypes.Structure):
    """exl3_paged_batch: the sequences of a call (device arrays)."""
    _fields_ = [("q_start", ctypes.c_void_p), ("kv_len", ctypes.c_void_p), ("page_table", ctypes.c_void_p),
                ("batch", ctypes.c_int), ("max_pages", ctypes.c_int)]


class _Made(ctypes.Structure):
    """A descriptor made for tensors of certain sizes: those fields stay as they are, since the
    kernels go by them and the checks of a call by the tensors' shapes."""
    _sizes: tuple = ()

    def __setattr__(self, name, value):
        if name in self._sizes and "_address" in self.__dict__:
            raise AttributeError(f"{name} is a size of the {type(self).__name__}'s tensors: make another one")
        super().__setattr__(name, value)


class Router(_Made):
    """exl3_router: a row of weights per expert (device pointers)."""
    _sizes = ("E", "k")
    _fields_ = [("w", ctypes.c_void_p), ("w_scale", ctypes.c_void_p), ("bias", ctypes.c_void_p), ("E", ctypes.c_int),
                ("k", ctypes.c_int)]


class RouteRule(ctypes.Structure):
    """exl3_route_rule: how experts are chosen from logits."""
    _fields_ = [("score", ctypes.c_int), ("bias", ctypes.c_void_p), ("groups", ctypes.c_int),
                ("groups_kept", ctypes.c_int), ("group_score", ctypes.c_int), ("topk", ctypes.c_int),
                ("renormalise", ctypes.c_int), ("scale", ctypes.c_float)]


class Adapters(_Made):
    """exl3_adapters: a pool of low-rank adapters for one linear (device pointers)."""
    _sizes = ("count", "max_rank", "k", "n")
    _fields_ = [("a", ctypes.c_void_p), ("b", ctypes.c_void_p), ("scale", ctypes.c_void_p), ("rank", ctypes.c_void_p),
                ("count", ctypes.c_int), ("max_rank", ctypes.c_int), ("k", ctypes.c_int), ("n", ctypes.c_int)]


class Exl3Error(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"libexl3 error {code}: {msg}")
        self.code = code


def lib_path() -> str:
    return _build.LIB


def lib():
    """Load libexl3.so (building it first if it is missing or stale)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        path = _build.build()
        L = ctypes.CDLL(path)
        P, I, Z, L64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_int64
        L.exl3_last_error.restype = ctypes.c_char_p
        L.exl3_version.restype = I
        L.exl3_workspace_clear.argtypes = [P, Z, P]
        L.exl3_relax_capture.argtypes = [I, ctypes.POINTER(I)]
        L.exl3_copy_in.argtypes = [P, P, Z, P]
        L.exl3_check_device_error.argtypes = [P, Z, P, ctypes.POINTER(I)]
        L.exl3_decode_tile.argtypes = [P, I, I, I, I, I, I, I, I, P, L64, P]
        L.exl3_input_rht.argtypes = [P, I, I, P, P, I, P]
        L.exl3_linear_workspace_size.argtypes = [I, I, I, I]
        L.exl3_linear_workspace_size.restype = Z
        L.exl3_linear.argtypes = [P, I, I, I, P, P, P, I, I, P, I, P, Z, P]
        L.exl3_linear_bias.argtypes = [P, I, I, I, P, P, P, P, I, I, P, I, P, Z, P]
        L.exl3_linear_int8_workspace_size.argtypes = [I, I, I, I]
        L.exl3_linear_int8_workspace_size.restype = Z
        L.exl3_linear_int8.argtypes = [P, I, I, I, P, P, P, I, I, ctypes.c_float, P, P, P, P, P, Z, P]
        L.exl3_linear_int8_bias.argtypes = [P, I, I, I, P, P, P, P, I, I, ctypes.c_float, P, P, P, P, P, Z, P]
        L.exl3_moe_workspace_size.argtypes = [I, I, I, P, P]
        L.exl3_moe_workspace_size.restype = Z
        L.exl3_moe_grouped.argtypes = [P, I, I, P, P, I, I, P, P, P, I, P, Z, P]
        L.exl3_linear_gemv_noalloc.argtypes = [P, I, I, P, P, P, I, I, P, I, P]
        L.exl3_noalloc_device_error.argtypes = [P, ctypes.POINTER(I)]
        L.exl3_linear_shards_workspace_size.argtypes = [I, I, I, I, I]
        L.exl3_linear_shards_workspace_size.restype = Z
        L.exl3_linear_shards.argtypes = [P, I, I, I, I, P, P, P, I, I, P, I, P, Z, P]
        L.exl3_linear_shards_var_workspace_size.argtypes = [I, I, I, P, I]
        L.exl3_linear_shards_var_workspace_size.restype = Z
        L.exl3_linear_shards_var.argtypes = [P, I, I, I, P, P, P, P, I, I, P, I, P, Z, P]
        L.exl3_moe_mixed_workspace_size.argtypes = [I, I, I, P, P]
        L.exl3_moe_mixed_workspace_size.restype = Z
        L.exl3_moe_grouped_mixed.argtypes = [P, I, I, P, P, I, I, P, P, P, I, P, Z, P]
        L.exl3_set_weight_prefetch.argtypes = [I]
        L.exl3_set_weight_prefetch.restype = I
        L.exl3_set_row_invariant.argtypes = [I]
        L.exl3_set_row_invariant.restype = I
        L.exl3_rope_frequencies.argtypes = [I, ctypes.c_double, I, ctypes.c_double, I, ctypes.c_double,
                                            ctypes.c_double, P, P]
        L.exl3_qk_norm_rope.argtypes = [P, L64, P, L64, I, I, I, I, I, P, P, P, P, I, P]
        L.exl3_qkv_append_workspace_size.argtypes = []
        L.exl3_qkv_append_workspace_size.restype = Z
        L.exl3_qkv_append.argtypes = [P, L64, P, L64, P, L64, I, I, I, P, P, P, P, P, P, Z, P]
        L.exl3_paged_attention_workspace_size.argtypes = [I, I, I, I, I]
        L.exl3_paged_attention_workspace_size.restype = Z
        L.exl3_paged_attention.argtypes = [P, L64, I, I, P, P, ctypes.c_float, I, I, P, I, P, P, Z, P]
        L.exl3_router_pack.argtypes = [P, I, I, P, P, P]
        L.exl3_router_logits_workspace_size.argtypes = []
        L.exl3_router_logits_workspace_size.restype = Z
        L.exl3_router_logits.argtypes = [P, L64, I, P, P, P, Z, P]
        L.exl3_route.argtypes = [P, L64, I, I, I, P, P, P, P]
        L.exl3_adapter_plan_size.argtypes = [I, I, I]
        L.exl3_adapter_plan_size.restype = Z
        L.exl3_adapter_plan.argtypes = [P, P, I, I, I, P, Z, P]
        L.exl3_adapter_add_workspace_size.argtypes = [I, I]
        L.exl3_adapter_add_workspace_size.restype = Z
        L.exl3_adapter_add.argtypes = [P, L64, P, L64, P, L64, I, P, P, I, I, P, Z, P]
        L.exl3_adapter_scratch_size.argtypes = [I, I, I]
        L.exl3_adapter_scratch_size.restype = Z
        L.exl3_adapter_add_scratch.argtypes = [P, L64, P, L64, P, L64, I, P, P, I, I, P, Z, P, Z, P]
        _lib = L
        return L


def _check(rc: int):
    if rc != EXL3_OK:
        raise Exl3Error(rc, lib().exl3_last_error().decode())


def _ptr(t, name: str, itemsize: int | None = None):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if itemsize is not None and t.element_size() != itemsize:
        raise TypeError(f"{name} must have {itemsize}-byte elements, got {t.dtype}")
    return ctypes.c_void_p(t.data_ptr())


def _ptr_pinned(t, name: str):
    """A pinned host tensor's address (the device addresses pinned memory directly)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    # (is_pinned asks the driver about the address; skipped while a CUDA
    # graph is being captured)
    if t.is_cuda or (not torch.cuda.is_current_stream_capturing() and not t.is_pinned()):
        raise ValueError(f"{name} must be a pinned host tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _raw_stream(stream=None) -> int:
    """The stream's handle: the given one, or the current device's current one."""
    if stream is not None:
        return stream.cuda_stream
    return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())


def _made_on(stream):
    """Context in which tensors are the given stream's (None: the current one's); as everywhere, all
    that it has to have is its handle."""
    if stream is None or isinstance(stream, torch.cuda.Stream):
        return torch.cuda.stream(stream)
    return torch.cuda.stream(torch.cuda.ExternalStream(stream.cuda_stream))


def _stream(stream=None):
    return ctypes.c_void_p(_raw_stream(stream))


_ws_cache: dict = {}                      # (device, stream): (buffer, address, bytes)
_ws_outgrown: list = []                   # buffers that captured graphs may go on using


def workspace(nbytes: int, device=None, stream=None) -> torch.Tensor:
    """A zero-initialised workspace of at least nbytes, cached per (device, stream).

    Every libexl3 call leaves its counters at zero again, so one cleared
    workspace serves any number of calls made in stream order.  A buffer whose
    place a larger one takes stays alive, since a captured graph may hold its
    address; its successor is at least twice as large, so that all that are
    kept are no more than the present one.  (Nothing is captured on the default
    stream: its buffers grow as asked and go.)"""
    if device is None:
        index = torch.cuda.current_device()
    else:
        device = torch.device(device)
        index = torch.cuda.current_device() if device.index is None else device.index
    raw = stream.cuda_stream if stream is not None else torch._C._cuda_getCurrentRawStream(index)
    key = (index, raw)
    buf, _, size = _ws_cache.get(key, (None, 0, -1))
    if size < nbytes:
        dev = torch.device("cuda", index)
        on = stream if stream is not None else torch.cuda.current_stream(dev)
        sizes = [max(nbytes, 256)]
        if buf is not None and raw:
            _ws_outgrown.append(buf)
            sizes.insert(0, max(nbytes, 2 * size))
        for n in sizes:
            try:
                buf = _cleared(n, dev, on, raw)
                break
            except torch.OutOfMemoryError:
                if n == sizes[-1]:
                    raise
        _ws_cache[key] = (buf, buf.data_ptr(), buf.numel())
    return buf


def _cleared(nbytes: int, device, on, raw: int) -> torch.Tensor:
    """A zero-filled buffer of the given stream's memory (what another stream freed may still be in
    use there)."""
    with _made_on(on):
        if not raw or not torch.cuda.is_current_stream_capturing():
            buf = torch.empty(nbytes, dtype=torch.uint8, device=device)
            exl3_workspace_clear(buf, stream=on)
            return buf
    return _outside_captures(nbytes, device)


def _outside_captures(nbytes: int, device) -> torch.Tensor:
    """A workspace first needed during a capture: cleared now, for all who will use it, and of
    memory that is no graph's (a graph's temporaries take turns in theirs, at every replay)."""
    with exl3_relax_capture():
        for _ in range(64):              # (streams come from a pool; one of them is being captured)
            s = torch.cuda.Stream(device)
            with torch.cuda.stream(s):
                if not torch.cuda.is_current_stream_capturing():
                    buf = torch.empty(nbytes, dtype=torch.uint8, device=device)
                    exl3_workspace_clear(buf, stream=s)
                    s.synchronize()
                    return buf
    raise RuntimeError("every stream is being captured: make a first call before the capture")


# ------------------------------------------------------------------ entry points

def exl3_version() -> int:
    return lib().exl3_version()


def exl3_workspace_clear(ws: torch.Tensor, stream=None):
    _check(lib().exl3_workspace_clear(_ptr(ws, "workspace"), ws.numel() * ws.element_size(), _stream(stream)))


@contextlib.contextmanager
def exl3_relax_capture():
    """The calling thread may allocate and wait on streams that no capture under way includes."""
    previous = ctypes.c_int(0)
    _check(lib().exl3_relax_capture(1, ctypes.byref(previous)))
    try:
        yield
    finally:
        _check(lib().exl3_relax_capture(0, ctypes.byref(previous)))


def exl3_copy_in(src: torch.Tensor, dst: torch.Tensor, stream=None) -> torch.Tensor:
    """Copy a pinned host tensor into a device tensor of the same byte size with
    a kernel chained by programmatic dependent launch (see exl3_copy_in in exl3.h)."""
    nbytes = src.numel() * src.element_size()
    if dst.numel() * dst.element_size() != nbytes:
        raise ValueError("src and dst must have the same size in bytes")
    _check(lib().exl3_copy_in(_ptr_pinned(src, "src"), _ptr(dst, "dst"), nbytes, _stream(stream)))
    return dst


def exl3_check_device_error(ws: torch.Tensor, stream=None) -> int:
    err = ctypes.c_int(0)
    _check(lib().exl3_check_device_error(_ptr(ws, "workspace"), ws.numel() * ws.element_size(),
                                         _stream(stream), ctypes.byref(err)))
    return err.value


def exl3_decode_tile(trellis, k: int, n: int, K: int, codebook: int = EXL3_CB_MUL1, tk0: int = 0,
                     tk_cnt: int | None = None, tn0: int = 0, tn_cnt: int | None = None,
                     w_out=None, ld: int | None = None, stream=None) -> torch.Tensor:
    """Dequantised fp16 weights of a tile range (the whole tensor by default)."""
    tk_cnt = k // 16 - tk0 if tk_cnt is None else tk_cnt
    tn_cnt = n // 16 - tn0 if tn_cnt is None else tn_cnt
    if w_out is None:
        ld = 16 * tn_cnt if ld is None else ld
        w_out = torch.empty((16 * tk_cnt, ld), dtype=torch.float16, device=trellis.device)
    elif ld is None:
        ld = w_out.shape[-1]
    _check(lib().exl3_decode_tile(_ptr(trellis, "trellis", 2), k, n, K, codebook, tk0, tk_cnt, tn0, tn_cnt,
                                  _ptr(w_out, "w_out", 2), ld, _stream(stream)))
    return w_out


def exl3_input_rht(x, suh, out_dtype: int = EXL3_OUT_F32, out=None, stream=None) -> torch.Tensor:
    M, k = x.shape
    if out is None:
        out = torch.empty((M, k), dtype=torch.float32 if out_dtype == EXL3_OUT_F32 else torch.float16,
                          device=x.device)
    _check(lib().exl3_input_rht(_ptr(x, "x", 2), M, k, _ptr(suh, "suh", 2), _ptr(out, "out"), out_dtype,
                                _stream(stream)))
    return out


def exl3_linear_workspace_size(M: int, k: int, n: int, K: int) -> int:
    return lib().exl3_linear_workspace_size(M, k, n, K)


def exl3_linear(x, trellis, suh, svh, K: int, codebook: int = EXL3_CB_MUL1, out_dtype: int = EXL3_OUT_F16,
                y=None, workspace_buf=None, stream=None) -> torch.Tensor:
    """y = RHT_out(RHT_in(x . suh) @ W) . svh for x [M, k] fp16.  At M = 1, y may be
    a pinned host tensor: the kernels write the result straight into it."""
    M, k = x.shape
    n = trellis.shape[1] * 16
    if y is None:
        y = torch.empty((M, n), dtype=torch.float32 if out_dtype == EXL3_OUT_F32 else torch.float16,
                        device=x.device)
    need = exl3_linear_workspace_size(M, k, n, K)
    ws = workspace_buf if workspace_buf is not None else workspace(need, x.device, stream)
    yp = _ptr_pinned(y, "y") if (M == 1 and not y.is_cuda) else _ptr(y, "y")
    _check(lib().exl3_linear(_ptr(x, "x", 2), M, k, n, _ptr(trellis, "trellis", 2), _ptr(suh, "suh", 2),
                             _ptr(svh, "svh", 2), K, codebook, yp, out_dtype, _ptr(ws, "workspace"),
                             ws.numel() * ws.element_size(), _stream(stream)))
    return y


def exl3_linear_bias(x, trellis, suh, svh, bias, K: int, codebook: int = EXL3_CB_MUL1,
                     out_dtype: int = EXL3_OUT_F16, y=None, workspace_buf=None, stream=None) -> torch.Tensor:
    """y = RHT_out(RHT_in(x . suh) @ W) . svh + bias for x [M, k] fp16, bias [n] fp16."""
    M, k = x.shape
    n = trellis.shape[1] * 16
    if y is None:
        y = torch.empty((M, n), dtype=torch.float32 if out_dtype == EXL3_OUT_F32 else torch.float16,
                        device=x.device)
    need = exl3_linear_workspace_size(M, k, n, K)
    ws = workspace_buf if workspace_buf is not None else workspace(need, x.device, stream)
    _check(lib().exl3_linear_bias(_ptr(x, "x", 2), M, k, n, _ptr(trellis, "trellis", 2), _ptr(suh, "suh", 2),
                                  _ptr(svh, "svh", 2), _ptr(bias, "bias", 2), K, codebook, _ptr(y, "y"), out_dtype,
                                  _ptr(ws, "workspace"), ws.numel() * ws.element_size(), _stream(stream)))
    return y


def exl3_linear_shards_workspace_size(M: int, k: int, n: int, K: int, nshards: int) -> int:
    return lib().exl3_linear_shards_workspace_size(M, k, n, K, nshards)


def exl3_linear_shards(x, trellis, suh, svh, K: int, codebook: int = EXL3_CB_MUL1, out_dtype: int = EXL3_OUT_F16,
                       y=None, workspace_buf=None, stream=None) -> torch.Tensor:
    """Fused shards over one input: trellis [S, k/16, n/16, 16K], suh [S, k], svh [S, n];
    returns y [S, M, n]."""
    M, k = x.shape
    S = trellis.shape[0]
    n = trellis.shape[2] * 16
    if y is None:
        y = torch.empty((S, M, n), dtype=torch.float32 if out_dtype == EXL3_OUT_F32 else torch.float16,
                        device=x.device)
    need = exl3_linear_shards_workspace_size(M, k, n, K, S)
    ws = workspace_buf if workspace_buf is not None else workspace(need, x.device, stream)
    _check(lib().exl3_linear_shards(_ptr(x, "x", 2), M, k, n, S, _ptr(trellis, "trellis", 2), _ptr(suh, "suh", 2),
                                    _ptr(svh, "svh", 2), K, codebook, _ptr(y, "y"), out_dtype, _ptr(ws, "workspace"),
                                    ws.numel() * ws.element_size(), _stream(stream)))
    return y


def exl3_linear_shards_var_workspace_size(M: int, k: int, widths, K: int) -> int:
    n = (ctypes.c_int * len(widths))(*[int(w) for w in widths])
    return lib().exl3_linear_shards_var_workspace_size(M, k, len(widths), n, K)


def exl3_linear_shards_var(x, trellis, suh, svh, widths, K: int, codebook: int = EXL3_CB_MUL1,
                           out_dtype: int = EXL3_OUT_F16, y=None, workspace_buf=None, stream=None) -> torch.Tensor:
    """Fused shards of different widths over one input: trellis flat (shard s's
    [k/16, n_s/16, 16K] tensor right after shard s-1's), suh [S, k], svh [sum n];
    returns y flat, shard-major (shard s an [M, n_s] block)."""
    M, k = x.shape
    S = len(widths)
    n = (ctypes.c_int * S)(*[int(w) for w in widths])
    total = M * sum(int(w) for w in widths)
    if y is None:
        y = torch.empty(total, dtype=torch.float32 if out_dtype == EXL3_OUT_F32 else torch.float16, device=x.device)
    need = lib().exl3_linear_shards_var_workspace_size(M, k, S, n, K)
    ws = workspace_buf if workspace_buf is not None else workspace(need, x.device, stream)
    _check(lib().exl3_linear_shards_var(_ptr(x, "x", 2), M, k, S, n, _ptr(trellis, "trellis", 2), _ptr(suh, "suh", 2),
                                        _ptr(svh, "svh", 2), K, codebook, _ptr(y, "y"), out_dtype,
                                        _ptr(ws, "workspace"), ws.numel() * ws.element_size(), _stream(stream)))
    return y


def exl3_set_row_invariant(enable: bool) -> bool:
    """Make each row of an exl3_linear result independent of the row count and
    of the other rows (same bits at every M); returns the previous setting."""
    return bool(lib().exl3_set_row_invariant(1 if enable else 0))


def exl3_set_weight_prefetch(enable: bool) -> bool:
    """Let M = 1 linears stream their weights while the kernel ahead of them
    on the stream finishes (CUDA programmatic dependent launch); returns the
    previous setting.  Weight buffers must not be written by kernels still in
    flight when a linear reading them is launched."""
    return bool(lib().exl3_set_weight_prefetch(1 if enable else 0))


def exl3_linear_int8_workspace_size(M: int, k: int, n: int, K: int) -> int:
    return lib().exl3_linear_int8_workspace_size(M, k, n, K)


WEIGHT_SCALE = 3.453125 / 127.0


def exl3_linear_int8(x, trellis, suh, svh, K: int, codebook: int = EXL3_CB_MUL1,
                     weight_scale: float = WEIGHT_SCALE, y=None, xq_out=None, row_scale_out=None,
                     acc_out=None, workspace_buf=None, stream=None) -> torch.Tensor:
    """int8 prefill linear: y fp16 [M, n]; optional int8 q_x, fp32 row scales and
    int32 accumulators are written to the given tensors."""
    M, k = x.shape
    n = trellis.shape[1] * 16
    if y is None:
        y = torch.empty((M, n), dtype=torch.float16, device=x.device)
    need = exl3_linear_int8_workspace_size(M, k, n, K)
    ws = workspace_buf if workspace_buf is not None else workspace(need, x.device, stream)
    _check(lib().exl3_linear_int8(_ptr(x, "x", 2), M, k, n, _ptr(trellis, "trellis", 2), _ptr(suh, "suh", 2),
                                  _ptr(svh, "svh", 2), K, codebook, weight_scale, _ptr(y, "y", 2),
                                  _ptr(xq_out, "xq_out", 1), _ptr(row_scale_out, "row_scale_out", 4),
                                  _ptr(acc_out, "acc_out", 4), _ptr(ws, "workspace"),
                                  ws.numel() * ws.element_size(), _stream(stream)))
    return y


def exl3_linear_int8_bias(x, trellis, suh, svh, bias, K: int, codebook: int = EXL3_CB_MUL1,
                          weight_scale: float = WEIGHT_SCALE, y=None, xq_out=None, row_scale_out=None,
                          acc_out=None, workspace_buf=None, stream=None) -> torch.Tensor:
    """int8 prefill linear plus an output bias [n] fp16: y fp16 [M, n]."""
    M, k = x.shape
    n = trellis.shape[1] * 16
    if y is None:
        y = torch.empty((M, n), dtype=torch.float16, device=x.device)
    need = exl3_linear_int8_workspace_size(M, k, n, K)
    ws = workspace_buf if workspace_buf is not None else workspace(need, x.device, stream)
    _check(lib().exl3_linear_int8_bias(_ptr(x, "x", 2), M, k, n, _ptr(trellis, "trellis", 2),
                                       _ptr(suh, "suh", 2), _ptr(svh, "svh", 2), _ptr(bias, "bias", 2), K,
                                       codebook, weight_scale, _ptr(y, "y", 2), _ptr(xq_out, "xq_out", 1),
                                       _ptr(row_scale_out, "row_scale_out", 4), _ptr(acc_out, "acc_out", 4),
                                       _ptr(ws, "workspace"), ws.numel() * ws.element_size(), _stream(stream)))
    return y


def expert_proj(trellis, suh, svh, K: int, codebook: int = EXL3_CB_MUL1) -> ExpertProj:
    """Descriptor of a projection arena: trellis [E, nslots, k/16, n/16, 16K], suh [E, nslots, k],
    svh [E, nslots, n] (CUDA tensors kept alive by the caller)."""
    E, nslots, tk, tn, _ = trellis.shape
    return ExpertProj(_ptr(trellis, "trellis", 2).value, _ptr(suh, "suh", 2).value, _ptr(svh, "svh", 2).value,
                      tk * 16, tn * 16, K, codebook, nslots)


def exl3_moe_workspace_size(T: int, topk: int, E: int, w13: ExpertProj, w2: ExpertProj) -> int:
    return lib().exl3_moe_workspace_size(T, topk, E, ctypes.byref(w13), ctypes.byref(w2))


def exl3_moe_grouped(x, topk_ids, topk_weights, w13: ExpertProj, w2: ExpertProj, E: int,
                     out_dtype: int = EXL3_OUT_F16, y=None, workspace_buf=None, stream=None) -> torch.Tensor:
    """Routed-expert contribution y [T, hidden] (gate+up, SiLU, down, weighted combine)."""
    T, hidden = x.shape
    topk = topk_ids.shape[1]
    if y is None:
        y = torch.empty((T, hidden), dtype=torch.float32 if out_dtype == EXL3_OUT_F32 else torch.float16,
                        device=x.device)
    need = exl3_moe_workspace_size(T, topk, E, w13, w2)
    ws = workspace_buf if workspace_buf is not None else workspace(need, x.device, stream)
    _check(lib().exl3_moe_grouped(_ptr(x, "x", 2), T, hidden, _ptr(topk_ids, "topk_ids", 4),
                                  _ptr(topk_weights, "topk_weights", 4), topk, E, ctypes.byref(w13),
                                  ctypes.byref(w2), _ptr(y, "y"), out_dtype, _ptr(ws, "workspace"),
                                  ws.numel() * ws.element_size(), _stream(stream)))
    return y


def expert_proj_mixed(trellis, suh, svh, K, k: int, n: int, codebook: int = EXL3_CB_MUL1) -> ExpertProjMixed:
    """Descriptor of a mixed-width projection arena: trellis flat (expert e's
    slots right after expert e-1's), suh [E, nslots, k], svh [E, nslots, n]
    (CUDA tensors kept alive by the caller), K the E widths (host)."""
    E, nslots, _ = suh.shape
    widths = (ctypes.c_int32 * E)(*[int(w) for w in K])
    d = ExpertProjMixed(_ptr(trellis, "trellis", 2).value, _ptr(suh, "suh", 2).value, _ptr(svh, "svh", 2).value,
                        ctypes.cast(widths, ctypes.POINTER(ctypes.c_int32)), k, n, codebook, nslots)
    d._widths = widths   # keep the host array alive with the descriptor
    return d


def exl3_moe_mixed_workspace_size(T: int, topk: int, E: int, w13: ExpertProjMixed, w2: ExpertProjMixed) -> int:
    return lib().exl3_moe_mixed_workspace_size(T, topk, E, ctypes.byref(w13), ctypes.byref(w2))


def exl3_moe_grouped_mixed(x, topk_ids, topk_weights, w13: ExpertProjMixed, w2: ExpertProjMixed, E: int,
                           out_dtype: int = EXL3_OUT_F16, y=None, workspace_buf=None, stream=None) -> torch.Tensor:
    """Routed-expert contribution y [T, hidden] with a width per expert."""
    T, hidden = x.shape
    topk = topk_ids.shape[1]
    if y is None:
        y = torch.empty((T, hidden), dtype=torch.float32 if out_dtype == EXL3_OUT_F32 else torch.float16,
                        device=x.device)
    need = exl3_moe_mixed_workspace_size(T, topk, E, w13, w2)
    ws = workspace_buf if workspace_buf is not None else workspace(need, x.device, stream)
    _check(lib().exl3_moe_grouped_mixed(_ptr(x, "x", 2), T, hidden, _ptr(topk_ids, "topk_ids", 4),
                                        _ptr(topk_weights, "topk_weights", 4), topk, E, ctypes.byref(w13),
                                        ctypes.byref(w2), _ptr(y, "y"), out_dtype, _ptr(ws, "workspace"),
                                        ws.numel() * ws.element_size(), _stream(stream)))
    return y


def exl3_linear_gemv_noalloc(x, trellis, suh, svh, K: int, codebook: int = EXL3_CB_MUL1,
                             out_dtype: int = EXL3_OUT_F16, y=None, stream=None) -> torch.Tensor:
    """M = 1 linear without a caller workspace, for callers that may not allocate
    device memory: the library's fixed scratch array is used instead."""
    k = x.numel()
    n = trellis.shape[1] * 16
    if y is None:
        y = torch.empty((1, n), dtype=torch.float32 if out_dtype == EXL3_OUT_F32 else torch.float16,
                        device=x.device)
    _check(lib().exl3_linear_gemv_noalloc(_ptr(x, "x", 2), k, n, _ptr(trellis, "trellis", 2),
                                          _ptr(suh, "suh", 2), _ptr(svh, "svh", 2), K, codebook,
                                          _ptr(y, "y"), out_dtype, _stream(stream)))
    return y


def exl3_noalloc_device_error(stream=None) -> int:
    """Device error word of the fixed scratch array used by
    exl3_linear_gemv_noalloc on the current device (waits for the stream,
    then reads and clears it; 0 = no device-side check failed)."""
    v = ctypes.c_int(0)
    _check(lib().exl3_noalloc_device_error(_stream(stream), ctypes.byref(v)))
    return v.value


# ------------------------------------------------------------------ attention

_FP16_BITS = (torch.float16, torch.int16, torch.uint16)      # fp16 values, or their bits in integers


def _check_fp16(t, name: str):
    """bfloat16 is as wide as fp16 and would be read as other numbers."""
    if isinstance(t, torch.Tensor) and t.dtype not in _FP16_BITS:
        raise TypeError(f"{name} must be torch.float16 (or its bits in a 16-bit integer type), got {t.dtype}")


def exl3_rope_frequencies(rotary_dim: int, base: float = 10000.0, scaling: int = EXL3_ROPE_NONE, factor: float = 1.0,
                          original_len: int = 4096, low: float = 1.0, high: float = 32.0):
    """Rotary frequencies of a model, (inv_freq [rotary_dim / 2] fp32 host tensor, magnitude)."""
    f = torch.empty(max(rotary_dim // 2, 1), dtype=torch.float32)
    mag = ctypes.c_float(1.0)
    _check(lib().exl3_rope_frequencies(rotary_dim, base, scaling, factor, original_len, low, high,
                                       ctypes.c_void_p(f.data_ptr()), ctypes.byref(mag)))
    return f, mag.value


def head_transform(q_norm=None, k_norm=None, eps: float = 1e-6, inv_freq=None, layout: int = EXL3_ROPE_HALF,
                   magnitude: float = 1.0) -> HeadTransform:
    """Descriptor of the head norms (fp16 weights [head_dim] or None) and the rotary
    positions (inv_freq fp32 [rotary_dim / 2] or None); the tensors are kept alive with it."""
    if inv_freq is not None and inv_freq.dtype != torch.float32:
        raise TypeError(f"inv_freq must be torch.float32, got {inv_freq.dtype}")
    _check_fp16(q_norm, "q_norm")
    _check_fp16(k_norm, "k_norm")
    p = lambda t, name, size: None if t is None else _ptr(t, name, size).value
    d = HeadTransform(p(q_norm, "q_norm", 2), p(k_norm, "k_norm", 2), eps, p(inv_freq, "inv_freq", 4),
                      0 if inv_freq is None else 2 * inv_freq.numel(), layout, magnitude)
    d._keep = (q_norm, k_norm, inv_freq)
    d._norm_sizes = tuple(None if t is None else t.numel() for t in (q_norm, k_norm))
    return d


def kv_cache(k, v) -> KvCache:
    """Descriptor of a paged cache from keys and values [pages, page_size, heads_kv, head_dim]
    fp16: any strides with dense head elements, the same for both (head-major pages and one
    allocation for both are transposed or sliced views); the tensors are kept alive with it."""
    for t, name in ((k, "k"), (v, "v")):
        _check_fp16(t, name)
        if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dim() != 4:
            raise ValueError(f"{name} must be a CUDA tensor [pages, page_size, heads_kv, head_dim]")
        if t.stride(3) != 1:
            raise ValueError(f"{name}'s head elements must be dense")
    if k.shape != v.shape or k.stride() != v.stride():
        raise ValueError("k and v must have the same shape and strides")
    pages, page, heads, dim = k.shape
    # torch gives a dimension of size one any stride: use the dense one
    stride = [s if n > 1 else heads * dim * page for s, n in zip(k.stride(), k.shape)]
    d = KvCache(k.data_ptr(), v.data_ptr(), pages, page, heads, dim, stride[0], stride[1], stride[2])
    d._keep = (k, v)
    return d


def paged_batch(q_start, kv_len, page_table) -> PagedBatch:
    """Descriptor of a call's sequences: q_start [B + 1], kv_len [B], page_table [B, max_pages],
    int32 on the device; the tensors are kept alive with it."""
    for t, name in ((q_start, "q_start"), (kv_len, "kv_len"), (page_table, "page_table")):
        if isinstance(t, torch.Tensor) and t.dtype != torch.int32:
            raise TypeError(f"{name} must be torch.int32, got {t.dtype}")
    B, max_pages = page_table.shape
    if q_start.shape != (B + 1,) or kv_len.shape != (B,):
        raise ValueError(f"q_start must be [{B + 1}] and kv_len [{B}] for a page table of {B} rows")
    d = PagedBatch(_ptr(q_start, "q_start").value, _ptr(kv_len, "kv_len").value, _ptr(page_table, "page_table").value,
                   B, max_pages)
    d._keep = (q_start, kv_len, page_table)
    return d


# (These run at every decode step: pointers as plain integers, each tensor
# property asked for once.)

def _rows(t, name: str, heads: int, dim: int, dtype):
    """Address and token stride of [T, heads, dim] CUDA rows whose heads are dense."""
    shape, s = t.shape, t.stride()
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if len(shape) != 3 or shape[1] != heads or shape[2] != dim:
        raise ValueError(f"{name} must be [T, {heads}, {dim}], got {tuple(shape)}")
    if s[2] != 1 or (s[1] != dim and heads > 1):
        raise ValueError(f"{name}'s heads must be dense")
    return t.data_ptr(), (s[0] if shape[0] > 1 else heads * dim)


_IO_DTYPES = {torch.float16: EXL3_OUT_F16, torch.float32: EXL3_OUT_F32}
_OUT_DTYPES = {EXL3_OUT_F16: torch.float16, EXL3_OUT_F32: torch.float32}


def _io_dtype(t, name: str) -> int:
    if not isinstance(t, torch.Tensor) or t.dtype not in _IO_DTYPES:
        raise TypeError(f"{name} must be a torch.float16 or torch.float32 tensor")
    return _IO_DTYPES[t.dtype]


def _out(t, name: str, shape, dtype) -> int:
    """Address of a dense CUDA output of the given shape and type."""
    if t.shape != shape or t.dtype != dtype or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA tensor {shape} {dtype}, got {tuple(t.shape)} {t.dtype}")
    return t.data_ptr()


def _workspace_arg(buf, nbytes: int, device, stream, raw: int):
    """Address and bytes of a call's workspace: the caller's, or the cached one."""
    if buf is not None:
        address = _ptr(buf, "workspace")
        if buf.get_device() != device.index:
            raise ValueError(f"the workspace is on {buf.device}, the call's tensors on {device}")
        return address, buf.numel() * buf.element_size()
    hit = _ws_cache.get((device.index, raw))
    if hit is None or hit[2] < nbytes:
        buf = workspace(nbytes, device, stream)
        return buf.data_ptr(), buf.numel()
    return hit[1], hit[2]


def _positions(t, T: int):
    if t is None:
        return None
    if t.dtype != torch.int32 or t.shape != (T,) or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"positions must be a contiguous CUDA int32 tensor of {T}")
    return t.data_ptr()


def _check_transform(transform: HeadTransform, dim: int):
    for n in transform._norm_sizes:
        if n is not None and n != dim:
            raise ValueError(f"norm weights must have {dim} elements, got {n}")


def exl3_qk_norm_rope(q, k, positions, transform: HeadTransform, q_out=None, k_out=None,
                      out_dtype: int = EXL3_OUT_F16, stream=None):
    """Head norms and rotary positions of q [T, Hq, D] and k [T, Hkv, D] (or None), fp16 or fp32;
    positions int32 [T] (None without rotation); returns (q_out, k_out), which may be q and k."""
    in_dtype, odt = _io_dtype(q, "q"), _OUT_DTYPES.get(out_dtype, torch.float16)
    T, Hq, D = q.shape
    Hkv = 0 if k is None else k.shape[1]
    if q_out is None:
        q_out = torch.empty((T, Hq, D), dtype=odt, device=q.device)
    if k_out is None and k is not None:
        k_out = torch.empty((T, Hkv, D), dtype=odt, device=q.device)
    _check_transform(transform, D)
    qp, qs = _rows(q, "q", Hq, D, q.dtype)
    kp, ks, kop = None, 0, None
    if k is not None:
        if k.shape[0] != T:
            raise ValueError(f"k must have {T} rows, got {k.shape[0]}")
        kp, ks = _rows(k, "k", Hkv, D, q.dtype)
        kop = _out(k_out, "k_out", (T, Hkv, D), odt)
    qop, pp = _out(q_out, "q_out", (T, Hq, D), odt), _positions(positions, T)
    if T:
        _check(lib().exl3_qk_norm_rope(qp, qs, kp, ks, in_dtype, T, Hq, Hkv, D, ctypes.byref(transform), pp, qop, kop,
                                       out_dtype, _raw_stream(stream)))
    return q_out, k_out


def exl3_qkv_append_workspace_size() -> int:
    return lib().exl3_qkv_append_workspace_size()


# (sizes of calls that a decode loop repeats)
_append_workspace = functools.cache(exl3_qkv_append_workspace_size)


def exl3_qkv_append(q, k, v, batch: PagedBatch, cache: KvCache, transform: HeadTransform, positions=None, q_out=None,
                    workspace_buf=None, stream=None) -> torch.Tensor:
    """Norm and rotate q [T, Hq, D], k and v [T, Hkv, D] (fp16 or fp32), write k and v to their
    places in the cache; returns q_out [T, Hq, D] fp16.  positions int32 [T], or None for the
    tokens' cache indexes."""
    in_dtype = _io_dtype(q, "q")
    T, Hq, D = q.shape
    if q_out is None:
        q_out = torch.empty((T, Hq, D), dtype=torch.float16, device=q.device)
    if D != cache.head_dim or k.shape[0] != T or v.shape[0] != T:
        raise ValueError(f"q, k and v must have {T} rows of heads of {cache.head_dim}")
    _check_transform(transform, D)
    qp, qs = _rows(q, "q", Hq, D, q.dtype)
    kp, ks = _rows(k, "k", cache.heads_kv, D, q.dtype)
    vp, vs = _rows(v, "v", cache.heads_kv, D, q.dtype)
    qop, pp = _out(q_out, "q_out", (T, Hq, D), torch.float16), _positions(positions, T)
    if T:
        raw = _raw_stream(stream)
        wp, wn = _workspace_arg(workspace_buf, _append_workspace(), q.device, stream, raw)
        _check(lib().exl3_qkv_append(qp, qs, kp, ks, vp, vs, in_dtype, T, Hq, ctypes.byref(transform), pp,
                                     ctypes.byref(batch), ctypes.byref(cache), qop, wp, wn, raw))
    return q_out


def exl3_paged_attention_workspace_size(T: int, heads_q: int, heads_kv: int, head_dim: int, batch: int) -> int:
    return lib().exl3_paged_attention_workspace_size(T, heads_q, heads_kv, head_dim, batch)


@functools.lru_cache(maxsize=4096)
def _attention_workspace(device: int, T: int, heads_q: int, heads_kv: int, head_dim: int, batch: int) -> int:
    """The size depends on the current device's number of SMs too: `device` is its index."""
    return exl3_paged_attention_workspace_size(T, heads_q, heads_kv, head_dim, batch)


def exl3_paged_attention(q, batch: PagedBatch, cache: KvCache, scale: float | None = None, causal: bool = True,
                         window: int = 0, out_dtype: int = EXL3_OUT_F16, y=None, lse=None, workspace_buf=None,
                         stream=None) -> torch.Tensor:
    """Attention of the new tokens q [T, Hq, D] fp16 over the paged cache that already holds their
    keys and values; returns y [T, Hq, D].  scale defaults to D ** -0.5; window > 0 keeps the last
    `window` tokens; lse, if given, is an fp32 [T, Hq] output (natural logarithm)."""
    T, Hq, D = q.shape
    odt = _OUT_DTYPES.get(out_dtype, torch.float16)
    if y is None:
        y = torch.empty((T, Hq, D), dtype=odt, device=q.device)
    if D != cache.head_dim:
        raise ValueError(f"q has heads of {D}, the cache of {cache.head_dim}")
    qp, qs = _rows(q, "q", Hq, D, torch.float16)
    yp = _out(y, "y", (T, Hq, D), odt)
    lp = None if lse is None else _out(lse, "lse", (T, Hq), torch.float32)
    if T:
        raw = _raw_stream(stream)
        need = _attention_workspace(torch.cuda.current_device(), T, Hq, cache.heads_kv, D, batch.batch)
        wp, wn = _workspace_arg(workspace_buf, need, q.device, stream, raw)
        _check(lib().exl3_paged_attention(qp, qs, T, Hq, ctypes.byref(batch), ctypes.byref(cache),
                                          D ** -0.5 if scale is None else scale, 1 if causal else 0, window, yp,
                                          out_dtype, lp, wp, wn, raw))
    return y


# -------------------------------------------------------- routing to experts

# (As above: pointers as plain integers, each property asked for once.)

def _on_current(t, name: str) -> int:
    """The current device, on which t has to be: its stream gets the kernels."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    d = t.get_device()
    if d < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    if d != torch._C._cuda_getDevice():
        raise ValueError(f"{name} is on {t.device}, the current device is cuda:{torch.cuda.current_device()}")
    return d


def _matrix(t, name: str, width: int, dtypes, device: int):
    """Address, row stride and number of rows of [rows, width] with dense rows on the given device."""
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(str(d) for d in dtypes)}, got {t.dtype}")
    shape = t.shape
    if len(shape) != 2 or shape[1] != width:
        raise ValueError(f"{name} must be [rows, {width}], got {tuple(shape)}")
    if t.get_device() != device:
        raise ValueError(f"{name} must be on the other tensors' device cuda:{device}, got {t.device}")
    s0, s1 = t.stride()
    if s1 != 1 and width > 1:
        raise ValueError(f"{name}'s rows must be dense")
    rows = shape[0]
    return t.data_ptr(), (s0 if rows > 1 else width), rows


def _dense(t, name: str, shape, dtype, device: int) -> int:
    """Address of a dense output of the given shape and type on the given device."""
    if t.shape != shape or t.dtype is not dtype or t.get_device() != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA tensor {shape} {dtype} on cuda:{device}, got "
                         f"{tuple(t.shape)} {t.dtype} on {t.device}")
    return t.data_ptr()


def _stream_of(stream, device: int) -> int:
    """The given stream's handle, or that of the device's current one."""
    return torch._C._cuda_getCurrentRawStream(device) if stream is None else stream.cuda_stream


_F16, _F32, _F16_F32 = (torch.float16,), (torch.float32,), (torch.float16, torch.float32)


def _vector(t, name: str, size: int, dtype):
    """Address of a dense [size] tensor, or None."""
    if t is None:
        return None
    _on_current(t, name)
    if t.dtype != dtype or t.shape != (size,) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of {size}, got {tuple(t.shape)} {t.dtype}")
    return t.data_ptr()


def router(w, bias=None, stream=None) -> Router:
    """Descriptor of a router: w [E, k] fp16, used as it is, or fp32, packed once into two fp16
    parts (exl3_router_pack); bias fp32 [E] or None.  The tensors are kept alive with it."""
    if not isinstance(w, torch.Tensor) or w.dim() != 2 or w.dtype not in (torch.float16, torch.float32):
        raise TypeError("w must be a torch.float16 or torch.float32 tensor [E, k]")
    E, k = w.shape
    _on_current(w, "w")
    parts, scale = w, None
    if w.dtype == torch.float32:
        with _made_on(stream):
            parts = torch.empty((2, E, k), dtype=torch.float16, device=w.device)
            scale = torch.empty(E, dtype=torch.float32, device=w.device)
        _check(lib().exl3_router_pack(_ptr(w, "w"), E, k, _ptr(parts, "packed"), _ptr(scale, "scale"), _stream(stream)))
    d = Router(_ptr(parts, "w").value, None if scale is None else scale.data_ptr(),
               _vector(bias, "bias", E, torch.float32), E, k)
    d._keep, d._address, d._device, d._shape = (parts, scale, bias), ctypes.addressof(d), w.get_device(), (E, k)
    return d


def exl3_router_pack(w, packed=None, scale=None, stream=None):
    """fp32 router weights [E, k] as two fp16 parts [2, E, k] and powers of two [E]; returns both."""
    E, k = w.shape
    _on_current(w, "w")
    if w.dtype != torch.float32:
        raise TypeError(f"w must be torch.float32, got {w.dtype}")
    if packed is None:
        packed = torch.empty((2, E, k), dtype=torch.float16, device=w.device)
    if scale is None:
        scale = torch.empty(E, dtype=torch.float32, device=w.device)
    _check(lib().exl3_router_pack(_ptr(w, "w"), E, k, _out(packed, "packed", (2, E, k), torch.float16),
                                  _vector(scale, "scale", E, torch.float32), _raw_stream(stream)))
    return packed, scale


def exl3_router_logits_workspace_size() -> int:
    return lib().exl3_router_logits_workspace_size()


_logits_workspace = functools.cache(exl3_router_logits_workspace_size)


def exl3_router_logits(x, router: Router, logits=None, workspace_buf=None, stream=None) -> torch.Tensor:
    """logits [T, E] fp32 = x @ w^T (+ bias) for x [T, k] fp16 with dense rows."""
    device = _on_current(x, "x")
    E, k = router._shape
    xp, xs, T = _matrix(x, "x", k, _F16, device)
    if router._device != device:
        raise ValueError(f"the router is on cuda:{router._device}, x on cuda:{device}")
    if logits is None:
        logits = torch.empty((T, E), dtype=torch.float32, device=x.device)
    lp = _dense(logits, "logits", (T, E), torch.float32, device)
    if T:
        raw = _stream_of(stream, device)
        wp, wn = _workspace_arg(workspace_buf, _logits_workspace(), x.device, stream, raw)
        rc = lib().exl3_router_logits(xp, xs, T, router._address, lp, wp, wn, raw)
        if rc:
            _check(rc)
    return logits


def route_rule(topk: int, score: int = EXL3_SCORE_SOFTMAX, bias=None, groups: int = 1, groups_kept: int | None = None,
               group_score: int = EXL3_GROUP_MAX, renormalise: bool = True, scale: float = 1.0) -> RouteRule:
    """Descriptor of how experts are chosen: softmax or sigmoid scores, a bias fp32 [E] (or None)
    added for the choice only, groups of consecutive experts of which groups_kept stay, topk
    experts, weights divided by their sum and multiplied by scale."""
    bp = None
    if bias is not None:
        if not isinstance(bias, torch.Tensor) or bias.dim() != 1:
            raise TypeError("bias must be a torch tensor [E]")
        bp = _vector(bias, "bias", bias.shape[0], torch.float32)
    d = RouteRule(score, bp, groups, groups if groups_kept is None else groups_kept, group_score, topk,
                  1 if renormalise else 0, scale)
    d._keep, d._address = (bias,), ctypes.addressof(d)
    d._experts, d._device = (None, None) if bias is None else (bias.shape[0], bias.get_device())
    return d


def exl3_route(logits, rule: RouteRule, ids=None, weights=None, stream=None):
    """Experts and weights of each token from logits [T, E] (fp32 or fp16, dense rows): ids int32
    and weights fp32, [T, topk], as exl3_moe_grouped takes them."""
    device = _on_current(logits, "logits")
    shape, topk, bias = logits.shape, rule.topk, rule._experts
    if len(shape) != 2:
        raise ValueError(f"logits must be [T, E], got {tuple(shape)}")
    T, E = shape
    lp, ls, _ = _matrix(logits, "logits", E, _F16_F32, device)
    if bias is not None and (bias != E or rule._device != device):
        raise ValueError(f"the rule's bias has {bias} experts on cuda:{rule._device}, the logits {E} on cuda:{device}")
    if ids is None:
        ids = torch.empty((T, topk), dtype=torch.int32, device=logits.device)
    if weights is None:
        weights = torch.empty((T, topk), dtype=torch.float32, device=logits.device)
    out = (T, topk)
    ip, wp = _dense(ids, "ids", out, torch.int32, device), _dense(weights, "weights", out, torch.float32, device)
    if T:
        rc = lib().exl3_route(lp, ls, _IO_DTYPES[logits.dtype], T, E, rule._address, ip, wp, _stream_of(stream, device))
        if rc:
            _check(rc)
    return ids, weights


# --------------------------------------------------------- low-rank adapters

def adapters(a, b, scale, rank=None) -> Adapters:
    """Descriptor of a pool of adapters for one linear: a [count, max_rank, k] and b [count, n,
    max_rank] fp16, scale fp32 [count], rank int32 [count] or None (all of max_rank); the tensors
    are kept alive with it."""
    for t, name in ((a, "a"), (b, "b")):
        _check_fp16(t, name)
        _on_current(t, name)
        if t.dim() != 3:
            raise ValueError(f"{name} must have three dimensions, got {tuple(t.shape)}")
    N, R, k = a.shape
    n = b.shape[1]
    if b.shape != (N, n, R):
        raise ValueError(f"b must be [{N}, n, {R}] for a {tuple(a.shape)}, got {tuple(b.shape)}")
    if scale is None:
        raise TypeError("scale must be a torch tensor")
    d = Adapters(_ptr(a, "a", 2).value, _ptr(b, "b", 2).value, _vector(scale, "scale", N, torch.float32),
                 _vector(rank, "rank", N, torch.int32), N, R, k, n)
    d._keep, d._address, d._device, d._shape = (a, b, scale, rank), ctypes.addressof(d), a.get_device(), (N, R, k, n)
    return d


class AdapterPlan:
    """A step's rows in the order of their adapters (exl3_adapter_plan): the device buffer and what
    it was made for."""
    def __init__(self, T: int, batch: int, count: int, device, stream=None):
        nbytes = exl3_adapter_plan_size(T, batch, count)
        if nbytes == 0:
            raise ValueError(f"T = {T}, batch = {batch} or count = {count} out of range")
        self.T, self.batch, self.count = T, batch, count
        with _made_on(stream):               # (the memory of the stream that fills it)
            self.data = torch.empty(nbytes, dtype=torch.uint8, device=device)
        self.address, self.device = self.data.data_ptr(), self.data.get_device()
        exl3_workspace_clear(self.data, stream=stream)


def exl3_adapter_plan_size(T: int, batch: int, count: int) -> int:
    return lib().exl3_adapter_plan_size(T, batch, count)


def exl3_adapter_plan(q_start, adapter, T: int, count: int, plan: AdapterPlan | None = None, stream=None) -> AdapterPlan:
    """Plan of a step: sequence b is rows q_start[b] .. q_start[b + 1] - 1 of T and uses adapter[b]
    of `count` (-1: none); int32 device tensors [B + 1] and [B].  `plan`, made for the same sizes,
    is filled again."""
    for t, name in ((q_start, "q_start"), (adapter, "adapter")):
        _on_current(t, name)
        if t.dtype != torch.int32 or t.dim() != 1:
            raise TypeError(f"{name} must be a torch.int32 tensor of one dimension, got {t.dtype} {tuple(t.shape)}")
    B = adapter.shape[0]
    if q_start.shape[0] != B + 1:
        raise ValueError(f"q_start must have {B + 1} elements for {B} adapters, got {q_start.shape[0]}")
    if plan is None:
        plan = AdapterPlan(T, B, count, adapter.device, stream)
    elif (plan.T, plan.batch, plan.count) != (T, B, count):
        raise ValueError(f"plan was made for T = {plan.T}, batch = {plan.batch}, count = {plan.count}")
    elif plan.device != adapter.get_device():
        raise ValueError(f"plan is on cuda:{plan.device}, q_start and adapter on {adapter.device}")
    _check(lib().exl3_adapter_plan(_ptr(q_start, "q_start"), _ptr(adapter, "adapter"), T, B, count,
                                   plan.address, plan.data.numel(), _raw_stream(stream)))
    return plan


def exl3_adapter_add_workspace_size(T: int, max_rank: int) -> int:
    return lib().exl3_adapter_add_workspace_size(T, max_rank)


def exl3_adapter_scratch_size(T: int, max_rank: int, n: int) -> int:
    return lib().exl3_adapter_scratch_size(T, max_rank, n)


@functools.lru_cache(maxsize=4096)
def _adapter_sizes(T: int, max_rank: int, n: int):
    return exl3_adapter_add_workspace_size(T, max_rank), exl3_adapter_scratch_size(T, max_rank, n)


def _capturing(stream, raw: int, device: int) -> bool:
    """Is the stream of a call being captured?  (Never the default one; asking takes the driver 0.4 us.)"""
    if raw == 0:
        return False
    if stream is None or raw == torch._C._cuda_getCurrentRawStream(device):
        return torch._C._cuda_isCurrentStreamCapturing()
    with _made_on(stream):
        return torch._C._cuda_isCurrentStreamCapturing()


def exl3_adapter_add(x, y, adapters: Adapters, plan: AdapterPlan, out=None, workspace_buf=None,
                     stream=None) -> torch.Tensor:
    """y + scale (x A^T) B^T for each row's adapter: x [T, k] fp16, y [T, n] fp16 or fp32, dense
    rows; written to `out`, or to y itself (rows of no sequence are left as they were)."""
    return _adapter_add(x, y, adapters, plan, out, workspace_buf, stream, None, False)


def exl3_adapter_add_scratch(x, y, adapters: Adapters, plan: AdapterPlan, scratch, out=None, workspace_buf=None,
                             stream=None) -> torch.Tensor:
    """exl3_adapter_add with a buffer of exl3_adapter_scratch_size(T, max_rank, n) bytes that no call
    running at once shares, or None where that is 0; the workspace holds the error word only."""
    return _adapter_add(x, y, adapters, plan, out, workspace_buf, stream, scratch, True)


def _adapter_add(x, y, adapters: Adapters, plan: AdapterPlan, out, workspace_buf, stream, scratch, apart: bool):
    device, dtype, T = _on_current(x, "x"), y.dtype, plan.T
    N, R, k, n = adapters._shape
    xp, xs, xr = _matrix(x, "x", k, _F16, device)
    yp, ys, yr = _matrix(y, "y", n, _F16_F32, device)
    if out is None or out is y:
        out, op, os_, rows = y, yp, ys, yr
    else:
        op, os_, rows = _matrix(out, "out", n, _F16 if dtype is torch.float16 else _F32, device)
    if not xr == yr == rows == T:
        raise ValueError(f"x has {xr} rows, y {yr}, out {rows}, the plan {T}")
    if T == 0:
        return out
    if plan.device != device or adapters._device != device or plan.count != N:
        raise ValueError(f"x is on cuda:{device}; the plan is for {plan.count} adapters on cuda:{plan.device}, the pool "
                         f"has {N} on cuda:{adapters._device}")
    raw, (need, scratch_need) = _stream_of(stream, device), _adapter_sizes(T, R, n)
    if not apart and workspace_buf is None and scratch_need and _capturing(stream, raw, device):
        # a graph gets scratch of its own, in its own memory: two that share the stream's would race when they
        # run at once.  Errors are found in the stream's workspace, as every captured call's are.
        with _made_on(stream):
            scratch = torch.empty(scratch_need, dtype=torch.uint8, device=x.device)
        apart = True
    if apart:
        wp, wn = _workspace_arg(workspace_buf, 256, x.device, stream, raw)
        sp, sn = (None, 0) if scratch is None else (_ptr(scratch, "scratch"), scratch.numel() * scratch.element_size())
        if scratch is not None and scratch.get_device() != device:
            raise ValueError(f"the scratch is on {scratch.device}, x on cuda:{device}")
        rc = lib().exl3_adapter_add_scratch(xp, xs, yp, ys, op, os_, _IO_DTYPES[dtype], adapters._address, plan.address, T,
                                            plan.batch, wp, wn, sp, sn, raw)
    else:
        wp, wn = _workspace_arg(workspace_buf, need, x.device, stream, raw)
        rc = lib().exl3_adapter_add(xp, xs, yp, ys, op, os_, _IO_DTYPES[dtype], adapters._address, plan.address, T,
                                    plan.batch, wp, wn, raw)
    if rc:
        _check(rc)
    return out
