"""ctypes binding of libattn.so (include/attn.h).

Argument marshalling only: tensors become device pointers, the torch stream
becomes a ``cudaStream_t``; every step of the computation runs in the
library's CUDA kernels.  There is no fallback: if the library is missing or
cannot be loaded, every call raises.
"""
from __future__ import annotations

import ctypes
import math
import os
import threading

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libattn.so")

ATTN_STATUS = {
    0: "ATTN_OK", -1: "ATTN_ERR_NULL", -2: "ATTN_ERR_ALIGN", -3: "ATTN_ERR_SHAPE",
    -4: "ATTN_ERR_DEVICE", -5: "ATTN_ERR_LAUNCH", -6: "ATTN_ERR_ALLOC", -7: "ATTN_ERR_TMA",
    -8: "ATTN_ERR_CUDA", -9: "ATTN_ERR_SCRATCH",
}
EXPORTED = ["attn_fwd", "attn_fwd_rows", "attn_fwd_fp8", "attn_fwd_host", "attn_fwd_host_workspace_bytes",
            "attn_decode_splitkv", "attn_decode_splitkv_noalloc",
            "attn_status_string", "attn_get_device_error", "attn_decode_workspace_bytes",
            "attn_selftest_wait_timeout", "attn_decode_splitkv_states", "attn_combine_states",
            "attn_decode_graph_create", "attn_decode_graph_launch", "attn_decode_graph_destroy",
            "attn_fwd_mod", "attn_row_ranges", "attn_decode_varlen", "attn_decode_prefix"]
DEVERR_SELFTEST = 0x10
NOALLOC_SCRATCH_BYTES = 8 * 1024 * 1024

_lock = threading.Lock()
_lib = None


class AttnError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(msg)
        self.status = status


def load(path: str = LIB_PATH):
    """Load libattn.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(path):
            raise RuntimeError(f"{path} is missing: build it with "
                               "`python -m attention_forward_sm_gb300._build`")
        lib = ctypes.CDLL(path)
        vp, i, f = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
        lib.attn_fwd.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, i, i, f, vp]
        lib.attn_fwd.restype = i
        lib.attn_fwd_rows.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, i, i, i, f, vp]
        lib.attn_fwd_rows.restype = i
        lib.attn_fwd_host.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, i, i, f, vp]
        lib.attn_fwd_host.restype = i
        lib.attn_fwd_host_workspace_bytes.argtypes = [i, i, i, i, i, i]
        lib.attn_fwd_host_workspace_bytes.restype = ctypes.c_longlong
        lib.attn_fwd_fp8.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, i, i, f, f, f, f, vp]
        lib.attn_fwd_fp8.restype = i
        lib.attn_decode_splitkv.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, i, vp]
        lib.attn_decode_splitkv.restype = i
        lib.attn_decode_splitkv_noalloc.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, i, vp]
        lib.attn_decode_splitkv_noalloc.restype = i
        lib.attn_status_string.argtypes = [i]
        lib.attn_status_string.restype = ctypes.c_char_p
        lib.attn_get_device_error.argtypes = [vp]
        lib.attn_get_device_error.restype = i
        lib.attn_decode_splitkv_states.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, i, vp]
        lib.attn_decode_splitkv_states.restype = i
        lib.attn_combine_states.argtypes = [vp, vp, vp, vp, i, i, i, vp]
        lib.attn_combine_states.restype = i
        lib.attn_selftest_wait_timeout.argtypes = [ctypes.c_uint, vp]
        lib.attn_selftest_wait_timeout.restype = i
        lib.attn_decode_graph_create.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, i,
                                                 ctypes.POINTER(vp)]
        lib.attn_decode_graph_create.restype = i
        lib.attn_decode_graph_launch.argtypes = [vp, vp]
        lib.attn_decode_graph_launch.restype = i
        lib.attn_decode_graph_destroy.argtypes = [vp]
        lib.attn_decode_graph_destroy.restype = i
        lib.attn_fwd_mod.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, i, i, i, f, f, vp, vp, vp]
        lib.attn_fwd_mod.restype = i
        lib.attn_row_ranges.argtypes = [vp, vp, vp, i, i, i, i, vp]
        lib.attn_row_ranges.restype = i
        lib.attn_decode_varlen.argtypes = [vp, vp, vp, vp, vp, vp, i, i, i, i, i, f, f, vp, vp]
        lib.attn_decode_varlen.restype = i
        lib.attn_decode_prefix.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, f, f,
                                           vp, vp]
        lib.attn_decode_prefix.restype = i
        lib.attn_decode_workspace_bytes.argtypes = [i, i, i, i]
        lib.attn_decode_workspace_bytes.restype = ctypes.c_longlong
        _lib = lib
        return lib


def _ptr(x) -> int:
    if x is None:
        return 0
    if isinstance(x, int):
        return x
    return x.data_ptr()


def _int(x) -> int:
    """A size for a C int, which would take what does not fit modulo 2^32."""
    x = int(x)
    if not -2**31 <= x < 2**31:
        _check(-3)  # ATTN_ERR_SHAPE
    return x


_LEAST_CAP = 2.0 ** -149  # below it a float would round to 0, which stands for no cap


def _cap(softcap) -> float:
    softcap = float(softcap)
    if 0 < softcap < _LEAST_CAP:
        _check(-3)  # ATTN_ERR_SHAPE
    return softcap


def _stream(stream) -> int:
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(rc: int):
    if rc != 0:
        msg = load().attn_status_string(rc).decode()
        raise AttnError(rc, msg)


# ----------------------------------------------------------------------------- C-ABI names


def attn_fwd(q, k, v, o, lse, B, Hq, Hkv, Nq, Nk, D, causal, scale, stream=None) -> None:
    """``attn_fwd`` of include/attn.h: tensors (or raw device pointers), sizes,
    causal flag, scale, and a torch stream / raw handle (None = current)."""
    _check(load().attn_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), int(B), int(Hq),
                           int(Hkv), int(Nq), int(Nk), int(D), int(bool(causal)), float(scale),
                           _stream(stream)))


def attn_fwd_rows(q, k, v, o, lse, B, Hq, Hkv, Nq, Nk, D, causal, q_offset, scale,
                  stream=None) -> None:
    """``attn_fwd_rows`` of include/attn.h: ``attn_fwd`` for query rows
    q_offset .. q_offset+Nq-1 of a longer sequence (the causal mask uses the
    global row index)."""
    _check(load().attn_fwd_rows(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), int(B), int(Hq),
                                int(Hkv), int(Nq), int(Nk), int(D), int(bool(causal)),
                                int(q_offset), float(scale), _stream(stream)))


def attn_fwd_host(q, k, v, o, lse, B, Hq, Hkv, Nq, Nk, D, causal, scale, stream=None) -> None:
    """``attn_fwd_host`` of include/attn.h: host (CPU, ideally pinned) tensors
    in and out; asynchronous on the stream."""
    _check(load().attn_fwd_host(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), int(B), int(Hq),
                                int(Hkv), int(Nq), int(Nk), int(D), int(bool(causal)),
                                float(scale), _stream(stream)))


def attn_fwd_host_workspace_bytes(B, Hq, Hkv, Nq, Nk, D) -> int:
    return int(load().attn_fwd_host_workspace_bytes(int(B), int(Hq), int(Hkv), int(Nq), int(Nk),
                                                    int(D)))


def attn_fwd_fp8(q, k, vt, o, lse, B, Hq, Hkv, Nq, Nk, D, causal, scale, q_scale, k_scale,
                 v_scale, stream=None) -> None:
    """``attn_fwd_fp8`` of include/attn.h: e4m3 q, k and V transposed
    ([B, Hkv, D, Nk]), per-tensor dequantisation scales, bf16 o."""
    _check(load().attn_fwd_fp8(_ptr(q), _ptr(k), _ptr(vt), _ptr(o), _ptr(lse), int(B), int(Hq),
                               int(Hkv), int(Nq), int(Nk), int(D), int(bool(causal)),
                               float(scale), float(q_scale), float(k_scale), float(v_scale),
                               _stream(stream)))


def attn_decode_splitkv(q, kcache, vcache, o, lse, B, Hq, Hkv, Nk, D, nsplit, stream=None) -> None:
    """``attn_decode_splitkv`` of include/attn.h."""
    _check(load().attn_decode_splitkv(_ptr(q), _ptr(kcache), _ptr(vcache), _ptr(o), _ptr(lse),
                                      int(B), int(Hq), int(Hkv), int(Nk), int(D), int(nsplit),
                                      _stream(stream)))


def attn_decode_splitkv_noalloc(q, kcache, vcache, o, lse, B, Hq, Hkv, Nk, D, nsplit,
                                stream=None) -> None:
    """``attn_decode_splitkv_noalloc`` of include/attn.h: the same decode for
    callers that cannot allocate device memory during the call; its scratch
    is a fixed 8 MiB device array shared by all calls on a device (order
    calls that could overlap on the GPU)."""
    _check(load().attn_decode_splitkv_noalloc(_ptr(q), _ptr(kcache), _ptr(vcache), _ptr(o),
                                              _ptr(lse), int(B), int(Hq), int(Hkv), int(Nk),
                                              int(D), int(nsplit), _stream(stream)))


def attn_status_string(status: int) -> str:
    return load().attn_status_string(int(status)).decode()


def attn_get_device_error(stream=None) -> int:
    """Synchronise the stream, return and clear the device error word."""
    rc = load().attn_get_device_error(_stream(stream))
    if rc < 0:
        _check(rc)
    return rc


def attn_decode_splitkv_states(q, kcache, vcache, o_state, lse, B, Hq, Hkv, Nk, D, nsplit,
                               stream=None) -> None:
    """``attn_decode_splitkv_states`` of include/attn.h (fp32 state output)."""
    _check(load().attn_decode_splitkv_states(_ptr(q), _ptr(kcache), _ptr(vcache), _ptr(o_state),
                                             _ptr(lse), int(B), int(Hq), int(Hkv), int(Nk),
                                             int(D), int(nsplit), _stream(stream)))


def attn_combine_states(part_o, part_lse, o, lse, rows, nparts, D, stream=None) -> None:
    """``attn_combine_states`` of include/attn.h."""
    _check(load().attn_combine_states(_ptr(part_o), _ptr(part_lse), _ptr(o), _ptr(lse), int(rows),
                                      int(nparts), int(D), _stream(stream)))


def attn_selftest_wait_timeout(limit_us: int, stream=None) -> None:
    """Launch the bounded-wait self-test (a wait that is meant to run out)."""
    _check(load().attn_selftest_wait_timeout(int(limit_us), _stream(stream)))


def attn_decode_graph_create(q, kcache, vcache, o, lse, B, Hq, Hkv, Nk, D, nsplit) -> int:
    """``attn_decode_graph_create`` of include/attn.h; returns the handle (an
    integer).  The buffers are bound by address until the handle is
    destroyed: keep the tensors alive."""
    h = ctypes.c_void_p()
    _check(load().attn_decode_graph_create(_ptr(q), _ptr(kcache), _ptr(vcache), _ptr(o),
                                           _ptr(lse), int(B), int(Hq), int(Hkv), int(Nk), int(D),
                                           int(nsplit), ctypes.byref(h)))
    return int(h.value)


def attn_decode_graph_launch(handle: int, stream=None) -> None:
    """``attn_decode_graph_launch`` of include/attn.h: replay one decode step."""
    _check(load().attn_decode_graph_launch(handle or None, _stream(stream)))


def attn_decode_graph_destroy(handle: int) -> None:
    """``attn_decode_graph_destroy`` of include/attn.h."""
    _check(load().attn_decode_graph_destroy(handle or None))


def attn_fwd_mod(q, k, v, o, lse, B, Hq, Hkv, Nq, Nk, D, causal, q_offset, scale, softcap=0.0,
                 slopes=None, ranges=None, stream=None) -> None:
    """``attn_fwd_mod`` of include/attn.h: ``attn_fwd_rows`` with capped scores,
    a distance bias (``slopes`` [Hq] fp32) and a key range per query row
    (``ranges`` [B, Nq, 2] int32)."""
    _check(load().attn_fwd_mod(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _int(B), _int(Hq),
                               _int(Hkv), _int(Nq), _int(Nk), _int(D), int(bool(causal)),
                               _int(q_offset), float(scale), _cap(softcap), _ptr(slopes),
                               _ptr(ranges), _stream(stream)))


def attn_row_ranges(doc_lens, prefix_lens, ranges, B, N, M, causal, stream=None) -> None:
    """``attn_row_ranges`` of include/attn.h: the key ranges of packed documents."""
    _check(load().attn_row_ranges(_ptr(doc_lens), _ptr(prefix_lens), _ptr(ranges), _int(B), _int(N),
                                  _int(M), int(bool(causal)), _stream(stream)))


def attn_decode_varlen(q, kcache, vcache, lens, o, lse, B, Hq, Hkv, Ncap, D, scale, softcap=0.0,
                       slopes=None, stream=None) -> None:
    """``attn_decode_varlen`` of include/attn.h: decode with a length per
    request (``lens`` [B] int32 on the device, or None: all Ncap keys)."""
    _check(load().attn_decode_varlen(_ptr(q), _ptr(kcache), _ptr(vcache), _ptr(lens), _ptr(o),
                                     _ptr(lse), _int(B), _int(Hq), _int(Hkv), _int(Ncap), _int(D),
                                     float(scale), _cap(softcap), _ptr(slopes),
                                     _stream(stream)))


def attn_decode_prefix(q, kprefix, vprefix, kcache, vcache, lens, o, lse, B, Hq, Hkv, Np, Ncap, D,
                       scale, softcap=0.0, slopes=None, stream=None) -> None:
    """``attn_decode_prefix`` of include/attn.h: ``attn_decode_varlen`` behind a
    prefix (``kprefix`` / ``vprefix`` [Hkv, Np, D]) that all requests share."""
    _check(load().attn_decode_prefix(_ptr(q), _ptr(kprefix), _ptr(vprefix), _ptr(kcache),
                                     _ptr(vcache), _ptr(lens), _ptr(o), _ptr(lse), _int(B), _int(Hq),
                                     _int(Hkv), _int(Np), _int(Ncap), _int(D), float(scale),
                                     _cap(softcap), _ptr(slopes), _stream(stream)))


def attn_decode_workspace_bytes(B, Hq, D, nsplit) -> int:
    return int(load().attn_decode_workspace_bytes(int(B), int(Hq), int(D), int(nsplit)))


# ----------------------------------------------------------------------------- tensor helpers


def _check_ranks(tensors: dict, ranks: dict):
    import torch
    for name, x in tensors.items():
        if not isinstance(x, torch.Tensor):
            raise TypeError(f"{name} must be a torch tensor")
        if x.dim() != ranks[name]:
            raise ValueError(f"{name} must have {ranks[name]} dimensions, got {x.dim()}")


def _check_inputs(tensors: dict, shapes: dict):
    """The helpers below pass raw pointers to the library, which cannot see
    dtypes or strides: check here that every input is a contiguous bf16 CUDA
    tensor, all on one device, with the expected ranks and matching sizes
    (``shapes`` maps a size name to the values the tensors give it)."""
    import torch
    dev = None
    for name, x in tensors.items():
        if x.dtype != torch.bfloat16:
            raise TypeError(f"{name} must be bfloat16, got {x.dtype}")
        if not x.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
        if not x.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        if dev is None:
            dev = x.device
        elif x.device != dev:
            raise ValueError(f"{name} is on {x.device}, expected {dev}")
    for size, values in shapes.items():
        if len(set(values)) != 1:
            raise ValueError(f"inconsistent {size}: {values}")



def forward(q, k, v, causal: bool = False, scale: float | None = None, stream=None):
    """O, LSE = attention(q [B,Hq,Nq,D], k/v [B,Hkv,Nk,D]) with outputs
    allocated by torch on q's device."""
    import torch
    _check_ranks({"q": q, "k": k, "v": v}, {"q": 4, "k": 4, "v": 4})  # [B, H, N, D]
    _check_inputs({"q": q, "k": k, "v": v},
                  {"B": (q.shape[0], k.shape[0], v.shape[0]), "D": (q.shape[3], k.shape[3], v.shape[3]),
                   "Hkv": (k.shape[1], v.shape[1]), "Nk": (k.shape[2], v.shape[2])})
    B, Hq, Nq, D = q.shape
    Hkv, Nk = k.shape[1], k.shape[2]
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    o = torch.empty_like(q)
    lse = torch.empty((B, Hq, Nq), dtype=torch.float32, device=q.device)
    attn_fwd(q, k, v, o, lse, B, Hq, Hkv, Nq, Nk, D, causal, scale, stream)
    return o, lse


class DecodeGraph:
    """One decode step captured as a CUDA graph for fixed q / cache / output
    tensors (held here, so their addresses stay valid); ``replay()`` runs the
    step on the buffers' current contents."""

    def __init__(self, q, kcache, vcache, nsplit: int):
        import torch
        self.handle = 0
        _check_decode_inputs(q, kcache, vcache)
        B, Hq, D = q.shape
        Hkv, Nk = kcache.shape[1], kcache.shape[2]
        self.q, self.kcache, self.vcache = q, kcache, vcache
        self.o = torch.empty_like(q)
        self.lse = torch.empty((B, Hq), dtype=torch.float32, device=q.device)
        self.handle = attn_decode_graph_create(q, kcache, vcache, self.o, self.lse, B, Hq, Hkv,
                                               Nk, D, nsplit)

    def replay(self, stream=None):
        attn_decode_graph_launch(self.handle, stream)
        return self.o, self.lse

    def close(self):
        if self.handle:
            h, self.handle = self.handle, 0
            attn_decode_graph_destroy(h)

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def _check_decode_inputs(q, kcache, vcache):
    # q [B, Hq, D], caches [B, Hkv, Nk, D]
    _check_ranks({"q": q, "kcache": kcache, "vcache": vcache}, {"q": 3, "kcache": 4, "vcache": 4})
    _check_inputs({"q": q, "kcache": kcache, "vcache": vcache},
                  {"B": (q.shape[0], kcache.shape[0], vcache.shape[0]),
                   "D": (q.shape[2], kcache.shape[3], vcache.shape[3]),
                   "Hkv": (kcache.shape[1], vcache.shape[1]), "Nk": (kcache.shape[2], vcache.shape[2])})


def decode(q, kcache, vcache, nsplit: int, stream=None):
    """O, LSE = split-KV decode(q [B,Hq,D], caches [B,Hkv,Nk,D])."""
    import torch
    _check_decode_inputs(q, kcache, vcache)
    B, Hq, D = q.shape
    Hkv, Nk = kcache.shape[1], kcache.shape[2]
    o = torch.empty_like(q)
    lse = torch.empty((B, Hq), dtype=torch.float32, device=q.device)
    attn_decode_splitkv(q, kcache, vcache, o, lse, B, Hq, Hkv, Nk, D, nsplit, stream)
    return o, lse


# ------------------------------------------------------- modified scores: tensor helpers
#
# These calls are short enough (a decode step: 10 us on the GPU) that the host's
# part of them shows.  So every argument is checked by plain attribute
# comparisons first, and only a call that fails them goes through the checks that
# find the words for it.

_torch = None


def _import_torch():
    global _torch
    if _torch is None:
        import torch
        _torch = torch
    return _torch


def _aux_bad(x, dtype, shape, dev: int) -> bool:
    return not (isinstance(x, _torch.Tensor) and x.dtype is dtype and x.shape == shape
                and x.get_device() == dev and x.is_contiguous())


def _check_aux(dev, **tensors):
    """The optional int32 / fp32 device arrays of the calls below:
    name=(tensor or None, dtype, shape)."""
    torch = _import_torch()
    for name, (x, dtype, shape) in tensors.items():
        if x is None:
            continue
        if not isinstance(x, torch.Tensor):
            raise TypeError(f"{name} must be a torch tensor")
        if x.dtype != dtype:
            raise TypeError(f"{name} must be {dtype}, got {x.dtype}")
        if tuple(x.shape) != tuple(shape):
            raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(x.shape)}")
        if not x.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
        if x.device != dev:
            raise ValueError(f"{name} is on {x.device}, expected {dev}")
        if not x.is_contiguous():
            raise ValueError(f"{name} must be contiguous")


def _current_raw_stream(dev: int) -> int:
    return _torch.cuda.current_stream(dev).cuda_stream


def _elsewhere(call, dev: int, stream, inputs):
    """``call()`` with ``dev`` current, on ``stream`` (None: the device's current
    one).  On another stream than the current one the outputs are allocated there
    too: the caching allocator may give memory out again that kernels of the
    current stream are still to read, which only that stream waits for.  The
    inputs are marked as used on the other stream and the outputs as used on the
    current one, so that neither's memory is handed out while it is in use."""
    cuda = _torch.cuda
    if _current_device() != dev:
        with cuda.device(dev):
            return _elsewhere(call, dev, stream, inputs)
    if stream is None:
        return call()
    if isinstance(stream, int):
        stream = cuda.ExternalStream(stream, device=dev) if stream else cuda.default_stream(dev)
    elif stream.device_index != dev:
        raise ValueError(f"the stream is on {stream.device}, the tensors on cuda:{dev}")
    current = cuda.current_stream(dev)
    if stream.cuda_stream == current.cuda_stream:
        return call()
    cuda.set_stream(stream)  # (and back: 10 us less than by a context)
    try:
        out = call()
    finally:
        cuda.set_stream(current)
    for x in inputs:
        if x is not None:
            x.record_stream(stream)
    for x in out if isinstance(out, tuple) else (out,):
        x.record_stream(current)
    return out


# The first call of each of these two puts the quickest way there is in its place.
def _current_device() -> int:
    global _current_device
    torch = _import_torch()
    _current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
    return _current_device()


def _raw_stream(dev: int) -> int:
    global _raw_stream
    _raw_stream = getattr(_import_torch()._C, "_cuda_getCurrentRawStream", _current_raw_stream)
    return _raw_stream(dev)


def forward_mod(q, k, v, *, causal: bool = False, scale: float | None = None,
                softcap: float = 0.0, slopes=None, ranges=None, q_offset: int = 0, stream=None):
    """O, LSE = attention(q [B,Hq,Nq,D], k/v [B,Hkv,Nk,D]) with modified scores:
    capped at ``softcap`` by a tanh (0: not), biased by ``-slopes[h] * distance``
    (``slopes`` [Hq] fp32, query row i at position ``q_offset + i``), row i of
    batch b seeing keys ``ranges[b, i, 0] <= j < ranges[b, i, 1]`` (``ranges``
    [B,Nq,2] int32, see ``row_ranges``; None: all) and, with ``causal``, of
    these those at or before its position.  Rows that see nothing give 0 and
    -inf."""
    torch = _torch or _import_torch()
    try:
        B, Hq, Nq, D = q.shape
        Bk, Hkv, Nk, Dk = k.shape
        dev, bf16 = q.get_device(), torch.bfloat16
        fine = (v.shape == k.shape and Bk == B and Dk == D and dev >= 0
                and q.dtype is bf16 and k.dtype is bf16 and v.dtype is bf16
                and k.get_device() == dev and v.get_device() == dev
                and q.is_contiguous() and k.is_contiguous() and v.is_contiguous())
    except (AttributeError, ValueError):
        fine = False
    if not fine or slopes is not None and _aux_bad(slopes, torch.float32, (Hq,), dev) \
            or ranges is not None and _aux_bad(ranges, torch.int32, (B, Nq, 2), dev):
        _check_ranks({"q": q, "k": k, "v": v}, {"q": 4, "k": 4, "v": 4})
        _check_inputs({"q": q, "k": k, "v": v},
                      {"B": (q.shape[0], k.shape[0], v.shape[0]),
                       "D": (q.shape[3], k.shape[3], v.shape[3]),
                       "Hkv": (k.shape[1], v.shape[1]), "Nk": (k.shape[2], v.shape[2])})
        _check_aux(q.device, slopes=(slopes, torch.float32, (Hq,)),
                   ranges=(ranges, torch.int32, (B, Nq, 2)))
    if stream is not None or _current_device() != dev:
        return _elsewhere(lambda: forward_mod(q, k, v, causal=causal, scale=scale, softcap=softcap,
                                              slopes=slopes, ranges=ranges, q_offset=q_offset),
                          dev, stream, (q, k, v, slopes, ranges))
    if q_offset >> 31 or 0 < softcap < _LEAST_CAP:
        _check(-3)  # ATTN_ERR_SHAPE: ctypes would pass it modulo 2^32, or as no cap
    device = q.device
    o = torch.empty_strided((B, Hq, Nq, D), (Hq * Nq * D, Nq * D, D, 1), dtype=bf16, device=device)
    lse = torch.empty_strided((B, Hq, Nq), (Hq * Nq, Nq, 1), dtype=torch.float32, device=device)
    rc = (_lib or load()).attn_fwd_mod(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(), B, Hq, Hkv, Nq, Nk,
        D, bool(causal), q_offset, D ** -0.5 if scale is None else scale, softcap,
        None if slopes is None else slopes.data_ptr(), None if ranges is None else ranges.data_ptr(),
        _raw_stream(dev))
    if rc:
        _check(rc)
    return o, lse


def row_ranges(doc_lens, N: int, *, prefix_lens=None, causal: bool = True, stream=None):
    """[B, N, 2] int32 key ranges for ``forward_mod`` from the lengths of the
    documents packed into each row (``doc_lens`` [B, M] int32, CUDA): a token
    sees its own document, with ``causal`` up to itself or to the end of the
    document's bidirectional prefix (``prefix_lens`` [B, M] int32).  Tokens
    behind the last document (padding) see nothing."""
    torch = _torch or _import_torch()
    i32 = torch.int32
    try:
        B, M = doc_lens.shape
        dev = doc_lens.get_device()
        fine = dev >= 0 and doc_lens.dtype is i32 and doc_lens.is_contiguous()
    except (AttributeError, ValueError):
        fine = False
    if not fine or prefix_lens is not None and _aux_bad(prefix_lens, i32, (B, M), dev):
        _check_ranks({"doc_lens": doc_lens}, {"doc_lens": 2})
        _check_aux(doc_lens.device, doc_lens=(doc_lens, i32, (B, M)),
                   prefix_lens=(prefix_lens, i32, (B, M)))
    if stream is not None or _current_device() != dev:
        return _elsewhere(lambda: row_ranges(doc_lens, N, prefix_lens=prefix_lens, causal=causal),
                          dev, stream, (doc_lens, prefix_lens))
    if N >> 31 or M >> 31:
        _check(-3)  # ATTN_ERR_SHAPE: ctypes would pass it modulo 2^32
    out = torch.empty((B, N, 2), dtype=i32, device=doc_lens.device)
    rc = (_lib or load()).attn_row_ranges(
        doc_lens.data_ptr(), None if prefix_lens is None else prefix_lens.data_ptr(),
        out.data_ptr(), B, N, M, bool(causal), _raw_stream(dev))
    if rc:
        _check(rc)
    return out


def _decode(fn, q, pre, kcache, vcache, lens, scale, softcap, slopes, stream):
    """What the two decode calls share; pre: () or (kprefix, vprefix)."""
    torch = _torch
    try:
        B, Hq, D = q.shape
        Bk, Hkv, Ncap, Dk = kcache.shape
        dev, bf16 = q.get_device(), torch.bfloat16
        fine = (vcache.shape == kcache.shape and Bk == B and Dk == D and dev >= 0
                and q.dtype is bf16 and kcache.dtype is bf16 and vcache.dtype is bf16
                and kcache.get_device() == dev and vcache.get_device() == dev
                and q.is_contiguous() and kcache.is_contiguous() and vcache.is_contiguous())
        if pre:
            kprefix, vprefix = pre
            Hp, Np, Dp = kprefix.shape
            fine = (fine and vprefix.shape == kprefix.shape and Hp == Hkv and Dp == D
                    and kprefix.dtype is bf16 and vprefix.dtype is bf16
                    and kprefix.get_device() == dev and vprefix.get_device() == dev
                    and kprefix.is_contiguous() and vprefix.is_contiguous())
    except (AttributeError, ValueError):
        fine = False
    if not fine or lens is not None and _aux_bad(lens, torch.int32, (B,), dev) \
            or slopes is not None and _aux_bad(slopes, torch.float32, (Hq,), dev):
        if pre:
            _check_ranks({"kprefix": pre[0], "vprefix": pre[1]}, {"kprefix": 3, "vprefix": 3})
        _check_decode_inputs(q, kcache, vcache)
        if pre:
            _check_inputs({"q": q, "kprefix": pre[0], "vprefix": pre[1]},
                          {"Hkv": (Hkv, pre[0].shape[0], pre[1].shape[0]),
                           "Np": (pre[0].shape[1], pre[1].shape[1]),
                           "D": (D, pre[0].shape[2], pre[1].shape[2])})
        _check_aux(q.device, slopes=(slopes, torch.float32, (Hq,)), lens=(lens, torch.int32, (B,)))
    if stream is not None or _current_device() != dev:
        return _elsewhere(lambda: _decode(fn, q, pre, kcache, vcache, lens, scale, softcap, slopes, None),
                          dev, stream, (q, *pre, kcache, vcache, lens, slopes))
    if 0 < softcap < _LEAST_CAP:
        _check(-3)  # ATTN_ERR_SHAPE: ctypes would pass it as no cap
    device = q.device
    o = torch.empty_strided((B, Hq, D), (Hq * D, D, 1), dtype=bf16, device=device)
    lse = torch.empty_strided((B, Hq), (Hq, 1), dtype=torch.float32, device=device)
    tail = (None if lens is None else lens.data_ptr(), o.data_ptr(), lse.data_ptr(), B, Hq, Hkv)
    score = (Ncap, D, D ** -0.5 if scale is None else scale, softcap,
             None if slopes is None else slopes.data_ptr())
    if pre:
        args = (q.data_ptr(), kprefix.data_ptr(), vprefix.data_ptr(), kcache.data_ptr(),
                vcache.data_ptr(), *tail, Np, *score)
    else:
        args = (q.data_ptr(), kcache.data_ptr(), vcache.data_ptr(), *tail, *score)
    rc = fn(*args, _raw_stream(dev))
    if rc:
        _check(rc)
    return o, lse


def decode_varlen(q, kcache, vcache, lens=None, *, scale: float | None = None,
                  softcap: float = 0.0, slopes=None, stream=None):
    """O, LSE = decode(q [B,Hq,D], caches [B,Hkv,Ncap,D]) over the first
    ``lens[b]`` keys of request b (``lens`` [B] int32, CUDA; None: all), with
    the score modifications of ``forward_mod``; the query is at position
    ``lens[b] - 1``."""
    _torch or _import_torch()
    return _decode((_lib or load()).attn_decode_varlen, q, (), kcache, vcache, lens, scale, softcap,
                   slopes, stream)


def decode_prefix(q, kprefix, vprefix, kcache, vcache, lens=None, *, scale: float | None = None,
                  softcap: float = 0.0, slopes=None, stream=None):
    """``decode_varlen`` for requests that share a prefix: ``kprefix`` /
    ``vprefix`` [Hkv,Np,D] are seen by every request before its own
    ``lens[b]`` cache keys, and read once for the whole batch; the query is at
    position ``Np + lens[b] - 1``."""
    _torch or _import_torch()
    return _decode((_lib or load()).attn_decode_prefix, q, (kprefix, vprefix), kcache, vcache, lens,
                   scale, softcap, slopes, stream)
