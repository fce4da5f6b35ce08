"""Thin ctypes binding of libkmip (the C ABI declared in include/kmip.h).

Argument marshalling only: every step of the computation runs in the CUDA
kernels of libkmip.so.  torch provides device memory and streams.  There is
no CPU fallback -- if the library is missing, or the tensors are not on a
CUDA device, the call raises.
"""
from __future__ import annotations

import ctypes
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
# KMIP_DEBUG_BOUNDS=1 loads the build with device-side index checks
# (python -m graph_transformer_sparse_kmip_b200.build --debug-bounds).
LIB_PATH = os.path.join(_PKG, "libkmip_debug.so" if os.environ.get("KMIP_DEBUG_BOUNDS") == "1"
                        else "libkmip.so")
# KMIP_NVTX=1 wraps every library call in an NVTX range (for nsys/ncu timelines).
_NVTX = os.environ.get("KMIP_NVTX") == "1"

KMIP_BF16, KMIP_F32 = 0, 1
POS_TYPES = {torch.float32: 0, torch.int32: 1, torch.int64: 2}
ACTS = {"none": 0, "silu": 1, "gelu": 2, "relu": 3}
STATUS_NAMES = {0: "KMIP_OK", 1: "KMIP_ERR_INVALID_ARG", 2: "KMIP_ERR_UNSUPPORTED",
                3: "KMIP_ERR_CUDA", 4: "KMIP_ERR_BAD_OFFSETS", 5: "KMIP_ERR_TIMEOUT",
                6: "KMIP_ERR_BAD_INDEX", 7: "KMIP_ERR_SCRATCH_LIMIT"}
EXPORTED = ("kmip_attn_fwd", "kmip_attn_fwd_noalloc", "kmip_attn_fwd_diag", "kmip_attn_bwd",
            "kmip_attn_bwd_deterministic", "kmip_attn_gather", "kmip_get_status",
            "kmip_rotary", "kmip_group_norm_fwd", "kmip_group_norm_bwd",
            "kmip_ffn_fwd", "kmip_ffn_bwd",
            "kmip_scratch_usage", "kmip_scratch_trim", "kmip_error_string",
            "kmip_fwd_path", "kmip_version")

_lib = None


class KmipError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {STATUS_NAMES.get(code, code)}")


def load() -> ctypes.CDLL:
    """Load libkmip.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"libkmip.so not found at {LIB_PATH}; build it with "
                          "`python -m graph_transformer_sparse_kmip_b200.build`")
    lib = ctypes.CDLL(LIB_PATH)
    P, I32, I64, F32 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float
    lib.kmip_attn_fwd.argtypes = [P, P, P, P, I64, I32, I32, I32, F32, P, P, P, P, I32, I32]
    lib.kmip_attn_fwd.restype = I32
    lib.kmip_attn_fwd_noalloc.argtypes = lib.kmip_attn_fwd.argtypes
    lib.kmip_attn_fwd_noalloc.restype = I32
    lib.kmip_attn_fwd_diag.argtypes = [P, P, P, P, I64, I32, I32, I32, F32, P, P, P, P, P, I32,
                                       I32]
    lib.kmip_attn_fwd_diag.restype = I32
    lib.kmip_attn_bwd.argtypes = [P, P, P, P, P, P, P, P, P, P, I64, I32, I32, I32, F32, I32]
    lib.kmip_attn_bwd.restype = I32
    lib.kmip_attn_bwd_deterministic.argtypes = lib.kmip_attn_bwd.argtypes
    lib.kmip_attn_bwd_deterministic.restype = I32
    lib.kmip_attn_gather.argtypes = [P, P, P, P, I64, I32, I32, I32, F32, P, P, P, I32]
    lib.kmip_attn_gather.restype = I32
    lib.kmip_rotary.argtypes = [P, I64, I64, P, I32, I32, P, P, I32, I32, I32, I64, I32, I32, P,
                                I64, I64, P, I32]
    lib.kmip_rotary.restype = I32
    lib.kmip_group_norm_fwd.argtypes = [P, P, P, P, I64, I32, I32, F32, I32, P, P, P, P, I32, I32]
    lib.kmip_group_norm_fwd.restype = I32
    lib.kmip_group_norm_bwd.argtypes = [P, P, P, P, P, P, P, I64, I32, I32, I32, P, P, P, P, I32,
                                        I32]
    lib.kmip_group_norm_bwd.restype = I32
    lib.kmip_ffn_fwd.argtypes = [P, P, P, P, I64, I32, I32, I32, P, P, I32]
    lib.kmip_ffn_fwd.restype = I32
    lib.kmip_ffn_bwd.argtypes = [P, P, P, P, P, I64, I32, I32, I32, P, P, P, P, P, I32]
    lib.kmip_ffn_bwd.restype = I32
    lib.kmip_get_status.argtypes = [P]
    lib.kmip_get_status.restype = I32
    lib.kmip_scratch_usage.argtypes = [P, P, I32]
    lib.kmip_scratch_usage.restype = I32
    lib.kmip_scratch_trim.argtypes = []
    lib.kmip_scratch_trim.restype = I32
    lib.kmip_error_string.argtypes = [I32]
    lib.kmip_error_string.restype = ctypes.c_char_p
    lib.kmip_test_wait_timeout.argtypes = [P, I32]
    lib.kmip_test_wait_timeout.restype = I32
    lib.kmip_fwd_path.argtypes = [I32, I32, I32]
    lib.kmip_fwd_path.restype = I32
    lib.kmip_version.argtypes = []
    lib.kmip_version.restype = I32
    _lib = lib
    return lib


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _call(name, *args):
    """Calls the C entry point `name` (inside an NVTX range when KMIP_NVTX=1)."""
    fn = getattr(load(), name)
    if not _NVTX:
        return fn(*args)
    torch.cuda.nvtx.range_push(name)
    try:
        return fn(*args)
    finally:
        torch.cuda.nvtx.range_pop()


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def dtype_code(t: torch.dtype) -> int:
    if t == torch.bfloat16:
        return KMIP_BF16
    if t == torch.float32:
        return KMIP_F32
    raise TypeError(f"unsupported dtype {t} (bf16 or fp32)")


def _check_cuda(*ts):
    for t in ts:
        if t is not None and (not t.is_cuda or not t.is_contiguous()):
            raise ValueError("libkmip takes contiguous CUDA tensors")


# --- the C entry points, same names, torch tensors in place of pointers ---

def kmip_attn_fwd(Q, K, V, graph_offsets, N, H, d, k, scale, out, idx, lse, stream=None,
                  num_graphs=None, dtype=None) -> int:
    _check_cuda(Q, K, V, graph_offsets, out, idx, lse)
    G = (graph_offsets.numel() - 1) if graph_offsets is not None else 1
    if num_graphs is None:
        num_graphs = G
    if dtype is None:
        dtype = dtype_code(Q.dtype)
    return _call("kmip_attn_fwd", _ptr(Q), _ptr(K), _ptr(V), _ptr(graph_offsets), int(N), int(H),
                                int(d), int(k), float(scale), _ptr(out), _ptr(idx), _ptr(lse),
                                _stream(stream), int(num_graphs), int(dtype))


def kmip_attn_fwd_noalloc(Q, K, V, graph_offsets, N, H, d, k, scale, out, idx, lse,
                          stream=None, num_graphs=None, dtype=None) -> int:
    """kmip_attn_fwd without any device allocation inside the library: the
    work list lives in a fixed device array of the library (for callers whose
    memory is fully owned by their own pool, or who must not allocate after
    start-up).  Calls on one device must not overlap on the GPU."""
    _check_cuda(Q, K, V, graph_offsets, out, idx, lse)
    G = (graph_offsets.numel() - 1) if graph_offsets is not None else 1
    if num_graphs is None:
        num_graphs = G
    if dtype is None:
        dtype = dtype_code(Q.dtype)
    return _call("kmip_attn_fwd_noalloc", _ptr(Q), _ptr(K), _ptr(V), _ptr(graph_offsets), int(N),
                                        int(H), int(d), int(k), float(scale), _ptr(out),
                                        _ptr(idx), _ptr(lse), _stream(stream), int(num_graphs),
                                        int(dtype))


def kmip_attn_fwd_diag(Q, K, V, graph_offsets, N, H, d, k, scale, out, idx, lse, lse_all,
                       stream=None, num_graphs=None, dtype=None) -> int:
    """kmip_attn_fwd plus lse_all [N, H]: the log-sum-exp over every key of
    the query's graph (the normaliser of full softmax attention)."""
    _check_cuda(Q, K, V, graph_offsets, out, idx, lse, lse_all)
    G = (graph_offsets.numel() - 1) if graph_offsets is not None else 1
    if num_graphs is None:
        num_graphs = G
    if dtype is None:
        dtype = dtype_code(Q.dtype)
    return _call("kmip_attn_fwd_diag", _ptr(Q), _ptr(K), _ptr(V), _ptr(graph_offsets), int(N),
                                     int(H), int(d), int(k), float(scale), _ptr(out), _ptr(idx),
                                     _ptr(lse), _ptr(lse_all), _stream(stream), int(num_graphs),
                                     int(dtype))


def kmip_attn_bwd(dOut, Q, K, V, idx, lse, dQ, dK, dV, stream=None, N=None, H=None, d=None,
                  k=None, scale=None, dtype=None) -> int:
    _check_cuda(dOut, Q, K, V, idx, lse, dQ, dK, dV)
    N_, H_, d_ = Q.shape
    N = N_ if N is None else N
    H = H_ if H is None else H
    d = d_ if d is None else d
    k = idx.shape[-1] if k is None else k
    if dtype is None:
        dtype = dtype_code(Q.dtype)
    return _call("kmip_attn_bwd", _ptr(dOut), _ptr(Q), _ptr(K), _ptr(V), _ptr(idx), _ptr(lse),
                                _ptr(dQ), _ptr(dK), _ptr(dV), _stream(stream), int(N), int(H),
                                int(d), int(k), float(scale), int(dtype))


def kmip_attn_bwd_deterministic(dOut, Q, K, V, idx, lse, dQ, dK, dV, stream=None, N=None,
                                H=None, d=None, k=None, scale=None, dtype=None) -> int:
    """kmip_attn_bwd with bitwise reproducible dK/dV (sorted gather, no
    atomics)."""
    _check_cuda(dOut, Q, K, V, idx, lse, dQ, dK, dV)
    N_, H_, d_ = Q.shape
    N = N_ if N is None else N
    H = H_ if H is None else H
    d = d_ if d is None else d
    k = idx.shape[-1] if k is None else k
    if dtype is None:
        dtype = dtype_code(Q.dtype)
    return _call(
        "kmip_attn_bwd_deterministic", _ptr(dOut), _ptr(Q), _ptr(K), _ptr(V), _ptr(idx), _ptr(lse), _ptr(dQ), _ptr(dK),
        _ptr(dV), _stream(stream), int(N), int(H), int(d), int(k), float(scale), int(dtype))


def kmip_attn_gather(Q, K, V, idx, N, H, d, k, scale, out, lse, stream=None, dtype=None) -> int:
    """Softmax and V gather over the given key sets (idx), scores recomputed."""
    _check_cuda(Q, K, V, idx, out, lse)
    if dtype is None:
        dtype = dtype_code(Q.dtype)
    return _call("kmip_attn_gather", _ptr(Q), _ptr(K), _ptr(V), _ptr(idx), int(N), int(H),
                 int(d), int(k), float(scale), _ptr(out), _ptr(lse), _stream(stream), int(dtype))


def attn_gather(Q, K, V, idx, scale: float, stream=None):
    """Returns (out, lse) of attention over the given sets idx [N, H, k]."""
    N, H, d = Q.shape
    out = torch.empty_like(Q)
    lse = torch.empty((N, H), dtype=torch.float32, device=Q.device)
    rc = kmip_attn_gather(Q, K, V, idx, N, H, d, idx.shape[-1], scale, out, lse, stream)
    if rc:
        raise KmipError(rc, "kmip_attn_gather")
    return out, lse


def kmip_get_status(stream=None) -> int:
    return load().kmip_get_status(_stream(stream))


def kmip_error_string(code: int) -> str:
    return load().kmip_error_string(int(code)).decode()


def kmip_scratch_usage(reset_high: bool = False):
    """(reserved, used_high) bytes of the library's scratch pool on the
    current device."""
    r, h = ctypes.c_uint64(0), ctypes.c_uint64(0)
    rc = load().kmip_scratch_usage(ctypes.byref(r), ctypes.byref(h), int(bool(reset_high)))
    if rc:
        raise KmipError(rc, "kmip_scratch_usage")
    return int(r.value), int(h.value)


def kmip_scratch_trim():
    """Return the library's unused pool memory on the current device (after
    the streams that used the library have been synchronised)."""
    rc = load().kmip_scratch_trim()
    if rc:
        raise KmipError(rc, "kmip_scratch_trim")


def kmip_version() -> int:
    return load().kmip_version()


def kmip_fwd_path(d: int, k: int, dtype: int = KMIP_BF16) -> int:
    """1 = tcgen05 tensor-core forward, 0 = fp32-FMA forward, -1 = unsupported."""
    return load().kmip_fwd_path(int(d), int(k), int(dtype))


def kmip_test_wait_timeout(timeout_us: int, stream=None) -> int:
    """Test hook (include/kmip_testing.h): a bounded wait that must run out."""
    return load().kmip_test_wait_timeout(_stream(stream), int(timeout_us))


# --- convenience wrappers that allocate the outputs with torch ---

def attn_fwd(Q, K, V, k: int, scale: float, graph_offsets=None, stream=None):
    """Returns (out [N,H,d] like Q, idx [N,H,k] int32, lse [N,H] fp32)."""
    N, H, d = Q.shape
    out = torch.empty_like(Q)
    idx = torch.empty((N, H, k), dtype=torch.int32, device=Q.device)
    lse = torch.empty((N, H), dtype=torch.float32, device=Q.device)
    rc = kmip_attn_fwd(Q, K, V, graph_offsets, N, H, d, k, scale, out, idx, lse, stream)
    if rc:
        raise KmipError(rc, "kmip_attn_fwd")
    return out, idx, lse


def attn_fwd_diag(Q, K, V, k: int, scale: float, graph_offsets=None, stream=None):
    """Returns (out, idx, lse, lse_all): kmip_attn_fwd's outputs and the
    log-sum-exp over every key of the query's graph."""
    N, H, d = Q.shape
    out = torch.empty_like(Q)
    idx = torch.empty((N, H, k), dtype=torch.int32, device=Q.device)
    lse = torch.empty((N, H), dtype=torch.float32, device=Q.device)
    lse_all = torch.empty((N, H), dtype=torch.float32, device=Q.device)
    rc = kmip_attn_fwd_diag(Q, K, V, graph_offsets, N, H, d, k, scale, out, idx, lse, lse_all,
                            stream)
    if rc:
        raise KmipError(rc, "kmip_attn_fwd_diag")
    return out, idx, lse, lse_all


def attn_bwd(dOut, Q, K, V, idx, lse, scale: float, stream=None, deterministic=False):
    """Returns (dQ, dK, dV), fp32 [N,H,d]."""
    dQ = torch.empty(Q.shape, dtype=torch.float32, device=Q.device)
    dK = torch.empty_like(dQ)
    dV = torch.empty_like(dQ)
    fn = kmip_attn_bwd_deterministic if deterministic else kmip_attn_bwd
    rc = fn(dOut, Q, K, V, idx, lse, dQ, dK, dV, stream, scale=scale)
    if rc:
        raise KmipError(rc, fn.__name__)
    return dQ, dK, dV


# --- the operators around the attention: positions, norm, feed-forward ---

# A small call is bound by what happens before its launch: these helpers stay
# with integers (device indices, addresses, raw stream handles) and make no
# torch.device, torch.cuda.Stream or ctypes objects on the way.

def _same_device(x, *ts):
    """Every tensor on x's CUDA device and contiguous (x itself may be
    strided)."""
    dev = x.get_device()
    if dev < 0:
        raise ValueError("libkmip takes CUDA tensors")
    for t in ts:
        if t is not None and (t.get_device() != dev or not t.is_contiguous()):
            raise ValueError(f"expected a contiguous tensor on {x.device}")


def _expect(t, name, shape, dtype):
    if t is not None and (t.shape != shape or t.dtype != dtype):
        raise ValueError(f"{name}: expected {tuple(shape)} {dtype}, got {tuple(t.shape)} {t.dtype}")


def _act_code(act: str) -> int:
    if act not in ACTS:
        raise ValueError(f"unknown activation {act!r} (one of {', '.join(ACTS)})")
    return ACTS[act]


def _offsets(graph_offsets):
    """Checks graph_offsets (int32 [G+1] or None); returns G."""
    if graph_offsets is None:
        return 1
    shape = graph_offsets.shape
    if graph_offsets.dtype != torch.int32 or len(shape) != 1 or shape[0] < 2:
        raise ValueError("graph_offsets: expected int32 [G + 1] with G >= 1")
    return shape[0] - 1


def _addr(t):
    return None if t is None else t.data_ptr()


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _launch(x, name, stream, args, tail, *used):
    """Calls entry point `name` with args, the stream and tail, with x's
    device current: on `stream`, or on that device's current stream.  Raises
    on a status.  `used` (and x): the call's tensors, which torch's allocator
    is told of when the call goes to a stream that is not theirs."""
    dev = x.get_device()
    if dev != _device():
        with torch.cuda.device(dev):
            return _launch(x, name, stream, args, tail, *used)
    if stream is not None:
        s = stream.cuda_stream
        for t in (x, *used):
            if t is not None:
                t.record_stream(stream)
    elif _raw_stream is not None:
        s = _raw_stream(dev)
    else:
        s = torch.cuda.current_stream().cuda_stream
    rc = _call(name, *args, s, *tail) if _NVTX else getattr(_lib or load(), name)(*args, s, *tail)
    if rc:
        raise KmipError(rc, name)


def rotary(x, pos, freq, axis, inverse: bool = False, interleaved: bool = False, out=None,
           stream=None):
    """Rotary positions with several axes (kmip_rotary): pair p of every head
    of node n turns by pos[n, axis[p]] * freq[p].

    x: [N, H, d] bf16 or fp32, rows and heads at any stride, elements of a
    head adjacent; pos: [N, A] fp32, int32 or int64; freq: fp64 [P]; axis:
    int32 [P].  out: a new contiguous tensor, or a tensor like x (x itself:
    in place).  inverse=True is the gradient with respect to x."""
    if x.dim() != 3:
        raise ValueError("x: expected [N, H, d]")
    (N, H, d), xs, P = x.shape, x.stride(), freq.numel()
    if xs[2] != 1 and d > 1 and N * H:
        raise ValueError("x: expected adjacent elements in a head")
    pos_type = POS_TYPES.get(pos.dtype)
    if pos_type is None:
        raise TypeError(f"unsupported position dtype {pos.dtype} (fp32, int32 or int64)")
    if pos.dim() != 2 or pos.shape[0] != N:
        raise ValueError(f"pos: expected [{N}, axes], got {tuple(pos.shape)}")
    _expect(freq, "freq", (P,), torch.float64)
    _expect(axis, "axis", (P,), torch.int32)
    _same_device(x, pos, freq, axis)
    if out is None:
        out = torch.empty_like(x, memory_format=torch.contiguous_format)
    elif (out.shape != x.shape or out.dtype != x.dtype or out.device != x.device
          or (out.stride(2) != 1 and d > 1 and N * H)):
        raise ValueError("out: expected a tensor like x")
    os = out.stride()
    _launch(x, "kmip_rotary", stream,
            (x.data_ptr(), xs[0], xs[1], pos.data_ptr(), pos_type, pos.shape[1], freq.data_ptr(),
             axis.data_ptr(), P, bool(interleaved), bool(inverse), N, H, d, out.data_ptr(), os[0],
             os[1]), (dtype_code(x.dtype),), pos, freq, axis, out)
    return out


def group_norm_fwd(x, weight, bias, groups: int, eps: float = 1e-5, act: str = "none",
                   graph_offsets=None, stream=None):
    """Group norm per graph with an activation (kmip_group_norm_fwd).

    x: [N, C] bf16 or fp32, contiguous; weight, bias: [C] like x, or both
    None; graph_offsets: int32 [G+1] or None (one graph).  Returns (y,
    mean, rstd), the last two fp32 [G, groups]."""
    if x.dim() != 2:
        raise ValueError("x: expected [N, C]")
    N, C = x.shape
    G = _offsets(graph_offsets)
    _same_device(x, x, weight, bias, graph_offsets)
    _expect(weight, "weight", (C,), x.dtype)
    _expect(bias, "bias", (C,), x.dtype)
    y = torch.empty_like(x)
    mean = x.new_empty((G, groups), dtype=torch.float32)
    rstd = torch.empty_like(mean)
    _launch(x, "kmip_group_norm_fwd", stream,
            (x.data_ptr(), _addr(weight), _addr(bias), _addr(graph_offsets), N, C, groups, eps,
             _act_code(act), y.data_ptr(), mean.data_ptr(), rstd.data_ptr()),
            (G, dtype_code(x.dtype)), weight, bias, graph_offsets, y, mean, rstd)
    return y, mean, rstd


def group_norm_bwd(dy, x, weight, bias, mean, rstd, groups: int, act: str = "none",
                   graph_offsets=None, stream=None):
    """Backward of group_norm_fwd: (dx, dweight, dbias) in x's type; the last
    two are None when there is no weight."""
    if x.dim() != 2:
        raise ValueError("x: expected [N, C]")
    N, C = x.shape
    G = _offsets(graph_offsets)
    _same_device(x, x, dy, weight, bias, graph_offsets, mean, rstd)
    _expect(dy, "dy", (N, C), x.dtype)
    _expect(weight, "weight", (C,), x.dtype)
    _expect(bias, "bias", (C,), x.dtype)
    _expect(mean, "mean", (G, groups), torch.float32)
    _expect(rstd, "rstd", (G, groups), torch.float32)
    dx = torch.empty_like(x)
    dw = db = None
    if weight is not None:
        dw, db = torch.empty_like(weight), torch.empty_like(weight)
    _launch(x, "kmip_group_norm_bwd", stream,
            (dy.data_ptr(), x.data_ptr(), _addr(weight), _addr(bias), _addr(graph_offsets),
             mean.data_ptr(), rstd.data_ptr(), N, C, groups, _act_code(act), dx.data_ptr(),
             _addr(dw), _addr(db)), (G, dtype_code(x.dtype)), dy, weight, bias, graph_offsets,
            mean, rstd, dx, dw, db)
    return dx, dw, db


def _ffn_args(x, wg, wu, wd):
    if x.dim() != 2 or wg.dim() != 2:
        raise ValueError("x: expected [N, C]; wg, wu: [F, C]; wd: [C, F]")
    (N, C), F = x.shape, wg.shape[0]
    _same_device(x, x, wg, wu, wd)
    _expect(wg, "wg", (F, C), x.dtype)
    _expect(wu, "wu", (F, C), x.dtype)
    _expect(wd, "wd", (C, F), x.dtype)
    return N, C, F


def ffn_fwd(x, wg, wu, wd, act: str = "silu", stream=None):
    """Gated feed-forward block y = (act(x wg^T) * (x wu^T)) wd^T
    (kmip_ffn_fwd).  x: [N, C] bf16 or fp32; wg, wu: [F, C]; wd: [C, F]."""
    N, C, F = _ffn_args(x, wg, wu, wd)
    y = torch.empty_like(x)
    _launch(x, "kmip_ffn_fwd", stream,
            (x.data_ptr(), wg.data_ptr(), wu.data_ptr(), wd.data_ptr(), N, C, F, _act_code(act),
             y.data_ptr()), (dtype_code(x.dtype),), wg, wu, wd, y)
    return y


def ffn_bwd(dy, x, wg, wu, wd, act: str = "silu", stream=None):
    """Backward of ffn_fwd: (dx, dwg, dwu, dwd) in x's type."""
    N, C, F = _ffn_args(x, wg, wu, wd)
    _same_device(x, dy)
    _expect(dy, "dy", (N, C), x.dtype)
    dx = torch.empty_like(x)
    dwg, dwu, dwd = torch.empty_like(wg), torch.empty_like(wu), torch.empty_like(wd)
    _launch(x, "kmip_ffn_bwd", stream,
            (dy.data_ptr(), x.data_ptr(), wg.data_ptr(), wu.data_ptr(), wd.data_ptr(), N, C, F,
             _act_code(act), dx.data_ptr(), dwg.data_ptr(), dwu.data_ptr(), dwd.data_ptr()),
            (dtype_code(x.dtype),), dy, wg, wu, wd, dx, dwg, dwu, dwd)
    return dx, dwg, dwu, dwd


def check_status(stream=None):
    rc = kmip_get_status(stream)
    if rc:
        raise KmipError(rc, "device status")
