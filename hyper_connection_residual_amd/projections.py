"""Thin Python binding of the C ABI in include/hc_proj.h (libhc_proj.so): the
projections around the hyper-connection read.

    project(x, W, adapter, A, B, scale)    a shared projection with the adapters of many requests
    route(logits, k)                       the k best experts per token, and the rows sorted by expert
    expert_project(x, W, offsets, rows)    products grouped by expert, plain or gated
    expert_combine(y, pos, weights)        each token's expert rows, weighted and summed

Argument checks and marshalling only: every step runs in the HIP kernels.
Inference only: results carry no gradients, whatever the inputs require.  An
`out` must not overlap the inputs.  PyTorch provides device memory and the
current stream.  A call on another stream (`stream=`) neither waits for the
current one nor makes it wait, and does not tell PyTorch that the inputs are in
use there: the caller keeps them until the call's work is done, temporaries too
(or calls their `record_stream`); results are allocated on that stream.  There
is no CPU fallback: if the library is missing or the device is not a gfx950 GPU
the calls raise.
"""
from __future__ import annotations

import ctypes
import os

import torch  # loaded first: the library then binds to the HIP runtime torch uses

from .binding import HC_OK

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libhc_proj.so")

HC_BF16, HC_FP16, HC_FP32 = 0, 1, 2
HC_MAX_RANK = 128
HC_MAX_EXPERTS = 512
HC_MAX_TOPK = 32

# Every function the header exports, with its ctypes signature.
_P, _L, _I = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
SIGNATURES = {
    "hc_project": (_I, [_L, _L, _L, _I, _P, _L, _P, _P, _L, _L, _P, _P, _P, _P, _L, _I, _P, _L, _P]),
    "hc_project_work": (_L, [_L, _L, _L, _L]),
    "hc_route": (_I, [_L, _L, _L, _P, _L, _I, _I, _P, _P, _P, _P, _P, _P, _L, _P]),
    "hc_route_work": (_L, [_L, _L, _L]),
    "hc_expert_project": (_I, [_L, _L, _L, _L, _I, _P, _L, _L, _P, _P, _P, _I, _P, _L, _I, _P]),
    "hc_expert_combine": (_I, [_L, _L, _L, _P, _L, _L, _I, _P, _P, _P, _L, _I, _P]),
    "hc_proj_status_string": (ctypes.c_char_p, [_I]),
    "hc_proj_last_hip_error": (_I, []),
}

_lib = None


class ProjectionError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__("%s: %s (status %d, hip error %d)" % (
            what, hc_proj_status_string(status), status, library().hc_proj_last_hip_error()))
        self.status = status


def library():
    """Load libhc_proj.so (it must have been built: python -m hyper_connection_residual_amd.build)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                "libhc_proj.so is not built; run `python -m hyper_connection_residual_amd.build` "
                "(the projections have no CPU implementation)")
        lib = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
    return _lib


def hc_proj_status_string(status: int) -> str:
    return library().hc_proj_status_string(int(status)).decode()


_TYPE = {torch.bfloat16: HC_BF16, torch.float16: HC_FP16, torch.float32: HC_FP32}
_TYPES = tuple(_TYPE)
_HALF = (torch.bfloat16, torch.float16)
_INT, _FLOAT = (torch.int32,), (torch.float32,)


def _check(t, name, dtypes, shape, strided=False):
    """Type, shape and layout; `strided`: rows may be further apart than they are long.  Returns the elements from
    row to row (a single row's own stride means nothing, nor does a single column's)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch tensor" % name)
    if t.dtype not in dtypes:
        raise TypeError("%s must be one of %s, got %s" % (name, dtypes, t.dtype))
    if t.shape != shape:
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    if t.is_contiguous():
        return shape[-1]
    if not (strided and (shape[1] == 1 or t.stride(1) == 1) and t.stride(0) >= shape[1]):
        raise ValueError("%s must be contiguous%s" % (name, " in its rows, and its rows apart" if strided else ""))
    return t.stride(0) if shape[0] > 1 else shape[1]


def _place(device, *tensors):
    """All tensors on one GPU."""
    for t in tensors:
        if t is not None and t.device != device:
            raise ValueError("the tensors must all be on %s, got one on %s" % (device, t.device))
    if device.type != "cuda":
        raise ValueError("the tensors must be on the GPU, not on %s" % device)


def _matrix(t, name):
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch tensor" % name)
    if t.dim() != 2:
        raise ValueError("%s must have two dimensions, got %s" % (name, tuple(t.shape)))
    return t.shape


# (torch.cuda.current_stream makes a Stream object for its handle, and
# torch.cuda.current_device asks whether CUDA is set up: 3 us of a call's 10)
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _launch(call, device, stream):
    """call(handle of the stream) with the tensors' device and the call's stream current: what it allocates
    belongs to that stream."""
    if stream is None:
        index = device.index
        if index == _current_device():
            return call(_current_stream(index))
        with torch.cuda.device(device):
            return call(_current_stream(index))
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device=device)
    elif stream.device != device:
        raise ValueError("the stream must be on %s, not on %s" % (device, stream.device))
    with torch.cuda.stream(stream):
        return call(stream.cuda_stream)


def _raise(status, what):
    if status != HC_OK:
        raise ProjectionError(status, what)


def _out(out, shape, dtypes, dtype):
    """(type, row stride) of the output: out's, else `dtype` or the first type of those that the call takes."""
    if out is None:
        if dtype is None:
            dtype = dtypes[0]
        elif dtype not in dtypes:
            raise TypeError("out_dtype must be one of %s, got %s" % (dtypes, dtype))
        return dtype, shape[1]
    ldo = _check(out, "out", dtypes, shape, strided=True)
    if dtype is not None and dtype != out.dtype:
        raise TypeError("out_dtype is %s, but out is %s" % (dtype, out.dtype))
    return out.dtype, ldo


def project(x, W, adapter=None, A=None, B=None, scale=None, out=None, out_dtype=None, stream=None):
    """y[t] = W x[t] + scale[a] * B[a] (A[a] x[t]), a = adapter[t], on the current stream.

    x: [T, K] bfloat16 or float16 (rows may be strided); W: [N, K] of x's type.
    adapter: int32 [T], each token's adapter, or None; a value outside [0, n)
    means none.  With it, A: [n, r, K] and B: [n, N, r] of x's type, scale:
    float32 [n] or None for 1.  K and r are multiples of 8, r up to 128.
    out: optional [T, N] tensor (rows may be strided), of x's type or float32;
    else one of out_dtype (default: x's type) is made.  Returns it.
    """
    T, K = _matrix(x, "x")
    N = _matrix(W, "W")[0]
    half = (x.dtype,)
    if x.dtype not in _HALF:
        raise TypeError("x must be one of %s, got %s" % (_HALF, x.dtype))
    ldx = _check(x, "x", half, (T, K), strided=True)
    _check(W, "W", half, (N, K))
    n = r = 0
    if adapter is not None:
        if not isinstance(A, torch.Tensor) or A.dim() != 3:
            raise ValueError("A must be a [adapters, rank, %d] tensor" % K)
        n, r = A.shape[0], A.shape[1]
        _check(adapter, "adapter", _INT, (T,))
        _check(A, "A", half, (n, r, K))
        _check(B, "B", half, (n, N, r))
        if scale is not None:
            _check(scale, "scale", _FLOAT, (n,))
        if n == 0:
            adapter, r = None, 0
    elif A is not None or B is not None or scale is not None:
        raise ValueError("A, B and scale come with adapter")
    device = x.device
    out_dtype, ldo = _out(out, (T, N), (x.dtype, torch.float32), out_dtype)
    _place(device, W, out, *((adapter, A, B, scale) if adapter is not None else ()))

    def call(handle):
        to = torch.empty(T, N, dtype=out_dtype, device=device) if out is None else out
        if T == 0 or N == 0:  # nothing to compute: no launch
            return to
        lib = library()
        size = lib.hc_project_work(T, K, N, r)
        work = torch.empty(size, dtype=torch.uint8, device=device) if size else None
        status = lib.hc_project(
            T, K, N, _TYPE[x.dtype], x.data_ptr(), ldx, W.data_ptr(),
            None if adapter is None else adapter.data_ptr(), n, r,
            None if adapter is None else A.data_ptr(), None if adapter is None else B.data_ptr(),
            None if scale is None else scale.data_ptr(), to.data_ptr(), ldo, _TYPE[out_dtype],
            None if work is None else work.data_ptr(), size, handle)
        _raise(status, "hc_project")
        return to

    return _launch(call, device, stream)


def route(logits, k, renorm=True, stream=None):
    """The k largest of E logits per token, and the rows sorted by expert.

    logits: [T, E] float32, bfloat16 or float16 (rows may be strided), E up to
    512, k up to 32.  Equal logits go to the lower expert; -inf and NaN mask an
    expert out.  renorm: weights are the softmax over the token's chosen
    experts; else over all of its unmasked experts.

    Returns (ids int32 [T, k], best first, -1 where fewer than k are unmasked;
    weights float32 [T, k]; offsets int32 [E + 1], expert e's rows being
    offsets[e] <= i < offsets[e + 1]; rows int32 [T * k], the token of each
    row, -1 from offsets[E] on; pos int32 [T, k], the row of each slot, or -1).
    """
    T, E = _matrix(logits, "logits")
    ldl = _check(logits, "logits", _TYPES, (T, E), strided=True)
    if not 1 <= k <= min(E, HC_MAX_TOPK) or E > HC_MAX_EXPERTS:
        raise ValueError("k must be in 1..min(E, %d) and E up to %d, got k = %d, E = %d" % (
            HC_MAX_TOPK, HC_MAX_EXPERTS, k, E))
    device = logits.device
    _place(device)

    def call(handle):
        if T == 0:
            none = torch.empty((0, k), dtype=torch.int32, device=device)
            return (none, none.float(), torch.zeros(E + 1, dtype=torch.int32, device=device),
                    none.flatten(), none.clone())
        lib = library()
        size = lib.hc_route_work(T, E, k)
        slots = T * k
        # two allocations, cut up (each costs a short call a microsecond and more, and so does each view); the
        # scratch lies behind the offsets, 16-byte aligned
        head = (E + 4) // 4 * 4
        slots_of = torch.empty(4, T, k, dtype=torch.int32, device=device)
        offsets = torch.empty(head + (size + 3) // 4 if size else E + 1, dtype=torch.int32, device=device)
        at, rest = slots_of.data_ptr(), offsets.data_ptr()
        _raise(lib.hc_route(
            T, E, k, logits.data_ptr(), ldl, _TYPE[logits.dtype], bool(renorm), at, at + 4 * slots,
            rest, at + 12 * slots, at + 8 * slots, rest + 4 * head if size else None, size, handle), "hc_route")
        ids, weights, pos, rows = slots_of.unbind(0)
        return ids, weights.view(torch.float32), offsets[:E + 1] if size else offsets, rows.view(-1), pos

    return _launch(call, device, stream)


def expert_project(x, W, offsets, rows=None, gate=False, out=None, out_dtype=None, stream=None):
    """y[i] = W[e] x[rows[i]] for offsets[e] <= i < offsets[e + 1]; gated:
    silu(W[e, :N] x) * (W[e, N:] x).

    x: [rows of x, K] bfloat16 or float16 (rows may be strided), K a multiple of
    8; W: [E, N, K], gated [E, 2 N, K], of x's type; offsets: int32 [E + 1],
    non-decreasing; rows: int32 [R], or None: row i of x for row i.
    out: optional [R, N] tensor (rows may be strided), of x's type or float32,
    whose rows in no group are left as they were; else one of out_dtype
    (default: x's type) is made, whose rows in no group hold anything.
    """
    X, K = _matrix(x, "x")
    if x.dtype not in _HALF:
        raise TypeError("x must be one of %s, got %s" % (_HALF, x.dtype))
    half = (x.dtype,)
    ldx = _check(x, "x", half, (X, K), strided=True)
    if not isinstance(W, torch.Tensor) or W.dim() != 3 or (gate and W.shape[1] % 2):
        raise ValueError("W must be a [experts, %s, %d] tensor" % ("2 N" if gate else "N", K))
    E, N = W.shape[0], W.shape[1] // 2 if gate else W.shape[1]
    _check(W, "W", half, (E, W.shape[1], K))
    _check(offsets, "offsets", _INT, (E + 1,))
    R = X
    if rows is not None:
        R = rows.numel() if isinstance(rows, torch.Tensor) else 0
        _check(rows, "rows", _INT, (R,))
    if X == 0 and R > 0:
        raise ValueError("rows has %d rows of an x without any" % R)
    device = x.device
    out_dtype, ldo = _out(out, (R, N), (x.dtype, torch.float32), out_dtype)
    _place(device, W, offsets, rows, out)

    def call(handle):
        to = torch.empty(R, N, dtype=out_dtype, device=device) if out is None else out
        if R == 0 or N == 0 or E == 0:
            return to
        _raise(library().hc_expert_project(
            R, K, N, E, _TYPE[x.dtype], x.data_ptr(), X, ldx, None if rows is None else rows.data_ptr(),
            W.data_ptr(), offsets.data_ptr(), bool(gate), to.data_ptr(), ldo, _TYPE[out_dtype], handle),
            "hc_expert_project")
        return to

    return _launch(call, device, stream)


def expert_combine(y, pos, weights, out=None, out_dtype=None, stream=None):
    """out[t] = sum over s of weights[t, s] * y[pos[t, s]], in fp32.

    y: [rows, C] bfloat16, float16 or float32 (rows may be strided); pos: int32
    [T, k], a position outside y adds nothing; weights: float32 [T, k].
    out: optional [T, C] tensor of any of the three types (rows may be
    strided); else one of out_dtype (default: y's type) is made.
    """
    Y, C = _matrix(y, "y")
    T, k = _matrix(pos, "pos")
    ldy = _check(y, "y", _TYPES, (Y, C), strided=True)
    _check(pos, "pos", _INT, (T, k))
    _check(weights, "weights", _FLOAT, (T, k))
    device = y.device
    out_dtype, ldo = _out(out, (T, C), (y.dtype,) + _TYPES, out_dtype)
    _place(device, pos, weights, out)

    def call(handle):
        to = torch.empty(T, C, dtype=out_dtype, device=device) if out is None else out
        if T == 0 or C == 0:
            return to
        if k == 0 or Y == 0:
            return to.zero_()
        _raise(library().hc_expert_combine(
            T, k, C, y.data_ptr(), Y, ldy, _TYPE[y.dtype], pos.data_ptr(), weights.data_ptr(),
            to.data_ptr(), ldo, _TYPE[out_dtype], handle), "hc_expert_combine")
        return to

    return _launch(call, device, stream)
