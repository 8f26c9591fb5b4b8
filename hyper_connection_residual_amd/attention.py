"""Thin Python binding of the C ABI in include/hc_attn.h (libhc_attn.so): the
attention between the projections of a layer.

    PagedCache(keys, values)               keys and values of many requests, in pages
    Batch(offsets, lengths, table)         the requests of a call, and their pages
    SharedPrefix(starts, lengths, table)   prefixes that requests share, and their pages
    rotate_heads(x, positions, f)          heads normed and turned by their positions
    append_heads(q, k, v, cache, batch, f) the same for queries and keys; keys and values go to the cache
    attend(q, cache, batch)                softmax(q k) v over each token's positions
    attend_shared(q, cache, batch, prefix) the same where requests begin with shared prefixes

Argument checks and marshalling only: every step runs in the HIP kernels.
Inference only: results carry no gradients, whatever the inputs require.  The
three descriptions check their tensors once and hold them; the tensors' contents
may change between calls (new lengths, new pages), their sizes not.  An `out` must not overlap the inputs, but that
of rotate_heads and append_heads may be the x or q given.  PyTorch provides device memory and the
current stream.  A call on another stream (`stream=`) neither waits for the
current one nor makes it wait, and does not tell PyTorch that the inputs are in
use there: the caller keeps them until the call's work is done, temporaries too
(or calls their `record_stream`); results are allocated on that stream.  There
is no CPU fallback: if the library is missing or the device is not a gfx950 GPU
the calls raise.
"""
from __future__ import annotations

import ctypes
import math
import os

import torch  # loaded first: the library then binds to the HIP runtime torch uses

from .binding import HC_OK
from .projections import HC_BF16, HC_FP16, _check, _launch, _place

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libhc_attn.so")

HC_MAX_HEAD = 256
HC_MAX_REQUESTS = 2048
HC_MAX_ROWS = 262144
HC_MIN_PAGE, HC_MAX_PAGE = 16, 65536
_MOST_SCALE = 2.0 ** 100  # of scale and cap

_P, _L, _I, _F = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float


class hc_cache(ctypes.Structure):
    _fields_ = [("keys", _P), ("values", _P)] + [(n, _L) for n in (
        "pages", "page_size", "heads", "dim", "key_page", "key_row", "key_head", "value_page", "value_row", "value_head",
        "type")]


class hc_batch(ctypes.Structure):
    _fields_ = [("requests", _L), ("offsets", _P), ("lengths", _P), ("table", _P), ("width", _L), ("table_row", _L)]


class hc_prefix(ctypes.Structure):
    _fields_ = [("groups", _L), ("starts", _P), ("lengths", _P), ("table", _P), ("width", _L), ("table_row", _L)]


# Every function the header exports, with its ctypes signature.
_ATTEND = [_F, _F, _P, _P, _P, _P, _L, _L, _P, _L, _P]
SIGNATURES = {
    "hc_rotate_heads": (_I, [_L, _L, _L, _I, _P, _L, _L, _P, _P, _L, _I, _P, _F, _P, _L, _L, _P]),
    "hc_append_heads": (_I, [_L, _L, _P, _L, _L, _P, _L, _L, _P, _L, _L, _P, _P, _P, _P, _L, _I, _P, _P, _F, _P, _L, _L, _P]),
    "hc_attend": (_I, [_L, _L, _P, _L, _L, _P, _P] + _ATTEND),
    "hc_attend_shared": (_I, [_L, _L, _P, _L, _L, _P, _P, _P] + _ATTEND),
    "hc_attend_work": (_L, [_L, _L, _L, _L, _L, _L]),
    "hc_attn_status_string": (ctypes.c_char_p, [_I]),
    "hc_attn_last_hip_error": (_I, []),
}

_lib = None


class AttentionError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__("%s: %s (status %d, hip error %d)" % (
            what, hc_attn_status_string(status), status, library().hc_attn_last_hip_error()))
        self.status = status


def library():
    """Load libhc_attn.so (it must have been built: python -m hyper_connection_residual_amd.build)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                "libhc_attn.so is not built; run `python -m hyper_connection_residual_amd.build` "
                "(the attention has no CPU implementation)")
        lib = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
    return _lib


def hc_attn_status_string(status: int) -> str:
    return library().hc_attn_status_string(int(status)).decode()


_TYPE = {torch.bfloat16: HC_BF16, torch.float16: HC_FP16}
_HALF = tuple(_TYPE)
_INT, _FLOAT = (torch.int32,), (torch.float32,)


def _raise(status, what):
    if status != HC_OK:
        raise AttentionError(status, what)


def _heads(t, name, dtypes, shape=None):
    """(token stride, head stride) of [tokens, heads, columns], whose columns are contiguous.  (The stride of a
    dimension of one means nothing.)"""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch tensor" % name)
    if t.dtype not in dtypes:
        raise TypeError("%s must be one of %s, got %s" % (name, dtypes, t.dtype))
    if t.dim() != 3 or (shape is not None and t.shape != shape):
        raise ValueError("%s must have shape %s, got %s" % (
            name, "[tokens, heads, columns]" if shape is None else tuple(shape), tuple(t.shape)))
    T, H, D = t.shape
    if D < 1 or D > HC_MAX_HEAD or D % 8:
        raise ValueError("%s must have heads of a multiple of 8 columns up to %d, got %d" % (name, HC_MAX_HEAD, D))
    row, head, col = t.stride()
    if t.numel() == 0:
        return max(H, 1) * D, D
    if H == 1:
        head = D
    if T == 1:
        row = H * head
    if col != 1 or row % 8 or head % 8 or head < D or row < D:
        raise ValueError("%s must have contiguous columns, heads and tokens apart and at multiples of 8 elements, got "
                         "strides %s" % (name, t.stride()))
    return row, head


def _list(t, name, shape):
    _check(t, name, _INT, shape)
    return t.data_ptr()


def _table(table, rows, name):
    """(pointer, width, row stride) of a table of pages."""
    if not isinstance(table, torch.Tensor):
        raise TypeError("%s must be a torch tensor" % name)
    if table.dim() != 2:
        raise ValueError("%s must have two dimensions, got %s" % (name, tuple(table.shape)))
    row = _check(table, name, _INT, (rows, table.shape[1]), strided=True)
    return table.data_ptr(), table.shape[1], row


class PagedCache:
    """keys, values: [pages, page_size, heads, columns] of bfloat16 or float16, in any strides of multiples of 8 with
    contiguous columns (a view of one tensor that holds both, or heads before rows, will do).  page_size is a power of
    two from 16, columns a multiple of 8 up to 256."""

    def __init__(self, keys, values):
        for t, name in ((keys, "keys"), (values, "values")):
            if not isinstance(t, torch.Tensor):
                raise TypeError("%s must be a torch tensor" % name)
            if t.dtype not in _HALF:
                raise TypeError("%s must be one of %s, got %s" % (name, _HALF, t.dtype))
            if t.dim() != 4 or 0 in t.shape:
                raise ValueError("%s must be [pages, page size, heads, columns], got %s" % (name, tuple(t.shape)))
        if values.dtype != keys.dtype:
            raise TypeError("values must be %s as the keys, got %s" % (keys.dtype, values.dtype))
        if values.shape != keys.shape:
            raise ValueError("values must have shape %s, got %s" % (tuple(keys.shape), tuple(values.shape)))
        pages, size, heads, dim = keys.shape
        if size & (size - 1) or not HC_MIN_PAGE <= size <= HC_MAX_PAGE:
            raise ValueError("a page must hold a power of two of positions, from %d to %d, got %d" % (HC_MIN_PAGE, HC_MAX_PAGE, size))
        if dim % 8 or dim > HC_MAX_HEAD:
            raise ValueError("heads must have a multiple of 8 columns up to %d, got %d" % (HC_MAX_HEAD, dim))
        strides = []
        for t, name in ((keys, "keys"), (values, "values")):
            page, row, head, col = t.stride()
            if pages == 1:
                page = 0
            if heads == 1:
                head = dim
            if (col != 1 and dim > 1) or page % 8 or row % 8 or head % 8 or row < dim or head < dim or page < 0 or page >= (1 << 31) - 65536 or max(row, head) >= 1 << 23:
                raise ValueError("%s must have contiguous columns and pages, rows and heads apart and at multiples of 8 "
                                 "elements, got strides %s" % (name, t.stride()))
            strides += [page, row, head]
        _place(keys.device, values)
        self.keys, self.values = keys, values
        self.device, self.dtype, self.heads, self.dim = keys.device, keys.dtype, heads, dim
        self._c = hc_cache(keys.data_ptr(), values.data_ptr(), pages, size, heads, dim, *strides, _TYPE[keys.dtype])
        self._at = ctypes.addressof(self._c)


class Batch:
    """offsets: int32 [requests + 1], request b's new tokens being offsets[b] <= t < offsets[b + 1]; lengths: int32
    [requests], its positions, the new tokens being the last ones; table: int32 [requests, width] (rows may be
    strided), the page of each page_size positions.  Up to 2048 requests."""

    def __init__(self, offsets, lengths, table):
        if not isinstance(lengths, torch.Tensor) or not isinstance(offsets, torch.Tensor):
            raise TypeError("offsets and lengths must be torch tensors")
        B = lengths.numel()
        if not 1 <= B <= HC_MAX_REQUESTS:
            raise ValueError("a batch has 1 to %d requests, got %d" % (HC_MAX_REQUESTS, B))
        at = _list(offsets, "offsets", (B + 1,)), _list(lengths, "lengths", (B,)), *_table(table, B, "table")
        _place(offsets.device, lengths, table)
        self.offsets, self.lengths, self.table, self.device, self.requests = offsets, lengths, table, offsets.device, B
        self._c = hc_batch(B, *at)
        self._at = ctypes.addressof(self._c)


class SharedPrefix:
    """starts: int32 [groups + 1], the requests starts[g] <= b < starts[g + 1] beginning with prefix g; lengths: int32
    [groups], its positions; table: int32 [groups, width] (rows may be strided), their pages."""

    def __init__(self, starts, lengths, table):
        if not isinstance(lengths, torch.Tensor) or not isinstance(starts, torch.Tensor):
            raise TypeError("starts and lengths must be torch tensors")
        G = lengths.numel()
        if not 1 <= G <= HC_MAX_REQUESTS:
            raise ValueError("there are 1 to %d prefixes, got %d" % (HC_MAX_REQUESTS, G))
        at = _list(starts, "starts", (G + 1,)), _list(lengths, "lengths", (G,)), *_table(table, G, "table")
        _place(starts.device, lengths, table)
        self.starts, self.lengths, self.table, self.device, self.groups = starts, lengths, table, starts.device, G
        self._c = hc_prefix(G, *at)
        self._at = ctypes.addressof(self._c)


def _rotation(frequencies, dim, device):
    """(pointer, rotated columns)"""
    if frequencies is None:
        return None, 0
    if not isinstance(frequencies, torch.Tensor):
        raise TypeError("frequencies must be a torch tensor")
    n = frequencies.numel()
    _check(frequencies, "frequencies", _FLOAT, (n,))
    if n < 1 or n % 4 or 2 * n > dim:
        raise ValueError("frequencies must be a multiple of 4, of up to half of a head's %d columns, got %d" % (dim, n))
    return frequencies.data_ptr(), 2 * n


def _weight(w, name, dim):
    if w is None:
        return None
    _check(w, name, _FLOAT, (dim,))
    return w.data_ptr()


def _eps(eps):
    if not (isinstance(eps, (int, float)) and 0.0 <= eps < math.inf):
        raise ValueError("eps must be a number from 0, got %s" % (eps,))
    return eps


def _tokens(t, name, T):
    if t is None:
        return None
    _check(t, name, _INT, (T,))
    return t.data_ptr()


def _out_heads(out, q, strides):
    """(token stride, head stride) of the output, of q's shape: out's, else those of a new one."""
    if out is None:
        return q.shape[1] * q.shape[2], q.shape[2]
    if out is q:
        return strides
    return _heads(out, "out", (q.dtype,), q.shape)


def rotate_heads(x, positions=None, frequencies=None, weight=None, eps=1e-6, interleaved=False, out=None, stream=None):
    """Every head normed, x / sqrt(mean x^2 + eps) * weight, and turned by its token's position.

    x: [T, heads, columns] bfloat16 or float16 (tokens and heads may be strided).
    frequencies: float32 [n] in radians per position, or None for no rotation:
    the pair i of the first 2 n columns, (i, i + n) or, interleaved, (2 i, 2 i +
    1), turns by positions[t] * frequencies[i]; n is a multiple of 4.
    positions: int32 [T].  weight: float32 [columns], or None for no norm.
    out: optional tensor of x's shape and type, or x itself; else one is made.
    Returns it.
    """
    row, head = strides = _heads(x, "x", _HALF)
    T, H, D = x.shape
    device = x.device
    f, rotated = _rotation(frequencies, D, device)
    if f is not None and positions is None:
        raise ValueError("frequencies come with positions")
    at = _tokens(positions, "positions", T)
    w = _weight(weight, "weight", D)
    out_row, out_head = _out_heads(out, x, strides)
    _eps(eps)
    _place(device, positions, frequencies, weight, out)

    def call(handle):
        to = torch.empty(x.shape, dtype=x.dtype, device=device) if out is None else out
        if T == 0 or H == 0:
            return to
        _raise(library().hc_rotate_heads(T, H, D, _TYPE[x.dtype], x.data_ptr(), row, head, at, f, rotated, bool(interleaved), w,
                                         eps, to.data_ptr(), out_row, out_head, handle), "hc_rotate_heads")
        return to

    return _launch(call, device, stream)


def append_heads(q, k, v, cache, batch, frequencies=None, positions=None, q_weight=None, k_weight=None, eps=1e-6,
                 interleaved=False, out=None, stream=None):
    """A batch's new tokens: keys normed, turned and stored in the cache, values stored there, queries normed, turned and
    returned.

    q: [T, q_heads, columns], or None; k, v: [T, cache heads, columns] of the
    cache's type (tokens and heads may be strided: views of one projection's
    rows will do).  Token t goes to its request's position lengths[b] -
    offsets[b + 1] + t; one that the table or the cache has no place for is not
    stored.  positions: int32 [T], what the angles go by, where it is not that
    position (requests under a shared prefix).  frequencies, weights, eps and
    interleaved as for rotate_heads.  out: optional tensor like q, or q itself;
    its tokens of no request are left as they were.  Returns it (None without q).
    """
    if not isinstance(cache, PagedCache) or not isinstance(batch, Batch):
        raise TypeError("cache must be a PagedCache and batch a Batch")
    half = (cache.dtype,)
    D, device = cache.dim, cache.device
    k_row, k_head = _heads(k, "k", half)
    T = k.shape[0]
    if k.shape != (T, cache.heads, D):
        raise ValueError("k must have shape %s, got %s" % ((T, cache.heads, D), tuple(k.shape)))
    v_row, v_head = _heads(v, "v", half, (T, cache.heads, D))
    H = row = head = out_row = out_head = 0
    if q is not None:
        row, head = strides = _heads(q, "q", half)
        H = q.shape[1]
        if q.shape != (T, H, D):
            raise ValueError("q must have shape %s, got %s" % ((T, H, D), tuple(q.shape)))
        out_row, out_head = _out_heads(out, q, strides)
    elif out is not None:
        raise ValueError("out comes with q")
    f, rotated = _rotation(frequencies, D, device)
    at = _tokens(positions, "positions", T)
    qw, kw = _weight(q_weight, "q_weight", D), _weight(k_weight, "k_weight", D)
    _eps(eps)
    _place(device, q, k, v, batch, positions, frequencies, q_weight, k_weight, out)

    def call(handle):
        to = out
        if q is not None and out is None:
            to = torch.empty((T, H, D), dtype=q.dtype, device=device)
        if T == 0:
            return to
        _raise(library().hc_append_heads(
            T, H, q.data_ptr() if H else None, row, head, k.data_ptr(), k_row, k_head, v.data_ptr(), v_row, v_head, cache._at,
            batch._at, at, f, rotated, bool(interleaved), qw, kw, eps, to.data_ptr() if H else None, out_row, out_head, handle),
            "hc_append_heads")
        return to

    return _launch(call, device, stream)


def _attend(q, cache, batch, prefix, scale, cap, slopes, first, last, out, stream):
    if not isinstance(cache, PagedCache) or not isinstance(batch, Batch):
        raise TypeError("cache must be a PagedCache and batch a Batch")
    row, head = strides = _heads(q, "q", (cache.dtype,))
    T, H, D = q.shape
    device = cache.device
    if D != cache.dim or H < 1 or H % cache.heads:
        raise ValueError("q must have heads of %d columns, a multiple of the cache's %d, got %s" % (cache.dim, cache.heads, tuple(q.shape)))
    if T * (H // cache.heads) > HC_MAX_ROWS:
        raise ValueError("a call has up to %d tokens times query heads by cache heads, got %d" % (HC_MAX_ROWS, T * (H // cache.heads)))
    scale = D ** -0.5 if scale is None else float(scale)
    cap = 0.0 if cap is None else float(cap)
    if not (abs(scale) <= _MOST_SCALE and 0.0 <= cap <= _MOST_SCALE):
        raise ValueError("scale must be within -2^100 and 2^100 and cap within 0 and 2^100, got %s and %s" % (scale, cap))
    if slopes is not None:
        _check(slopes, "slopes", _FLOAT, (H,))
    lo, hi = _tokens(first, "first", T), _tokens(last, "last", T)
    out_row, out_head = _out_heads(out, q, strides)
    if out is q:
        raise ValueError("out must not be q")
    _place(device, q, batch, prefix, slopes, first, last, out)

    def call(handle):
        to = torch.empty((T, H, D), dtype=q.dtype, device=device) if out is None else out
        if T == 0:
            return to
        lib = library()
        size = lib.hc_attend_work(T, H, cache.heads, D, batch.requests, 0 if prefix is None else prefix.groups)
        work = torch.empty(size, dtype=torch.uint8, device=device)
        rest = (scale, cap, None if slopes is None else slopes.data_ptr(), lo, hi, to.data_ptr(), out_row, out_head,
                work.data_ptr(), size, handle)
        if prefix is None:
            _raise(lib.hc_attend(T, H, q.data_ptr(), row, head, cache._at, batch._at, *rest), "hc_attend")
        else:
            _raise(lib.hc_attend_shared(T, H, q.data_ptr(), row, head, cache._at, batch._at, prefix._at, *rest), "hc_attend_shared")
        return to

    return _launch(call, device, stream)


def attend(q, cache, batch, scale=None, cap=None, slopes=None, first=None, last=None, out=None, stream=None):
    """out[t, h] = sum_j softmax_j(score) v[j] over the positions j that the token sees.

    q: [T, q_heads, columns] of the cache's type (tokens and heads may be
    strided), q_heads a multiple of the cache's heads, T * q_heads / heads up to
    262144; tables of up to 2^31 - 65536 positions, with their prefixes'.  score =
    scale * q k[j] (scale: default columns ** -0.5); with cap, cap * tanh(score /
    cap); with slopes (float32 [q_heads]), less slopes[h] * |p - j|, p being the
    token's position.  first, last: int32 [T], token t sees
    first[t] <= j < last[t] of its request's positions, by default 0 and p + 1:
    causal; windows and packed documents by first, prefixes that see each other
    and no causality at all by last.  A token that sees none gives zeros.
    out: optional tensor of q's shape and type, whose tokens of no request are
    left as they were; else one is made.  Returns it.
    """
    return _attend(q, cache, batch, None, scale, cap, slopes, first, last, out, stream)


def attend_shared(q, cache, batch, prefix, scale=None, cap=None, slopes=None, first=None, last=None, out=None, stream=None):
    """attend, where groups of requests begin with prefixes that they share: each prefix's keys and values are read once
    for all of its requests' tokens.

    A request's sequence is its prefix's positions and then its own, those of
    the batch; positions (p, j, first and last) count from the prefix's first.
    By default a token sees the whole prefix and its request's own positions up
    to its own.  Every row leaves two partial results in scratch (8192 tokens of 20
    heads of 128 columns: 239 MB, attend 68): for prompts of hundreds of tokens per
    request, attend with the prefix's pages in every request's own table is faster.
    """
    if not isinstance(prefix, SharedPrefix):
        raise TypeError("prefix must be a SharedPrefix")
    return _attend(q, cache, batch, prefix, scale, cap, slopes, first, last, out, stream)
