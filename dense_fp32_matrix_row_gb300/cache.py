"""Python binding of the attention operators over an 8-bit paged key-value cache
(``include/sgemm_gb300.h``): norms of query and key heads with the position
rotation, the cache's write and read, and attention of one new token per
sequence.

As in ``q8``, outputs are the caller's tensors, calls are enqueued on ``stream``
(default: the current torch stream of the output's device) and return without
waiting.  Heads are tensors of (tokens, heads, dim) with contiguous dims; tokens
and heads may be strided, as the views of a joint projection's rows are.
Positions, slots, page numbers and lengths stay on the device: one outside its
array is left out by the call and reported by the next ``status()``.
"""

from __future__ import annotations

import ctypes
import math
import struct

from . import q8

_i64, _vp, _int, _f32 = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int, ctypes.c_float
_HEADS = struct.Struct("Qqqq").pack                 # sgemm_heads
_ROTARY = struct.Struct("QQqqqQi4x").pack           # sgemm_rotary
_CACHE = struct.Struct("QQQQqqqqqqqq").pack         # sgemm_q8_cache

q8._SIGNATURES.update({
    "sgemm_norm_rope": [_i64, _i64, _int] + [_vp] * 6 + [_f32, _vp, _vp],
    "sgemm_q8_cache_write": [_i64, _int] + [_vp] * 5,
    "sgemm_q8_norm_rope_write": [_i64, _int] + [_vp] * 6 + [_f32, _vp, _vp, _vp, _vp],
    "sgemm_q8_cache_read": [_i64, _int] + [_vp] * 5,
    "sgemm_q8_attend": [_i64, _int, _vp, _vp, _vp, _i64, _i64, _vp, _f32, _i64, _vp, _vp, _vp],
})


_Tensor = None      # and the types below: set by the first call, like q8.torch


def _load():
    global _Tensor, _F32, _I32, _I64, _FLOATS, _TYPES
    if q8.torch is None:
        q8._load()
    t = q8.torch
    _F32, _I32, _I64, _FLOATS, _TYPES = t.float32, t.int32, t.int64, q8._FLOATS, q8._TYPES
    _Tensor = t.Tensor


# The helpers take a call's eight or ten tensors apart in the time that its launch
# leaves: each asks a tensor only for what it needs, at 0.1 us an answer.

def _heads(t, name, dtype, shape, index):
    """Checks heads of this type (None: type and shape are known to be right) and shape on
    CUDA device `index`; their sgemm_heads."""
    if dtype is not None:
        if not isinstance(t, _Tensor):
            raise TypeError(f"{name} must be a torch tensor")
        if t.dtype is not dtype:
            raise TypeError(f"{name} must be of type {dtype}, not {t.dtype}")
        if t.shape != shape:
            raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    T, H, D = shape
    if T == 0 or H == 0:
        return _HEADS(0, 0, 0, 0)
    if t.get_device() != index or index < 0:
        raise TypeError(f"{name} must live on the same CUDA device as the output")
    ld, hs, ds = t.stride()
    if ds != 1 and D > 1:
        raise ValueError(f"{name} must have contiguous heads (stride(2) == 1)")
    if H == 1:          # the strides of a single head or token are arbitrary in torch
        hs = D
    if T == 1:
        ld = (H - 1) * hs + D
    return _HEADS(t.data_ptr(), H, ld, hs)


def _vector(t, name, dtype, shape, index):
    """Checks a contiguous array of this shape; its address."""
    if not (isinstance(t, _Tensor) and t.dtype is dtype and t.shape == shape and t.get_device() == index >= 0
            and t.is_contiguous()):
        q8._packed(t, name, dtype, shape, index)        # says what is wrong (or lets an empty one pass)
    return t.data_ptr()


def _shape3(t, name):
    if not isinstance(t, _Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    shape = t.shape
    if len(shape) != 3:
        raise ValueError(f"{name} must be 3-D (tokens, heads, dim)")
    return shape


def _type(t, name):
    dtype = t.dtype
    if dtype not in _FLOATS:
        raise TypeError(f"{name} must be of type float32 or bfloat16, not {dtype}")
    return dtype


def _rotary(cos, sin, positions, interleaved, T, index):
    """The tables' sgemm_rotary (None without them)."""
    if cos is None and sin is None:
        return None
    if (isinstance(cos, _Tensor) and isinstance(sin, _Tensor) and cos.dtype is _F32 and sin.dtype is _F32
            and cos.get_device() == index == sin.get_device() and index >= 0 and cos.is_contiguous()
            and sin.is_contiguous() and cos.dim() == 2 and cos.shape == sin.shape):
        rows, ld = cos.shape
        half = ld
    else:                   # strided, empty, or wrong: says what
        rows, half = q8._shape2(cos, "cos")
        ld = q8._matrix(cos, "cos", (_F32,), (rows, half), index)
        if q8._matrix(sin, "sin", (_F32,), (rows, half), index) != ld:
            raise ValueError("cos and sin must have the same row stride")
    at = 0 if positions is None else _vector(positions, "positions", _I64, (T,), index)
    return _ROTARY(cos.data_ptr(), sin.data_ptr(), rows, ld, 2 * half, at, 1 if interleaved else 0)


class CacheQ8:
    """Keys and values of past tokens in pages of 8-bit rows, one scale per row.

    ``k`` and ``v`` are int8 (blocks, heads, page, dim), ``k_scale`` and
    ``v_scale`` float32 (blocks, heads, page), all on one CUDA device.  Pages may
    be strided (views of a larger pool); within a page the elements are
    contiguous.  The object keeps the tensors; it neither copies nor clears them.
    One that is given another storage, shape or strides, or is replaced, is checked
    again by the next call, which takes it as it then is.
    ``slot = block * page + row`` names a token's place."""

    __slots__ = ("k", "v", "k_scale", "v_scale", "heads", "page", "dim", "slots", "_device", "_c", "_of", "_ask", "_seen")

    def __init__(self, k, v, k_scale, v_scale):
        if _Tensor is None:
            _load()
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self._check()

    def _check(self):
        torch = q8.torch
        self._seen = None       # until everything is found to be fine
        self._of = of = (self.k, self.v, self.k_scale, self.v_scale)
        names = ("k", "v", "k_scale", "v_scale")
        for t, name in zip(of, names):
            if not isinstance(t, torch.Tensor):
                raise TypeError(f"{name} must be a torch tensor")
        if self.k.dim() != 4:
            raise ValueError("k must be 4-D (blocks, heads, page, dim)")
        shape = self.k.shape
        blocks, heads, page, dim = shape
        if 0 in shape[1:]:
            raise ValueError(f"a cache has heads, rows and elements: k of shape {tuple(shape)}")
        device = self.k.get_device()
        strides, ask = [], []
        for t, name, dtype, want in zip(of, names, (torch.int8, torch.int8, torch.float32, torch.float32),
                                        (shape, shape, shape[:3], shape[:3])):
            if t.dtype is not dtype:
                raise TypeError(f"{name} must be of type {dtype}, not {t.dtype}")
            if t.shape != want:
                raise ValueError(f"{name} must have shape {tuple(want)}, not {tuple(t.shape)}")
            if t.numel() and (device < 0 or t.get_device() != device):
                raise TypeError("the cache's tensors must live on one CUDA device")
            if blocks and not t[0].is_contiguous():
                raise ValueError(f"{name} must have contiguous pages")
            strides.append(t.stride(0) if blocks > 1 else t[0].numel() if blocks else 0)
            # what its place and layout are told by: a contiguous tensor's size says where its elements are
            ask += (t.data_ptr, t.size, t.is_contiguous if t.is_contiguous() else t.stride)
        self.heads, self.page, self.dim, self.slots = heads, page, dim, blocks * page
        self._device = device
        self._c = _CACHE(*(t.data_ptr() for t in of), blocks, heads, page, dim, *strides)
        self._ask = ask
        self._seen = [f() for f in ask]

    def _struct(self):
        """The sgemm_q8_cache; made again where a tensor's place or layout is another."""
        if self._seen is not None:
            k, v, ks, vs = self._of
            a, b, c, d, e, f, g, h, i, j, m, n = self._ask      # 0.1 us less than a loop
            if (self.k is k and self.v is v and self.k_scale is ks and self.v_scale is vs
                    and [a(), b(), c(), d(), e(), f(), g(), h(), i(), j(), m(), n()] == self._seen):
                return self._c
        self._check()
        return self._c


def _cache(cache):
    if type(cache) is not CacheQ8:
        raise TypeError("cache must be a CacheQ8")
    return cache._struct()


def norm_rope(q, k, cos, sin, q_out, k_out, positions=None, q_weight=None, k_weight=None, eps: float = 1e-6,
              interleaved: bool = False, stream=None) -> None:
    """RMS norm and position rotation of each head, in one pass:
    p = x * weight, p's pairs turned by their angles, result p / sqrt(mean(x^2) + eps).

    ``q`` (T, Hq, D) and ``k`` (T, Hk, D) are float32 or bfloat16 alike, like their
    results ``q_out`` and ``k_out`` (which may be q and k themselves); either pair may
    be None.  ``cos`` and ``sin`` (rows, R/2; float32) are the tables of the first R
    elements' angles; token t has row ``positions[t]`` (int64), or row t without
    ``positions``; both None: no rotation.  Pairs are (i, i + R/2), or (2i, 2i+1)
    with ``interleaved``.  ``q_weight`` and ``k_weight`` (D; float32): None: no norm.
    A token whose position is outside the tables is left out."""
    if _Tensor is None:
        _load()
    if q is None and k is None:
        raise ValueError("norm_rope needs q or k")
    lead, result, name = (q, q_out, "q") if q is not None else (k, k_out, "k")
    shape, dev, dt = _shape3(lead, name), q8._index(result, name + "_out"), _type(lead, name)
    T, _, D = shape
    cq = cqo = ck = cko = pq = pk = None
    if q is not None:
        cq, cqo = _heads(q, "q", None, shape, dev), _heads(q_out, "q_out", dt, shape, dev)
        if q_weight is not None:
            pq = _vector(q_weight, "q_weight", _F32, (D,), dev)
    if k is not None:
        kshape = _shape3(k, "k")
        if kshape[0] != T or kshape[2] != D:
            raise ValueError(f"k must have shape ({T}, heads, {D}), not {tuple(kshape)}")
        ck, cko = _heads(k, "k", dt if k is not lead else None, kshape, dev), _heads(k_out, "k_out", dt, kshape, dev)
        if k_weight is not None:
            pk = _vector(k_weight, "k_weight", _F32, (D,), dev)
    rotary = _rotary(cos, sin, positions, interleaved, T, dev)
    q8._launch(dev, "sgemm_norm_rope", T, D, _TYPES[dt], cq, cqo, pq, ck, cko, pk, eps, rotary,
               q8._stream(stream, dev))


def cache_write_q8(k, v, cache, slots, stream=None) -> None:
    """Keys and values ``k`` and ``v`` (T, heads, dim; float32 or bfloat16 alike) into
    ``cache`` at ``slots`` (T; int64): each row as 8-bit whole numbers with one scale,
    max|row| / 127.  A token with a negative slot is not stored; slots that are not
    negative have to differ."""
    norm_rope_write_q8(None, k, v, None, None, None, cache, slots, stream=stream)


def norm_rope_write_q8(q, k, v, cos, sin, q_out, cache, slots, positions=None, q_weight=None, k_weight=None,
                       eps: float = 1e-6, interleaved: bool = False, stream=None) -> None:
    """``norm_rope`` of ``q`` into ``q_out`` and of ``k`` into ``cache``, with ``v`` as it
    is, in one pass: what a decoder layer does between its first product and
    attention.  The keys are not rounded to ``k``'s type on their way into 8 bits.
    ``q`` and ``q_out`` may be None; the other arguments are those of ``norm_rope``
    and ``cache_write_q8``."""
    if _Tensor is None:
        _load()
    c = _cache(cache)
    shape, dev, dt = _shape3(k, "k"), cache._device, _type(k, "k")
    T = shape[0]
    want = (T, cache.heads, cache.dim)
    if shape != want:
        raise ValueError(f"k must have shape {want}, not {tuple(shape)}")
    ck, cv = _heads(k, "k", None, want, dev), _heads(v, "v", dt, want, dev)
    at = _vector(slots, "slots", _I64, (T,), dev)
    cq = cqo = pq = pk = None
    if q is not None:
        qshape = _shape3(q, "q")
        if qshape[0] != T or qshape[2] != cache.dim:
            raise ValueError(f"q must have shape ({T}, heads, {cache.dim}), not {tuple(qshape)}")
        cq, cqo = _heads(q, "q", dt, qshape, dev), _heads(q_out, "q_out", dt, qshape, dev)
        if q_weight is not None:
            pq = _vector(q_weight, "q_weight", _F32, (cache.dim,), dev)
    if k_weight is not None:
        pk = _vector(k_weight, "k_weight", _F32, (cache.dim,), dev)
    rotary = _rotary(cos, sin, positions, interleaved, T, dev)
    q8._launch(dev, "sgemm_q8_norm_rope_write", T, _TYPES[dt], cq, cqo, pq, ck, pk, cv, eps, rotary, at, c,
               q8._stream(stream, dev))


def cache_read_q8(cache, slots, k_out=None, v_out=None, stream=None) -> None:
    """The rows at ``slots`` (N; int64) as floats, whole number * scale, into ``k_out``
    and ``v_out`` (N, heads, dim; float32 or bfloat16 alike; either may be None).  A
    row whose slot is negative stays as it was."""
    if _Tensor is None:
        _load()
    c = _cache(cache)
    lead = k_out if k_out is not None else v_out
    if lead is None:
        raise ValueError("cache_read_q8 needs k_out or v_out")
    name = "k_out" if k_out is not None else "v_out"
    shape, dev, dt = _shape3(lead, name), lead.get_device(), _type(lead, name)
    N = shape[0]
    want = (N, cache.heads, cache.dim)
    if shape != want:
        raise ValueError(f"{name} must have shape {want}, not {tuple(shape)}")
    if N and cache._device != dev:
        raise TypeError("the cache must live on the same CUDA device as the output")
    ck = None if k_out is None else _heads(k_out, "k_out", None, want, dev)
    cv = None if v_out is None else _heads(v_out, "v_out", None if k_out is None else dt, want, dev)
    at = _vector(slots, "slots", _I64, (N,), dev)
    q8._launch(dev, "sgemm_q8_cache_read", N, _TYPES[dt], c, at, ck, cv, q8._stream(stream, dev))


def attend_q8(q, cache, table, lens, out, scale=None, window: int = 0, lse=None, stream=None) -> None:
    """Attention of one new token per sequence over ``cache``:
    out = softmax(scale * q k^T) v over the sequence's tokens.

    ``q`` and ``out`` (B, heads, dim) are float32 or bfloat16 alike, ``heads`` a
    multiple of the cache's: query head h reads key head h * cache.heads // heads.
    Token t of sequence b is row t % page of page ``table[b, t // page]``; ``table``
    (B, pages) and ``lens`` (B) are int32.  ``window`` > 0: only the last ``window``
    tokens.  ``scale`` defaults to 1 / sqrt(dim).  ``lse`` (B, heads; float32) takes the
    logarithm of the sum of exp(scores).  A sequence of length 0 gives zeros and -inf."""
    if _Tensor is None:
        _load()
    c = _cache(cache)
    shape, dev, dt = _shape3(q, "q"), q8._index(out, "out"), _type(q, "q")
    B, H, D = shape
    if D != cache.dim or H % cache.heads != 0 or H == 0:
        raise ValueError(f"q must have shape (sequences, a multiple of {cache.heads} heads, {cache.dim}), not {tuple(shape)}")
    if B and cache._device != dev:
        raise TypeError("the cache must live on the same CUDA device as the output")
    cq, co = _heads(q, "q", None, shape, dev), _heads(out, "out", dt, shape, dev)
    tshape = q8._shape2(table, "table")
    if tshape[0] != B:
        raise ValueError(f"table must have shape ({B}, pages), not {tuple(tshape)}")
    if table.dtype is _I32 and table.get_device() == dev >= 0 and table.is_contiguous():
        ldt = tshape[1] or 1
    else:                   # strided, empty, or wrong: says what
        ldt = q8._matrix(table, "table", (_I32,), tshape, dev)
    pl = _vector(lens, "lens", _I32, (B,), dev)
    ps = None if lse is None else _vector(lse, "lse", _F32, (B, H), dev)
    q8._launch(dev, "sgemm_q8_attend", B, _TYPES[dt], cq, c, table.data_ptr(), ldt, tshape[1], pl,
               1.0 / math.sqrt(D) if scale is None else scale, window, co, ps,
               q8._stream(stream, dev))
