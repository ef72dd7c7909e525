"""Python binding of the 8-bit serving operators (``sgemm_q8_*`` in
``include/sgemm_gb300.h``): row quantisation, RMS norm with quantisation, the
8-bit linear product and the expert layer for a few tokens.

Like the rest of the package it only marshals torch CUDA tensors into the C
ABI: outputs are the caller's, calls are enqueued on ``stream`` (default: the
current torch stream of the output's device) and return without waiting.
"""

from __future__ import annotations

import ctypes

_i64, _vp, _int, _f32 = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int, ctypes.c_float
TYPE_FP32, TYPE_BF16 = 0, 1
ACTIVATIONS = {"none": 0, "relu": 1, "gelu": 2, "silu": 3}

_SIGNATURES = {
    "sgemm_q8_quantize": [_i64, _i64, _vp, _i64, _int, _vp, _i64, _vp, _vp],
    "sgemm_q8_rmsnorm": [_i64, _i64, _vp, _i64, _vp, _i64, _int, _vp, _f32, _vp, _i64, _vp, _i64,
                         _vp, _i64, _vp, _vp],
    "sgemm_q8_linear": [_i64, _i64, _i64, _vp, _i64, _vp, _vp, _i64, _vp, _vp, _int, _vp, _i64,
                        _int, _vp],
    "sgemm_q8_moe": [_i64] * 5 + [_vp, _i64, _int, _vp, _i64, _vp, _i64, _vp, _vp, _i64, _vp, _int,
                                  _vp, _i64, _vp, _vp, _vp],
}
_fn = {}


def _entry(name):
    f = _fn.get(name)
    if f is None:
        from . import lib
        f = getattr(lib(), name)
        f.argtypes, f.restype = _SIGNATURES[name], _int
        _fn[name] = f
    return f


def _launch(index, name, *args):
    """Calls an entry point with the tensors' device current."""
    f = _fn.get(name) or _entry(name)
    if index < 0 or index == _current_device():
        rc = f(*args)
    else:
        with torch.cuda.device(index):
            rc = f(*args)
    if rc:
        from . import SgemmError
        raise SgemmError(rc, name)


torch = None    # imported by the first call: the package can be imported without it


def _load():
    global torch, _TYPES, _FLOATS, _INT8, _raw_stream, _current_device
    import torch as t
    _TYPES = {t.float32: TYPE_FP32, t.bfloat16: TYPE_BF16}
    _FLOATS = (t.float32, t.bfloat16)
    _INT8 = (t.int8,)
    # torch's own accessors behind torch.cuda.current_stream and current_device,
    # without the objects those make (2 us a call); the public ones otherwise
    _raw_stream = getattr(t._C, "_cuda_getCurrentRawStream", None)
    _current_device = getattr(t._C, "_cuda_getDevice", None) or t.cuda.current_device
    torch = t      # last: the sign that the rest is there


def _stream(stream, index):
    if stream is None:
        if index < 0:
            return 0
        return _raw_stream(index) if _raw_stream else torch.cuda.current_stream(index).cuda_stream
    return stream if isinstance(stream, int) else stream.cuda_stream


def _matrix(t, name, dtypes, shape, index):
    """Checks a 2-D operand on CUDA device `index` (-1: the output is not on
    one) of this shape; its row stride."""
    if (type(t) is torch.Tensor and t.dtype in dtypes and t.shape == shape and t.get_device() == index >= 0
            and t.is_contiguous()):
        return shape[1] or 1
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be of type {' or '.join(str(d) for d in dtypes)}, not {t.dtype}")
    if t.dim() != 2 or t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    rows, cols = t.shape
    if t.numel() == 0:
        return max(cols, 1)
    if index < 0 or t.get_device() != index:
        raise TypeError(f"{name} must live on the same CUDA device as the output")
    if cols > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} must be row-major with contiguous rows (stride(1) == 1)")
    return max(t.stride(0), cols) if rows == 1 else t.stride(0)


def _packed(t, name, dtype, shape, index):
    """Checks a contiguous operand of exactly this type and shape."""
    if (type(t) is torch.Tensor and t.dtype is dtype and t.shape == shape and t.get_device() == index >= 0
            and t.is_contiguous()):
        return
    if not isinstance(t, torch.Tensor) or t.dtype != dtype:
        raise TypeError(f"{name} must be a torch tensor of type {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    if t.numel() and (index < 0 or t.get_device() != index):
        raise TypeError(f"{name} must live on the same CUDA device as the output")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _shape2(t, name):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D")
    return t.shape


def _index(t, name):
    """CUDA device of an output (-1: on none)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    return t.get_device()


def quantize_q8(x, q, scale, stream=None) -> None:
    """Each row of ``x`` (M, K; float32 or bfloat16) as 8-bit whole numbers
    ``q`` (M, K; int8) and one ``scale`` (M; float32): x is about q * scale,
    scale = max|row| / 127.  Rows of ``x`` and ``q`` may be strided."""
    if torch is None:
        _load()
    dev, shape = _index(q, "q"), _shape2(x, "x")
    M, K = shape
    ldx = _matrix(x, "x", _FLOATS, shape, dev)
    ldq = _matrix(q, "q", _INT8, shape, dev)
    _packed(scale, "scale", torch.float32, (M,), dev)
    _launch(dev, "sgemm_q8_quantize", M, K, x.data_ptr(), ldx, _TYPES[x.dtype], q.data_ptr(), ldq,
            scale.data_ptr(), _stream(stream, dev))


def rmsnorm_q8(x, weight, q, scale, residual=None, h=None, y=None, eps: float = 1e-6,
               stream=None) -> None:
    """h = x + residual; y = h * weight / sqrt(mean(h^2) + eps); ``q`` and
    ``scale`` are y's 8-bit rows.

    ``x``, ``residual``, ``h`` and ``y`` are (M, K) of one type (float32 or
    bfloat16), ``weight`` K float32 values.  ``residual``, ``h`` and ``y`` may
    be left out; ``h`` may be ``x`` or ``residual`` itself."""
    if torch is None:
        _load()
    dev, shape = _index(q, "q"), _shape2(x, "x")
    M, K = shape
    ldx = _matrix(x, "x", _FLOATS, shape, dev)
    ldq = _matrix(q, "q", _INT8, shape, dev)
    _packed(weight, "weight", torch.float32, (K,), dev)
    _packed(scale, "scale", torch.float32, (M,), dev)
    pr = ph = py = None
    ldr = ldh = ldy = 0
    like = (x.dtype,)
    if residual is not None:
        ldr, pr = _matrix(residual, "residual", like, shape, dev), residual.data_ptr()
    if h is not None:
        ldh, ph = _matrix(h, "h", like, shape, dev), h.data_ptr()
    if y is not None:
        ldy, py = _matrix(y, "y", like, shape, dev), y.data_ptr()
    _launch(dev, "sgemm_q8_rmsnorm", M, K, x.data_ptr(), ldx, pr, ldr, _TYPES[x.dtype],
            weight.data_ptr(), eps, ph, ldh, py, ldy, q.data_ptr(), ldq, scale.data_ptr(),
            _stream(stream, dev))


def linear_q8(xq, xs, wq, ws, out, bias=None, activation: str = "none", stream=None) -> None:
    """out = act((xq @ wq^T) * xs[:, None] * ws[None, :] + bias).

    ``xq`` (M, K) and ``wq`` (N, K) are int8 with the float32 scales ``xs``
    (M) and ``ws`` (N); ``out`` (M, N) is float32 or bfloat16; ``bias`` is N
    float32 values or None; ``activation`` is a key of ``ACTIVATIONS``."""
    if torch is None:
        _load()
    act = ACTIVATIONS.get(activation)
    if act is None:
        raise ValueError(f"unknown activation {activation!r}; one of {sorted(ACTIVATIONS)}")
    dev, xshape, wshape = _index(out, "out"), _shape2(xq, "xq"), _shape2(wq, "wq")
    M, K = xshape
    N = wshape[0]
    if wshape[1] != K:
        raise ValueError(f"shape mismatch: xq {tuple(xshape)}, wq {tuple(wshape)}")
    ldx = _matrix(xq, "xq", _INT8, xshape, dev)
    ldw = _matrix(wq, "wq", _INT8, wshape, dev)
    ldc = _matrix(out, "out", _FLOATS, (M, N), dev)
    _packed(xs, "xs", torch.float32, (M,), dev)
    _packed(ws, "ws", torch.float32, (N,), dev)
    if bias is not None:
        _packed(bias, "bias", torch.float32, (N,), dev)
    _launch(dev, "sgemm_q8_linear", M, N, K, xq.data_ptr(), ldx, xs.data_ptr(), wq.data_ptr(), ldw,
            ws.data_ptr(), None if bias is None else bias.data_ptr(), act, out.data_ptr(), ldc,
            _TYPES[out.dtype], _stream(stream, dev))


def moe_q8(x, router, w_up, s_up, w_down, s_down, out, top_k: int, renormalize: bool = True,
           ids=None, gates=None, stream=None) -> None:
    """A mixture-of-experts layer for up to 64 tokens.

    ``x`` and ``out`` (T, H) are float32 or bfloat16 alike; ``router`` (E, H)
    float32; ``w_up`` (E, 2I, H) and ``w_down`` (E, H, I) int8 with the float32
    scales ``s_up`` (E, 2I) and ``s_down`` (E, H).  The first I rows of an
    expert's ``w_up`` are its gate, the last I its up projection:
    out[t] = sum over the top_k experts of gate * down(silu(gate) * up), with
    the token and the hidden row in 8 bits.  ``ids`` (T, top_k; int32) and
    ``gates`` (T, top_k; float32) take the routing if given."""
    if torch is None:
        _load()
    dev, shape, rshape = _index(out, "out"), _shape2(x, "x"), _shape2(router, "router")
    T, H = shape
    E = rshape[0]
    if rshape[1] != H:
        raise ValueError(f"router must have shape (E, {H}), not {tuple(rshape)}")
    ldx = _matrix(x, "x", _FLOATS, shape, dev)
    ldo = _matrix(out, "out", (x.dtype,), shape, dev)
    ldr = _matrix(router, "router", (torch.float32,), rshape, dev)
    for t, name in ((w_up, "w_up"), (w_down, "w_down")):
        if not isinstance(t, torch.Tensor) or t.dim() != 3:
            raise ValueError(f"{name} must be a torch tensor of three dimensions")
    inner = w_down.shape[2]
    _packed(w_up, "w_up", torch.int8, (E, 2 * inner, H), dev)
    _packed(w_down, "w_down", torch.int8, (E, H, inner), dev)
    _packed(s_up, "s_up", torch.float32, (E, 2 * inner), dev)
    _packed(s_down, "s_down", torch.float32, (E, H), dev)
    if ids is not None:
        _packed(ids, "ids", torch.int32, (T, top_k), dev)
    if gates is not None:
        _packed(gates, "gates", torch.float32, (T, top_k), dev)
    _launch(dev, "sgemm_q8_moe", T, E, top_k, H, inner, x.data_ptr(), ldx, _TYPES[x.dtype],
            router.data_ptr(), ldr, w_up.data_ptr(), H, s_up.data_ptr(), w_down.data_ptr(), inner,
            s_down.data_ptr(), 1 if renormalize else 0, out.data_ptr(), ldo,
            None if ids is None else ids.data_ptr(), None if gates is None else gates.data_ptr(),
            _stream(stream, dev))
