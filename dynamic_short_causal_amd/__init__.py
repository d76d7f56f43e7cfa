"""Python binding of ``libdsc.so``, the gfx950 dynamic short causal convolution.

Argument marshalling only: every step of the computation runs in the HIP
kernels behind the C ABI of ``include/dsc.h``.  PyTorch supplies device memory
and the current stream.  There is no CPU or PyTorch fallback: if the library
is missing, importing this package raises.

The functions named like the C entry points (``dsc_headwise_fwd`` ...) take
pre-allocated output tensors; ``headwise_fwd`` and friends allocate them with
``torch.empty``, on the stream of the call, and call the former.
"""
import ctypes
import functools
import inspect
import math
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libdsc.so")

DSC_OK, DSC_ERR_INVALID_ARG, DSC_ERR_UNSUPPORTED, DSC_ERR_WORKSPACE, DSC_ERR_HIP = range(5)
DSC_F32, DSC_BF16 = 0, 1
DSC_RESIDUAL, DSC_ACT_SILU = 1, 2

# every symbol declared in include/dsc.h
EXPORTS = ("dsc_version", "dsc_status_string", "dsc_last_error", "dsc_headwise_fwd",
           "dsc_headwise_bwd", "dsc_lowrank_fwd", "dsc_lowrank_bwd_workspace_bytes",
           "dsc_lowrank_bwd", "dsc_headwise_decode", "dsc_lowrank_decode",
           "dsc_decode_state", "dsc_static_fwd", "dsc_static_bwd_workspace_bytes",
           "dsc_static_bwd", "dsc_headwise_fwd_varlen", "dsc_headwise_bwd_varlen",
           "dsc_lowrank_fwd_varlen", "dsc_lowrank_bwd_varlen", "dsc_headwise_gen_fwd",
           "dsc_lowrank_bwd_noalloc", "dsc_scan_fwd_workspace_bytes", "dsc_scan_fwd",
           "dsc_scan_bwd_workspace_bytes", "dsc_scan_bwd", "dsc_scan_decode",
           "dsc_layernorm_fwd", "dsc_layernorm_bwd_workspace_bytes", "dsc_layernorm_bwd")

# bytes of the library-owned buffer behind dsc_lowrank_bwd_noalloc (include/dsc.h)
NOALLOC_SCRATCH_BYTES = 128 << 20


class ScanShape(ctypes.Structure):
    """dsc_scan_shape of include/dsc.h."""
    _fields_ = [("B", ctypes.c_int64), ("T", ctypes.c_int64), ("D", ctypes.c_int64),
                ("x_row", ctypes.c_int64), ("delta_row", ctypes.c_int64),
                ("z_row", ctypes.c_int64), ("b_row", ctypes.c_int64), ("c_row", ctypes.c_int64),
                ("N", ctypes.c_int), ("G", ctypes.c_int), ("W", ctypes.c_int),
                ("dtype", ctypes.c_int), ("flags", ctypes.c_uint)]


class DscError(RuntimeError):
    def __init__(self, status, msg):
        super().__init__(f"{_status_name(status)}: {msg}")
        self.status = status


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is missing: build it with dynamic_short_causal_amd/build.py "
            "(or __graft_entry__.build()); there is no fallback path")
    lib = ctypes.CDLL(LIB_PATH)
    vp, i64, ci, cu = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_uint
    lib.dsc_version.restype = ci
    lib.dsc_status_string.restype = ctypes.c_char_p
    lib.dsc_status_string.argtypes = [ci]
    lib.dsc_last_error.restype = ctypes.c_char_p
    lib.dsc_headwise_fwd.argtypes = [vp, vp, vp, i64, i64, i64, ci, ci, ci, cu, vp]
    lib.dsc_headwise_bwd.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, ci, ci, ci, cu, vp]
    lib.dsc_lowrank_fwd.argtypes = [vp, vp, vp, vp, i64, i64, i64, ci, ci, ci, ci, cu, vp]
    lib.dsc_lowrank_bwd_workspace_bytes.argtypes = [i64, i64, i64, ci, ci, ci, ci]
    lib.dsc_lowrank_bwd_workspace_bytes.restype = ctypes.c_size_t
    lib.dsc_lowrank_bwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, ctypes.c_size_t, i64, i64,
                                    i64, ci, ci, ci, ci, cu, vp]
    lib.dsc_lowrank_bwd_noalloc.argtypes = [vp, vp, vp, vp, vp, vp, vp, i64, i64, i64, ci, ci,
                                            ci, ci, cu, vp]
    lib.dsc_headwise_decode.argtypes = [vp, vp, vp, vp, i64, i64, ci, ci, ci, cu, vp]
    lib.dsc_lowrank_decode.argtypes = [vp, vp, vp, vp, vp, i64, i64, ci, ci, ci, ci, cu, vp]
    lib.dsc_decode_state.argtypes = [vp, vp, i64, i64, i64, ci, ci, vp]
    lib.dsc_static_fwd.argtypes = [vp, vp, vp, i64, i64, i64, ci, ci, ci, cu, vp]
    lib.dsc_static_bwd_workspace_bytes.argtypes = [i64, i64, i64, ci, ci, ci]
    lib.dsc_static_bwd_workspace_bytes.restype = ctypes.c_size_t
    lib.dsc_static_bwd.argtypes = [vp, vp, vp, vp, vp, vp, ctypes.c_size_t, i64, i64, i64, ci,
                                   ci, ci, cu, vp]
    lib.dsc_headwise_gen_fwd.argtypes = [vp, vp, vp, vp, i64, i64, i64, i64, ci, ci, ci, cu, vp]
    lib.dsc_headwise_fwd_varlen.argtypes = [vp, vp, vp, vp, i64, i64, i64, ci, ci, ci, cu, vp]
    lib.dsc_headwise_bwd_varlen.argtypes = [vp, vp, vp, vp, vp, vp, i64, i64, i64, ci, ci, ci,
                                            cu, vp]
    lib.dsc_lowrank_fwd_varlen.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, ci, ci, ci, ci,
                                           cu, vp]
    lib.dsc_lowrank_bwd_varlen.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, ctypes.c_size_t,
                                           i64, i64, i64, ci, ci, ci, ci, cu, vp]
    lib.dsc_scan_fwd_workspace_bytes.argtypes = [vp]
    lib.dsc_scan_fwd_workspace_bytes.restype = ctypes.c_size_t
    lib.dsc_scan_fwd.argtypes = [vp] * 17 + [vp, ctypes.c_size_t, vp]
    lib.dsc_scan_bwd_workspace_bytes.argtypes = [vp]
    lib.dsc_scan_bwd_workspace_bytes.restype = ctypes.c_size_t
    lib.dsc_scan_bwd.argtypes = [vp] * 24 + [ctypes.c_size_t, vp]
    lib.dsc_scan_decode.argtypes = [vp] * 15
    lib.dsc_layernorm_fwd.argtypes = [vp] * 6 + [i64, i64, ctypes.c_float, ci, vp]
    lib.dsc_layernorm_bwd_workspace_bytes.argtypes = [i64, i64, ci]
    lib.dsc_layernorm_bwd_workspace_bytes.restype = ctypes.c_size_t
    lib.dsc_layernorm_bwd.argtypes = [vp] * 9 + [ctypes.c_size_t, i64, i64, ci, vp]
    for name in ("dsc_headwise_fwd", "dsc_headwise_bwd", "dsc_lowrank_fwd",
                 "dsc_scan_fwd", "dsc_scan_bwd", "dsc_scan_decode", "dsc_layernorm_fwd",
                 "dsc_layernorm_bwd",
                 "dsc_lowrank_bwd", "dsc_headwise_decode", "dsc_lowrank_decode",
                 "dsc_decode_state", "dsc_static_fwd", "dsc_static_bwd",
                 "dsc_headwise_fwd_varlen", "dsc_headwise_bwd_varlen",
                 "dsc_lowrank_fwd_varlen", "dsc_lowrank_bwd_varlen", "dsc_headwise_gen_fwd",
                 "dsc_lowrank_bwd_noalloc"):
        getattr(lib, name).restype = ci
    return lib


LIB = _load()


def _status_name(s):
    return LIB.dsc_status_string(int(s)).decode()


def version():
    return int(LIB.dsc_version())


def _check(status):
    if status != DSC_OK:
        raise DscError(status, LIB.dsc_last_error().decode())


def _dtype(t):
    if t.dtype == torch.bfloat16:
        return DSC_BF16
    if t.dtype == torch.float32:
        return DSC_F32
    raise TypeError(f"unsupported dtype {t.dtype}")


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(stream):
    if stream is None:  # torch.cuda.current_stream() builds a Stream object first: 3 us
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    return stream.cuda_stream


def _flags(residual, act):
    return (DSC_RESIDUAL if residual else 0) | (DSC_ACT_SILU if act else 0)


def _need(t, name, shape, dtype):
    if t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")


# --------------------------------------------------------------- C-named calls
def dsc_headwise_fwd(x, w, y, H, residual=False, act=False, stream=None):
    B, T, D = x.shape
    W = w.shape[-1]
    for n, t, s in (("x", x, (B, T, D)), ("w", w, (B, T, D // H, W)), ("y", y, (B, T, D))):
        _need(t, n, s, x.dtype)
    _check(LIB.dsc_headwise_fwd(_ptr(x), _ptr(w), _ptr(y), B, T, D, W, H, _dtype(x),
                                _flags(residual, act), _stream(stream)))
    return y


def dsc_headwise_bwd(x, w, dy, dx, dw, H, residual=False, act=False, stream=None):
    B, T, D = x.shape
    W = w.shape[-1]
    for n, t, s in (("x", x, (B, T, D)), ("w", w, (B, T, D // H, W)), ("dy", dy, (B, T, D)),
                    ("dx", dx, (B, T, D)), ("dw", dw, (B, T, D // H, W))):
        _need(t, n, s, x.dtype)
    _check(LIB.dsc_headwise_bwd(_ptr(x), _ptr(w), _ptr(dy), _ptr(dx), _ptr(dw), B, T, D, W, H,
                                _dtype(x), _flags(residual, act), _stream(stream)))
    return dx, dw


def dsc_lowrank_fwd(x, z, U, y, W, H, residual=False, act=False, stream=None):
    B, T, D = x.shape
    R = z.shape[-1]
    for n, t, s in (("x", x, (B, T, D)), ("z", z, (B, T, R)), ("U", U, (R, (D // H) * W)),
                    ("y", y, (B, T, D))):
        _need(t, n, s, x.dtype)
    _check(LIB.dsc_lowrank_fwd(_ptr(x), _ptr(z), _ptr(U), _ptr(y), B, T, D, W, H, R,
                               _dtype(x), _flags(residual, act), _stream(stream)))
    return y


def dsc_lowrank_bwd_workspace_bytes(B, T, D, W, H, R, dtype):
    d = DSC_BF16 if dtype == torch.bfloat16 else DSC_F32
    return int(LIB.dsc_lowrank_bwd_workspace_bytes(B, T, D, W, H, R, d))


def dsc_lowrank_bwd(x, z, U, dy, dx, dz, dU, workspace, W, H, residual=False, act=False,
                    stream=None):
    B, T, D = x.shape
    R = z.shape[-1]
    for n, t, s in (("x", x, (B, T, D)), ("z", z, (B, T, R)), ("U", U, (R, (D // H) * W)),
                    ("dy", dy, (B, T, D)), ("dx", dx, (B, T, D)), ("dz", dz, (B, T, R)),
                    ("dU", dU, (R, (D // H) * W))):
        _need(t, n, s, x.dtype)
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(LIB.dsc_lowrank_bwd(_ptr(x), _ptr(z), _ptr(U), _ptr(dy), _ptr(dx), _ptr(dz),
                               _ptr(dU), _ptr(workspace), nbytes, B, T, D, W, H, R,
                               _dtype(x), _flags(residual, act), _stream(stream)))
    return dx, dz, dU


def dsc_lowrank_bwd_noalloc(x, z, U, dy, dx, dz, dU, W, H, residual=False, act=False,
                            stream=None):
    """dsc_lowrank_bwd with the library's own partial-sum buffer (no workspace)."""
    B, T, D = x.shape
    R = z.shape[-1]
    for n, t, s in (("x", x, (B, T, D)), ("z", z, (B, T, R)), ("U", U, (R, (D // H) * W)),
                    ("dy", dy, (B, T, D)), ("dx", dx, (B, T, D)), ("dz", dz, (B, T, R)),
                    ("dU", dU, (R, (D // H) * W))):
        _need(t, n, s, x.dtype)
    _check(LIB.dsc_lowrank_bwd_noalloc(_ptr(x), _ptr(z), _ptr(U), _ptr(dy), _ptr(dx), _ptr(dz),
                                       _ptr(dU), B, T, D, W, H, R, _dtype(x),
                                       _flags(residual, act), _stream(stream)))
    return dx, dz, dU


def dsc_headwise_decode(x, w, state, y, H, residual=False, act=False, stream=None):
    """One token: x (B, D), w (B, G, W); state (B, W-1, D) is advanced in place."""
    B, D = x.shape
    W = w.shape[-1]
    for n, t, s in (("x", x, (B, D)), ("w", w, (B, D // H, W)), ("state", state, (B, W - 1, D)),
                    ("y", y, (B, D))):
        _need(t, n, s, x.dtype)
    _check(LIB.dsc_headwise_decode(_ptr(x), _ptr(w), _ptr(state), _ptr(y), B, D, W, H,
                                   _dtype(x), _flags(residual, act), _stream(stream)))
    return y


def dsc_lowrank_decode(x, z, U, state, y, W, H, residual=False, act=False, stream=None):
    """One token: x (B, D), z (B, R), U (R, G*W); state (B, W-1, D) advanced in place."""
    B, D = x.shape
    R = z.shape[-1]
    for n, t, s in (("x", x, (B, D)), ("z", z, (B, R)), ("U", U, (R, (D // H) * W)),
                    ("state", state, (B, W - 1, D)), ("y", y, (B, D))):
        _need(t, n, s, x.dtype)
    _check(LIB.dsc_lowrank_decode(_ptr(x), _ptr(z), _ptr(U), _ptr(state), _ptr(y), B, D, W, H,
                                  R, _dtype(x), _flags(residual, act), _stream(stream)))
    return y


def dsc_decode_state(x, state, stream=None):
    """The (B, W-1, D) state left by a prompt x (B, T, D)."""
    B, T, D = x.shape
    W = state.shape[1] + 1
    for n, t, s in (("x", x, (B, T, D)), ("state", state, (B, W - 1, D))):
        _need(t, n, s, x.dtype)
    _check(LIB.dsc_decode_state(_ptr(x), _ptr(state), B, T, D, W, _dtype(x), _stream(stream)))
    return state


def dsc_static_fwd(x, w, y, H, residual=False, act=False, stream=None):
    """Static filter w (G, W) for every sequence and token."""
    B, T, D = x.shape
    W = w.shape[-1]
    for n, t, s in (("x", x, (B, T, D)), ("w", w, (D // H, W)), ("y", y, (B, T, D))):
        _need(t, n, s, x.dtype)
    _check(LIB.dsc_static_fwd(_ptr(x), _ptr(w), _ptr(y), B, T, D, W, H, _dtype(x),
                              _flags(residual, act), _stream(stream)))
    return y


def dsc_static_bwd_workspace_bytes(B, T, D, W, H, dtype):
    d = DSC_BF16 if dtype == torch.bfloat16 else DSC_F32
    return int(LIB.dsc_static_bwd_workspace_bytes(B, T, D, W, H, d))


def dsc_static_bwd(x, w, dy, dx, dw, workspace, H, residual=False, act=False, stream=None):
    B, T, D = x.shape
    W = w.shape[-1]
    for n, t, s in (("x", x, (B, T, D)), ("w", w, (D // H, W)), ("dy", dy, (B, T, D)),
                    ("dx", dx, (B, T, D)), ("dw", dw, (D // H, W))):
        _need(t, n, s, x.dtype)
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(LIB.dsc_static_bwd(_ptr(x), _ptr(w), _ptr(dy), _ptr(dx), _ptr(dw), _ptr(workspace),
                              nbytes, B, T, D, W, H, _dtype(x), _flags(residual, act),
                              _stream(stream)))
    return dx, dw


def _need_pos(pos, B, T):
    if pos.dtype != torch.int32:
        raise TypeError(f"pos has dtype {pos.dtype}, expected torch.int32")
    if tuple(pos.shape) != (B, T):
        raise ValueError(f"pos has shape {tuple(pos.shape)}, expected {(B, T)}")
    if not pos.is_contiguous() or not pos.is_cuda:
        raise ValueError("pos must be a contiguous device tensor")


def dsc_headwise_fwd_varlen(x, w, pos, y, H, residual=False, act=False, stream=None):
    """Packed rows: pos (B, T) int32 holds each token's index in its document."""
    B, T, D = x.shape
    W = w.shape[-1]
    for n, t, s in (("x", x, (B, T, D)), ("w", w, (B, T, D // H, W)), ("y", y, (B, T, D))):
        _need(t, n, s, x.dtype)
    _need_pos(pos, B, T)
    _check(LIB.dsc_headwise_fwd_varlen(_ptr(x), _ptr(w), _ptr(pos), _ptr(y), B, T, D, W, H,
                                       _dtype(x), _flags(residual, act), _stream(stream)))
    return y


def dsc_headwise_bwd_varlen(x, w, pos, dy, dx, dw, H, residual=False, act=False, stream=None):
    B, T, D = x.shape
    W = w.shape[-1]
    for n, t, s in (("x", x, (B, T, D)), ("w", w, (B, T, D // H, W)), ("dy", dy, (B, T, D)),
                    ("dx", dx, (B, T, D)), ("dw", dw, (B, T, D // H, W))):
        _need(t, n, s, x.dtype)
    _need_pos(pos, B, T)
    _check(LIB.dsc_headwise_bwd_varlen(_ptr(x), _ptr(w), _ptr(pos), _ptr(dy), _ptr(dx),
                                       _ptr(dw), B, T, D, W, H, _dtype(x), _flags(residual, act),
                                       _stream(stream)))
    return dx, dw


def dsc_lowrank_fwd_varlen(x, z, U, pos, y, W, H, residual=False, act=False, stream=None):
    B, T, D = x.shape
    R = z.shape[-1]
    for n, t, s in (("x", x, (B, T, D)), ("z", z, (B, T, R)), ("U", U, (R, (D // H) * W)),
                    ("y", y, (B, T, D))):
        _need(t, n, s, x.dtype)
    _need_pos(pos, B, T)
    _check(LIB.dsc_lowrank_fwd_varlen(_ptr(x), _ptr(z), _ptr(U), _ptr(pos), _ptr(y), B, T, D,
                                      W, H, R, _dtype(x), _flags(residual, act),
                                      _stream(stream)))
    return y


def dsc_lowrank_bwd_varlen(x, z, U, pos, dy, dx, dz, dU, workspace, W, H, residual=False,
                           act=False, stream=None):
    B, T, D = x.shape
    R = z.shape[-1]
    for n, t, s in (("x", x, (B, T, D)), ("z", z, (B, T, R)), ("U", U, (R, (D // H) * W)),
                    ("dy", dy, (B, T, D)), ("dx", dx, (B, T, D)), ("dz", dz, (B, T, R)),
                    ("dU", dU, (R, (D // H) * W))):
        _need(t, n, s, x.dtype)
    _need_pos(pos, B, T)
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(LIB.dsc_lowrank_bwd_varlen(_ptr(x), _ptr(z), _ptr(U), _ptr(pos), _ptr(dy), _ptr(dx),
                                      _ptr(dz), _ptr(dU), _ptr(workspace), nbytes, B, T, D, W,
                                      H, R, _dtype(x), _flags(residual, act), _stream(stream)))
    return dx, dz, dU


def dsc_headwise_gen_fwd(x, xh, Mt, y, W, H, residual=False, act=False, stream=None):
    """Filters generated on chip: w = xh M with xh (B, T, Dh) and M given
    transposed, Mt (G*W, Dh) (a linear layer's weight layout)."""
    B, T, D = x.shape
    Dh = xh.shape[-1]
    for n, t, s in (("x", x, (B, T, D)), ("xh", xh, (B, T, Dh)), ("Mt", Mt, ((D // H) * W, Dh)),
                    ("y", y, (B, T, D))):
        _need(t, n, s, x.dtype)
    _check(LIB.dsc_headwise_gen_fwd(_ptr(x), _ptr(xh), _ptr(Mt), _ptr(y), B, T, D, Dh, W, H,
                                    _dtype(x), _flags(residual, act), _stream(stream)))
    return y


# --------------------------------------------------------------- selective scan
def _rows(t, name, shape, dtype, lead):
    """Elements from one token of t to the next, for a tensor whose axes after the
    first `lead` are dense and whose sequences follow each other (a dense one,
    or a slice of wider rows)."""
    if t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    width = math.prod(shape[lead:])
    if t.is_contiguous():
        return width
    strides, n = t.stride(), width
    for size, st in zip(shape[lead:], strides[lead:]):
        n //= size
        if size > 1 and st != n:
            raise ValueError(f"{name} must be dense within a token")
    B, T = shape[0], shape[1] if lead == 2 else 1
    row = strides[1] if T > 1 else strides[0] if B > 1 else width
    if B > 1 and T > 1 and strides[0] != T * row:
        raise ValueError(f"the sequences of {name} must follow each other")
    if row < width:  # an expanded tensor
        raise ValueError(f"the tokens of {name} overlap")
    return row


def _opt(t, name, shape, dtype):
    if t is not None:
        _need(t, name, shape, dtype)


def _scan_shape(x, delta, A, Bm, Cm, w, cb, Dk, z, dt_bias, residual, act):
    """The ScanShape of a call with (B, T, ...) inputs, or (B, ...) ones of one
    token, after their checks."""
    lead, shape, dtype = x.dim() - 1, x.shape, x.dtype
    D, N, G = shape[-1], A.shape[-1], Bm.shape[-2]
    W = 0 if w is None else w.shape[-1]
    bc = (*shape[:-1], G, N)
    s = ScanShape(shape[0], shape[1] if lead == 2 else 1, D,
                  _rows(x, "x", shape, dtype, lead), _rows(delta, "delta", shape, dtype, lead),
                  0 if z is None else _rows(z, "z", shape, dtype, lead),
                  _rows(Bm, "Bm", bc, dtype, lead), _rows(Cm, "Cm", bc, dtype, lead),
                  N, G, W, _dtype(x), _flags(residual, act))
    _need(A, "A", (D, N), torch.float32)
    _opt(w, "w", (D, W), dtype)
    _opt(cb, "cb", (D,), dtype)
    _opt(Dk, "Dk", (D,), torch.float32)
    _opt(dt_bias, "dt_bias", (D,), torch.float32)
    return s


def _shape_ptr(s):
    return ctypes.addressof(s)


def _bytes_of(t):
    return 0 if t is None else t.numel() * t.element_size()


def dsc_scan_fwd(x, delta, A, Bm, Cm, y, w=None, cb=None, Dk=None, z=None, dt_bias=None,
                 h0=None, conv0=None, pos=None, hT=None, convT=None, workspace=None,
                 residual=False, act=False, stream=None):
    """Selective scan behind its short convolution: x, delta, z, y (B, T, D),
    Bm, Cm (B, T, G, N), w (D, W), cb (D) of one dtype; A (D, N), Dk, dt_bias (D)
    and the states h0, hT (B, D, N) in fp32; conv0, convT (B, W-1, D)."""
    B, T, D = x.shape
    s = _scan_shape(x, delta, A, Bm, Cm, w, cb, Dk, z, dt_bias, residual, act)
    _need(y, "y", (B, T, D), x.dtype)
    for n, t in (("h0", h0), ("hT", hT)):
        _opt(t, n, (B, D, s.N), torch.float32)
    for n, t in (("conv0", conv0), ("convT", convT)):
        _opt(t, n, (B, max(s.W - 1, 0), D), x.dtype)
    if pos is not None:
        _need_pos(pos, B, T)
    _check(LIB.dsc_scan_fwd(_shape_ptr(s), _ptr(x), _ptr(delta), _ptr(A), _ptr(Bm), _ptr(Cm),
                            _ptr(w), _ptr(cb), _ptr(Dk), _ptr(z), _ptr(dt_bias), _ptr(h0),
                            _ptr(conv0), _ptr(pos), _ptr(y), _ptr(hT), _ptr(convT),
                            _ptr(workspace), _bytes_of(workspace), _stream(stream)))
    return y


def dsc_scan_bwd(x, delta, A, Bm, Cm, dy, grads, workspace, w=None, cb=None, Dk=None, z=None,
                 dt_bias=None, pos=None, residual=False, act=False, stream=None):
    """Gradients of dsc_scan_fwd from a zero state, written to the tensors of
    `grads`: dx, ddelta, dA, dBm, dCm, and dw, dcb, dDk, dz, ddt_bias where
    their inputs are given; all dense, in the inputs' dtypes."""
    B, T, D = x.shape
    s = _scan_shape(x, delta, A, Bm, Cm, w, cb, Dk, z, dt_bias, residual, act)
    _need(dy, "dy", (B, T, D), x.dtype)
    if pos is not None:
        _need_pos(pos, B, T)
    inputs = dict(dx=x, ddelta=delta, dA=A, dBm=Bm, dCm=Cm, dw=w, dcb=cb, dDk=Dk, dz=z,
                  ddt_bias=dt_bias)
    outs = []
    for n, t in inputs.items():
        if t is not None:
            _need(grads[n], n, t.shape, t.dtype)
        outs.append(_ptr(None if t is None else grads[n]))
    _check(LIB.dsc_scan_bwd(_shape_ptr(s), _ptr(x), _ptr(delta), _ptr(A), _ptr(Bm), _ptr(Cm),
                            _ptr(w), _ptr(cb), _ptr(Dk), _ptr(z), _ptr(dt_bias), _ptr(pos),
                            _ptr(dy), *outs, _ptr(workspace), _bytes_of(workspace),
                            _stream(stream)))
    return grads


def dsc_scan_decode(x, delta, A, Bm, Cm, h, conv, y, w=None, cb=None, Dk=None, z=None,
                    dt_bias=None, residual=False, act=False, stream=None):
    """One token: x, delta, z, y (B, D), Bm, Cm (B, G, N); the states h (B, D, N)
    in fp32 and conv (B, W-1, D) are advanced in place."""
    B, D = x.shape
    s = _scan_shape(x, delta, A, Bm, Cm, w, cb, Dk, z, dt_bias, residual, act)
    _need(y, "y", (B, D), x.dtype)
    _need(h, "h", (B, D, s.N), torch.float32)
    if s.W > 1:
        if conv is None:
            raise ValueError("conv is needed for W > 1")
        _need(conv, "conv", (B, s.W - 1, D), x.dtype)
    _check(LIB.dsc_scan_decode(_shape_ptr(s), _ptr(x), _ptr(delta), _ptr(A), _ptr(Bm), _ptr(Cm),
                               _ptr(w), _ptr(cb), _ptr(Dk), _ptr(z), _ptr(dt_bias), _ptr(h),
                               _ptr(conv if s.W > 1 else None), _ptr(y), _stream(stream)))
    return y


# --------------------------------------------------------------- layer norm
def _norm_params(x, w, b):
    for n, t in (("w", w), ("b", b)):
        _opt(t, n, (x.shape[-1],), x.dtype)


def dsc_layernorm_fwd(x, w, b, y, mean, rstd, eps=1e-5, stream=None):
    """Layer norm of the rows of x (M, D); mean and rstd (M) in fp32."""
    M, D = x.shape
    _need(x, "x", (M, D), x.dtype)
    _norm_params(x, w, b)
    _need(y, "y", (M, D), x.dtype)
    _need(mean, "mean", (M,), torch.float32)
    _need(rstd, "rstd", (M,), torch.float32)
    _check(LIB.dsc_layernorm_fwd(_ptr(x), _ptr(w), _ptr(b), _ptr(y), _ptr(mean), _ptr(rstd), M,
                                 D, eps, _dtype(x), _stream(stream)))
    return y, mean, rstd


def dsc_layernorm_bwd_workspace_bytes(M, D, dtype):
    d = DSC_BF16 if dtype == torch.bfloat16 else DSC_F32
    return int(LIB.dsc_layernorm_bwd_workspace_bytes(M, D, d))


def dsc_layernorm_bwd(x, w, dy, mean, rstd, dx, dw, db, workspace, stream=None):
    M, D = x.shape
    for n, t in (("x", x), ("dy", dy), ("dx", dx)):
        _need(t, n, (M, D), x.dtype)
    for n, t in (("w", w), ("dw", dw), ("db", db)):
        _opt(t, n, (D,), x.dtype)
    for n, t in (("mean", mean), ("rstd", rstd)):
        _need(t, n, (M,), torch.float32)
    _check(LIB.dsc_layernorm_bwd(_ptr(x), _ptr(w), _ptr(dy), _ptr(mean), _ptr(rstd), _ptr(dx),
                                 _ptr(dw), _ptr(db), _ptr(workspace), _bytes_of(workspace), M, D,
                                 _dtype(x), _stream(stream)))
    return dx, dw, db


# --------------------------------------------------------------- allocating forms
def _on_stream(call):
    """An allocating form whose tensors belong to the stream that it is queued on.

    Memory from the current stream's pool would go back to it as soon as a
    workspace (or an output that the caller drops) is released, and to that
    stream's next tensor while the kernels on the other stream still use it.
    Outputs are recorded on the current stream too, where the caller reads them."""
    at = list(inspect.signature(call).parameters).index("stream")

    @functools.wraps(call)
    def run(*args, **kwargs):
        stream = args[at] if len(args) > at else kwargs.get("stream")
        if stream is None or stream.cuda_stream == _stream(None):
            return call(*args, **kwargs)
        current = torch.cuda.current_stream()
        with torch.cuda.stream(stream):
            out = call(*args, **kwargs)
        outs = out.values() if isinstance(out, dict) else out if isinstance(out, tuple) else (out,)
        for t in outs:
            t.record_stream(current)
        return out
    return run


@_on_stream
def headwise_fwd(x, w, H, residual=False, act=False, stream=None):
    return dsc_headwise_fwd(x, w, torch.empty_like(x), H, residual, act, stream)


@_on_stream
def headwise_bwd(x, w, dy, H, residual=False, act=False, stream=None):
    return dsc_headwise_bwd(x, w, dy, torch.empty_like(x), torch.empty_like(w), H, residual,
                            act, stream)


@_on_stream
def lowrank_fwd(x, z, U, W, H, residual=False, act=False, stream=None):
    return dsc_lowrank_fwd(x, z, U, torch.empty_like(x), W, H, residual, act, stream)


def lowrank_workspace(x, z, W, H):
    B, T, D = x.shape
    n = dsc_lowrank_bwd_workspace_bytes(B, T, D, W, H, z.shape[-1], x.dtype)
    return torch.empty(max(n, 1), dtype=torch.uint8, device=x.device)


@_on_stream
def lowrank_bwd(x, z, U, dy, W, H, residual=False, act=False, workspace=None, stream=None):
    if workspace is None:
        workspace = lowrank_workspace(x, z, W, H)
    return dsc_lowrank_bwd(x, z, U, dy, torch.empty_like(x), torch.empty_like(z),
                           torch.empty_like(U), workspace, W, H, residual, act, stream)


@_on_stream
def decode_state(x, W, stream=None):
    B, T, D = x.shape
    return dsc_decode_state(x, torch.empty(B, W - 1, D, dtype=x.dtype, device=x.device), stream)


@_on_stream
def headwise_decode(x, w, state, H, residual=False, act=False, stream=None):
    return dsc_headwise_decode(x, w, state, torch.empty_like(x), H, residual, act, stream)


@_on_stream
def lowrank_decode(x, z, U, state, W, H, residual=False, act=False, stream=None):
    return dsc_lowrank_decode(x, z, U, state, torch.empty_like(x), W, H, residual, act, stream)


@_on_stream
def static_fwd(x, w, H, residual=False, act=False, stream=None):
    return dsc_static_fwd(x, w, torch.empty_like(x), H, residual, act, stream)


def static_workspace(x, W, H):
    B, T, D = x.shape
    n = dsc_static_bwd_workspace_bytes(B, T, D, W, H, x.dtype)
    return torch.empty(max(n, 1), dtype=torch.uint8, device=x.device)


@_on_stream
def static_bwd(x, w, dy, H, residual=False, act=False, workspace=None, stream=None):
    if workspace is None:
        workspace = static_workspace(x, w.shape[-1], H)
    return dsc_static_bwd(x, w, dy, torch.empty_like(x), torch.empty_like(w), workspace, H,
                          residual, act, stream)


@_on_stream
def headwise_fwd_varlen(x, w, pos, H, residual=False, act=False, stream=None):
    return dsc_headwise_fwd_varlen(x, w, pos, torch.empty_like(x), H, residual, act, stream)


@_on_stream
def headwise_bwd_varlen(x, w, pos, dy, H, residual=False, act=False, stream=None):
    return dsc_headwise_bwd_varlen(x, w, pos, dy, torch.empty_like(x), torch.empty_like(w), H,
                                   residual, act, stream)


@_on_stream
def lowrank_fwd_varlen(x, z, U, pos, W, H, residual=False, act=False, stream=None):
    return dsc_lowrank_fwd_varlen(x, z, U, pos, torch.empty_like(x), W, H, residual, act, stream)


@_on_stream
def lowrank_bwd_varlen(x, z, U, pos, dy, W, H, residual=False, act=False, workspace=None,
                       stream=None):
    if workspace is None:
        workspace = lowrank_workspace(x, z, W, H)
    return dsc_lowrank_bwd_varlen(x, z, U, pos, dy, torch.empty_like(x), torch.empty_like(z),
                                  torch.empty_like(U), workspace, W, H, residual, act, stream)


@_on_stream
def headwise_gen_fwd(x, xh, Mt, W, H, residual=False, act=False, stream=None):
    return dsc_headwise_gen_fwd(x, xh, Mt, torch.empty_like(x), W, H, residual, act, stream)


def scan_workspace(x, N, G):
    """Workspace of scan_fwd, or None where it needs none."""
    B, T, D = x.shape
    s = ScanShape(B=B, T=T, D=D, N=N, G=G, dtype=_dtype(x))
    n = int(LIB.dsc_scan_fwd_workspace_bytes(_shape_ptr(s)))
    return x.new_empty(n, dtype=torch.uint8) if n else None


@_on_stream
def scan_fwd(x, delta, A, Bm, Cm, w=None, cb=None, Dk=None, z=None, dt_bias=None, h0=None,
             conv0=None, pos=None, residual=False, act=False, final_state=False, workspace=None,
             stream=None):
    """y, or (y, hT, convT) with final_state: what scan_decode, or the next part
    of a prompt (as h0 and conv0), goes on from.  With pos, convT holds the row's
    last inputs whatever their document: before a scan_decode, clear those from
    before a last document of fewer than W - 1 tokens."""
    B, T, D = x.shape
    N, W = A.shape[-1], 0 if w is None else w.shape[-1]
    if workspace is None:
        workspace = scan_workspace(x, N, Bm.shape[-2])
    y = x.new_empty(B, T, D)
    hT = convT = None
    if final_state:
        if T == 0:
            raise ValueError("an empty call leaves no final state")
        hT = A.new_empty(B, D, N)
        convT = x.new_empty(B, max(W - 1, 0), D)
    dsc_scan_fwd(x, delta, A, Bm, Cm, y, w, cb, Dk, z, dt_bias, h0, conv0, pos, hT, convT,
                 workspace, residual, act, stream)
    return (y, hT, convT) if final_state else y


def scan_bwd_workspace(x, N, G, W=None):
    """Workspace of scan_bwd with W taps, or (None) with any number of them."""
    B, T, D = x.shape
    n = 0
    for taps in (0, 8) if W is None else (W,):
        s = ScanShape(B=B, T=T, D=D, N=N, G=G, W=taps, dtype=_dtype(x))
        n = max(n, int(LIB.dsc_scan_bwd_workspace_bytes(_shape_ptr(s))))
    return x.new_empty(n, dtype=torch.uint8) if n else None


@_on_stream
def scan_bwd(x, delta, A, Bm, Cm, dy, w=None, cb=None, Dk=None, z=None, dt_bias=None, pos=None,
             residual=False, act=False, workspace=None, stream=None):
    """The gradients of scan_fwd by name: dx, ddelta, dA, dBm, dCm, and dw, dcb,
    dDk, dz, ddt_bias of the inputs given."""
    if workspace is None:
        workspace = scan_bwd_workspace(x, A.shape[-1], Bm.shape[-2],
                                       0 if w is None else w.shape[-1])
    inputs = dict(dx=x, ddelta=delta, dA=A, dBm=Bm, dCm=Cm, dw=w, dcb=cb, dDk=Dk, dz=z,
                  ddt_bias=dt_bias)
    grads = {n: t.new_empty(t.shape)
             for n, t in inputs.items() if t is not None}
    return dsc_scan_bwd(x, delta, A, Bm, Cm, dy, grads, workspace, w, cb, Dk, z, dt_bias, pos,
                        residual, act, stream)


@_on_stream
def scan_decode(x, delta, A, Bm, Cm, h, conv=None, w=None, cb=None, Dk=None, z=None,
                dt_bias=None, residual=False, act=False, stream=None):
    y = x.new_empty(x.shape)
    return dsc_scan_decode(x, delta, A, Bm, Cm, h, conv, y, w, cb, Dk, z, dt_bias, residual, act,
                           stream)


@_on_stream
def layernorm_fwd(x, w=None, b=None, eps=1e-5, stream=None):
    """y, mean, rstd of the rows of x (M, D)."""
    mean = x.new_empty(x.shape[0], dtype=torch.float32)
    return dsc_layernorm_fwd(x, w, b, torch.empty_like(x), mean, torch.empty_like(mean), eps,
                             stream)


def layernorm_workspace(x):
    n = dsc_layernorm_bwd_workspace_bytes(x.shape[0], x.shape[1], x.dtype)
    return x.new_empty(max(n, 1), dtype=torch.uint8)


@_on_stream
def layernorm_bwd(x, w, dy, mean, rstd, workspace=None, stream=None):
    """dx, dw, db (the latter two also where w is None: the gradients at w = 1, b = 0)."""
    if workspace is None:
        workspace = layernorm_workspace(x)
    dw = x.new_empty(x.shape[1])
    return dsc_layernorm_bwd(x, w, dy, mean, rstd, torch.empty_like(x), dw, torch.empty_like(dw),
                             workspace, stream)
