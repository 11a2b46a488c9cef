"""MI355X (gfx950) quantized-weight GEMV: Python binding of libqgemv.so.

Argument marshalling only.  Every step of the computation runs in the HIP
kernels of ``libqgemv.so``; there is no CPU or PyTorch fallback: if the
library is missing or a call is refused, an exception is raised.

Two layers:
* ``qgemv_*`` -- the C ABI under the same names, taking raw device pointers
  (ints), sizes and a stream handle, returning the status code;
* ``i4g``, ``fp8b128``, ``mq4v2``, ``fwht256``, ``moe_topk``, ``dequant_*``,
  ``i4g_linear``, ``fp8b128_linear``, ``moe_group``, ``i4g_grouped``,
  ``moe_combine`` -- take torch tensors on the current CUDA (HIP) device, allocate the output
  with ``torch.empty``, launch on ``torch.cuda.current_stream()`` and raise
  ``QgemvError`` on a refusal.  No call records a gradient; the products with
  an epilogue and ``moe_combine`` refuse arguments that ask for one.
"""
from __future__ import annotations

import contextlib
import ctypes as C
import operator
import os

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libqgemv.so")

QGEMV_MAX_S = 8

# qgemv_act
ACTIVATIONS = {None: 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4}


class Epilogue(C.Structure):
    """qgemv_epilogue (host struct of device pointers)."""
    _fields_ = [("act", C.c_int), ("gated", C.c_int), ("bias", C.c_void_p),
                ("residual", C.c_void_p), ("ld_residual", C.c_longlong)]


# every entry point declared in include/qgemv.h
_SIGS = {
    "qgemv_strerror": (C.c_char_p, [C.c_int]),
    "qgemv_version": (C.c_char_p, []),
    "qgemv_i4g": (C.c_int, [C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p,
                            C.c_int, C.c_int, C.c_int, C.c_int, C.c_void_p]),
    "qgemv_i4g_prefill": (C.c_int, [C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p,
                                    C.c_int, C.c_int, C.c_int, C.c_int, C.c_void_p]),
    "qgemv_fp8b128": (C.c_int, [C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p,
                                C.c_int, C.c_int, C.c_int, C.c_void_p]),
    "qgemv_fp8b128_ue8m0": (C.c_int, [C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p,
                                      C.c_int, C.c_int, C.c_int, C.c_void_p]),
    "qgemv_mq4v2": (C.c_int, [C.c_void_p, C.c_void_p, C.c_void_p,
                              C.c_int, C.c_int, C.c_int, C.c_void_p]),
    "qgemv_mq4v1": (C.c_int, [C.c_void_p, C.c_void_p, C.c_void_p,
                              C.c_int, C.c_int, C.c_int, C.c_void_p]),
    "qgemv_mq4c": (C.c_int, [C.c_void_p, C.c_void_p, C.c_void_p,
                             C.c_int, C.c_int, C.c_int, C.c_void_p]),
    "qgemv_mq4v2_encode": (C.c_int, [C.c_void_p, C.c_void_p, C.c_int, C.c_int, C.c_void_p]),
    "qgemv_mq4v2_rot": (C.c_int, [C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p,
                                  C.c_int, C.c_int, C.c_int, C.c_void_p]),
    "qgemv_fwht256": (C.c_int, [C.c_void_p, C.c_void_p, C.c_void_p,
                                C.c_int, C.c_int, C.c_void_p]),
    "qgemv_router_topk": (C.c_int, [C.c_void_p, C.c_int, C.c_int, C.c_int, C.c_int,
                                    C.c_void_p, C.c_void_p, C.c_void_p]),
    "qgemv_moe_topk_workspace": (C.c_size_t, [C.c_int, C.c_int, C.c_int]),
    "qgemv_moe_topk": (C.c_int, [C.c_void_p, C.c_void_p, C.c_longlong, C.c_longlong,
                                 C.c_int, C.c_void_p, C.c_void_p, C.c_int, C.c_int,
                                 C.c_void_p, C.c_void_p, C.c_int, C.c_int, C.c_int,
                                 C.c_void_p, C.c_size_t, C.c_void_p]),
    "qgemv_moe_topk_error": (C.c_int, [C.c_void_p, C.POINTER(C.c_int), C.c_void_p]),
    "qgemv_moe_topk_noalloc": (C.c_int, [C.c_void_p, C.c_void_p, C.c_longlong, C.c_longlong,
                                         C.c_int, C.c_void_p, C.c_void_p, C.c_int, C.c_int,
                                         C.c_void_p, C.c_void_p, C.c_int, C.c_int, C.c_int,
                                         C.c_void_p]),
    "qgemv_linear_workspace": (C.c_size_t, [C.c_int, C.c_int, C.c_int, C.c_int]),
    "qgemv_i4g_linear": (C.c_int, [C.c_void_p, C.c_void_p, C.c_void_p, C.c_longlong, C.c_void_p,
                                   C.c_longlong, C.c_int, C.c_int, C.c_int, C.c_int, C.c_int,
                                   C.c_void_p, C.c_void_p, C.c_size_t, C.c_void_p]),
    "qgemv_fp8b128_linear": (C.c_int, [C.c_void_p, C.c_void_p, C.c_void_p, C.c_longlong,
                                       C.c_void_p, C.c_longlong, C.c_int, C.c_int, C.c_int,
                                       C.c_int, C.c_void_p, C.c_void_p, C.c_size_t, C.c_void_p]),
    "qgemv_moe_group_workspace": (C.c_size_t, [C.c_int, C.c_int, C.c_int]),
    "qgemv_moe_group": (C.c_int, [C.c_void_p, C.c_int, C.c_int, C.c_int, C.c_void_p, C.c_void_p,
                                  C.c_void_p, C.c_void_p, C.c_size_t, C.c_void_p]),
    "qgemv_grouped_workspace": (C.c_size_t, [C.c_int, C.c_int, C.c_int, C.c_int, C.c_int,
                                             C.c_int]),
    "qgemv_i4g_grouped": (C.c_int, [C.c_void_p, C.c_void_p, C.c_longlong, C.c_longlong, C.c_int,
                                    C.c_void_p, C.c_void_p, C.c_void_p, C.c_longlong, C.c_int,
                                    C.c_void_p, C.c_longlong, C.c_int, C.c_int, C.c_int, C.c_int,
                                    C.c_int, C.c_void_p, C.c_void_p, C.c_size_t, C.c_void_p]),
    "qgemv_moe_combine": (C.c_int, [C.c_void_p, C.c_longlong, C.c_int, C.c_void_p, C.c_void_p,
                                    C.c_int, C.c_int, C.c_int, C.c_void_p, C.c_longlong,
                                    C.c_void_p, C.c_longlong, C.c_int, C.c_void_p]),
    "qgemv_dequant_i4g": (C.c_int, [C.c_void_p, C.c_void_p, C.c_void_p,
                                    C.c_int, C.c_int, C.c_int, C.c_void_p]),
    "qgemv_dequant_fp8b128": (C.c_int, [C.c_void_p, C.c_void_p, C.c_void_p,
                                        C.c_int, C.c_int, C.c_void_p]),
    "qgemv_dequant_fp8b128_ue8m0": (C.c_int, [C.c_void_p, C.c_void_p, C.c_void_p,
                                              C.c_int, C.c_int, C.c_void_p]),
    "qgemv_dequant_mq4v2": (C.c_int, [C.c_void_p, C.c_void_p,
                                      C.c_int, C.c_int, C.c_void_p]),
    "qgemv_dequant_mq4v1": (C.c_int, [C.c_void_p, C.c_void_p, C.c_int, C.c_int, C.c_void_p]),
    "qgemv_dequant_mq4c": (C.c_int, [C.c_void_p, C.c_void_p, C.c_int, C.c_int, C.c_void_p]),
}

ENTRY_POINTS = tuple(_SIGS)


class QgemvError(RuntimeError):
    def __init__(self, fn, status, msg):
        super().__init__(f"{fn}: status {status}: {msg}")
        self.status = status


_lib = None


def lib(path: str = LIB_PATH):
    """The loaded libqgemv.so (raises if it was never built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(path):
            raise ImportError(f"{path} is not built: run quantized_weight_decode_amd.build.build()")
        L = C.CDLL(path)
        for name, (res, args) in _SIGS.items():
            if not hasattr(L, name):
                continue  # reported by exported_symbols(); calling it raises
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


def exported_symbols(path: str = LIB_PATH):
    """Entry points of include/qgemv.h that the built library exports."""
    L = lib(path)
    return [n for n in ENTRY_POINTS if hasattr(L, n)]


def strerror(status: int) -> str:
    return lib().qgemv_strerror(status).decode()


def version() -> str:
    return lib().qgemv_version().decode()


def _call(name, *args):
    st = getattr(lib(), name)(*args)
    if st != 0:
        raise QgemvError(name, st, strerror(st))
    return st


# -- raw C ABI, same names -------------------------------------------------
def qgemv_i4g(w, scales, x, y, S, I, O, gs, stream):
    return lib().qgemv_i4g(w, scales, x, y, S, I, O, gs, stream)


def qgemv_i4g_prefill(w, scales, x, y, S, I, O, gs, stream):
    return lib().qgemv_i4g_prefill(w, scales, x, y, S, I, O, gs, stream)


def qgemv_fp8b128(w, scale_inv, x, y, S, I, O, stream):
    return lib().qgemv_fp8b128(w, scale_inv, x, y, S, I, O, stream)


def qgemv_fp8b128_ue8m0(w, scale_e8m0, x, y, S, I, O, stream):
    return lib().qgemv_fp8b128_ue8m0(w, scale_e8m0, x, y, S, I, O, stream)


def qgemv_mq4v2(w, x_rot, y, S, I, O, stream):
    return lib().qgemv_mq4v2(w, x_rot, y, S, I, O, stream)


def qgemv_mq4v1(w, x_rot, y, S, I, O, stream):
    return lib().qgemv_mq4v1(w, x_rot, y, S, I, O, stream)


def qgemv_mq4c(w, x_rot, y, S, I, O, stream):
    return lib().qgemv_mq4c(w, x_rot, y, S, I, O, stream)


def qgemv_mq4v2_encode(W, w_out, I, O, stream):
    return lib().qgemv_mq4v2_encode(W, w_out, I, O, stream)


def qgemv_mq4v2_rot(w, x, signs, y, S, I, O, stream):
    return lib().qgemv_mq4v2_rot(w, x, signs, y, S, I, O, stream)


def qgemv_fwht256(x, signs, x_rot, S, I, stream):
    return lib().qgemv_fwht256(x, signs, x_rot, S, I, stream)


def qgemv_router_topk(logits, T, E, ld, K, ids, gates, stream):
    return lib().qgemv_router_topk(logits, T, E, ld, K, ids, gates, stream)


def qgemv_moe_topk_workspace(T, K, O):
    return lib().qgemv_moe_topk_workspace(T, K, O)


def qgemv_moe_topk(w, scales, w_stride, s_stride, E, ids, gates, T, K, x, y, I, O, gs,
                   workspace, ws_bytes, stream):
    return lib().qgemv_moe_topk(w, scales, w_stride, s_stride, E, ids, gates, T, K, x, y,
                                I, O, gs, workspace, ws_bytes, stream)


def qgemv_moe_topk_noalloc(w, scales, w_stride, s_stride, E, ids, gates, T, K, x, y, I, O, gs,
                           stream):
    return lib().qgemv_moe_topk_noalloc(w, scales, w_stride, s_stride, E, ids, gates, T, K, x, y,
                                        I, O, gs, stream)


def qgemv_linear_workspace(S, I, O, dtype):
    return lib().qgemv_linear_workspace(S, I, O, dtype)


def qgemv_i4g_linear(w, scales, x, ldx, y, ldy, S, I, O, gs, dtype, epilogue, workspace, ws_bytes,
                     stream):
    return lib().qgemv_i4g_linear(w, scales, x, ldx, y, ldy, S, I, O, gs, dtype, epilogue,
                                  workspace, ws_bytes, stream)


def qgemv_fp8b128_linear(w, scale_inv, x, ldx, y, ldy, S, I, O, dtype, epilogue, workspace,
                         ws_bytes, stream):
    return lib().qgemv_fp8b128_linear(w, scale_inv, x, ldx, y, ldy, S, I, O, dtype, epilogue,
                                      workspace, ws_bytes, stream)


def qgemv_moe_group_workspace(T, K, E):
    return lib().qgemv_moe_group_workspace(T, K, E)


def qgemv_moe_group(ids, T, K, E, offsets, tokens, pos, workspace, ws_bytes, stream):
    return lib().qgemv_moe_group(ids, T, K, E, offsets, tokens, pos, workspace, ws_bytes, stream)


def qgemv_grouped_workspace(T, R, E, I, O, dtype):
    return lib().qgemv_grouped_workspace(T, R, E, I, O, dtype)


def qgemv_i4g_grouped(w, scales, w_stride, s_stride, E, offsets, rows, x, ldx, T, y, ldy, R, I, O,
                      gs, dtype, epilogue, workspace, ws_bytes, stream):
    return lib().qgemv_i4g_grouped(w, scales, w_stride, s_stride, E, offsets, rows, x, ldx, T, y,
                                   ldy, R, I, O, gs, dtype, epilogue, workspace, ws_bytes, stream)


def qgemv_moe_combine(h, ldh, R, pos, gates, T, K, O, residual, ldr, y, ldy, dtype, stream):
    return lib().qgemv_moe_combine(h, ldh, R, pos, gates, T, K, O, residual, ldr, y, ldy, dtype,
                                   stream)


def qgemv_dequant_i4g(w, scales, W, I, O, gs, stream):
    return lib().qgemv_dequant_i4g(w, scales, W, I, O, gs, stream)


def qgemv_dequant_fp8b128(w, scale_inv, W, I, O, stream):
    return lib().qgemv_dequant_fp8b128(w, scale_inv, W, I, O, stream)


def qgemv_dequant_fp8b128_ue8m0(w, scale_e8m0, W, I, O, stream):
    return lib().qgemv_dequant_fp8b128_ue8m0(w, scale_e8m0, W, I, O, stream)


def qgemv_dequant_mq4v2(w, W, I, O, stream):
    return lib().qgemv_dequant_mq4v2(w, W, I, O, stream)


def qgemv_dequant_mq4v1(w, W, I, O, stream):
    return lib().qgemv_dequant_mq4v1(w, W, I, O, stream)


def qgemv_dequant_mq4c(w, W, I, O, stream):
    return lib().qgemv_dequant_mq4c(w, W, I, O, stream)


# -- torch-tensor layer ----------------------------------------------------
_torch_module = None


def _torch():
    """torch, imported by the first call that needs it."""
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


def _stream():
    return _torch().cuda.current_stream().cuda_stream


def _dev(t, name, dtype=None):
    torch = _torch()
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA (HIP) tensor")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _shape(t, name, shape):
    """t must have exactly this shape (a tuple of ints)."""
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _one_device(*ts):
    devs = [t.device for t in ts if t is not None]
    if devs.count(devs[0]) != len(devs):
        raise ValueError(f"tensors are on different devices: {sorted(set(map(str, devs)))}")


def _out(out, S, O, like):
    """The caller's y (checked: f32 [S][O] on like's device) or a new one."""
    torch = _torch()
    if out is None:
        return torch.empty((S, O), dtype=torch.float32, device=like.device)
    if out.numel() != S * O or out.dim() not in (1, 2) or \
            (out.dim() == 2 and tuple(out.shape) != (S, O)) or (out.dim() == 1 and S != 1):
        raise ValueError(f"out must have shape ({S}, {O})" + (f" or ({O},)" if S == 1 else ""))
    return out


_MAX_DIM = 1 << 24


def _gs(gs):
    gs = operator.index(gs)
    if gs < 2 or gs % 2 or gs > _MAX_DIM:               # (above 2^31 the C call would wrap)
        raise QgemvError("argument check", 3, "group size must be an even number in 2 .. 2^24")
    return gs


def _vecs(x, I, name="x"):
    if x.dim() == 1:
        return 1
    if x.dim() == 2 and x.shape[1] == I:
        return x.shape[0]
    raise ValueError(f"{name} must be [I] or [S, I]")


def _i4g_check(w, scales, x, gs, S, I):
    O = w.shape[0]
    _gs(gs)
    _shape(w, "w", (O, (I + 1) // 2))
    if scales.numel() != O * ((I + gs - 1) // gs):
        raise ValueError(f"scales must hold {O} x {(I + gs - 1) // gs} floats")
    return O


def i4g(w, scales, x, gs, out=None):
    """y[S][O] = grouped-int4 W[O][I] . x[S][I]; w u8 [O][(I+1)//2], scales f32 [O][ng]."""
    torch = _torch()
    I = x.shape[-1]
    S = _vecs(x, I)
    O = _i4g_check(w, scales, x, gs, S, I)
    _one_device(w, scales, x, out)
    y = _out(out, S, O, x)
    _call("qgemv_i4g", _dev(w, "w", torch.uint8), _dev(scales, "scales", torch.float32),
          _dev(x, "x", torch.float32), _dev(y, "y", torch.float32), S, I, O, gs, _stream())
    return y


def i4g_prefill(w, scales, x, gs, out=None):
    """Grouped-int4 product for many tokens (MFMA): x f32 [S][I] -> y f32 [S][O].

    Decodes and multiplies in f32; ``i4g_linear`` is the faster product for many
    tokens."""
    torch = _torch()
    I = x.shape[-1]
    S = x.reshape(-1, I).shape[0]
    O = _i4g_check(w, scales, x, gs, S, I)
    _one_device(w, scales, x, out)
    y = _out(out, S, O, x)
    _call("qgemv_i4g_prefill", _dev(w, "w", torch.uint8), _dev(scales, "scales", torch.float32),
          _dev(x, "x", torch.float32), _dev(y, "y", torch.float32), S, I, O, gs, _stream())
    return y


def _fp8_check(w, sc, I, name):
    O = w.shape[0]
    _shape(w, "w", (O, I))
    if sc.numel() != ((O + 127) // 128) * ((I + 127) // 128):
        raise ValueError(f"{name} must hold {(O + 127) // 128} x {(I + 127) // 128} block scales")
    return O


def fp8b128(w, scale_inv, x, out=None):
    torch = _torch()
    I = x.shape[-1]
    S = _vecs(x, I)
    O = _fp8_check(w, scale_inv, I, "scale_inv")
    _one_device(w, scale_inv, x, out)
    y = _out(out, S, O, x)
    _call("qgemv_fp8b128", _dev(w, "w", torch.uint8), _dev(scale_inv, "scale_inv", torch.float32),
          _dev(x, "x", torch.float32), _dev(y, "y", torch.float32), S, I, O, _stream())
    return y


def fp8b128_ue8m0(w, scale_e8m0, x, out=None):
    """fp8-e4m3 GEMV with UE8M0 (power-of-two byte) block scales."""
    torch = _torch()
    I = x.shape[-1]
    S = _vecs(x, I)
    O = _fp8_check(w, scale_e8m0, I, "scale_e8m0")
    _one_device(w, scale_e8m0, x, out)
    y = _out(out, S, O, x)
    _call("qgemv_fp8b128_ue8m0", _dev(w, "w", torch.uint8),
          _dev(scale_e8m0, "scale_e8m0", torch.uint8), _dev(x, "x", torch.float32),
          _dev(y, "y", torch.float32), S, I, O, _stream())
    return y


def _mq4_check(w, I):
    O = w.shape[0]
    if I % 256 == 0:  # otherwise the library refuses the call by name
        if w.numel() != O * (I // 256) * 136:
            raise ValueError(f"w must hold {O} rows of {I // 256} 136-byte groups")
    return O


def mq4v2(w, x_rot, out=None):
    torch = _torch()
    I = x_rot.shape[-1]
    S = _vecs(x_rot, I, "x_rot")
    O = _mq4_check(w, I)
    _one_device(w, x_rot, out)
    y = _out(out, S, O, x_rot)
    _call("qgemv_mq4v2", _dev(w, "w", torch.uint8), _dev(x_rot, "x_rot", torch.float32),
          _dev(y, "y", torch.float32), S, I, O, _stream())
    return y


def _mq4_any(fn, w, x_rot, out):
    torch = _torch()
    I = x_rot.shape[-1]
    S = _vecs(x_rot, I, "x_rot")
    O = _mq4_check(w, I)
    _one_device(w, x_rot, out)
    y = _out(out, S, O, x_rot)
    _call(fn, _dev(w, "w", torch.uint8), _dev(x_rot, "x_rot", torch.float32),
          _dev(y, "y", torch.float32), S, I, O, _stream())
    return y


def mq4v1(w, x_rot, out=None):
    """MQ4 v1 (f32 scale and zero per 256 weights) GEMV on rotated x."""
    return _mq4_any("qgemv_mq4v1", w, x_rot, out)


def mq4c(w, x_rot, out=None):
    """MQ4C pad (one fp16 scale/zero pair per 256 weights) GEMV on rotated x."""
    return _mq4_any("qgemv_mq4c", w, x_rot, out)


def mq4v2_encode(W, out=None):
    """MQ4-v2 groups [O][I/256*136] u8 from rotated-space weights W f32 [O][I]."""
    torch = _torch()
    O, I = W.shape
    _one_device(W, out)
    if out is not None and out.numel() != O * (I // 256) * 136:
        raise ValueError(f"out must hold {O} rows of {I // 256} 136-byte groups")
    w = out if out is not None else torch.empty((O, (I // 256) * 136), dtype=torch.uint8,
                                                 device=W.device)
    _call("qgemv_mq4v2_encode", _dev(W, "W", torch.float32), _dev(w, "w_out", torch.uint8),
          I, O, _stream())
    return w


def mq4v2_rot(w, x, signs, out=None):
    """MQ4-v2 GEMV on unrotated x: the FWHT-256 pre-rotation fused in."""
    torch = _torch()
    I = x.shape[-1]
    S = _vecs(x, I)
    O = _mq4_check(w, I)
    if signs.numel() != I:
        raise ValueError(f"signs must hold {I} values")
    _one_device(w, x, signs, out)
    y = _out(out, S, O, x)
    _call("qgemv_mq4v2_rot", _dev(w, "w", torch.uint8), _dev(x, "x", torch.float32),
          _dev(signs, "signs", torch.int8), _dev(y, "y", torch.float32), S, I, O, _stream())
    return y


def fwht256(x, signs, out=None):
    torch = _torch()
    I = x.shape[-1]
    S = _vecs(x, I)
    if signs.numel() != I:
        raise ValueError(f"signs must hold {I} values")
    _one_device(x, signs, out)
    if out is not None and out.numel() != x.numel():
        raise ValueError(f"out must hold {x.numel()} floats")
    y = out if out is not None else torch.empty_like(x)
    _call("qgemv_fwht256", _dev(x, "x", torch.float32), _dev(signs, "signs", torch.int8),
          _dev(y, "x_rot", torch.float32), S, I, _stream())
    return y


def router_topk(logits, E, K):
    """logits f32 [T][ld] (experts 0..E-1 valid) -> (ids int32 [T][K], gates f32 [T][K])."""
    torch = _torch()
    T, ld = logits.shape
    if not (1 <= E <= ld):
        raise ValueError(f"E must be in 1..{ld} (the row stride of logits)")
    ids = torch.empty((T, K), dtype=torch.int32, device=logits.device)
    gates = torch.empty((T, K), dtype=torch.float32, device=logits.device)
    _call("qgemv_router_topk", _dev(logits, "logits", torch.float32), T, E, ld, K,
          _dev(ids, "ids", torch.int32), _dev(gates, "gates", torch.float32), _stream())
    return ids, gates


def moe_topk_workspace(T, K, O, device):
    torch = _torch()
    n = qgemv_moe_topk_workspace(T, K, O)
    return torch.zeros(max(int(n), 1), dtype=torch.uint8, device=device)


def moe_topk(w, scales, ids, gates, x, gs, workspace=None, out=None):
    """w u8 [E][O][rb], scales f32 [E][O][ng], ids int32 [T][K], gates f32 [T][K], x f32 [T][I]."""
    torch = _torch()
    E, O = w.shape[0], w.shape[1]
    T, K = ids.shape
    I = x.shape[-1]
    _gs(gs)
    _shape(w, "w", (E, O, (I + 1) // 2))
    _shape(scales, "scales", (E, O, (I + gs - 1) // gs))
    _shape(gates, "gates", (T, K))
    _shape(x, "x", (T, I))
    _one_device(w, scales, ids, gates, x, workspace, out)
    ws = workspace if workspace is not None else moe_topk_workspace(T, K, O, x.device)
    if ws.numel() < qgemv_moe_topk_workspace(T, K, O):
        raise ValueError(f"workspace must hold {qgemv_moe_topk_workspace(T, K, O)} bytes")
    y = _out(out, T, O, x)
    _call("qgemv_moe_topk", _dev(w, "w", torch.uint8), _dev(scales, "scales", torch.float32),
          w[0].numel(), scales[0].numel(), E, _dev(ids, "ids", torch.int32),
          _dev(gates, "gates", torch.float32), T, K, _dev(x, "x", torch.float32),
          _dev(y, "y", torch.float32), I, O, gs, _dev(ws, "workspace", torch.uint8),
          ws.numel(), _stream())
    return y


def moe_topk_error(workspace):
    flag = C.c_int(0)
    _call("qgemv_moe_topk_error", _dev(workspace, "workspace"), C.byref(flag), _stream())
    return flag.value


# -- products with an epilogue, routed slots -------------------------------
# x, bias, residual and y of one call share a type, float32 or bfloat16.
# x, residual, h and a caller's out may be row-strided views (columns
# contiguous); everything else is contiguous.  out must not share elements with
# another argument, but for residual, which may be out itself.  The launch goes
# to the device of the tensors, on its current stream.  There is no backward pass: a call that
# autograd would have to record is refused (torch.no_grad(), or detach()).
_NO_GUARD = contextlib.nullcontext()


def _sizes(fn, *sizes):
    """Refuses sizes that no call takes, before a C int could wrap them."""
    for n in sizes:
        if not 0 <= n <= _MAX_DIM:
            raise QgemvError(fn, 2, strerror(2))


def _no_gradient(*ts):
    for t in ts:
        if t is not None and t.requires_grad and _torch().is_grad_enabled():
            raise ValueError("an argument requires a gradient, and this call has no backward "
                             "pass: detach it or use torch.no_grad()")


def _on(device):
    """Makes `device` current for a launch (nothing to do where it is)."""
    cuda = _torch().cuda
    return _NO_GUARD if device.index == cuda.current_device() else cuda.device(device)


def _raw_stream(device):
    """The device's current stream handle, without building a Stream object."""
    return _torch()._C._cuda_getCurrentRawStream(device.index)


def _dtype_code(t, name):
    torch = _torch()
    if isinstance(t, torch.Tensor):
        if t.dtype == torch.float32:
            return 0
        if t.dtype == torch.bfloat16:
            return 1
        raise TypeError(f"{name} must be float32 or bfloat16, got {t.dtype}")
    raise TypeError(f"{name} must be a CUDA (HIP) tensor")


def _rows(t, name, dtype, shape=None):
    """(pointer, row stride in elements) of a 2-D tensor with contiguous rows."""
    torch = _torch()
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA (HIP) tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != 2:
        raise ValueError(f"{name} must have two dimensions")
    if shape is not None:
        _shape(t, name, shape)
    n, width = t.shape
    if width > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} must have contiguous rows")
    if n <= 1:
        return t.data_ptr(), max(t.stride(0), width)
    if t.stride(0) < width:
        raise ValueError(f"{name}'s rows must not overlap")
    return t.data_ptr(), t.stride(0)


def _epilogue(dtype, O, bias, act, gated, residual, rows, E=None):
    """(Epilogue or None, columns of y); E: bias is [E][O]."""
    if act not in ACTIVATIONS:
        raise ValueError(f"act must be one of {sorted(k for k in ACTIVATIONS if k)} or None")
    if gated and O % 2:
        raise ValueError("a gated product needs an even number of rows in w")
    oc = O // 2 if gated else O
    if bias is None and act is None and not gated and residual is None:
        return None, oc
    e = Epilogue(ACTIVATIONS[act], int(bool(gated)), None, None, 0)
    if bias is not None:
        e.bias = _dev(bias, "bias", dtype)
        _shape(bias, "bias", (O,) if E is None else (E, O))
    if residual is not None:
        e.residual, e.ld_residual = _rows(residual, "residual", dtype, (rows, oc))
    return e, oc


def _ref(e):
    return C.addressof(e) if e is not None else None


def _scratch(workspace, need, device):
    """The caller's workspace (checked) or a new one, none where none is needed;
    (tensor, pointer, bytes)."""
    torch = _torch()
    if workspace is None:
        if need == 0:
            return None, None, 0
        workspace = torch.empty(int(need), dtype=torch.uint8, device=device)
        return workspace, workspace.data_ptr(), need
    if workspace.numel() < need:
        raise ValueError(f"workspace must hold {need} bytes")
    return workspace, _dev(workspace, "workspace", torch.uint8), workspace.numel()


def _new_rows(out, name, n, width, like):
    """(y, pointer, row stride): the caller's out (checked) or new rows of like's
    type."""
    if out is None:
        out = _torch().empty((n, width), dtype=like.dtype, device=like.device)
        return out, out.data_ptr(), width
    return (out, *_rows(out, name, like.dtype, (n, width)))


def _linear(fn, w, scales, x, gs, bias, act, gated, residual, workspace, out):
    torch = _torch()
    code = _dtype_code(x, "x")
    one = x.dim() == 1
    if one:
        x = x.unsqueeze(0)
        residual = residual.unsqueeze(0) if residual is not None and residual.dim() == 1 \
            else residual
        out = out.unsqueeze(0) if out is not None and out.dim() == 1 else out
    if x.dim() != 2:
        raise ValueError("x must be [I] or [S, I]")
    S, I = x.shape
    O = _i4g_check(w, scales, x, gs, S, I) if gs is not None else _fp8_check(w, scales, I,
                                                                             "scale_inv")
    _sizes(fn, S, I, O)
    _no_gradient(scales, x, bias, residual, out)
    _one_device(w, scales, x, bias, residual, workspace, out)
    xp, ldx = _rows(x, "x", x.dtype)
    epi, oc = _epilogue(x.dtype, O, bias, act, gated, residual, S)
    y, yp, ldy = _new_rows(out, "out", S, oc, x)
    wp, sp = _dev(w, "w", torch.uint8), _dev(scales, "scales", torch.float32)
    with _on(x.device):
        ws, wsp, nbytes = _scratch(workspace, qgemv_linear_workspace(S, I, O, code), x.device)
        args = (wp, sp, xp, ldx, yp, ldy, S, I, O) + ((gs,) if gs is not None else ())
        _call(fn, *args, code, _ref(epi), wsp, nbytes, _raw_stream(x.device))
    return y[0] if one else y


def linear_workspace(S, I, O, dtype, device):
    """Scratch for one i4g_linear or fp8b128_linear call of these sizes."""
    torch = _torch()
    code = _dtype_code(torch.empty(0, dtype=dtype), "dtype")
    return torch.empty(max(int(qgemv_linear_workspace(S, I, O, code)), 1), dtype=torch.uint8,
                       device=device)


def i4g_linear(w, scales, x, gs, bias=None, act=None, gated=False, residual=None, workspace=None,
               out=None):
    """y = act(x W^T + bias) + residual with grouped-int4 W, any number of rows.

    w u8 [O][(I+1)//2], scales f32 [O][ng], x [S][I] (or [I]) f32 or bf16, bias
    [O], residual and y [S][O] of x's type.  gated: w holds the gate rows, then
    the up rows, y = act(gate) * up (+ residual) has O/2 columns.  act: None,
    "relu", "silu", "gelu" or "gelu_tanh".  One or two plain f32 vectors run
    faster through ``i4g``.
    """
    return _linear("qgemv_i4g_linear", w, scales, x, _gs(gs), bias, act, gated, residual,
                   workspace, out)


def fp8b128_linear(w, scale_inv, x, bias=None, act=None, gated=False, residual=None,
                   workspace=None, out=None):
    """i4g_linear's product with fp8-e4m3 W [O][I] and 128x128 block scales."""
    return _linear("qgemv_fp8b128_linear", w, scale_inv, x, None, bias, act, gated, residual,
                   workspace, out)


def moe_group(ids, E, workspace=None):
    """Routed slots sorted by expert: ids int32 [T][K] -> (offsets int32 [E+1],
    tokens int32 [T*K], pos int32 [T][K]); see qgemv_moe_group."""
    torch = _torch()
    if ids.dim() != 2:
        raise ValueError("ids must be [T, K]")
    T, K = ids.shape
    E = operator.index(E)
    _sizes("qgemv_moe_group", T, K, E)
    _one_device(ids, workspace)
    ip = _dev(ids, "ids", torch.int32)
    offsets = torch.empty(min(E, 1024) + 1, dtype=torch.int32, device=ids.device)
    tokens = torch.empty(T * K, dtype=torch.int32, device=ids.device)
    pos = torch.empty((T, K), dtype=torch.int32, device=ids.device)
    with _on(ids.device):
        ws, wsp, nbytes = _scratch(workspace, qgemv_moe_group_workspace(T, K, E), ids.device)
        _call("qgemv_moe_group", ip, T, K, E, offsets.data_ptr(), tokens.data_ptr(),
              pos.data_ptr(), wsp, nbytes, _raw_stream(ids.device))
    return offsets, tokens, pos


def grouped_workspace(T, R, E, I, O, dtype, device):
    """Scratch for one i4g_grouped call of these sizes."""
    torch = _torch()
    code = _dtype_code(torch.empty(0, dtype=dtype), "dtype")
    return torch.empty(max(int(qgemv_grouped_workspace(T, R, E, I, O, code)), 1),
                       dtype=torch.uint8, device=device)


def i4g_grouped(w, scales, x, offsets, gs, rows=None, bias=None, act=None, gated=False,
                workspace=None, out=None):
    """Each expert's rows times its grouped-int4 matrix, with i4g_linear's bias,
    activation and gate: w u8 [E][O][rb], scales f32 [E][O][ng], offsets int32
    [E+1], bias [E][O].  Row r of y belongs to the expert e with offsets[e] <=
    r < offsets[e+1] and reads x[rows[r]] (x[r] without rows); rows of no
    expert are left as they are in ``out``."""
    torch = _torch()
    code = _dtype_code(x, "x")
    gs = _gs(gs)
    if w.dim() != 3 or x.dim() != 2:
        raise ValueError("w must be [E, O, (I + 1) // 2] and x [T, I]")
    E, O = w.shape[0], w.shape[1]
    T, I = x.shape
    R = T if rows is None else rows.numel()
    _sizes("qgemv_i4g_grouped", T, R, E, I, O)
    _shape(w, "w", (E, O, (I + 1) // 2))
    _shape(scales, "scales", (E, O, (I + gs - 1) // gs))
    _shape(offsets, "offsets", (E + 1,))
    if rows is not None:
        _shape(rows, "rows", (R,))
    _no_gradient(scales, x, bias, out)
    _one_device(w, scales, x, offsets, rows, bias, workspace, out)
    xp, ldx = _rows(x, "x", x.dtype)
    epi, oc = _epilogue(x.dtype, O, bias, act, gated, None, R, E)
    y, yp, ldy = _new_rows(out, "out", R, oc, x)
    wp, sp = _dev(w, "w", torch.uint8), _dev(scales, "scales", torch.float32)
    op = _dev(offsets, "offsets", torch.int32)
    rp = _dev(rows, "rows", torch.int32) if rows is not None else None
    with _on(x.device):
        ws, wsp, nbytes = _scratch(workspace, qgemv_grouped_workspace(T, R, E, I, O, code),
                                   x.device)
        _call("qgemv_i4g_grouped", wp, sp, O * w.shape[2], O * scales.shape[2], E, op, rp, xp,
              ldx, T, yp, ldy, R, I, O, gs, code, _ref(epi), wsp, nbytes,
              _raw_stream(x.device))
    return y


def moe_combine(h, pos, gates, residual=None, out=None):
    """y[t] = sum_k gates[t][k] h[pos[t][k]] (+ residual[t]): h [R][O] f32 or
    bf16, pos int32 [T][K], gates f32 [T][K], residual and y [T][O]."""
    torch = _torch()
    code = _dtype_code(h, "h")
    if pos.dim() != 2 or h.dim() != 2:
        raise ValueError("h must be [R, O] and pos [T, K]")
    T, K = pos.shape
    R, O = h.shape
    _sizes("qgemv_moe_combine", T, K, R, O)
    _shape(gates, "gates", (T, K))
    _no_gradient(h, gates, residual, out)
    _one_device(h, pos, gates, residual, out)
    hp, ldh = _rows(h, "h", h.dtype)
    rp, ldr = _rows(residual, "residual", h.dtype, (T, O)) if residual is not None else (None, 0)
    y, yp, ldy = _new_rows(out, "out", T, O, h)
    with _on(h.device):
        _call("qgemv_moe_combine", hp, ldh, R, _dev(pos, "pos", torch.int32),
              _dev(gates, "gates", torch.float32), T, K, O, rp, ldr, yp, ldy, code,
              _raw_stream(h.device))
    return y


def dequant_i4g(w, scales, I, gs):
    torch = _torch()
    O = _i4g_check(w, scales, None, gs, 1, I)
    _one_device(w, scales)
    W = torch.empty((O, I), dtype=torch.float32, device=w.device)
    _call("qgemv_dequant_i4g", _dev(w, "w", torch.uint8), _dev(scales, "scales", torch.float32),
          _dev(W, "W"), I, O, gs, _stream())
    return W


def dequant_fp8b128(w, scale_inv):
    torch = _torch()
    O, I = w.shape
    _fp8_check(w, scale_inv, I, "scale_inv")
    _one_device(w, scale_inv)
    W = torch.empty((O, I), dtype=torch.float32, device=w.device)
    _call("qgemv_dequant_fp8b128", _dev(w, "w", torch.uint8),
          _dev(scale_inv, "scale_inv", torch.float32), _dev(W, "W"), I, O, _stream())
    return W


def dequant_fp8b128_ue8m0(w, scale_e8m0):
    torch = _torch()
    O, I = w.shape
    _fp8_check(w, scale_e8m0, I, "scale_e8m0")
    _one_device(w, scale_e8m0)
    W = torch.empty((O, I), dtype=torch.float32, device=w.device)
    _call("qgemv_dequant_fp8b128_ue8m0", _dev(w, "w", torch.uint8),
          _dev(scale_e8m0, "scale_e8m0", torch.uint8), _dev(W, "W"), I, O, _stream())
    return W


def _dequant_mq4_any(fn, w, I):
    torch = _torch()
    O = _mq4_check(w, I)
    W = torch.empty((O, I), dtype=torch.float32, device=w.device)
    _call(fn, _dev(w, "w", torch.uint8), _dev(W, "W"), I, O, _stream())
    return W


def dequant_mq4v1(w, I):
    return _dequant_mq4_any("qgemv_dequant_mq4v1", w, I)


def dequant_mq4c(w, I):
    return _dequant_mq4_any("qgemv_dequant_mq4c", w, I)


def dequant_mq4v2(w, I):
    torch = _torch()
    O = _mq4_check(w, I)
    W = torch.empty((O, I), dtype=torch.float32, device=w.device)
    _call("qgemv_dequant_mq4v2", _dev(w, "w", torch.uint8), _dev(W, "W"), I, O, _stream())
    return W
