"""Thin ctypes binding of libhyena_b200.so (declared in include/hyena.h).

Argument marshalling only: every step of the operator runs in the CUDA
library.  Tensors are torch CUDA tensors (torch supplies device memory and
streams); the functions take the same names as the C entry points.  There
is no fallback: if the shared library is missing, loading raises.
"""
from __future__ import annotations

import ctypes
import os
import struct
import threading

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libhyena_b200.so")

HYENA_F32, HYENA_BF16 = 0, 1
STATUS = {0: "HYENA_OK", 1: "HYENA_ERR_INVALID_ARG", 2: "HYENA_ERR_UNSUPPORTED_SHAPE",
          3: "HYENA_ERR_MISALIGNED", 4: "HYENA_ERR_SPECTRUM_MISMATCH",
          5: "HYENA_ERR_WORKSPACE_TOO_SMALL", 6: "HYENA_ERR_CUDA", 7: "HYENA_ERR_INTERNAL",
          8: "HYENA_ERR_TIMEOUT"}

# every symbol include/hyena.h declares
EXPORTS = ["hyena_version", "hyena_status_string", "hyena_last_error_detail", "hyena_spectrum_bytes",
           "hyena_filter_spectrum", "hyena_shortconv", "hyena_gated_fftconv_workspace_bytes",
           "hyena_gated_fftconv_workspace_min_bytes", "hyena_gated_fftconv", "hyena_gated_fftconv_noalloc",
           "hyena_gated_fftconv_per_sample", "hyena_gated_fftconv_host", "hyena_spectrum_check",
           "hyena_debug_conv_tc", "hyena_debug_conv_cluster", "hyena_debug_conv_2d_tc", "hyena_debug_conv_2dc_tc", "hyena_gated_fftconv_ex", "hyena_kernel_status", "hyena_in_proj",
           "hyena_out_proj", "hyena_implicit_filter_workspace_bytes", "hyena_filter_spectrum_implicit",
           "hyena_delta_rule_workspace_bytes", "hyena_delta_rule", "hyena_delta_rule_step", "hyena_quantize_fp8",
           "hyena_quantize_fp8_weight", "hyena_proj_fp8", "hyena_debug_delta_rule", "hyena_debug_proj_fp8"]

_lock = threading.Lock()
_lib = None


class HyenaError(RuntimeError):
    def __init__(self, status: int, detail: str):
        super().__init__(f"{STATUS.get(status, status)}: {detail}")
        self.status = status
        self.detail = detail


def load(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load the CUDA library (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(path):
            raise RuntimeError(f"{path} is missing: build it with "
                               "`python -m fft_long_convolution_02_b200.build`")
        lib = ctypes.CDLL(path)
        i64, vp, sz, fp = ctypes.c_int64, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p
        i64p = ctypes.POINTER(ctypes.c_int64)
        lib.hyena_version.restype = ctypes.c_int
        lib.hyena_status_string.restype = ctypes.c_char_p
        lib.hyena_status_string.argtypes = [ctypes.c_int]
        lib.hyena_last_error_detail.restype = ctypes.c_char_p
        lib.hyena_spectrum_bytes.restype = sz
        lib.hyena_spectrum_bytes.argtypes = [i64, ctypes.c_int, i64p, ctypes.c_int]
        lib.hyena_filter_spectrum.restype = ctypes.c_int
        lib.hyena_filter_spectrum.argtypes = [vp, ctypes.c_int, fp, i64, ctypes.c_int, i64p, ctypes.c_int,
                                              vp, sz, vp]
        lib.hyena_shortconv.restype = ctypes.c_int
        lib.hyena_shortconv.argtypes = [vp, vp, fp, fp, i64, i64, i64, ctypes.c_int, vp]
        lib.hyena_gated_fftconv_workspace_bytes.restype = sz
        lib.hyena_gated_fftconv_workspace_bytes.argtypes = [i64, i64, ctypes.c_int, i64p, ctypes.c_int]
        lib.hyena_gated_fftconv_workspace_min_bytes.restype = sz
        lib.hyena_gated_fftconv_workspace_min_bytes.argtypes = [i64, ctypes.c_int, i64p, ctypes.c_int]
        lib.hyena_gated_fftconv.restype = ctypes.c_int
        lib.hyena_gated_fftconv.argtypes = [vp, vp, vp, sz, fp, fp, i64, i64, ctypes.c_int, i64p, ctypes.c_int,
                                            ctypes.c_int, vp, sz, vp]
        lib.hyena_gated_fftconv_per_sample.restype = ctypes.c_int
        lib.hyena_gated_fftconv_per_sample.argtypes = [vp, vp, vp, sz, fp, fp, i64, i64, ctypes.c_int, i64p,
                                                       ctypes.c_int, ctypes.c_int, vp, sz, vp]
        lib.hyena_gated_fftconv_host.restype = ctypes.c_int
        lib.hyena_gated_fftconv_host.argtypes = [vp, vp, vp, vp, vp, sz, fp, fp, i64, i64, ctypes.c_int, i64p,
                                                 ctypes.c_int, ctypes.c_int, vp, sz, i64, vp]
        lib.hyena_gated_fftconv_noalloc.restype = ctypes.c_int
        lib.hyena_gated_fftconv_noalloc.argtypes = [vp, vp, vp, sz, fp, fp, i64, i64, ctypes.c_int, i64p,
                                                    ctypes.c_int, ctypes.c_int, vp]
        lib.hyena_gated_fftconv_ex.restype = ctypes.c_int
        lib.hyena_gated_fftconv_ex.argtypes = [vp, vp, vp, sz, fp, fp, i64, i64, ctypes.c_int, i64p, ctypes.c_int,
                                               ctypes.c_int, vp, sz, ctypes.c_uint, vp]
        lib.hyena_in_proj.restype = ctypes.c_int
        lib.hyena_in_proj.argtypes = [vp, vp, fp, vp, i64, i64, i64, ctypes.c_int, vp]
        lib.hyena_out_proj.restype = ctypes.c_int
        lib.hyena_out_proj.argtypes = [vp, vp, fp, vp, i64, i64, i64, vp]
        lib.hyena_implicit_filter_workspace_bytes.restype = sz
        lib.hyena_implicit_filter_workspace_bytes.argtypes = [i64, ctypes.c_int]
        lib.hyena_filter_spectrum_implicit.restype = ctypes.c_int
        lib.hyena_filter_spectrum_implicit.argtypes = [ctypes.POINTER(ImplicitFilter), fp, i64, i64, ctypes.c_int, vp,
                                                       sz, vp, sz, fp, vp]
        lib.hyena_kernel_status.restype = ctypes.c_int
        lib.hyena_kernel_status.argtypes = [vp]
        lib.hyena_spectrum_check.restype = ctypes.c_int
        lib.hyena_spectrum_check.argtypes = [vp, i64, ctypes.c_int, i64p, ctypes.c_int, vp]
        lib.hyena_debug_conv_tc.restype = ctypes.c_int
        lib.hyena_debug_conv_tc.argtypes = [vp, vp, vp, sz, fp, fp, i64, i64, ctypes.c_int, ctypes.c_uint64,
                                            ctypes.c_int, vp]
        lib.hyena_debug_conv_cluster.restype = ctypes.c_int
        lib.hyena_debug_conv_cluster.argtypes = [vp, vp, vp, sz, fp, fp, i64, i64, ctypes.c_int, vp, sz,
                                                 ctypes.c_uint64, ctypes.c_int, vp]
        lib.hyena_debug_conv_2d_tc.restype = ctypes.c_int
        lib.hyena_debug_conv_2d_tc.argtypes = [vp, vp, vp, sz, i64, i64, i64, ctypes.c_int, vp, sz,
                                               ctypes.c_uint64, ctypes.c_int, vp]
        lib.hyena_debug_conv_2dc_tc.restype = ctypes.c_int
        lib.hyena_debug_conv_2dc_tc.argtypes = [vp, vp, vp, sz, i64, i64, ctypes.c_int, vp, sz,
                                                ctypes.c_uint64, ctypes.c_int, vp]
        lib.hyena_delta_rule_workspace_bytes.restype = sz
        lib.hyena_delta_rule_workspace_bytes.argtypes = [i64, i64] + [ctypes.c_int] * 5
        lib.hyena_delta_rule.restype = ctypes.c_int
        lib.hyena_delta_rule.argtypes = [vp, vp, sz, vp]
        lib.hyena_debug_delta_rule.restype = ctypes.c_int
        lib.hyena_debug_delta_rule.argtypes = [vp, vp, sz, ctypes.c_uint64, i64, vp]
        lib.hyena_delta_rule_step.restype = ctypes.c_int
        lib.hyena_delta_rule_step.argtypes = [vp, vp, i64, vp, vp]
        lib.hyena_quantize_fp8.restype = ctypes.c_int
        lib.hyena_quantize_fp8.argtypes = [vp, vp, fp, i64, i64, i64, ctypes.c_int, ctypes.c_int, vp]
        lib.hyena_quantize_fp8_weight.restype = ctypes.c_int
        lib.hyena_quantize_fp8_weight.argtypes = [vp, vp, fp, i64, i64, ctypes.c_int, vp]
        lib.hyena_proj_fp8.restype = ctypes.c_int
        lib.hyena_proj_fp8.argtypes = [vp, fp, vp, fp, fp, vp, i64, i64, i64, i64, ctypes.c_int, vp]
        lib.hyena_debug_proj_fp8.restype = ctypes.c_int
        lib.hyena_debug_proj_fp8.argtypes = [vp, fp, vp, fp, fp, vp, i64, i64, i64, i64, ctypes.c_int, ctypes.c_uint64,
                                             ctypes.c_int, vp]
        _lib = lib
    return _lib


HYENA_CIRCULAR = 0x100   # include/hyena.h: OR-ed into ndim for the circular 2-D form


class Circular(tuple):
    """sizes (H, W) of the circular (periodic) 2-D form: pass Circular((H, W))
    wherever a shape is taken."""


def _sizes(sizes):
    circ = isinstance(sizes, Circular)
    sizes = [int(s) for s in sizes]
    nd = len(sizes)
    if circ:
        if nd != 2:
            raise ValueError("the circular form is 2-D")
        nd |= HYENA_CIRCULAR
    return (ctypes.c_int64 * len(sizes))(*sizes), nd


def _ptr(x):
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


def _stream(stream):
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _dtype_code(t) -> int:
    import torch
    if t.dtype == torch.float32:
        return HYENA_F32
    if t.dtype == torch.bfloat16:
        return HYENA_BF16
    raise TypeError(f"unsupported tensor dtype {t.dtype}")


def _check(rc: int):
    if rc != 0:
        detail = load().hyena_last_error_detail().decode()
        raise HyenaError(rc, detail)


def hyena_version() -> int:
    return load().hyena_version()


def hyena_spectrum_bytes(C: int, sizes, order: int) -> int:
    arr, nd = _sizes(sizes)
    return int(load().hyena_spectrum_bytes(C, nd, arr, order))


def hyena_gated_fftconv_workspace_bytes(B: int, C: int, sizes, order: int) -> int:
    arr, nd = _sizes(sizes)
    return int(load().hyena_gated_fftconv_workspace_bytes(B, C, nd, arr, order))


def hyena_gated_fftconv_workspace_min_bytes(C: int, sizes, order: int) -> int:
    arr, nd = _sizes(sizes)
    return int(load().hyena_gated_fftconv_workspace_min_bytes(C, nd, arr, order))


def hyena_filter_spectrum(k, D, C: int, sizes, order: int, spectrum, stream=None) -> None:
    """k: [order-1, C, *sizes] (f32/bf16 CUDA), D: [order-1, C] f32 or None,
    spectrum: uint8 CUDA tensor of hyena_spectrum_bytes(...) bytes."""
    arr, nd = _sizes(sizes)
    _check(load().hyena_filter_spectrum(_ptr(k), _dtype_code(k), _ptr(D), C, nd, arr, order, _ptr(spectrum),
                                        spectrum.numel() * spectrum.element_size(), _stream(stream)))


def hyena_shortconv(u, out, w, bias=None, stream=None) -> None:
    """u, out: [B, Ctot, L]; w: [Ctot, 3] f32; bias: [Ctot] f32 or None."""
    B, Ctot, L = u.shape
    _check(load().hyena_shortconv(_ptr(u), _ptr(out), _ptr(w), _ptr(bias), B, Ctot, L, _dtype_code(u),
                                  _stream(stream)))


def hyena_gated_fftconv(u, y, spectrum, sc_w, sc_bias, B: int, C: int, sizes, order: int, workspace=None,
                        stream=None) -> None:
    """u: [B, (order+1)*C, *sizes], y: [B, C, *sizes] (same dtype), spectrum from
    hyena_filter_spectrum, sc_w [(order+1)*C, 3] f32 or None, workspace uint8 or None."""
    arr, nd = _sizes(sizes)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(load().hyena_gated_fftconv(_ptr(u), _ptr(y), _ptr(spectrum), spectrum.numel() * spectrum.element_size(),
                                      _ptr(sc_w), _ptr(sc_bias), B, C, nd, arr, order, _dtype_code(u),
                                      _ptr(workspace), ws_bytes, _stream(stream)))


HYENA_FLAG_FP32_TRANSFORM = 0x1


def hyena_gated_fftconv_ex(u, y, spectrum, sc_w, sc_bias, B: int, C: int, sizes, order: int, workspace=None,
                           flags: int = 0, stream=None) -> None:
    """hyena_gated_fftconv with flags (HYENA_FLAG_FP32_TRANSFORM: the fp32
    transform at L = 8192 with bf16 storage)."""
    arr, nd = _sizes(sizes)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(load().hyena_gated_fftconv_ex(_ptr(u), _ptr(y), _ptr(spectrum), spectrum.numel() * spectrum.element_size(),
                                         _ptr(sc_w), _ptr(sc_bias), B, C, nd, arr, order, _dtype_code(u),
                                         _ptr(workspace), ws_bytes, int(flags), _stream(stream)))


def hyena_in_proj(x, W, bias, u, order: int, stream=None) -> None:
    """x [B, L, D] bf16, W [(order+1)*D, D] bf16, bias [(order+1)*D] f32 or
    None -> u [B, (order+1)*D, L] bf16 (in_proj then 'b l d -> b d l')."""
    B, L, D = x.shape
    _check(load().hyena_in_proj(_ptr(x), _ptr(W), _ptr(bias), _ptr(u), B, L, D, int(order), _stream(stream)))


def hyena_out_proj(y, W, bias, out, stream=None) -> None:
    """y [B, D, L] bf16, W [D, D] bf16, bias [D] f32 or None -> out [B, L, D]
    bf16 ('b d l -> b l d' then out_proj)."""
    B, D, L = y.shape
    _check(load().hyena_out_proj(_ptr(y), _ptr(W), _ptr(bias), _ptr(out), B, L, D, _stream(stream)))


class ImplicitFilter(ctypes.Structure):
    """hyena_implicit_filter_t (device pointers)."""
    _fields_ = [("emb_dim", ctypes.c_int), ("width", ctypes.c_int), ("num_inner", ctypes.c_int),
                ("W_in", ctypes.c_void_p), ("b_in", ctypes.c_void_p), ("W_inner", ctypes.c_void_p),
                ("b_inner", ctypes.c_void_p), ("W_out", ctypes.c_void_p), ("w", ctypes.c_void_p),
                ("alpha", ctypes.c_void_p)]


def hyena_implicit_filter_workspace_bytes(L: int, width: int) -> int:
    return int(load().hyena_implicit_filter_workspace_bytes(L, width))


def hyena_filter_spectrum_implicit(params: dict, D, C: int, L: int, order: int, spectrum, workspace, k_out=None,
                                   stream=None) -> None:
    """params: emb_dim, width, num_inner (ints) and CUDA float32 tensors W_in,
    b_in, W_inner, b_inner (or None), W_out, w, alpha (hyena_implicit_filter_t)."""
    f = ImplicitFilter(int(params["emb_dim"]), int(params["width"]), int(params["num_inner"]),
                       _ptr(params["W_in"]), _ptr(params["b_in"]), _ptr(params.get("W_inner")),
                       _ptr(params.get("b_inner")), _ptr(params["W_out"]), _ptr(params["w"]), _ptr(params["alpha"]))
    ws_bytes = workspace.numel() * workspace.element_size()
    _check(load().hyena_filter_spectrum_implicit(ctypes.byref(f), _ptr(D), C, L, int(order), _ptr(spectrum),
                                                 spectrum.numel() * spectrum.element_size(), _ptr(workspace),
                                                 ws_bytes, _ptr(k_out), _stream(stream)))


HYENA_DELTA_L2NORM = 0x1


class DeltaRule(ctypes.Structure):
    """hyena_delta_rule_t (device pointers, element strides)."""
    _fields_ = ([("B", ctypes.c_int64), ("L", ctypes.c_int64)]
                + [(n, ctypes.c_int) for n in ("Hk", "Hv", "dk", "dv", "dtype")]
                + [("flags", ctypes.c_uint), ("scale", ctypes.c_float)]
                + [(n, ctypes.c_void_p) for n in ("q", "k", "v", "o", "g", "beta")]
                + [(n, ctypes.c_int64 * 3) for n in ("q_stride", "k_stride", "v_stride", "o_stride", "g_stride",
                                                     "beta_stride")]
                + [(n, ctypes.c_void_p) for n in ("state_in", "state_out", "lengths")])


# the same struct packed from plain numbers (a third of the time of filling it field by field)
_DELTA = struct.Struct("@qq5iIf4x6P18q3P")


_torch = None


def _lazy_torch():
    """torch, imported by the first call that needs it."""
    global _torch
    if _torch is None:
        import torch
        _torch = torch
    return _torch


def _on_device(first, *others) -> int:
    """The kernels run on the current device: its own tensors only (None passes)."""
    dev = first.get_device()
    if dev < 0 or dev != _torch._C._cuda_getDevice():
        raise ValueError(f"tensor on {first.device}, not on the current CUDA device")
    for t in others:
        if t is not None and t.get_device() != dev:
            raise ValueError(f"tensor on {t.device}, but the current device is cuda:{dev}")
    return dev


def _raw_stream(stream, dev: int) -> int:
    """The stream's handle; of the device's current stream without an object around it."""
    if stream is None:
        return _torch._C._cuda_getCurrentRawStream(dev)
    return stream if isinstance(stream, int) else stream.cuda_stream


def _plain(name, t, shape, dtype) -> None:
    """A contiguous tensor of this shape and dtype (None passes)."""
    if t is not None and (t.shape != shape or t.dtype != dtype or not t.is_contiguous()):
        raise ValueError(f"{name} must be contiguous {dtype} {shape}, got {t.dtype} {tuple(t.shape)}")


_NONE3 = (0, 0, 0)
_NONE_STATES = (None, None, None)


def _delta_args(q, k, v, g, beta, o, B, L, Hk, Hv, scale, l2norm, states, three):
    """Shapes checked, tensors and strides packed; (dk, dv) and the struct's
    bytes, with `states` (state_in, state_out, lengths).  three: [B, C, L] and
    [B, Hv, L]; otherwise [B, C] and [B, Hv]."""
    torch = _torch
    if Hk < 1 or Hv < 1 or q.shape[1] % Hk or v.shape[1] % Hv:
        raise ValueError("the channels of q and k must divide into Hk heads, those of v into Hv")
    dk, dv = q.shape[1] // Hk, v.shape[1] // Hv
    ck, cv, heads = ((B, Hk * dk, L), (B, Hv * dv, L), (B, Hv, L)) if three else ((B, Hk * dk), (B, Hv * dv), (B, Hv))
    dtype, f32 = q.dtype, torch.float32
    code = HYENA_BF16 if dtype is torch.bfloat16 else _dtype_code(q)
    if (q.shape != ck or k.shape != ck or v.shape != cv or o.shape != cv or k.dtype is not dtype or v.dtype is not dtype
            or o.dtype is not dtype or g is not None and (g.shape != heads or g.dtype is not f32)
            or beta is not None and (beta.shape != heads or beta.dtype is not f32)):
        for name, t, c, d in (("q", q, ck, dtype), ("k", k, ck, dtype), ("v", v, cv, dtype), ("o", o, cv, dtype),
                              ("g", g, heads, f32), ("beta", beta, heads, f32)):
            if t is not None and (t.shape != c or t.dtype is not d):
                raise ValueError(f"{name} must be {d} {c}, got {t.dtype} {tuple(t.shape)}")
    state_in, state_out, lengths = states
    if state_in is not None:
        _plain("state_in", state_in, (B, Hv, dk, dv), torch.float32)
    if state_out is not None:
        _plain("state_out", state_out, (B, Hv, dk, dv), torch.float32)
    if lengths is not None:
        _plain("lengths", lengths, (B,), torch.int32)
    last = () if three else (0,)                      # one token: the third stride
    try:
        packed = _DELTA.pack(
            B, L, Hk, Hv, dk, dv, code, HYENA_DELTA_L2NORM if l2norm else 0, 0.0 if scale is None else scale,
            q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), 0 if g is None else g.data_ptr(),
            0 if beta is None else beta.data_ptr(), *q.stride(), *last, *k.stride(), *last, *v.stride(), *last, *o.stride(),
            *last, *(_NONE3 if g is None else g.stride() + last), *(_NONE3 if beta is None else beta.stride() + last),
            0 if state_in is None else state_in.data_ptr(), 0 if state_out is None else state_out.data_ptr(),
            0 if lengths is None else lengths.data_ptr())
    except struct.error as e:
        raise ValueError(str(e)) from None
    return dk, dv, packed


def hyena_delta_rule_workspace_bytes(B: int, L: int, Hk: int, Hv: int, dk: int, dv: int, dtype) -> int:
    """dtype: torch.float32 or torch.bfloat16, the storage of q, k, v, o."""
    import torch
    code = {torch.float32: HYENA_F32, torch.bfloat16: HYENA_BF16}[dtype]
    return int(load().hyena_delta_rule_workspace_bytes(B, L, Hk, Hv, dk, dv, code))


def hyena_delta_rule(q, k, v, g, beta, o, Hk: int, Hv: int, state_in=None, state_out=None, lengths=None, scale=None,
                     l2norm: bool = False, workspace=None, stream=None) -> None:
    """q, k: [B, Hk*dk, L], v, o: [B, Hv*dv, L] (f32 or bf16, any strides: views
    of a projected stream; token-major tensors as x.transpose(1, 2)), g, beta:
    [B, Hv, L] f32 or None, state_in/state_out: [B, Hv, dk, dv] f32 or None,
    lengths: [B] int32 or None, workspace: uint8 of
    hyena_delta_rule_workspace_bytes(...) or None when that is 0."""
    torch = _lazy_torch()
    dev = _on_device(q, k, v, g, beta, o, state_in, state_out, lengths, workspace)
    B, _, L = q.shape
    _, _, packed = _delta_args(q, k, v, g, beta, o, B, L, Hk, Hv, scale, l2norm, (state_in, state_out, lengths), True)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(load().hyena_delta_rule(packed, _ptr(workspace), ws_bytes, _raw_stream(stream, dev)))


def hyena_delta_rule_step(q, k, v, g, beta, o, states, Hk: int, Hv: int, slots=None, scale=None, l2norm: bool = False,
                          stream=None) -> None:
    """One token a row: q, k: [B, Hk*dk], v, o: [B, Hv*dv], g, beta: [B, Hv] or
    None, states: [n, Hv, dk, dv] f32 updated in place, slots: [B] int32 (row b
    uses state slots[b], negative: padding) or None (row b uses state b)."""
    torch = _lazy_torch()
    dev = _on_device(q, k, v, g, beta, o, states, slots)
    B = q.shape[0]
    dk, dv, packed = _delta_args(q, k, v, g, beta, o, B, 1, Hk, Hv, scale, l2norm, _NONE_STATES, False)
    n = states.shape[0]
    _plain("states", states, (n, Hv, dk, dv), torch.float32)
    if slots is not None:
        _plain("slots", slots, (B,), torch.int32)
    _check(load().hyena_delta_rule_step(packed, states.data_ptr(), n, _ptr(slots), _raw_stream(stream, dev)))


def hyena_quantize_fp8(x, xq, xs, channels_first: bool = False, stream=None) -> None:
    """x [B, L, K] (or [B, K, L] with channels_first) f32 or bf16 -> xq [B, L, K]
    float8_e4m3fn, xs [B, ceil(K/128), L] f32."""
    torch = _lazy_torch()
    dev = _on_device(x, xq, xs)
    B, L, K = (x.shape[0], x.shape[2], x.shape[1]) if channels_first else x.shape
    _plain("x", x, x.shape, x.dtype)
    _plain("xq", xq, (B, L, K), torch.float8_e4m3fn)
    _plain("xs", xs, (B, -(-K // 128), L), torch.float32)
    _check(load().hyena_quantize_fp8(x.data_ptr(), xq.data_ptr(), xs.data_ptr(), B, L, K, _dtype_code(x),
                                     1 if channels_first else 0, _raw_stream(stream, dev)))


def hyena_quantize_fp8_weight(W, Wq, Ws, stream=None) -> None:
    """W [N, K] f32 or bf16 -> Wq [N, K] float8_e4m3fn, Ws [ceil(N/128), ceil(K/128)] f32."""
    torch = _lazy_torch()
    dev = _on_device(W, Wq, Ws)
    N, K = W.shape
    _plain("W", W, (N, K), W.dtype)
    _plain("Wq", Wq, (N, K), torch.float8_e4m3fn)
    _plain("Ws", Ws, (-(-N // 128), -(-K // 128)), torch.float32)
    _check(load().hyena_quantize_fp8_weight(W.data_ptr(), Wq.data_ptr(), Ws.data_ptr(), N, K, _dtype_code(W),
                                            _raw_stream(stream, dev)))


def _proj_fp8_sizes(xq, xs, Wq, Ws, bias, out, channels_first):
    torch = _torch
    B, L, K = xq.shape
    N = Wq.shape[0]
    _plain("xq", xq, (B, L, K), torch.float8_e4m3fn)
    _plain("xs", xs, (B, -(-K // 128), L), torch.float32)
    _plain("Wq", Wq, (N, K), torch.float8_e4m3fn)
    _plain("Ws", Ws, (-(-N // 128), -(-K // 128)), torch.float32)
    _plain("bias", bias, (N,), torch.float32)
    _plain("out", out, (B, N, L) if channels_first else (B, L, N), torch.bfloat16)
    return B, L, K, N


def hyena_proj_fp8(xq, xs, Wq, Ws, bias, out, channels_first: bool = False, stream=None) -> None:
    """xq [B, L, K], Wq [N, K] float8_e4m3fn with their scales, bias [N] f32 or
    None -> out bf16 [B, L, N], or [B, N, L] with channels_first."""
    _lazy_torch()
    dev = _on_device(xq, xs, Wq, Ws, bias, out)
    B, L, K, N = _proj_fp8_sizes(xq, xs, Wq, Ws, bias, out, channels_first)
    _check(load().hyena_proj_fp8(xq.data_ptr(), xs.data_ptr(), Wq.data_ptr(), Ws.data_ptr(), _ptr(bias),
                                 out.data_ptr(), B, L, K, N, 1 if channels_first else 0, _raw_stream(stream, dev)))


def hyena_kernel_status(stream=None) -> None:
    """Raises HyenaError (HYENA_ERR_TIMEOUT, HYENA_ERR_SPECTRUM_MISMATCH, or
    HYENA_ERR_INVALID_ARG for a bad slot of hyena_delta_rule_step)
    when a kernel on the current device recorded one since the
    last call; synchronises the stream and clears the record."""
    _check(load().hyena_kernel_status(_stream(stream)))


def hyena_gated_fftconv_per_sample(u, y, spectrum, sc_w, sc_bias, B: int, C: int, sizes, order: int,
                                   workspace=None, stream=None) -> None:
    """hyena_gated_fftconv with one filter per (b, c) row: spectrum from
    hyena_filter_spectrum over B*C channels (k [order-1, B, C, *sizes])."""
    arr, nd = _sizes(sizes)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(load().hyena_gated_fftconv_per_sample(_ptr(u), _ptr(y), _ptr(spectrum),
                                                 spectrum.numel() * spectrum.element_size(), _ptr(sc_w),
                                                 _ptr(sc_bias), B, C, nd, arr, order, _dtype_code(u),
                                                 _ptr(workspace), ws_bytes, _stream(stream)))


def hyena_gated_fftconv_host(u_host, y_host, u_dev, y_dev, spectrum, sc_w, sc_bias, B: int, C: int, sizes,
                             order: int, workspace=None, chunk_rows: int = 0, stream=None) -> None:
    """u_host / y_host: CPU tensors (pinned for overlap); u_dev / y_dev: CUDA
    tensors of the same shapes; the copies are pipelined against the kernels."""
    if u_host.is_cuda or y_host.is_cuda:
        raise ValueError("u_host and y_host must be host (CPU) tensors")
    if not (u_host.is_contiguous() and y_host.is_contiguous()):
        raise ValueError("u_host and y_host must be contiguous")
    arr, nd = _sizes(sizes)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(load().hyena_gated_fftconv_host(u_host.data_ptr(), y_host.data_ptr(), _ptr(u_dev), _ptr(y_dev),
                                           _ptr(spectrum), spectrum.numel() * spectrum.element_size(), _ptr(sc_w),
                                           _ptr(sc_bias), B, C, nd, arr, order, _dtype_code(u_dev),
                                           _ptr(workspace), ws_bytes, int(chunk_rows), _stream(stream)))


def hyena_gated_fftconv_noalloc(u, y, spectrum, sc_w, sc_bias, B: int, C: int, sizes, order: int,
                                stream=None) -> None:
    """hyena_gated_fftconv without a workspace argument: the library's fixed
    scratch array is used instead (for callers that cannot allocate)."""
    arr, nd = _sizes(sizes)
    _check(load().hyena_gated_fftconv_noalloc(_ptr(u), _ptr(y), _ptr(spectrum),
                                              spectrum.numel() * spectrum.element_size(), _ptr(sc_w),
                                              _ptr(sc_bias), B, C, nd, arr, order, _dtype_code(u),
                                              _stream(stream)))


def hyena_spectrum_check(spectrum, C: int, sizes, order: int, stream=None) -> None:
    arr, nd = _sizes(sizes)
    _check(load().hyena_spectrum_check(_ptr(spectrum), C, nd, arr, order, _stream(stream)))


def hyena_debug_conv_tc(u, y, spectrum, sc_w, sc_bias, B: int, C: int, order: int, wait_budget_ns: int,
                        issue_mma: bool = True, stream=None) -> None:
    """Test hook of the L = 8192 bf16 tensor-core kernel: its bounded waits give
    up after wait_budget_ns; issue_mma=False issues no tensor-core work, so the
    first wait runs out (read back with hyena_kernel_status)."""
    _check(load().hyena_debug_conv_tc(_ptr(u), _ptr(y), _ptr(spectrum), spectrum.numel() * spectrum.element_size(),
                                      _ptr(sc_w), _ptr(sc_bias), B, C, order, int(wait_budget_ns),
                                      1 if issue_mma else 0, _stream(stream)))


def hyena_debug_conv_2d_tc(u, y, spectrum, B: int, C: int, W: int, order: int, workspace, wait_budget_ns: int,
                           issue_mma: bool = True, stream=None) -> None:
    """The same test hook for the 2-D tensor-core column pass (H = 256, bf16)."""
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(load().hyena_debug_conv_2d_tc(_ptr(u), _ptr(y), _ptr(spectrum), spectrum.numel() * spectrum.element_size(),
                                         B, C, W, order, _ptr(workspace), ws_bytes, int(wait_budget_ns),
                                         1 if issue_mma else 0, _stream(stream)))


def hyena_debug_conv_2dc_tc(u, y, spectrum, B: int, C: int, order: int, workspace, wait_budget_ns: int,
                            issue_mma: bool = True, stream=None) -> None:
    """The same test hook for the circular form's paired tensor-core passes
    (256 x 256, bf16, even B)."""
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(load().hyena_debug_conv_2dc_tc(_ptr(u), _ptr(y), _ptr(spectrum), spectrum.numel() * spectrum.element_size(),
                                          B, C, order, _ptr(workspace), ws_bytes, int(wait_budget_ns),
                                          1 if issue_mma else 0, _stream(stream)))


def hyena_debug_conv_cluster(u, y, spectrum, sc_w, sc_bias, B: int, C: int, order: int, workspace,
                             wait_budget_ns: int, issue_mma: bool = True, stream=None) -> None:
    """The same test hook for the L = 65536 bf16 cluster kernel."""
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(load().hyena_debug_conv_cluster(_ptr(u), _ptr(y), _ptr(spectrum),
                                           spectrum.numel() * spectrum.element_size(), _ptr(sc_w), _ptr(sc_bias), B,
                                           C, order, _ptr(workspace), ws_bytes, int(wait_budget_ns),
                                           1 if issue_mma else 0, _stream(stream)))


def hyena_debug_delta_rule(q, k, v, g, beta, o, Hk: int, Hv: int, state_in, state_out, workspace, wait_budget_ns: int,
                           hold_chunk: int = -1, l2norm: bool = False, stream=None) -> None:
    """The same test hook for the scans of hyena_delta_rule: the stage of chunk hold_chunk (-1: none) is never freed."""
    _lazy_torch()
    dev = _on_device(q, k, v, g, beta, o, state_in, state_out, workspace)
    B, _, L = q.shape
    _, _, packed = _delta_args(q, k, v, g, beta, o, B, L, Hk, Hv, None, l2norm, (state_in, state_out, None), True)
    _check(load().hyena_debug_delta_rule(packed, _ptr(workspace), workspace.numel() * workspace.element_size(),
                                         int(wait_budget_ns), hold_chunk, _raw_stream(stream, dev)))


def hyena_debug_proj_fp8(xq, xs, Wq, Ws, bias, out, wait_budget_ns: int, hold: int = 0, channels_first: bool = False,
                         stream=None) -> None:
    """The same test hook for hyena_proj_fp8 (more than 16 rows): hold 1 issues no products, 2 keeps a warp's staged part back."""
    _lazy_torch()
    dev = _on_device(xq, xs, Wq, Ws, bias, out)
    B, L, K, N = _proj_fp8_sizes(xq, xs, Wq, Ws, bias, out, channels_first)
    _check(load().hyena_debug_proj_fp8(xq.data_ptr(), xs.data_ptr(), Wq.data_ptr(), Ws.data_ptr(), _ptr(bias), out.data_ptr(),
                                       B, L, K, N, 1 if channels_first else 0, int(wait_budget_ns), hold,
                                       _raw_stream(stream, dev)))
