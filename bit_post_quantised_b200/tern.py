"""Python binding of libtern (include/tern.h): argument marshalling only.

Every step of the ternary linear path runs in the library's sm_100a kernels;
this module only turns torch tensors into pointers, sizes and the current
CUDA stream, calls the C ABI, and raises on a non-OK status.  There is no
fallback: if libtern.so is missing or the device is not an sm_100 GPU, the
calls fail loudly.
"""
from __future__ import annotations

import ctypes
import os
import struct
from typing import Optional, Sequence

import torch

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libtern.so")
_lib = None

TERN_OK = 0
STATUS_NAMES = {0: "TERN_OK", -1: "TERN_ERR_INVALID_ARG", -2: "TERN_ERR_UNSUPPORTED_SHAPE",
                -3: "TERN_ERR_MISALIGNED", -4: "TERN_ERR_CUDA", -5: "TERN_ERR_TIMEOUT",
                -6: "TERN_ERR_NO_DEVICE", -7: "TERN_ERR_LAUNCH_CONFIG"}

EXPORTED = ("tern_packed_bytes", "tern_quantize_pack", "tern_linear", "tern_linear_noalloc",
            "tern_linear_act", "tern_linear_epilogue", "tern_linear_batch", "tern_linear_batch_act",
            "tern_linear_batch_epilogue", "tern_linear_strided", "tern_linear_batch_strided",
            "tern_adaln_modulate", "tern_quantize_act_e4m3", "tern_linear_e4m3",
            "tern_rope_table", "tern_rope", "tern_attention", "tern_attention_plan", "tern_gated_residual_norm",
            "tern_dequantize", "tern_get_device_status", "tern_set_wait_limit_ns",
            "tern_selftest_wait_timeout", "tern_status_string", "tern_last_error")


class TernError(RuntimeError):
    def __init__(self, status: int, detail: str):
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {detail}")
        self.status = status


class LinearArgs(ctypes.Structure):
    """Mirror of tern_linear_args."""
    _fields_ = [("x", ctypes.c_void_p), ("packed", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("bias", ctypes.c_void_p), ("y", ctypes.c_void_p),
                ("M", ctypes.c_int64), ("N", ctypes.c_int64), ("K", ctypes.c_int64)]


class LinearActArgs(ctypes.Structure):
    """Mirror of tern_linear_act_args."""
    _fields_ = [("linear", LinearArgs), ("act", ctypes.c_int), ("act_col0", ctypes.c_int64)]


class LinearStridedArgs(ctypes.Structure):
    """Mirror of tern_linear_strided_args."""
    _fields_ = [("linear", LinearArgs), ("ldx", ctypes.c_int64), ("ldy", ctypes.c_int64)]


class Epilogue(ctypes.Structure):
    """Mirror of tern_epilogue."""
    _fields_ = [("act", ctypes.c_int), ("act_col0", ctypes.c_int64), ("residual", ctypes.c_void_p),
                ("gate", ctypes.c_void_p), ("norm_col0", ctypes.c_int64), ("norm_col1", ctypes.c_int64),
                ("norm_weight", ctypes.c_void_p), ("norm_eps", ctypes.c_float), ("rope_cs", ctypes.c_void_p)]


class RopeTensor(ctypes.Structure):
    """Mirror of tern_rope_tensor."""
    _fields_ = [("x", ctypes.c_void_p), ("y", ctypes.c_void_p)] + [
        (n, ctypes.c_int64) for n in ("heads", "x_b", "x_l", "x_h", "y_b", "y_l", "y_h")]


class AttentionArgs(ctypes.Structure):
    """Mirror of tern_attention_args."""
    _fields_ = [(n, ctypes.c_void_p) for n in ("q", "k", "v", "o")] + [
        (n, ctypes.c_int64) for n in ("B", "Lq", "Lk", "H", "Hkv", "D", "q_b", "q_l", "q_h", "k_b", "k_l", "k_h",
                                      "v_b", "v_l", "v_h", "o_b", "o_l", "o_h")] + [
        ("scale", ctypes.c_float), ("kv_len", ctypes.c_void_p), ("key_mask", ctypes.c_void_p),
        ("mask_ld", ctypes.c_int64)]


class GatedResidualNormArgs(ctypes.Structure):
    """Mirror of tern_gated_residual_norm_args."""
    _fields_ = [(n, ctypes.c_void_p) for n in ("x", "o", "x_out", "h")] + [
        (n, ctypes.c_int64) for n in ("M", "K", "ld_x", "ld_o", "ld_x_out", "ld_h")] + [
        ("residual_scale", ctypes.c_float), ("post_norm", ctypes.c_int), ("post_weight", ctypes.c_void_p),
        ("post_eps", ctypes.c_float), ("gate", ctypes.c_void_p), ("gate_tanh", ctypes.c_int),
        ("pre_norm", ctypes.c_int), ("pre_weight", ctypes.c_void_p), ("pre_eps", ctypes.c_float),
        ("scale", ctypes.c_void_p), ("shift", ctypes.c_void_p), ("mod_ld", ctypes.c_int64),
        ("tokens_per_row", ctypes.c_int64)]


# The same two layouts for struct.pack, which takes a fifth of the time.
_ATTENTION = struct.Struct("4P18qfPPq")
_RESIDUAL_NORM = struct.Struct("4P6qfiPfPiiPfPPqq")

ACT_NONE = 0       # tern_act values
ACT_GELU_TANH = 1

ATTENTION_NONE = 0  # tern_attention_kernel values
ATTENTION_ROWS = 1
ATTENTION_TILES = 2

NORM_NONE = 0      # tern_norm values
NORM_RMS = 1
NORM_LAYER = 2


def library_path() -> str:
    return _LIB_PATH


def lib() -> ctypes.CDLL:
    """Loads libtern.so (raising if it was not built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(_LIB_PATH):
            raise ImportError(f"libtern.so not found at {_LIB_PATH}; build it with "
                              "bit_post_quantised_b200._build.build()")
        L = ctypes.CDLL(_LIB_PATH)
        i64, vp, st = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int
        L.tern_packed_bytes.argtypes = [i64, i64]
        L.tern_packed_bytes.restype = ctypes.c_size_t
        L.tern_quantize_pack.argtypes = [vp, i64, i64, ctypes.c_float, vp, vp, vp]
        L.tern_quantize_pack.restype = st
        L.tern_linear.argtypes = [vp, i64, i64, vp, vp, vp, i64, vp, vp]
        L.tern_linear.restype = st
        L.tern_linear_noalloc.argtypes = [vp, i64, i64, vp, vp, vp, i64, vp, vp]
        L.tern_linear_noalloc.restype = st
        L.tern_linear_batch.argtypes = [ctypes.POINTER(LinearArgs), ctypes.c_int, vp]
        L.tern_linear_act.argtypes = [vp, i64, i64, vp, vp, vp, i64, ctypes.c_int, i64, vp, vp]
        L.tern_linear_act.restype = st
        L.tern_linear_batch_act.argtypes = [ctypes.POINTER(LinearActArgs), ctypes.c_int, vp]
        L.tern_linear_batch_act.restype = st
        L.tern_linear_epilogue.argtypes = [ctypes.POINTER(LinearArgs), ctypes.POINTER(Epilogue), vp]
        L.tern_linear_epilogue.restype = st
        L.tern_linear_batch_epilogue.argtypes = [ctypes.POINTER(LinearArgs), ctypes.POINTER(Epilogue), ctypes.c_int,
                                                 vp]
        L.tern_linear_batch_epilogue.restype = st
        L.tern_linear_strided.argtypes = [ctypes.POINTER(LinearStridedArgs), ctypes.POINTER(Epilogue), vp]
        L.tern_linear_strided.restype = st
        L.tern_linear_batch_strided.argtypes = [ctypes.POINTER(LinearStridedArgs), ctypes.POINTER(Epilogue),
                                                ctypes.c_int, vp]
        L.tern_linear_batch_strided.restype = st
        L.tern_linear_batch.restype = st
        L.tern_adaln_modulate.argtypes = [vp, i64, i64, vp, vp, i64, i64, ctypes.c_float, vp, vp]
        L.tern_adaln_modulate.restype = st
        L.tern_quantize_act_e4m3.argtypes = [vp, i64, i64, vp, vp, vp]
        L.tern_quantize_act_e4m3.restype = st
        L.tern_linear_e4m3.argtypes = [vp, vp, i64, i64, vp, vp, vp, i64, vp, vp]
        L.tern_linear_e4m3.restype = st
        L.tern_rope_table.argtypes = [vp, i64, ctypes.c_int, vp, ctypes.c_double, vp, vp]
        L.tern_rope_table.restype = st
        L.tern_rope.argtypes = [vp, ctypes.c_int, i64, i64, i64, vp, i64, i64, ctypes.c_int, vp]
        L.tern_rope.restype = st
        L.tern_attention.argtypes = [vp, vp]
        L.tern_attention.restype = st
        L.tern_attention_plan.argtypes = [vp, ctypes.c_int, vp, vp]
        L.tern_attention_plan.restype = st
        L.tern_gated_residual_norm.argtypes = [vp, vp]
        L.tern_gated_residual_norm.restype = st
        L.tern_dequantize.argtypes = [vp, vp, i64, i64, vp, vp]
        L.tern_dequantize.restype = st
        L.tern_get_device_status.argtypes = [vp]
        L.tern_get_device_status.restype = st
        L.tern_set_wait_limit_ns.argtypes = [ctypes.c_uint64]
        L.tern_set_wait_limit_ns.restype = None
        L.tern_selftest_wait_timeout.argtypes = [ctypes.c_uint64, vp]
        L.tern_selftest_wait_timeout.restype = st
        L.tern_status_string.argtypes = [st]
        L.tern_status_string.restype = ctypes.c_char_p
        L.tern_last_error.argtypes = []
        L.tern_last_error.restype = ctypes.c_char_p
        _lib = L
    return _lib


def _check(status: int) -> None:
    if status != TERN_OK:
        raise TernError(status, lib().tern_last_error().decode())


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream: Optional[torch.cuda.Stream]):
    if stream is not None:
        return stream.cuda_stream
    # The handle alone: a torch.cuda.Stream object around it costs 3 us.
    return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())


def _empty(*shape, dtype, device, stream=None) -> torch.Tensor:
    """An output buffer allocated on the stream the call launches on, so that
    the caching allocator orders its reuse after that stream's work."""
    if stream is None:
        return torch.empty(*shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(*shape, dtype=dtype, device=device)


def _empty_as(t: torch.Tensor, stream=None) -> torch.Tensor:
    """A contiguous output buffer of t's shape and type (see _empty)."""
    if stream is None:
        return torch.empty_like(t, memory_format=torch.contiguous_format)
    return _empty(t.shape, dtype=t.dtype, device=t.device, stream=stream)


def packed_bytes(N: int, K: int) -> int:
    return int(lib().tern_packed_bytes(N, K))


def quantize_pack(W: torch.Tensor, eps: float = 1e-5, packed: Optional[torch.Tensor] = None,
                  scales: Optional[torch.Tensor] = None, stream=None):
    """tern_quantize_pack: W bf16 [N,K] -> (packed uint8 [N*K/4], scales fp32 [N])."""
    N, K = W.shape
    if packed is None:
        packed = _empty(max(packed_bytes(N, K), 1), dtype=torch.uint8, device=W.device, stream=stream)
    if scales is None:
        scales = _empty(N, dtype=torch.float32, device=W.device, stream=stream)
    _check(lib().tern_quantize_pack(_ptr(W), N, K, float(eps), _ptr(packed), _ptr(scales),
                                    _stream(stream)))
    return packed, scales


def adaln_modulate(x: torch.Tensor, scale: torch.Tensor, shift: torch.Tensor, eps: float = 1e-6,
                   tokens_per_row: Optional[int] = None, mod_ld: Optional[int] = None,
                   out: Optional[torch.Tensor] = None, stream=None):
    """tern_adaln_modulate: out = LayerNorm(x) * (1 + scale[g]) + shift[g] per
    token row, g = row // tokens_per_row (default: every row uses row 0).
    scale and shift are bf16 with rows mod_ld elements apart (default: their
    own row stride), e.g. slices of the modulation output; out may be x."""
    M, K = x.shape
    T = M if tokens_per_row is None else int(tokens_per_row)
    if scale.stride(-1) != 1 or shift.stride(-1) != 1:
        raise ValueError("scale and shift rows must be contiguous")
    if mod_ld is None:
        mod_ld = scale.stride(0) if scale.dim() == 2 else K
        if shift.dim() == 2 and shift.stride(0) != mod_ld:
            raise ValueError("scale and shift rows must be the same distance apart")
    G = -(-M // max(T, 1)) if M else 0
    for name, t in (("scale", scale), ("shift", shift)):
        rows = t.shape[0] if t.dim() == 2 else 1
        if t.shape[-1] < K or (G and (G - 1) * int(mod_ld) + K > (rows - 1) * int(mod_ld) + t.shape[-1]):
            raise ValueError(f"{name} holds fewer than the {G} modulation rows of {K} values that "
                             f"{M} rows at {T} tokens per row need")
    if out is None:
        out = _empty(*x.shape, dtype=x.dtype, device=x.device, stream=stream)
    _check(lib().tern_adaln_modulate(_ptr(x), M, K, _ptr(scale), _ptr(shift), int(mod_ld), max(T, 1), float(eps),
                                     _ptr(out), _stream(stream)))
    return out


def _dense(*ts) -> None:
    """The dense entry points take row-major tensors without gaps; a view
    with a row stride goes through linear_strided / linear_batch_strided."""
    for t in ts:
        if t is not None and not t.is_contiguous():
            raise ValueError("x, y and residual must be dense row-major here; row-strided views go through "
                             "linear_strided / linear_batch_strided")


def linear(x: torch.Tensor, packed: torch.Tensor, scales: torch.Tensor,
           bias: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None, stream=None):
    """tern_linear: y = (x . T^T) * s + b, x bf16 [M,K] -> y bf16 [M,N]."""
    M, K = x.shape
    N = scales.shape[0]
    if out is None:
        out = _empty(M, N, dtype=torch.bfloat16, device=x.device, stream=stream)
    _dense(x, out)
    _check(lib().tern_linear(_ptr(x), M, K, _ptr(packed), _ptr(scales), _ptr(bias), N, _ptr(out),
                             _stream(stream)))
    return out


def linear_noalloc(x: torch.Tensor, packed: torch.Tensor, scales: torch.Tensor,
                   bias: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                   stream=None):
    """tern_linear_noalloc: tern_linear with its split-K scratch in the library's
    static device array (no device allocation by the library; `out` must be
    given by callers that cannot allocate)."""
    M, K = x.shape
    N = scales.shape[0]
    if out is None:
        out = _empty(M, N, dtype=torch.bfloat16, device=x.device, stream=stream)
    _dense(x, out)
    _check(lib().tern_linear_noalloc(_ptr(x), M, K, _ptr(packed), _ptr(scales), _ptr(bias), N,
                                     _ptr(out), _stream(stream)))
    return out


def linear_batch(problems: Sequence[dict], stream=None) -> None:
    """tern_linear_batch over dicts with keys x, packed, scales, bias (or None), y."""
    arr = (LinearArgs * max(1, len(problems)))()
    for i, p in enumerate(problems):
        _dense(p["x"], p["y"])
        M, K = p["x"].shape
        N = p["scales"].shape[0]
        arr[i] = LinearArgs(p["x"].data_ptr(), p["packed"].data_ptr(), p["scales"].data_ptr(),
                            None if p.get("bias") is None else p["bias"].data_ptr(),
                            p["y"].data_ptr(), M, N, K)
    _check(lib().tern_linear_batch(arr, len(problems), _stream(stream)))


def linear_act(x: torch.Tensor, packed: torch.Tensor, scales: torch.Tensor,
               bias: Optional[torch.Tensor] = None, act: int = ACT_GELU_TANH, act_col0: int = 0,
               out: Optional[torch.Tensor] = None, stream=None):
    """tern_linear_act: the linear with `act` fused into its epilogue on
    output columns [act_col0, N)."""
    M, K = x.shape
    N = scales.shape[0]
    if out is None:
        out = _empty(M, N, dtype=torch.bfloat16, device=x.device, stream=stream)
    _dense(x, out)
    _check(lib().tern_linear_act(_ptr(x), M, K, _ptr(packed), _ptr(scales), _ptr(bias), N, act, act_col0,
                                 _ptr(out), _stream(stream)))
    return out


def linear_batch_act(problems: Sequence[dict], stream=None) -> None:
    """tern_linear_batch_act over dicts as linear_batch's plus act (default
    none) and act_col0 (default 0)."""
    arr = (LinearActArgs * max(1, len(problems)))()
    for i, p in enumerate(problems):
        _dense(p["x"], p["y"])
        M, K = p["x"].shape
        N = p["scales"].shape[0]
        arr[i] = LinearActArgs(LinearArgs(p["x"].data_ptr(), p["packed"].data_ptr(), p["scales"].data_ptr(),
                                          None if p.get("bias") is None else p["bias"].data_ptr(),
                                          p["y"].data_ptr(), M, N, K),
                               p.get("act", ACT_NONE), p.get("act_col0", 0))
    _check(lib().tern_linear_batch_act(arr, len(problems), _stream(stream)))


def _linear_args(p: dict) -> LinearArgs:
    _dense(p["x"], p["y"])
    M, K = p["x"].shape
    N = p["scales"].shape[0]
    return LinearArgs(p["x"].data_ptr(), p["packed"].data_ptr(), p["scales"].data_ptr(),
                      None if p.get("bias") is None else p["bias"].data_ptr(), p["y"].data_ptr(), M, N, K)


def _epilogue(p: dict, strided: bool = False) -> Epilogue:
    if not strided:
        _dense(p.get("residual"))
    rope = p.get("rope_cs")
    if rope is not None and (rope.dtype != torch.float32 or not rope.is_contiguous() or rope.shape[-2:] != (64, 2)
                             or rope.shape[0] < p["y"].shape[0]):
        raise ValueError("rope_cs must be contiguous fp32 [>= M, 64, 2] (cos, sin) pairs")
    return Epilogue(p.get("act", ACT_NONE), p.get("act_col0", 0), _ptr(p.get("residual")), _ptr(p.get("gate")),
                    p.get("norm_col0", 0), p.get("norm_col1", 0), _ptr(p.get("norm_weight")),
                    p.get("norm_eps", 0.0), _ptr(rope))


def linear_epilogue(x: torch.Tensor, packed: torch.Tensor, scales: torch.Tensor,
                    bias: Optional[torch.Tensor] = None, act: int = ACT_NONE, act_col0: int = 0,
                    residual: Optional[torch.Tensor] = None, gate: Optional[torch.Tensor] = None,
                    norm_cols=(0, 0), norm_weight: Optional[torch.Tensor] = None, norm_eps: float = 0.0,
                    out: Optional[torch.Tensor] = None, stream=None, rope_cs: Optional[torch.Tensor] = None):
    """tern_linear_epilogue: y = residual + gate * act(norm(x . T^T * s + b))
    (see tern_epilogue); `out` may be `residual` itself for an in-place
    update; norm_cols = (first, end) of the RMS-normalised columns; rope_cs
    fp32 [M, 64, 2] (cos, sin) rotates the normalised columns' channel pairs."""
    M, K = x.shape
    N = scales.shape[0]
    if out is None:
        out = _empty(M, N, dtype=torch.bfloat16, device=x.device, stream=stream)
    a = _linear_args(dict(x=x, packed=packed, scales=scales, bias=bias, y=out))
    e = _epilogue(dict(act=act, act_col0=act_col0, residual=residual, gate=gate, norm_col0=norm_cols[0],
                       norm_col1=norm_cols[1], norm_weight=norm_weight, norm_eps=norm_eps, rope_cs=rope_cs, y=out))
    _check(lib().tern_linear_epilogue(ctypes.byref(a), ctypes.byref(e), _stream(stream)))
    return out


def linear_batch_epilogue(problems: Sequence[dict], stream=None) -> None:
    """tern_linear_batch_epilogue over dicts as linear_batch's plus the
    optional keys act, act_col0, residual, gate, norm_col0, norm_col1,
    norm_weight, norm_eps and rope_cs."""
    n = max(1, len(problems))
    args, epis = (LinearArgs * n)(), (Epilogue * n)()
    for i, p in enumerate(problems):
        args[i] = _linear_args(p)
        epis[i] = _epilogue(p)
    _check(lib().tern_linear_batch_epilogue(args, epis, len(problems), _stream(stream)))


def quantize_act_e4m3(x: torch.Tensor, xq: Optional[torch.Tensor] = None, a: Optional[torch.Tensor] = None,
                      stream=None):
    """tern_quantize_act_e4m3: x bf16 [M,K] -> (xq uint8 [M,K] E4M3 bytes in the
    interleaved k order of include/tern.h, a fp32 [M] per-token scales)."""
    M, K = x.shape
    if xq is None:
        xq = _empty(M, K, dtype=torch.uint8, device=x.device, stream=stream)
    if a is None:
        a = _empty(M, dtype=torch.float32, device=x.device, stream=stream)
    _check(lib().tern_quantize_act_e4m3(_ptr(x), M, K, _ptr(xq), _ptr(a), _stream(stream)))
    return xq, a


def linear_e4m3(xq: torch.Tensor, a: torch.Tensor, packed: torch.Tensor, scales: torch.Tensor,
                bias: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None, stream=None):
    """tern_linear_e4m3: y = a_m * s_n * sum_k xq[m,k] T[n,k] + b_n -> bf16 [M,N]."""
    M, K = xq.shape
    N = scales.shape[0]
    if out is None:
        out = _empty(M, N, dtype=torch.bfloat16, device=xq.device, stream=stream)
    _check(lib().tern_linear_e4m3(_ptr(xq), _ptr(a), M, K, _ptr(packed), _ptr(scales), _ptr(bias), N, _ptr(out),
                                  _stream(stream)))
    return out


def _strided_args(p: dict) -> LinearStridedArgs:
    x, y = p["x"], p["y"]
    if x.stride(1) != 1 or y.stride(1) != 1:
        raise ValueError("x and y rows must be contiguous (stride 1 along the last dimension)")
    M, K = x.shape
    N = p["scales"].shape[0]
    lin = LinearArgs(x.data_ptr(), p["packed"].data_ptr(), p["scales"].data_ptr(),
                     None if p.get("bias") is None else p["bias"].data_ptr(), y.data_ptr(), M, N, K)
    return LinearStridedArgs(lin, x.stride(0), y.stride(0))


def linear_strided(x: torch.Tensor, packed: torch.Tensor, scales: torch.Tensor, bias: Optional[torch.Tensor],
                   out: torch.Tensor, stream=None, **epilogue):
    """tern_linear_strided: x and out may be row-strided views (for instance
    column slices of wider tensors); their row strides are passed as ldx and
    ldy.  Keyword arguments are the epilogue's (act, act_col0, residual,
    gate, norm_col0, norm_col1, norm_weight, norm_eps); a residual has out's
    row stride."""
    a = _strided_args(dict(x=x, packed=packed, scales=scales, bias=bias, y=out))
    e = _epilogue(dict(epilogue, y=out), strided=True)
    _check(lib().tern_linear_strided(ctypes.byref(a), ctypes.byref(e), _stream(stream)))
    return out


def linear_batch_strided(problems: Sequence[dict], stream=None) -> None:
    """tern_linear_batch_strided over dicts as linear_batch_epilogue's, with x
    and y possibly row-strided views."""
    n = max(1, len(problems))
    args, epis = (LinearStridedArgs * n)(), (Epilogue * n)()
    for i, p in enumerate(problems):
        args[i] = _strided_args(p)
        epis[i] = _epilogue(p, strided=True)
    _check(lib().tern_linear_batch_strided(args, epis, len(problems), _stream(stream)))


def _launch_on(ts, stream) -> int:
    """The library launches on the current device: every tensor has to live
    there.  Returns the raw stream to launch on; where that is not the current
    one, the caching allocator is told that the tensors are in use on it."""
    dev = -2
    for t in ts:
        if t is not None:
            d = t.get_device()  # -1 on the host
            if d != dev:
                if d < 0 or dev >= 0 or d != torch.cuda.current_device():
                    raise ValueError(f"every tensor must be on the current CUDA device; got one on {t.device}")
                dev = d
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(dev)
    if stream.device.index != dev:
        raise ValueError(f"the stream belongs to device {stream.device.index}, the tensors to {dev}")
    if stream != torch.cuda.current_stream():
        for t in ts:
            if t is not None:
                t.record_stream(stream)
    return stream.cuda_stream


def _bf16(name: str, t: torch.Tensor, dims) -> tuple:
    """t's strides, once it is known to be bf16 with adjacent channels."""
    s = t.stride()
    if t.dtype is not torch.bfloat16 or len(s) not in dims or (s[-1] != 1 and t.shape[-1] > 1):
        raise ValueError(f"{name} must be bf16 with {' or '.join(map(str, dims))} dimensions and adjacent channels; got "
                         f"{t.dtype}, shape {tuple(t.shape)}, strides {s}")
    return s


def rope_table(ids: torch.Tensor, axes: Sequence[int], theta: float = 10000.0, out: Optional[torch.Tensor] = None,
               stream=None) -> torch.Tensor:
    """tern_rope_table: fp32 [L, P, 2] (cos, sin) of token positions ids fp32
    [L, len(axes)], P = sum(axes) / 2: axis a owns axes[a] channels, pair i of
    it turning by ids[:, a] * theta^(-2 i / axes[a]).  The table that `rope`
    and (with P = 64) the linears' rope_cs take."""
    n = len(axes)
    shape = ids.shape
    if ids.dtype is not torch.float32 or len(shape) != 2 or shape[1] != n or not ids.is_contiguous():
        raise ValueError(f"ids must be contiguous fp32 [L, {n}], got {ids.dtype} {tuple(shape)}")
    L, P = shape[0], sum(axes) // 2
    raw = _launch_on((ids, out), stream)
    if out is None:
        out = _empty(L, P, 2, dtype=torch.float32, device=ids.device, stream=stream)
    elif out.dtype is not torch.float32 or out.shape != (L, P, 2) or not out.is_contiguous():
        raise ValueError(f"out must be contiguous fp32 [{L}, {P}, 2]")
    _check(lib().tern_rope_table(ids.data_ptr(), L, n, struct.pack(f"{n}i", *axes), float(theta), out.data_ptr(), raw))
    return out


def rope(xs: Sequence[torch.Tensor], cs: torch.Tensor, halves: bool = False,
         outs: Optional[Sequence[torch.Tensor]] = None, stream=None):
    """tern_rope: the heads of up to four bf16 tensors [L, H, D] (or all
    [B, L, H, D]) of the same tokens, any strides with adjacent channels,
    rotated by cs fp32 [L, P, 2] (or [B * L, P, 2]): channels 2j and 2j + 1, or
    with `halves` j and P + j, turn by pair j; channels from 2P on are copied.
    Returns the rotated tensors (new and contiguous, or `outs`; an element of
    `outs` may be its input)."""
    if not xs:
        return []
    shape = xs[0].shape
    nd = len(shape)
    parts = []  # (address, heads, strides) of each
    for x in xs:
        st = _bf16("x", x, (nd,) if nd == 3 or nd == 4 else (3, 4))
        sh = x.shape
        if sh[0] != shape[0] or sh[-1] != shape[-1] or (nd == 4 and sh[1] != shape[1]):
            raise ValueError("the tensors must share their tokens and head size")
        parts.append((x.data_ptr(), sh[-2], st if nd == 4 else (0, *st)))
    table = cs.shape
    if cs.dtype is not torch.float32 or len(table) != 3 or table[2] != 2 or not cs.is_contiguous():
        raise ValueError("cs must be contiguous fp32 [rows, P, 2]")
    raw = _launch_on((*xs, cs, *(outs or ())), stream)
    B, L = (shape[0], shape[1]) if nd == 4 else (1, shape[0])
    D = shape[-1]
    args = []
    if outs is None:
        outs = [_empty_as(x, stream) for x in xs]
        for y, (at, heads, sx) in zip(outs, parts):
            args += (at, y.data_ptr(), heads, sx[0], sx[1], sx[2], L * heads * D, heads * D, D)
    else:
        if len(outs) != len(xs):
            raise ValueError("one output per tensor")
        for x, y, (at, heads, sx) in zip(xs, outs, parts):
            sy = y.stride()
            if y.shape != x.shape or y.dtype is not torch.bfloat16 or (sy[-1] != 1 and D > 1):
                raise ValueError("an output is bf16 of its input's shape with adjacent channels")
            if nd == 3:
                sy = (0, *sy)
            args += (at, y.data_ptr(), heads, sx[0], sx[1], sx[2], sy[0], sy[1], sy[2])
    _check(lib().tern_rope(struct.pack("2P7q" * len(xs), *args), len(xs), B, L, D, cs.data_ptr(), table[0],
                           table[1], 1 if halves else 0, raw))
    return list(outs)


def attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, scale: Optional[float] = None,
              kv_len: Optional[torch.Tensor] = None, key_mask: Optional[torch.Tensor] = None,
              out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """tern_attention: softmax(scale q k^T) v of q bf16 [B, Lq, H, D] to k, v
    bf16 [B, Lk, Hkv, D] (or all without B), any strides with adjacent
    channels; H / Hkv query heads share a key-value head; scale defaults to
    1 / sqrt(D).  kv_len int32 [B] and key_mask bool or uint8 [B, Lk] (without
    B: [1] and [Lk]) say which keys count; a batch entry without one gives
    zeros.  Where `attention_plan` says tiles, probabilities meet v as bf16;
    all else is fp32.  Returns [B, Lq, H, D] (contiguous, or `out`)."""
    sq, sk, sv = _bf16("q", q, (3, 4)), _bf16("k", k, (3, 4)), _bf16("v", v, (3, 4))
    nd = len(sq)
    if len(sk) != nd or len(sv) != nd:
        raise ValueError("q, k and v must all have a batch dimension, or none")
    qs, ks = q.shape, k.shape
    if nd == 4:
        (B, Lq, H, D), (Bk, Lk, Hkv, Dk) = qs, ks
    else:
        (Lq, H, D), (Lk, Hkv, Dk), B, Bk = qs, ks, 1, 1
        sq, sk, sv = (0, *sq), (0, *sk), (0, *sv)
    if v.shape != ks or Dk != D or Bk != B:
        raise ValueError(f"q {tuple(qs)}, k {tuple(ks)} and v {tuple(v.shape)} do not fit")
    lens = mask = mask_ld = 0
    if kv_len is not None:
        if kv_len.dtype is not torch.int32 or kv_len.shape != (B,) or not kv_len.is_contiguous():
            raise ValueError(f"kv_len must be contiguous int32 [{B}]")
        lens = kv_len.data_ptr()
    if key_mask is not None:
        if (key_mask.dtype not in (torch.bool, torch.uint8) or key_mask.shape != ((B, Lk) if nd == 4 else (Lk,))
                or (Lk > 1 and key_mask.stride(-1) != 1)):
            raise ValueError(f"key_mask must be bool or uint8 {'[B, Lk]' if nd == 4 else '[Lk]'} with adjacent keys")
        mask, mask_ld = key_mask.data_ptr(), key_mask.stride(0) if nd == 4 else 0
    raw = _launch_on((q, k, v, kv_len, key_mask, out), stream)
    if out is None:
        out = _empty_as(q, stream)
        so = out.stride()
    else:
        so = _bf16("out", out, (nd,))
        if out.shape != qs:
            raise ValueError("out has q's shape")
    if nd == 3:
        so = (0, *so)
    _check(lib().tern_attention(
        _ATTENTION.pack(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), B, Lq, Lk, H, Hkv, D, *sq[:3], *sk[:3],
                        *sv[:3], *so[:3], D ** -0.5 if scale is None else scale, lens, mask, mask_ld), raw))
    return out


def attention_plan(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, sms: int = 0):
    """tern_attention_plan: (ATTENTION_* kernel, CTAs that share the keys of a
    unit) that `attention` takes for tensors of these shapes and strides (on any
    device) on a GPU of `sms` SMs (0: the current one)."""
    q, k, v = (t if t.dim() == 4 else t[None] for t in (q, k, v))
    (B, Lq, H, D), (Lk, Hkv) = q.shape, k.shape[1:3]
    args = _ATTENTION.pack(0, 0, 0, 0, B, Lq, Lk, H, Hkv, D, *q.stride()[:3], *k.stride()[:3], *v.stride()[:3], 0, 0, 0, 1.0,
                           0, 0, 0)
    kernel, ctas = ctypes.c_int(), ctypes.c_int()
    _check(lib().tern_attention_plan(args, sms, ctypes.byref(kernel), ctypes.byref(ctas)))
    return kernel.value, ctas.value


def gated_residual_norm(x: torch.Tensor, o: torch.Tensor, *, gate: Optional[torch.Tensor] = None,
                        gate_tanh: bool = False, residual_scale: float = 1.0, post_norm: int = NORM_NONE,
                        post_weight: Optional[torch.Tensor] = None, post_eps: float = 1e-6, pre_norm: int = NORM_NONE,
                        pre_weight: Optional[torch.Tensor] = None, pre_eps: float = 1e-6,
                        scale: Optional[torch.Tensor] = None, shift: Optional[torch.Tensor] = None,
                        tokens_per_row: Optional[int] = None, x_out: Optional[torch.Tensor] = None,
                        h: Optional[torch.Tensor] = None, stream=None):
    """tern_gated_residual_norm: r = residual_scale * x + gate * post(o) per
    token row of x, o bf16 [M, K], stored to x_out, and h = pre(r) * (1 +
    scale) + shift.  gate, scale and shift are bf16 [G, K] (or [K]) rows
    equally far apart, row m // tokens_per_row each (default: row 0 for all),
    e.g. slices of a modulation output; the norms are NORM_* values.  x_out
    may be x, h may be o (or the reverse).  Returns (x_out, h); h is None, and
    not computed, where neither a pre norm, scale and shift, nor h is given."""
    sx, so = _bf16("x", x, (2,)), _bf16("o", o, (2,))
    shape = x.shape
    M, K = shape
    if o.shape != shape:
        raise ValueError("x and o must have one shape")
    T = max(M, 1) if tokens_per_row is None else int(tokens_per_row)
    G = -(-M // T) if T > 0 else 0
    mod_ld = K
    apart = None
    at = [0, 0, 0]  # addresses of the modulation rows
    for i, t in enumerate((gate, scale, shift)):
        if t is not None:
            s = _bf16("gate, scale or shift", t, (1, 2))
            sh = t.shape
            if sh[-1] != K or (sh[0] if len(sh) == 2 else 1) < G:
                raise ValueError(f"{('gate', 'scale', 'shift')[i]} holds fewer than the {G} modulation rows of {K} values that "
                                 f"{M} rows at {T} tokens per row need")
            if G > 1:
                if apart is not None and s[0] != apart:
                    raise ValueError("gate, scale and shift rows must be the same distance apart")
                apart = mod_ld = s[0]
            at[i] = t.data_ptr()
    post_at = pre_at = 0
    if post_weight is not None:
        _bf16("post_weight", post_weight, (1,))
        post_at = post_weight.data_ptr()
    if pre_weight is not None:
        _bf16("pre_weight", pre_weight, (1,))
        pre_at = pre_weight.data_ptr()
    for w in (post_weight, pre_weight):
        if w is not None and w.shape[0] != K:
            raise ValueError(f"post_weight and pre_weight must hold {K} values")
    raw = _launch_on((x, o, gate, scale, shift, post_weight, pre_weight, x_out, h), stream)
    ld_xo = ld_h = K
    if x_out is None:
        x_out = _empty_as(x, stream)
    else:
        ld_xo = _bf16("x_out", x_out, (2,))[0]
        if x_out.shape != shape:
            raise ValueError("x_out has x's shape")
    if h is not None:
        ld_h = _bf16("h", h, (2,))[0]
        if h.shape != shape:
            raise ValueError("h has x's shape")
    elif pre_norm != NORM_NONE or scale is not None or shift is not None:
        h = _empty_as(x, stream)
    ld_x, ld_o = sx[0], so[0]
    if M <= 1:
        ld_x = ld_o = ld_xo = ld_h = K
    _check(lib().tern_gated_residual_norm(
        _RESIDUAL_NORM.pack(x.data_ptr(), o.data_ptr(), x_out.data_ptr(), 0 if h is None else h.data_ptr(), M, K, ld_x, ld_o,
                            ld_xo, ld_h, residual_scale, post_norm, post_at, post_eps, at[0], 1 if gate_tanh else 0, pre_norm,
                            pre_at, pre_eps, at[1], at[2], mod_ld, T), raw))
    return x_out, h


def dequantize(packed: torch.Tensor, scales: torch.Tensor, K: int, out: Optional[torch.Tensor] = None,
               stream=None) -> torch.Tensor:
    """tern_dequantize: codes -> bf16 [N,K] with W'[n,k] = T[n,k] * s_n."""
    N = scales.shape[0]
    if out is None:
        out = _empty(N, K, dtype=torch.bfloat16, device=scales.device, stream=stream)
    _check(lib().tern_dequantize(_ptr(packed), _ptr(scales), N, K, _ptr(out), _stream(stream)))
    return out


def device_status(stream=None) -> int:
    """tern_get_device_status (synchronises the stream); returns the raw status."""
    return int(lib().tern_get_device_status(_stream(stream)))


def set_wait_limit_ns(limit_ns: int) -> None:
    lib().tern_set_wait_limit_ns(int(limit_ns))


def selftest_wait_timeout(limit_ns: int, stream=None) -> None:
    _check(lib().tern_selftest_wait_timeout(int(limit_ns), _stream(stream)))


def status_string(status: int) -> str:
    return lib().tern_status_string(int(status)).decode()
