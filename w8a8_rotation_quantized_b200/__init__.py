"""INT8 ConvRot (W8A8, Hadamard-256) linear layer on B200: Python binding of libh3q.so.

The functions carry the C ABI's names (include/h3q.h) and only marshal
arguments: torch tensors in device memory become pointers, the current CUDA
stream becomes the stream argument, and a non-OK status raises H3QError. Every
step of the computation runs in the library's kernels. There is no fallback:
if the library is missing or cannot be loaded, importing this package fails.
"""
from __future__ import annotations

import ctypes
import os
import re

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libh3q.so")
HEADER = os.path.join(os.path.dirname(HERE), "include", "h3q.h")

H3Q_OK, H3Q_ERR_INVALID_ARG, H3Q_ERR_UNSUPPORTED, H3Q_ERR_CUDA, H3Q_ERR_TIMEOUT = range(5)
H3Q_EPI_NONE, H3Q_EPI_SWIGLU = 0, 1
H3Q_DTYPE_BF16, H3Q_DTYPE_F32 = 0, 1
H3Q_MAX_K = 16384

if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is missing: build it with `python w8a8_rotation_quantized_b200/build.py` "
                      "(or __graft_entry__.build())")

lib = ctypes.CDLL(LIB_PATH)

_P, _I64, _SZ, _INT, _U64 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t, ctypes.c_int, ctypes.c_uint64
_SIGS = {
    "h3q_rotate_quant": (_INT, [_P, _I64, _I64, _P, _P, _P]),
    "h3q_prepare_weight": (_INT, [_P, _I64, _I64, _P, _P, _P]),
    "h3q_linear_w8a8": (_INT, [_P, _P, _I64, _I64, _P, _P, _I64, _P, _INT, _P, _P]),
    "h3q_ffn_workspace_size": (_SZ, [_I64, _I64, _I64]),
    "h3q_ffn": (_INT, [_P, _I64, _I64, _P, _P, _P, _I64, _P, _P, _P, _P, _P, _SZ, _P]),
    "h3q_ffn_static_scratch": (_INT, [_P, _I64, _I64, _P, _P, _P, _I64, _P, _P, _P, _P, _P]),
    "h3q_lora_workspace_size": (_SZ, [_I64, _I64]),
    "h3q_lora_merge": (_INT, [_P, _P, _I64, _I64, _P, _P, _I64, ctypes.c_float, _P, _SZ, _P]),
    "h3q_nvfp4_sf_bytes": (_SZ, [_I64, _I64]),
    "h3q_nvfp4_quantize": (_INT, [_P, _INT, _I64, _I64, _P, _P, _P, _P]),
    "h3q_linear_nvfp4": (_INT, [_P, _P, _P, _I64, _I64, _P, _P, _P, _I64, _P, _INT, _P, _P]),
    "h3q_gemm_nvfp4_f32": (_INT, [_P, _P, _I64, _I64, _P, _P, _I64, _P, _P]),
    "h3q_attention_workspace_size": (_SZ, [_I64, _I64]),
    "h3q_attention_int8": (_INT, [_P, _P, _P, _I64, _I64, _I64, _P, _I64, _P, _SZ, _P]),
    "h3q_attention_prep": (_INT, [_P, _P, _P, _I64, _I64, _I64, _P, _P, _P, _P, _P, _P]),
    "h3q_fp8_quantize": (_INT, [_P, _INT, _I64, _I64, _P, _P, _P]),
    "h3q_fp8_prepare_weight": (_INT, [_P, _INT, _I64, _I64, _P, _P, _P]),
    "h3q_linear_fp8": (_INT, [_P, _P, _I64, _I64, _P, _P, _I64, _P, _INT, _P, _P]),
    "h3q_linear_fp8_swiglu_quant": (_INT, [_P, _P, _I64, _I64, _P, _P, _I64, _P, _P, _P, _P]),
    "h3q_test_fp8_plan": (_INT, [_I64, _I64, _I64, _INT, _INT, _P]),
    "h3q_test_stalled_linear_fp8": (_INT, [_P, _P, _I64, _I64, _P, _P, _I64, _INT, _P, _U64, _P]),
    "h3q_qk_norm_rope": (_INT, [_P, _P, _I64, _I64, _I64, _I64, _I64, _I64, _P, _P, ctypes.c_float, _P, _P, _I64,
                                _I64, _INT, _P, _P, _P, _I64, _I64, _P]),
    "h3q_gemm_s32": (_INT, [_P, _P, _I64, _I64, _I64, _P, _P]),
    "h3q_get_device_status": (_INT, [_P]),
    "h3q_set_wait_limit_ns": (None, [_U64]),
    "h3q_test_stalled_wait": (_INT, [_U64, _P]),
    "h3q_status_string": (ctypes.c_char_p, [_INT]),
    "h3q_version": (ctypes.c_char_p, []),
}
for _name, (_res, _args) in _SIGS.items():
    _fn = getattr(lib, _name)
    _fn.restype, _fn.argtypes = _res, _args


class H3QError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {lib.h3q_status_string(status).decode()} (status {status})")


def header_functions() -> list[str]:
    """Names of the functions include/h3q.h declares."""
    text = open(HEADER).read()
    return sorted(set(re.findall(r"^\s*(?:const\s+)?[\w\s\*]*?\b(h3q_\w+)\s*\(", text, flags=re.M)))


def _check(status: int, where: str) -> None:
    if status != H3Q_OK:
        raise H3QError(status, where)


def _dtypes():
    import torch
    return {"bf16": torch.bfloat16, "f32": torch.float32, "i8": torch.int8, "u8": torch.uint8,
            "i32": torch.int32, "e4m3": torch.float8_e4m3fn}


def _need(where: str, name: str, t, dtype: str, shape, device=None, dense: bool = True):
    """Raises ValueError unless t is a CUDA tensor of `dtype` and `shape` (None entries
    match any size), dense (or, with dense=False, with unit column stride) and, when
    given, on `device`. The kernels index their operands from the sizes alone, so a
    tensor of another shape or layout would be read or written out of bounds."""
    if t is None:
        raise ValueError(f"{where}: {name} is required")
    want = _dtypes()[dtype]
    if t.dtype != want:
        raise ValueError(f"{where}: {name} must be {want}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{where}: {name} must be a CUDA tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{where}: {name} is on {t.device}, the other operands on {device}")
    if len(t.shape) != len(shape) or any(w is not None and int(g) != int(w) for g, w in zip(t.shape, shape)):
        raise ValueError(f"{where}: {name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if dense and not t.is_contiguous():
        raise ValueError(f"{where}: {name} must be contiguous (row-major, dense)")
    if not dense and t.dim() == 2 and t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError(f"{where}: {name} must have unit column stride")
    return t


def _nbytes(where: str, name: str, t, device) -> int:
    """Byte size of a caller-owned scratch tensor (any dtype, contiguous, on `device`)."""
    if t is None or not t.is_cuda or t.device != device or not t.is_contiguous():
        raise ValueError(f"{where}: {name} must be a contiguous CUDA tensor on {device}")
    return t.numel() * t.element_size()


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(stream):
    if stream is not None:
        return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    import torch
    return torch.cuda.current_stream().cuda_stream


def h3q_rotate_quant(x, xq, sx, stream=None) -> None:
    """x bf16 [M, K] -> xq int8 [M, K] (rotated codes), sx fp32 [M]."""
    w = "h3q_rotate_quant"
    M, K = _need(w, "x", x, "bf16", (None, None)).shape
    _need(w, "xq", xq, "i8", (M, K), x.device)
    _need(w, "sx", sx, "f32", (M,), x.device)
    _check(lib.h3q_rotate_quant(_ptr(x), M, K, _ptr(xq), _ptr(sx), _stream(stream)), "h3q_rotate_quant")


def h3q_prepare_weight(w, wq, sw, stream=None) -> None:
    """w fp32 [N, K] -> wq int8 [N, K] (rotated along K), sw fp32 [N]."""
    wh = "h3q_prepare_weight"
    N, K = _need(wh, "w", w, "f32", (None, None)).shape
    _need(wh, "wq", wq, "i8", (N, K), w.device)
    _need(wh, "sw", sw, "f32", (N,), w.device)
    _check(lib.h3q_prepare_weight(_ptr(w), N, K, _ptr(wq), _ptr(sw), _stream(stream)), "h3q_prepare_weight")


def h3q_linear_w8a8(xq, sx, wq, sw, y, bias=None, epilogue=H3Q_EPI_NONE, stream=None) -> None:
    """y bf16 = rescale(xq @ wq^T) (+ bias); SwiGLU epilogue: y [M, N/2]."""
    w = "h3q_linear_w8a8"
    M, K = _need(w, "xq", xq, "i8", (None, None)).shape
    dev = xq.device
    N = _need(w, "wq", wq, "i8", (None, K), dev).shape[0]
    _need(w, "sx", sx, "f32", (M,), dev)
    _need(w, "sw", sw, "f32", (N,), dev)
    if bias is not None:
        _need(w, "bias", bias, "bf16", (N,), dev)
    _need(w, "y", y, "bf16", (M, N // 2 if int(epilogue) == H3Q_EPI_SWIGLU else N), dev)
    _check(lib.h3q_linear_w8a8(_ptr(xq), _ptr(sx), M, K, _ptr(wq), _ptr(sw), N, _ptr(bias), int(epilogue),
                               _ptr(y), _stream(stream)), "h3q_linear_w8a8")


def h3q_ffn_workspace_size(M: int, K: int, F: int) -> int:
    return int(lib.h3q_ffn_workspace_size(M, K, F))


def _ffn_operands(w, x, w_gu, s_gu, w_down, s_down, y, b_gu, b_down):
    M, K = _need(w, "x", x, "bf16", (None, None)).shape
    dev = x.device
    F2 = _need(w, "w_gu", w_gu, "i8", (None, K), dev).shape[0]
    if F2 % 2:
        raise ValueError(f"{w}: w_gu must have an even row count (gate rows, then up rows), got {F2}")
    F = F2 // 2
    _need(w, "s_gu", s_gu, "f32", (2 * F,), dev)
    _need(w, "w_down", w_down, "i8", (K, F), dev)
    _need(w, "s_down", s_down, "f32", (K,), dev)
    _need(w, "y", y, "bf16", (M, K), dev)
    if b_gu is not None:
        _need(w, "b_gu", b_gu, "bf16", (2 * F,), dev)
    if b_down is not None:
        _need(w, "b_down", b_down, "bf16", (K,), dev)
    return M, K, F


def h3q_ffn(x, w_gu, s_gu, w_down, s_down, y, workspace, b_gu=None, b_down=None, stream=None) -> None:
    """y [M, K] = down(rotquant(swiglu(gate_up(rotquant(x)))))."""
    w = "h3q_ffn"
    M, K, F = _ffn_operands(w, x, w_gu, s_gu, w_down, s_down, y, b_gu, b_down)
    nbytes = _nbytes(w, "workspace", workspace, x.device)
    _check(lib.h3q_ffn(_ptr(x), M, K, _ptr(w_gu), _ptr(s_gu), _ptr(b_gu), F, _ptr(w_down), _ptr(s_down),
                       _ptr(b_down), _ptr(y), _ptr(workspace), nbytes, _stream(stream)), "h3q_ffn")


H3Q_STATIC_SCRATCH_BYTES = 64 << 20


def h3q_ffn_static_scratch(x, w_gu, s_gu, w_down, s_down, y, b_gu=None, b_down=None, stream=None) -> None:
    """h3q_ffn without a workspace, for callers that cannot allocate device memory:
    the intermediates live in the library's fixed 64 MiB device array, shared by
    all calls (calls that may overlap on the GPU must be serialized)."""
    M, K, F = _ffn_operands("h3q_ffn_static_scratch", x, w_gu, s_gu, w_down, s_down, y, b_gu, b_down)
    _check(lib.h3q_ffn_static_scratch(_ptr(x), M, K, _ptr(w_gu), _ptr(s_gu), _ptr(b_gu), F, _ptr(w_down),
                                      _ptr(s_down), _ptr(b_down), _ptr(y), _stream(stream)),
           "h3q_ffn_static_scratch")


H3Q_LORA_MAX_RANK = 512


def h3q_lora_workspace_size(r: int, K: int) -> int:
    return int(lib.h3q_lora_workspace_size(r, K))


def h3q_lora_merge(wq, sw, lora_a, lora_b, alpha: float, workspace, stream=None) -> None:
    """Merge alpha * lora_b @ lora_a (rotated along K) into the int8 weights
    wq [N, K] / sw [N], in place. lora_a [r, K], lora_b [N, r] fp32."""
    w = "h3q_lora_merge"
    N, K = _need(w, "wq", wq, "i8", (None, None)).shape
    dev = wq.device
    _need(w, "sw", sw, "f32", (N,), dev)
    r = _need(w, "lora_a", lora_a, "f32", (None, K), dev).shape[0]
    _need(w, "lora_b", lora_b, "f32", (N, r), dev)
    nbytes = _nbytes(w, "workspace", workspace, dev)
    _check(lib.h3q_lora_merge(_ptr(wq), _ptr(sw), N, K, _ptr(lora_a), _ptr(lora_b), r, float(alpha),
                              _ptr(workspace), nbytes, _stream(stream)), "h3q_lora_merge")


def h3q_nvfp4_sf_bytes(rows: int, K: int) -> int:
    return int(lib.h3q_nvfp4_sf_bytes(rows, K))


def h3q_nvfp4_quantize(x, codes, sf, scale, stream=None) -> None:
    """x [rows, K] bf16 or fp32 -> codes uint8 [rows, K/2], sf uint8 [h3q_nvfp4_sf_bytes],
    scale fp32 [2] (max|x|, s_enc)."""
    import torch
    w = "h3q_nvfp4_quantize"
    rows, K = _need(w, "x", x, "bf16" if x.dtype == torch.bfloat16 else "f32", (None, None)).shape
    dt = H3Q_DTYPE_BF16 if x.dtype == torch.bfloat16 else H3Q_DTYPE_F32
    _need(w, "codes", codes, "u8", (rows, K // 2), x.device)
    _need(w, "sf", sf, "u8", (h3q_nvfp4_sf_bytes(rows, K),), x.device)
    _need(w, "scale", scale, "f32", (2,), x.device)
    _check(lib.h3q_nvfp4_quantize(_ptr(x), dt, rows, K, _ptr(codes), _ptr(sf), _ptr(scale), _stream(stream)),
           "h3q_nvfp4_quantize")


def _nvfp4_operands(w, xc, xsf, wc, wsf):
    M, K2 = _need(w, "xc", xc, "u8", (None, None)).shape
    dev = xc.device
    N = _need(w, "wc", wc, "u8", (None, K2), dev).shape[0]
    _need(w, "xsf", xsf, "u8", (h3q_nvfp4_sf_bytes(M, 2 * K2),), dev)
    _need(w, "wsf", wsf, "u8", (h3q_nvfp4_sf_bytes(N, 2 * K2),), dev)
    return M, N, K2


def h3q_linear_nvfp4(xc, xsf, x_scale, wc, wsf, w_scale, y, bias=None, epilogue=H3Q_EPI_NONE, stream=None) -> None:
    """y bf16 = NVFP4 linear of x (codes xc [M, K/2]) with w (codes wc [N, K/2])."""
    w = "h3q_linear_nvfp4"
    M, N, K2 = _nvfp4_operands(w, xc, xsf, wc, wsf)
    _need(w, "x_scale", x_scale, "f32", (2,), xc.device)
    _need(w, "w_scale", w_scale, "f32", (2,), xc.device)
    if bias is not None:
        _need(w, "bias", bias, "bf16", (N,), xc.device)
    _need(w, "y", y, "bf16", (M, N // 2 if int(epilogue) == H3Q_EPI_SWIGLU else N), xc.device)
    _check(lib.h3q_linear_nvfp4(_ptr(xc), _ptr(xsf), _ptr(x_scale), M, 2 * K2, _ptr(wc), _ptr(wsf), _ptr(w_scale), N,
                                _ptr(bias), int(epilogue), _ptr(y), _stream(stream)), "h3q_linear_nvfp4")


def h3q_gemm_nvfp4_f32(xc, xsf, wc, wsf, acc, stream=None) -> None:
    """acc fp32 [M, N]: the raw NVFP4 accumulators (test hook)."""
    w = "h3q_gemm_nvfp4_f32"
    M, N, K2 = _nvfp4_operands(w, xc, xsf, wc, wsf)
    _need(w, "acc", acc, "f32", (M, N), xc.device)
    _check(lib.h3q_gemm_nvfp4_f32(_ptr(xc), _ptr(xsf), M, 2 * K2, _ptr(wc), _ptr(wsf), N, _ptr(acc),
                                  _stream(stream)), "h3q_gemm_nvfp4_f32")


def h3q_attention_workspace_size(S: int, H: int) -> int:
    return int(lib.h3q_attention_workspace_size(S, H))


def _ld(t):
    return t.stride(0)


def _attention_inputs(w, q, k, v, H):
    """q, k, v: [S, >= 128 H] bf16 views with unit column stride and one common row stride."""
    S = _need(w, "q", q, "bf16", (None, None), dense=False).shape[0]
    for name, t in (("k", k), ("v", v)):
        _need(w, name, t, "bf16", (S, None), q.device, dense=False)
    for name, t in (("q", q), ("k", k), ("v", v)):
        if t.shape[1] < 128 * H:
            raise ValueError(f"{w}: {name} must have at least {128 * H} columns, got {t.shape[1]}")
        if t.stride(0) != q.stride(0):
            raise ValueError(f"{w}: q, k and v must share one row stride")
    return S


def h3q_attention_int8(q, k, v, H, out, workspace, stream=None) -> None:
    """out [S, >= 128 H] bf16 = int8 attention of q, k, v ([S, ld] bf16 views, head h
    at columns h*128; q, k, v may be column slices of one matrix)."""
    w = "h3q_attention_int8"
    S = _attention_inputs(w, q, k, v, H)
    _need(w, "out", out, "bf16", (S, None), q.device, dense=False)
    if out.shape[1] < 128 * H:
        raise ValueError(f"{w}: out must have at least {128 * H} columns, got {out.shape[1]}")
    nbytes = _nbytes(w, "workspace", workspace, q.device)
    _check(lib.h3q_attention_int8(_ptr(q), _ptr(k), _ptr(v), S, H, _ld(q), _ptr(out), _ld(out), _ptr(workspace),
                                  nbytes, _stream(stream)), "h3q_attention_int8")


def h3q_attention_prep(q, k, v, H, qq, qs, kq, ks, vt, stream=None) -> None:
    """The attention's input pass: int8 Q codes and scales per token and head, K codes per
    head with one scale per block of 128 keys (ks [H, ceil(S/128)]), V^T per head."""
    w = "h3q_attention_prep"
    S = _attention_inputs(w, q, k, v, H)
    dev = q.device
    _need(w, "qq", qq, "i8", (H, S, 128), dev)
    _need(w, "kq", kq, "i8", (H, S, 128), dev)
    _need(w, "qs", qs, "f32", (H, S), dev)
    _need(w, "ks", ks, "f32", (H, (S + 127) // 128), dev)
    _need(w, "vt", vt, "bf16", (H * 128, S), dev)
    _check(lib.h3q_attention_prep(_ptr(q), _ptr(k), _ptr(v), S, H, _ld(q), _ptr(qq), _ptr(qs), _ptr(kq), _ptr(ks),
                                  _ptr(vt), _stream(stream)), "h3q_attention_prep")


# The fp8 and query/key calls are also made for single tokens, where the checks of their
# operands would cost more than the kernel: they test each operand in one expression and
# come to the checks above only to name the fault.
_torch = _raw_stream = _current_device = None


def _t():
    """torch, imported on first use."""
    global _torch, _raw_stream, _current_device
    if _torch is None:
        import torch
        # the handles without the Stream object around them, where this torch has them
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
            lambda index: torch.cuda.current_stream(index).cuda_stream)
        _current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
        _torch = torch
    return _torch


def _is(t, dtype, shape, index):
    """t is a dense tensor of this dtype and shape on CUDA device `index`."""
    return (t is not None and t.dtype is dtype and t.get_device() == index and t.shape == shape
            and t.is_contiguous())


def _row_stride(t, dtype, S, width, index):
    """The row stride of t if it is a [S, >= width] view of this dtype with unit column
    stride on CUDA device `index` (of a single row, whose stride means nothing, its width);
    else None."""
    if t is not None and t.dtype is dtype and t.get_device() == index:
        shape, stride = t.shape, t.stride()
        if len(shape) == 2 and shape[0] == S and shape[1] >= width and stride[1] == 1:
            return stride[0] if S > 1 else width
    return None


def _run(name, fn, index, stream, *args):
    """Calls fn(*args, stream) with CUDA device `index` current, on `stream` or that device's
    current stream."""
    if stream is None:
        stream = _raw_stream(index)
    else:
        stream = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    if _current_device() == index:
        status = fn(*args, stream)
    else:
        with _t().cuda.device(index):
            status = fn(*args, stream)
    if status != H3Q_OK:
        raise H3QError(status, name)


def _fp8_quantizer(w, fn, x, codes, scales, weight, stream):
    torch = _t()
    names = ("w", "wq", "sw") if weight else ("x", "xq", "sx")
    kind = "bf16" if x is not None and x.dtype is torch.bfloat16 else "f32"
    if x is None or x.dim() != 2 or not x.is_cuda or x.dtype not in (torch.bfloat16, torch.float32):
        _need(w, names[0], x, kind, (None, None))
    rows, K = x.shape
    index = x.get_device()
    KB = (K + 127) // 128
    shape = ((rows + 127) // 128, KB) if weight else (KB, rows)
    if not (x.is_contiguous() and _is(codes, torch.float8_e4m3fn, (rows, K), index)
            and _is(scales, torch.float32, shape, index)):
        _need(w, names[0], x, kind, (None, None))
        _need(w, names[1], codes, "e4m3", (rows, K), x.device)
        _need(w, names[2], scales, "f32", shape, x.device)
    _run(w, fn, index, stream, x.data_ptr(), H3Q_DTYPE_BF16 if kind == "bf16" else H3Q_DTYPE_F32, rows, K,
         codes.data_ptr(), scales.data_ptr())


def h3q_fp8_quantize(x, xq, sx, stream=None) -> None:
    """x [M, K] bf16 or fp32 -> xq float8_e4m3fn [M, K], sx fp32 [ceil(K/128), M]: one scale
    per token and 128 elements."""
    _fp8_quantizer("h3q_fp8_quantize", lib.h3q_fp8_quantize, x, xq, sx, False, stream)


def h3q_fp8_prepare_weight(w, wq, sw, stream=None) -> None:
    """w [N, K] bf16 or fp32 -> wq float8_e4m3fn [N, K], sw fp32 [ceil(N/128), ceil(K/128)]:
    one scale per 128 x 128 block."""
    _fp8_quantizer("h3q_fp8_prepare_weight", lib.h3q_fp8_prepare_weight, w, wq, sw, True, stream)


def _fp8_operands(w, xq, sx, wq, sw, bias, out, out_dtype, halved, sh=None):
    """M, K, N and the device's index of an fp8 product's operands; raises ValueError."""
    torch = _t()
    if xq is not None and wq is not None and xq.dim() == 2 and wq.dim() == 2 and xq.is_cuda:
        M, K = xq.shape
        N = wq.shape[0]
        index = xq.get_device()
        KB = (K + 127) // 128
        e4m3, f32 = torch.float8_e4m3fn, torch.float32
        out_shape = (M, N // 2 if halved else N)
        if (_is(xq, e4m3, (M, K), index) and _is(wq, e4m3, (N, K), index) and _is(sx, f32, (KB, M), index)
                and _is(sw, f32, ((N + 127) // 128, KB), index)
                and (bias is None or _is(bias, torch.bfloat16, (N,), index))
                and _is(out, torch.bfloat16 if out_dtype == "bf16" else e4m3, out_shape, index)
                and (out_dtype == "bf16" or _is(sh, f32, (N // 256, M), index))):
            return M, K, N, index
    M, K = _need(w, "xq", xq, "e4m3", (None, None)).shape
    dev = xq.device
    N = _need(w, "wq", wq, "e4m3", (None, K), dev).shape[0]
    KB = (K + 127) // 128
    _need(w, "sx", sx, "f32", (KB, M), dev)
    _need(w, "sw", sw, "f32", ((N + 127) // 128, KB), dev)
    if bias is not None:
        _need(w, "bias", bias, "bf16", (N,), dev)
    _need(w, "y" if out_dtype == "bf16" else "hq", out, out_dtype, (M, N // 2 if halved else N), dev)
    if out_dtype != "bf16":
        _need(w, "sh", sh, "f32", (N // 256, M), dev)
    return M, K, N, dev.index


def h3q_linear_fp8(xq, sx, wq, sw, y, bias=None, epilogue=H3Q_EPI_NONE, stream=None) -> None:
    """y bf16 [M, N] = block-scaled fp8 product of xq (sx) and wq (sw), + bias; SwiGLU
    epilogue: y [M, N/2]."""
    w = "h3q_linear_fp8"
    epilogue = int(epilogue)
    M, K, N, index = _fp8_operands(w, xq, sx, wq, sw, bias, y, "bf16", epilogue == H3Q_EPI_SWIGLU)
    _run(w, lib.h3q_linear_fp8, index, stream, xq.data_ptr(), sx.data_ptr(), M, K, wq.data_ptr(), sw.data_ptr(), N,
         _ptr(bias), epilogue, y.data_ptr())


def h3q_linear_fp8_swiglu_quant(xq, sx, wq, sw, hq, sh, bias=None, stream=None) -> None:
    """hq float8_e4m3fn [M, F], sh fp32 [F/128, M] = quantized SwiGLU of the gate/up product
    (wq [2F, K], gate rows first): the operands of the down projection."""
    w = "h3q_linear_fp8_swiglu_quant"
    M, K, N, index = _fp8_operands(w, xq, sx, wq, sw, bias, hq, "e4m3", True, sh)
    _run(w, lib.h3q_linear_fp8_swiglu_quant, index, stream, xq.data_ptr(), sx.data_ptr(), M, K, wq.data_ptr(),
         sw.data_ptr(), N, _ptr(bias), hq.data_ptr(), sh.data_ptr())


def h3q_test_fp8_plan(M, K, N, epilogue=H3Q_EPI_NONE, sms=148):
    """(tokens of a tile, 0 for the large kernel; CTAs along K; stages; shared-memory bytes;
    tensor-memory columns) of an fp8 product on a GPU of `sms` SMs. Host only."""
    plan = (ctypes.c_int32 * 5)()
    _check(lib.h3q_test_fp8_plan(M, K, N, int(epilogue), sms, plan), "h3q_test_fp8_plan")
    return tuple(plan)


H3Q_QK_MAX_D = 256


def h3q_qk_norm_rope(q, k, Hq, Hk, D, cos, sin, q_out, k_out, q_weight=None, k_weight=None, positions=None,
                     eps=1e-6, interleaved=False, stream=None) -> None:
    """RMS norm of every head of q ([S, >= Hq D] bf16 view) and k ([S, >= Hk D], or None with
    Hk = 0), then the rotation by row positions[t] (int32 [S]; None: row t) of cos, sin
    (fp32 [P, rot/2]; None: no rotation). q_out, k_out: the same shapes, may be q and k."""
    w = "h3q_qk_norm_rope"
    torch = _t()
    bf16, f32 = torch.bfloat16, torch.float32
    if q is None or q.dim() != 2 or not q.is_cuda:
        _need(w, "q", q, "bf16", (None, None), dense=False)
    S, index = q.shape[0], q.get_device()
    ldq, ldqo = _row_stride(q, bf16, S, Hq * D, index), _row_stride(q_out, bf16, S, Hq * D, index)
    ldk = ldko = 0
    if Hk:
        ldk, ldko = _row_stride(k, bf16, S, Hk * D, index), _row_stride(k_out, bf16, S, Hk * D, index)
    if ldq is None or ldqo is None or ldk is None or ldko is None:
        views = [("q", q, Hq), ("q_out", q_out, Hq)] + ([("k", k, Hk), ("k_out", k_out, Hk)] if Hk else [])
        for name, t, heads in views:
            _need(w, name, t, "bf16", (S, None), q.device, dense=False)
            if t.shape[1] < heads * D:
                raise ValueError(f"{w}: {name} must have at least {heads * D} columns, got {t.shape[1]}")
        raise ValueError(f"{w}: q, q_out, k and k_out must be [S, columns] views with unit column stride")
    qw = kw = c = s = at = None  # optional operands' pointers
    P = half = 0
    if q_weight is not None:
        if not _is(q_weight, bf16, (D,), index):
            _need(w, "q_weight", q_weight, "bf16", (D,), q.device)
        qw = q_weight.data_ptr()
    if k_weight is not None:
        if not _is(k_weight, bf16, (D,), index):
            _need(w, "k_weight", k_weight, "bf16", (D,), q.device)
        kw = k_weight.data_ptr()
    if cos is not None:
        shape = cos.shape
        if len(shape) != 2 or not (_is(cos, f32, shape, index) and _is(sin, f32, shape, index)):
            _need(w, "cos", cos, "f32", (None, None), q.device)
            _need(w, "sin", sin, "f32", tuple(shape), q.device)
        P, half = shape
        c, s = cos.data_ptr(), sin.data_ptr()
    elif sin is not None:
        raise ValueError(f"{w}: sin without cos")
    if positions is not None:
        if not _is(positions, torch.int32, (S,), index):
            _need(w, "positions", positions, "i32", (S,), q.device)
        at = positions.data_ptr()
    _run(w, lib.h3q_qk_norm_rope, index, stream, q.data_ptr(), k.data_ptr() if Hk else None, S, Hq, Hk, D, ldq, ldk,
         qw, kw, eps, c, s, P, 2 * half, 1 if interleaved else 0, at, q_out.data_ptr(),
         k_out.data_ptr() if Hk else None, ldqo, ldko)


def h3q_gemm_s32(xq, wq, acc, stream=None) -> None:
    """acc int32 [M, N] = xq [M, K] @ wq [N, K]^T."""
    w = "h3q_gemm_s32"
    M, K = _need(w, "xq", xq, "i8", (None, None)).shape
    N = _need(w, "wq", wq, "i8", (None, K), xq.device).shape[0]
    _need(w, "acc", acc, "i32", (M, N), xq.device)
    _check(lib.h3q_gemm_s32(_ptr(xq), _ptr(wq), M, N, K, _ptr(acc), _stream(stream)), "h3q_gemm_s32")


def h3q_get_device_status(stream=None) -> int:
    return int(lib.h3q_get_device_status(_stream(stream)))


def h3q_set_wait_limit_ns(ns: int) -> None:
    lib.h3q_set_wait_limit_ns(int(ns))


def h3q_test_stalled_wait(limit_ns: int, stream=None) -> None:
    _check(lib.h3q_test_stalled_wait(int(limit_ns), _stream(stream)), "h3q_test_stalled_wait")


def h3q_test_stalled_linear_fp8(xq, sx, wq, sw, y, limit_ns, epilogue=H3Q_EPI_NONE, stream=None) -> None:
    """h3q_linear_fp8 whose operands never count as complete: it gives up after limit_ns."""
    w = "h3q_test_stalled_linear_fp8"
    epilogue = int(epilogue)
    M, K, N, index = _fp8_operands(w, xq, sx, wq, sw, None, y, "bf16", epilogue == H3Q_EPI_SWIGLU)
    _run(w, lib.h3q_test_stalled_linear_fp8, index, stream, xq.data_ptr(), sx.data_ptr(), M, K, wq.data_ptr(),
         sw.data_ptr(), N, epilogue, y.data_ptr(), int(limit_ns))


def h3q_status_string(status: int) -> str:
    return lib.h3q_status_string(int(status)).decode()


def h3q_version() -> str:
    return lib.h3q_version().decode()
