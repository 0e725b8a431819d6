"""Python binding of libfp8q.so: per-token-group FP8 quantization, block-scaled FP8 GEMMs,
their 4-bit (MXFP4) counterparts, and the operators between them in a serving layer (quantizing
norm, 4-bit key/value cache with its page plan, attention over it) for AMD Instinct MI355X (gfx950).

This module only marshals torch tensors (device memory, strides, the current HIP
stream) into the C ABI declared in include/fp8q.h; every step of the computation runs
in the library's HIP kernels. The functions named fp8q_* mirror the C entry points one
to one and write into caller-allocated tensors; group_quant() additionally allocates
its outputs (the role of _allocate_outputs in the sglang PR #30924 design, prhub
report section "实现拆解" item 2), as do rms_norm_group_quant(), mxfp4_quant(), mxfp4_dequant(),
kv4_read(), kv4_attention(), kv4_window_attention(), kv4_tree_attention() and kv4_plan();
alloc_kv4_cache() allocates a cache.

The 4-bit products, the page plan and the attention run on their tensors' GPU, whichever is current; the other
calls on the current one.

There is no fallback: if libfp8q.so is missing or the device is not a gfx950, calls
raise.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import os
from typing import NamedTuple

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libfp8q.so")

# constants of include/fp8q.h
OK, EINVAL, EUNSUPPORTED, EALIGN, EDEVICE, ELAUNCH = 0, 1, 2, 3, 4, 5
DTYPE_BF16, DTYPE_F16, DTYPE_F32 = 0, 1, 2
SCALE_F32, SCALE_UE8M0, SCALE_UE8M0_PACKED = 0, 1, 2
GEMM_BLOCK128, GEMM_MX32 = 0, 1

_DTYPES = {torch.bfloat16: DTYPE_BF16, torch.float16: DTYPE_F16, torch.float32: DTYPE_F32}
_SCALE_FMT = {"f32": SCALE_F32, "ue8m0": SCALE_UE8M0, "ue8m0_packed": SCALE_UE8M0_PACKED}

_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_INT = ctypes.c_int
_F32 = ctypes.c_float

_SIGNATURES = {
    "fp8q_group_quant": [_P, _INT, _I64, _I64, _I64, _I64, _I64, _P, _I64, _I64, _P, _INT, _I64, _I64,
                         _I64, _INT, _P, _I64, _P],
    "fp8q_silu_mul_group_quant": [_P, _INT, _I64, _I64, _I64, _I64, _I64, _P, _I64, _I64, _P, _INT, _I64,
                                  _I64, _I64, _INT, _P, _I64, _P],
    "fp8q_group_quant_int8": [_P, _INT, _I64, _I64, _I64, _I64, _I64, _P, _I64, _I64, _P, _INT, _I64,
                              _I64, _I64, _INT, _P, _I64, _P],
    "fp8q_gemm_blockscaled": [_P, _I64, _P, _INT, _I64, _I64, _P, _I64, _P, _INT, _I64, _I64, _P, _I64,
                              _I64, _I64, _I64, _INT, _P],
    "fp8q_gemm_blockscaled_ws": [_P, _I64, _P, _INT, _I64, _I64, _P, _I64, _P, _INT, _I64, _I64, _P, _I64,
                                 _I64, _I64, _I64, _INT, _P, _I64, _P],
    "fp8q_gemm_workspace_size": [_I64, _I64, _I64, _INT],
    "fp8q_gemm_blockscaled_noalloc": [_P, _I64, _P, _INT, _I64, _I64, _P, _I64, _P, _INT, _I64, _I64, _P, _I64,
                                      _I64, _I64, _I64, _INT, _P],
    "fp8q_grouped_gemm_masked": [_P, _I64, _I64, _P, _INT, _I64, _I64, _I64, _P, _I64, _I64, _P, _INT,
                                 _I64, _I64, _I64, _P, _I64, _I64, _P, _I64, _I64, _I64, _I64, _I64, _P],
    "fp8q_grouped_gemm_segments": [_P, _I64, _P, _INT, _I64, _I64, _P, _I64, _I64, _P, _INT, _I64, _I64, _I64,
                                   _P, _I64, _P, _P, _I64, _I64, _I64, _I64, _I64, _I64, _P],
    "fp8q_grouped_gemm_contiguous": [_P, _I64, _P, _INT, _I64, _I64, _P, _I64, _I64, _P, _INT, _I64, _I64, _I64,
                                     _P, _I64, _P, _I64, _I64, _I64, _I64, _P],
    "fp8q_rms_norm_group_quant": [_P, _INT, _I64, _I64, _I64, _P, _I64, _P, _I64, _P, _F32, _P, _I64, _P, _INT,
                                  _I64, _I64, _INT, _P],
    "fp8q_kv4_write": [_P, _I64, _I64, _P, _I64, _I64, _INT, _I64, _I64, _I64, _P, _P, _P, _P, _P, _I64, _I64,
                       _I64, _I64, _I64, _I64, _I64, _I64, _P],
    "fp8q_kv4_read": [_P, _I64, _I64, _P, _I64, _I64, _INT, _I64, _I64, _I64, _P, _P, _P, _P, _P, _I64, _I64,
                      _I64, _I64, _I64, _I64, _I64, _I64, _P],
    "fp8q_kv4_attention": [_P, _INT, _I64, _I64, _P, _P, _P, _P, _I64, _I64, _I64, _I64, _I64, _I64, _I64, _I64,
                           _P, _I64, _I64, _P, _P, _P, _I64, _I64, _P, _I64, _I64, _I64, _I64, _I64, _I64, _F32,
                           _INT, _P, _I64, _P],
    "fp8q_kv4_attention_workspace_size": [_INT, _I64, _I64, _I64, _I64, _I64, _I64],
    "fp8q_kv4_window_attention": [_P, _INT, _I64, _I64, _P, _P, _P, _P, _I64, _I64, _I64, _I64, _I64, _I64, _I64, _I64,
                                  _P, _I64, _I64, _P, _P, _P, _I64, _I64, _P, _I64, _I64, _I64, _I64, _I64, _I64, _F32,
                                  _I64, _I64, _P, _I64, _P],
    "fp8q_kv4_window_attention_workspace_size": [_INT, _I64, _I64, _I64, _I64, _I64, _I64, _I64, _I64],
    "fp8q_kv4_tree_attention_workspace_size": [_INT, _I64, _I64, _I64, _I64, _I64, _I64],
    "fp8q_kv4_tree_attention": [_P, _INT, _I64, _I64, _P, _P, _P, _P, _I64, _I64, _I64, _I64, _I64, _I64, _I64, _I64,
                                _P, _I64, _I64, _P, _P, _P, _I64, _I64, _P, _I64, _I64, _I64, _I64, _I64, _I64, _F32,
                                _P, _I64, _I64, _P, _I64, _P],
    "fp8q_kv4_plan": [_P, _P, _I64, _P, _I64, _P, _I64, _I64, _I64, _I64, _P, _P, _P, _P, _I64, _P, _P],
    "fp8q_mxfp4_quant": [_P, _INT, _I64, _I64, _I64, _P, _I64, _P, _INT, _I64, _I64, _P],
    "fp8q_silu_mul_mxfp4_quant": [_P, _INT, _I64, _I64, _I64, _P, _I64, _P, _INT, _I64, _I64, _P],
    "fp8q_mxfp4_dequant": [_P, _I64, _P, _INT, _I64, _I64, _P, _INT, _I64, _I64, _I64, _P],
    "fp8q_gemm_mxfp4": [_P, _I64, _P, _INT, _I64, _I64, _P, _I64, _P, _INT, _I64, _I64, _P, _I64, _I64, _I64, _I64,
                        _P, _I64, _P],
    "fp8q_gemm_mxfp4_workspace_size": [_I64, _I64, _I64],
    "fp8q_status_string": [_INT],
    "fp8q_last_error": [],
    "fp8q_device_check": [_INT],
}


class Fp8qError(RuntimeError):
    def __init__(self, status: int, detail: str):
        super().__init__(f"{detail} [{_status_string(status)}]")
        self.status = status


_lib = None


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Loads libfp8q.so (built by fp8_group_quant_amd/build.py). Raises if it is missing."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise ImportError(f"{path} is not built; run fp8_group_quant_amd/build.py (there is no fallback)")
    lib = ctypes.CDLL(path)
    for name, args in _SIGNATURES.items():
        fn = getattr(lib, name, None)
        if fn is None:  # calling it later raises AttributeError; tests check every export
            continue
        fn.argtypes = args
        fn.restype = (ctypes.c_char_p if name in ("fp8q_status_string", "fp8q_last_error")
                      else _I64 if name.endswith("_workspace_size") else _INT)
    _lib = lib
    return lib


def _status_string(status: int) -> str:
    return load_library().fp8q_status_string(status).decode()


def _check(status: int) -> None:
    if status != OK:
        raise Fp8qError(status, load_library().fp8q_last_error().decode())


def _stream(stream) -> int:
    if stream is None:
        # the handle alone (a Stream object around it costs about 2 us)
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _stream_here(stream, device: int) -> int | None:
    """The stream's handle for a call whose tensors are on GPU `device`; None where another GPU is the current one:
    kernels, their shapes and the default stream go by that, so the call makes the tensors' current. (A handle that is
    given as a number does not say whose it is.)"""
    if stream is None:
        current = torch._C._cuda_getDevice()
        return torch._C._cuda_getCurrentRawStream(current) if current == device else None
    if isinstance(stream, torch.cuda.Stream) and stream.device_index != device:
        raise ValueError("the stream must be one of the tensors' GPU")
    if torch.cuda.is_initialized() and torch._C._cuda_getDevice() != device:
        return None
    return _stream(stream)


def _ptr(t: torch.Tensor | None) -> int | None:
    return None if t is None else t.data_ptr()


def _as3(t: torch.Tensor) -> tuple[int, int, int, int, int]:
    """(E, M, W, stride_e, stride_m) of a [M, W] or [E, M, W] tensor with unit inner stride."""
    if t.dim() == 2:
        if t.size(1) > 1 and t.stride(1) != 1:
            raise ValueError("innermost dimension must be contiguous")
        return 1, t.size(0), t.size(1), t.size(0) * t.stride(0), t.stride(0)
    if t.dim() == 3:
        if t.size(2) > 1 and t.stride(2) != 1:
            raise ValueError("innermost dimension must be contiguous")
        return t.size(0), t.size(1), t.size(2), t.stride(0), t.stride(1)
    raise ValueError("expected a 2-D or 3-D tensor")


def _scale_strides(s: torch.Tensor) -> tuple[int, int, int]:
    """(s_se, s_sm, s_sg) of the logical [M, ng] or [E, M, ng] scale view."""
    if s.dim() == 2:
        return 0, s.stride(0), s.stride(1)
    if s.dim() == 3:
        return s.stride(0), s.stride(1), s.stride(2)
    raise ValueError("expected a 2-D or 3-D scale view")


def _scale_fmt_of(s: torch.Tensor) -> int:
    if s.dtype == torch.float32:
        return SCALE_F32
    if s.dtype == torch.uint8:
        return SCALE_UE8M0
    if s.dtype == torch.int32:
        return SCALE_UE8M0_PACKED
    raise ValueError("scales must be float32 (fp32 scales), uint8 (UE8M0 bytes) or int32 "
                     "(UE8M0 bytes packed 4 groups per word)")


# ------------------------------------------------------------------------------ quant
def _quant(entry: str, x, q, s, group_size, masked_m, expected_m, stream, silu):
    E, M, W, x_se, x_sm = _as3(x)
    K = W // 2 if silu else W
    if x.dtype not in _DTYPES:
        raise ValueError(f"unsupported input dtype {x.dtype}")
    qE, qM, qK, q_se, q_sm = _as3(q.view(torch.uint8))
    if (qE, qM, qK) != (E, M, K):
        raise ValueError(f"q has shape {tuple(q.shape)}, expected {(E, M, K) if x.dim() == 3 else (M, K)}")
    s_se, s_sm, s_sg = _scale_strides(s)
    mm = None
    if masked_m is not None:
        if masked_m.dtype != torch.int32 or masked_m.numel() != E or not masked_m.is_cuda:
            raise ValueError("masked_m must be a device int32 tensor with one entry per expert")
        mm = masked_m
    fn = getattr(load_library(), entry)
    _check(fn(_ptr(x), _DTYPES[x.dtype], E, M, K, x_se, x_sm, _ptr(q), q_se, q_sm, _ptr(s),
              _scale_fmt_of(s), s_se, s_sm, s_sg, group_size, _ptr(mm), int(expected_m),
              _stream(stream)))


def fp8q_group_quant(x: torch.Tensor, q: torch.Tensor, s: torch.Tensor, group_size: int = 128,
                     masked_m: torch.Tensor | None = None, expected_m: int = 0, stream=None) -> None:
    """x [M, K] or [E, M, K] (bf16/f16/f32) -> q (uint8 or float8_e4m3fn, same shape) and
    s: a [.., M, K/G] view (float32 = fp32 scales, uint8 = UE8M0); its strides choose the
    row- or column-major layout. group_size == K is per-token quantization (s [.., M, 1])."""
    _quant("fp8q_group_quant", x, q, s, group_size, masked_m, expected_m, stream, False)


def fp8q_group_quant_int8(x: torch.Tensor, q: torch.Tensor, s: torch.Tensor, group_size: int = 128,
                          masked_m: torch.Tensor | None = None, expected_m: int = 0, stream=None) -> None:
    """As fp8q_group_quant with int8 codes in q (torch.int8) and float32 scales
    s = amax / 127."""
    if q.dtype != torch.int8:
        raise ValueError("q must be an int8 tensor")
    if s.dtype != torch.float32:
        raise ValueError("int8 output takes float32 scales")
    _quant("fp8q_group_quant_int8", x, q, s, group_size, masked_m, expected_m, stream, False)


def fp8q_silu_mul_group_quant(x: torch.Tensor, q: torch.Tensor, s: torch.Tensor, group_size: int = 128,
                              masked_m: torch.Tensor | None = None, expected_m: int = 0,
                              stream=None) -> None:
    """As fp8q_group_quant, with x [.., M, 2K] = gate | up and silu(gate) * up quantized."""
    _quant("fp8q_silu_mul_group_quant", x, q, s, group_size, masked_m, expected_m, stream, True)


def alloc_scales(E: int | None, M: int, ng: int, scale_fmt: str, layout: str, device) -> torch.Tensor:
    """Scale tensor viewed as [.., M, ng]: row-major storage, or column-major storage
    [.., ng, M] returned transposed (the strides carry the layout). "ue8m0_packed" returns
    int32 words of 4 groups each, viewed as [.., M, ng / 4]."""
    dt = {"f32": torch.float32, "ue8m0": torch.uint8, "ue8m0_packed": torch.int32}[scale_fmt]
    if scale_fmt == "ue8m0_packed":
        if ng % 4:
            raise ValueError("packed UE8M0 scales need a multiple of 4 groups per row")
        ng //= 4
    lead = () if E is None else (E,)
    if layout == "row":
        return torch.empty(*lead, M, ng, dtype=dt, device=device)
    return torch.empty(*lead, ng, M, dtype=dt, device=device).transpose(-1, -2)


def group_quant(x: torch.Tensor, group_size: int = 128, scale_fmt: str = "ue8m0", layout: str = "col",
                silu: bool = False, masked_m: torch.Tensor | None = None, expected_m: int = 0,
                stream=None, int8: bool = False) -> tuple[torch.Tensor, torch.Tensor]:
    """Allocating form: returns (q uint8 [.., M, K] of e4m3 bytes, or int8 codes with
    int8=True (fp32 scales), scales viewed as [.., M, K/G]). group_size == K is per-token."""
    W = x.shape[-1]
    K = W // 2 if silu else W
    lead = tuple(x.shape[:-2])
    M = x.shape[-2]
    q = torch.empty(*lead, M, K, dtype=torch.int8 if int8 else torch.uint8, device=x.device)
    s = alloc_scales(lead[0] if lead else None, M, K // group_size, scale_fmt, layout, x.device)
    if int8:
        if silu:
            raise ValueError("int8 output has no fused silu variant")
        fp8q_group_quant_int8(x, q, s, group_size, masked_m, expected_m, stream)
    elif silu:
        fp8q_silu_mul_group_quant(x, q, s, group_size, masked_m, expected_m, stream)
    else:
        fp8q_group_quant(x, q, s, group_size, masked_m, expected_m, stream)
    return q, s


# ------------------------------------------------------------------------------ GEMM
def _u8(t: torch.Tensor) -> torch.Tensor:
    return t.view(torch.uint8) if t.dtype != torch.uint8 else t


def _allocating_on(stream, device):
    """Context in which torch allocates on the stream that the kernels run on, so that the caching
    allocator hands the blocks to no other stream's work before they finish."""
    if stream is None:
        return contextlib.nullcontext()
    st = stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(int(stream), device=device)
    return torch.cuda.stream(st)


def _alloc_workspace(nbytes: int, device, stream) -> torch.Tensor | None:
    """nbytes of device memory (None for 0) for kernels on `stream`."""
    if nbytes <= 0:
        return None
    with _allocating_on(stream, device):
        return torch.empty(nbytes, dtype=torch.uint8, device=device)


def fp8q_gemm_workspace_size(M: int, N: int, K: int, mode: int = GEMM_BLOCK128) -> int:
    """Bytes of workspace with which fp8q_gemm_blockscaled_ws takes its split-K path for this
    shape on the current device (0: none needed)."""
    return _gemm_workspace_size(torch.cuda.current_device(), M, N, K, mode)


# A size depends on the shape and the device alone. A server's M takes many values: the least recently used go.
@functools.lru_cache(maxsize=8192)
def _gemm_workspace_size(device: int, M: int, N: int, K: int, mode: int) -> int:
    return int(load_library().fp8q_gemm_workspace_size(M, N, K, mode))


@functools.lru_cache(maxsize=8192)
def _gemm_mxfp4_workspace_size(device: int, M: int, N: int, K: int) -> int:
    return int(load_library().fp8q_gemm_mxfp4_workspace_size(M, N, K))


def fp8q_gemm_blockscaled(a: torch.Tensor, sa: torch.Tensor, b: torch.Tensor, sb: torch.Tensor,
                          y: torch.Tensor, mode: int = GEMM_BLOCK128, stream=None,
                          workspace: torch.Tensor | None = None) -> None:
    """Y[M, N] (bf16) = dequant(a [M, K]) @ dequant(b [N, K])^T.
    BLOCK128: sa viewed as [M, K/128], sb as [ceil(N/128), K/128] (float32 or uint8 UE8M0;
    sa may be int32 packed UE8M0 words [M, K/512]).
    MX32: sa [M, K/32], sb [N, K/32], uint8 E8M0; or either as int32 packed words [rows, K/128]
    (the four E8M0 bytes of one 128-wide K step per word; a [K/128, rows] storage viewed
    transposed gives the column-major words that load fastest).
    Calls fp8q_gemm_blockscaled_ws: when the shape can use a workspace and none is given, one
    is taken from torch's allocator on a's device (stream-ordered, capturable)."""
    a8, b8 = _u8(a), _u8(b)
    M, K = a8.shape
    N = b8.shape[0]
    if b8.shape[1] != K or tuple(y.shape) != (M, N):
        raise ValueError("shape mismatch")
    if a8.stride(1) != 1 or b8.stride(1) != 1 or y.stride(1) != 1:
        raise ValueError("innermost dimensions must be contiguous")
    if workspace is None and mode == GEMM_BLOCK128:
        workspace = _alloc_workspace(fp8q_gemm_workspace_size(M, N, K, mode), a8.device, stream)
    ws_ptr = None if workspace is None else workspace.data_ptr()
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(load_library().fp8q_gemm_blockscaled_ws(
        _ptr(a8), a8.stride(0), _ptr(sa), _scale_fmt_of(sa), sa.stride(0), sa.stride(1),
        _ptr(b8), b8.stride(0), _ptr(sb), _scale_fmt_of(sb), sb.stride(0), sb.stride(1),
        _ptr(y), y.stride(0), M, N, K, mode, ws_ptr, ws_bytes, _stream(stream)))


def fp8q_gemm_blockscaled_noalloc(a: torch.Tensor, sa: torch.Tensor, b: torch.Tensor, sb: torch.Tensor,
                                  y: torch.Tensor, mode: int = GEMM_BLOCK128, stream=None) -> None:
    """fp8q_gemm_blockscaled with the split-K partial sums in the library's own device array
    (no allocation anywhere; calls that overlap on one device race on that array)."""
    a8, b8 = _u8(a), _u8(b)
    M, K = a8.shape
    N = b8.shape[0]
    if b8.shape[1] != K or tuple(y.shape) != (M, N):
        raise ValueError("shape mismatch")
    if a8.stride(1) != 1 or b8.stride(1) != 1 or y.stride(1) != 1:
        raise ValueError("innermost dimensions must be contiguous")
    _check(load_library().fp8q_gemm_blockscaled_noalloc(
        _ptr(a8), a8.stride(0), _ptr(sa), _scale_fmt_of(sa), sa.stride(0), sa.stride(1),
        _ptr(b8), b8.stride(0), _ptr(sb), _scale_fmt_of(sb), sb.stride(0), sb.stride(1),
        _ptr(y), y.stride(0), M, N, K, mode, _stream(stream)))


def fp8q_grouped_gemm_masked(a: torch.Tensor, sa: torch.Tensor, b: torch.Tensor, sb: torch.Tensor,
                             y: torch.Tensor, masked_m: torch.Tensor, expected_m: int = 0,
                             stream=None) -> None:
    """Per expert e: Y[e, :masked_m[e]] = BLOCK128 product of a[e] [cap, K] and b[e] [N, K].
    sa viewed as [E, cap, K/128]; sb as [E, ceil(N/128), K/128]; y [E, cap, N] bf16."""
    a8, b8 = _u8(a), _u8(b)
    E, cap, K = a8.shape
    N = b8.shape[1]
    if b8.shape[0] != E or b8.shape[2] != K or tuple(y.shape) != (E, cap, N):
        raise ValueError("shape mismatch")
    if masked_m.dtype != torch.int32 or masked_m.numel() != E or not masked_m.is_cuda:
        raise ValueError("masked_m must be a device int32 tensor with one entry per expert")
    _check(load_library().fp8q_grouped_gemm_masked(
        _ptr(a8), a8.stride(0), a8.stride(1), _ptr(sa), _scale_fmt_of(sa), sa.stride(0), sa.stride(1),
        sa.stride(2), _ptr(b8), b8.stride(0), b8.stride(1), _ptr(sb), _scale_fmt_of(sb), sb.stride(0),
        sb.stride(1), sb.stride(2), _ptr(y), y.stride(0), y.stride(1), _ptr(masked_m), int(expected_m),
        E, cap, N, K, _stream(stream)))


def _packed_rows_operands(a, sa, b, sb, y):
    a8, b8 = _u8(a), _u8(b)
    T, K = a8.shape
    W, N = b8.shape[0], b8.shape[1]
    if b8.dim() != 3 or b8.shape[2] != K or tuple(y.shape) != (T, N) or sb.dim() != 3:
        raise ValueError("shape mismatch: a [T, K], b [W, N, K], sb [W, N/128, K/128], y [T, N]")
    if a8.stride(1) != 1 or b8.stride(2) != 1 or y.stride(1) != 1:
        raise ValueError("a, b and y must have unit stride along their last dimension")
    return a8, b8, T, K, W, N


def _dev_i32(t: torch.Tensor, what: str) -> torch.Tensor:
    if t.dtype != torch.int32 or not t.is_cuda or t.dim() != 1 or t.stride(0) != 1:
        raise ValueError(f"{what} must be a contiguous 1-D device int32 tensor")
    return t


def fp8q_grouped_gemm_segments(a: torch.Tensor, sa: torch.Tensor, b: torch.Tensor, sb: torch.Tensor,
                               y: torch.Tensor, seg_indptr: torch.Tensor, seg_weight: torch.Tensor | None = None,
                               expected_rows: int = 0, stream=None) -> None:
    """Rows [seg_indptr[s], seg_indptr[s+1]) of a [T, K] times weight seg_weight[s] (default s)
    of b [W, N, K] into the same rows of y [T, N] (bf16). sa viewed as [T, K/128] (or packed
    words [T, K/512]); sb as [W, N/128, K/128]."""
    a8, b8, T, K, W, N = _packed_rows_operands(a, sa, b, sb, y)
    si = _dev_i32(seg_indptr, "seg_indptr")
    sw = None if seg_weight is None else _dev_i32(seg_weight, "seg_weight")
    S = si.numel() - 1
    if S < 0 or (sw is not None and sw.numel() != S):
        raise ValueError("seg_indptr needs S + 1 entries and seg_weight S")
    _check(load_library().fp8q_grouped_gemm_segments(
        _ptr(a8), a8.stride(0), _ptr(sa), _scale_fmt_of(sa), sa.stride(0), sa.stride(1),
        _ptr(b8), b8.stride(0), b8.stride(1), _ptr(sb), _scale_fmt_of(sb), sb.stride(0), sb.stride(1),
        sb.stride(2), _ptr(y), y.stride(0), _ptr(si), _ptr(sw), S, T, W, N, K, int(expected_rows),
        _stream(stream)))


def fp8q_grouped_gemm_contiguous(a: torch.Tensor, sa: torch.Tensor, b: torch.Tensor, sb: torch.Tensor,
                                 y: torch.Tensor, m_indices: torch.Tensor, stream=None) -> None:
    """Rows of a [T, K] tagged m_indices[t] (-1: padding; blocks of 128 rows, see the header)
    times weight m_indices[t] of b [W, N, K] into y [T, N] (bf16)."""
    a8, b8, T, K, W, N = _packed_rows_operands(a, sa, b, sb, y)
    mi = _dev_i32(m_indices, "m_indices")
    if mi.numel() != T:
        raise ValueError("m_indices needs one entry per row of a")
    _check(load_library().fp8q_grouped_gemm_contiguous(
        _ptr(a8), a8.stride(0), _ptr(sa), _scale_fmt_of(sa), sa.stride(0), sa.stride(1),
        _ptr(b8), b8.stride(0), b8.stride(1), _ptr(sb), _scale_fmt_of(sb), sb.stride(0), sb.stride(1),
        sb.stride(2), _ptr(y), y.stride(0), _ptr(mi), T, W, N, K, _stream(stream)))


# Every operand of a call below is on one GPU: an address that is not the GPU's own is a memory fault in
# the kernel. (Compared in place, tensor by tensor: a helper with a loop takes up to 0.3 us more.)
_ELSEWHERE = "every tensor must be on one GPU"


# ------------------------------------------------------------------------------ MXFP4
def _mxfp4_rows(entry: str, x, q, s, width, stream) -> None:
    """The rows' checks and call of the quantizer (x of `width` elements per row, gate | up twice as many) and,
    with its own argument order, of the way back."""
    dt = _DTYPES.get(x.dtype)
    if dt is None or x.dim() != 2 or q.dim() != 2 or s.dim() != 2:
        raise ValueError("x (bf16, fp16 or fp32), q and s must be 2-D tensors")
    M = x.shape[0]
    rows, K = q.shape
    K *= 2
    if q.element_size() != 1 or rows != M or width != K:
        raise ValueError(f"q has shape {tuple(q.shape)} of {q.dtype}, expected bytes of {(M, width // 2)}")
    x_sm, x_in = x.stride()
    q_sm, q_in = q.stride()
    if (x_in != 1 and x.shape[1] > 1) or (q_in != 1 and K > 2):
        raise ValueError("innermost dimensions must be contiguous")
    fmt = _scale_fmt_of(s)
    if s.shape != (M, K // 128 if fmt == SCALE_UE8M0_PACKED else K // 32):
        raise ValueError(f"s has shape {tuple(s.shape)} of {s.dtype}, expected a scale per 32 of {(M, K)} elements")
    if not 0 <= x.get_device() == q.get_device() == s.get_device():
        raise ValueError(_ELSEWHERE)
    handle = _stream_here(stream, x.get_device())
    if handle is None:
        with torch.cuda.device(x.get_device()):
            return _mxfp4_rows(entry, x, q, s, width, stream)
    s_sm, s_sg = s.stride()
    if entry == "fp8q_mxfp4_dequant":
        _check(load_library().fp8q_mxfp4_dequant(q.data_ptr(), q_sm, s.data_ptr(), fmt, s_sm, s_sg, x.data_ptr(), dt, M, K,
                                                 x_sm, handle))
    else:
        _check(getattr(load_library(), entry)(x.data_ptr(), dt, M, K, x_sm, q.data_ptr(), q_sm, s.data_ptr(), fmt, s_sm, s_sg,
                                              handle))


def fp8q_mxfp4_quant(x: torch.Tensor, q: torch.Tensor, s: torch.Tensor, stream=None) -> None:
    """x [M, K] (bf16, fp16 or fp32) as e2m1 codes q (uint8 [M, K/2], element 2i in the low half of byte i) with one
    UE8M0 scale per 32 elements: s uint8 [M, K/32], or int32 words of four [M, K/128]; its strides choose the
    row- or column-major layout."""
    _mxfp4_rows("fp8q_mxfp4_quant", x, q, s, x.shape[-1], stream)


def fp8q_silu_mul_mxfp4_quant(x: torch.Tensor, q: torch.Tensor, s: torch.Tensor, stream=None) -> None:
    """As fp8q_mxfp4_quant, with x [M, 2K] = gate | up and silu(gate) * up quantized."""
    if x.shape[-1] % 2:
        raise ValueError("x must hold gate | up, two halves of one width")
    _mxfp4_rows("fp8q_silu_mul_mxfp4_quant", x, q, s, x.shape[-1] // 2, stream)


def fp8q_mxfp4_dequant(q: torch.Tensor, s: torch.Tensor, x: torch.Tensor, stream=None) -> None:
    """The rows x [M, K] (bf16, fp16 or fp32) that codes q and scales s stand for."""
    _mxfp4_rows("fp8q_mxfp4_dequant", x, q, s, x.shape[-1], stream)


def mxfp4_quant(x: torch.Tensor, scale_fmt: str = "ue8m0_packed", layout: str = "col", silu: bool = False,
                stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """Allocating form: (q uint8 [M, K/2], scales viewed as [M, K/32], or [M, K/128] words with "ue8m0_packed")."""
    M, W = x.shape
    K = W // 2 if silu else W
    if scale_fmt not in ("ue8m0", "ue8m0_packed"):
        raise ValueError("scale_fmt must be 'ue8m0' or 'ue8m0_packed'")
    with _allocating_on(stream, x.device):
        q = torch.empty(M, K // 2, dtype=torch.uint8, device=x.device)
        s = alloc_scales(None, M, K // 32, scale_fmt, layout, x.device)
    (fp8q_silu_mul_mxfp4_quant if silu else fp8q_mxfp4_quant)(x, q, s, stream)
    return q, s


def mxfp4_dequant(q: torch.Tensor, s: torch.Tensor, dtype: torch.dtype = torch.bfloat16, stream=None) -> torch.Tensor:
    """Allocating form of fp8q_mxfp4_dequant: [M, K] of dtype."""
    with _allocating_on(stream, q.device):
        x = torch.empty(q.shape[0], 2 * q.shape[1], dtype=dtype, device=q.device)
    fp8q_mxfp4_dequant(q, s, x, stream)
    return x


def fp8q_gemm_mxfp4_workspace_size(M: int, N: int, K: int) -> int:
    """Bytes of workspace with which fp8q_gemm_mxfp4 splits K over more of the current device (0: it does not)."""
    return int(load_library().fp8q_gemm_mxfp4_workspace_size(M, N, K))


def fp8q_gemm_mxfp4(a: torch.Tensor, sa: torch.Tensor, b: torch.Tensor, sb: torch.Tensor, y: torch.Tensor, stream=None,
                    workspace: torch.Tensor | None = None) -> None:
    """y [M, N] (bf16) = a b^T of MXFP4 operands: codes a [M, K/2], b [N, K/2] (uint8) with scales sa, sb as the
    quantizer gives them: int32 words [rows, K/128] of any strides (column-major ones are read fastest), or
    row-major uint8 [rows, K/32].
    When the shape can use a workspace and none is given, one is taken from torch's allocator."""
    M, kb = a.shape
    N, kb2 = b.shape
    K = 2 * kb
    if kb != kb2 or y.shape != (M, N) or y.dtype != torch.bfloat16 or a.element_size() != 1 or b.element_size() != 1:
        raise ValueError("shape mismatch: a [M, K/2] and b [N, K/2] of bytes, y [M, N] of bf16")
    lda, a_in = a.stride()
    ldb, b_in = b.stride()
    ldy, y_in = y.stride()
    if ((a_in != 1 or b_in != 1) and kb > 1) or (y_in != 1 and N > 1):
        raise ValueError("innermost dimensions must be contiguous")
    fa, fb = _scale_fmt_of(sa), _scale_fmt_of(sb)
    if sa.shape != (M, K // 128 if fa == SCALE_UE8M0_PACKED else K // 32) or \
            sb.shape != (N, K // 128 if fb == SCALE_UE8M0_PACKED else K // 32):
        raise ValueError("scales must be [rows, K/32] bytes or [rows, K/128] words")
    if not 0 <= a.get_device() == b.get_device() == y.get_device() == sa.get_device() == sb.get_device() \
            or (workspace is not None and workspace.get_device() != a.get_device()):
        raise ValueError(_ELSEWHERE)
    dev = a.get_device()
    handle = _stream_here(stream, dev)
    if handle is None:
        with torch.cuda.device(dev):
            return fp8q_gemm_mxfp4(a, sa, b, sb, y, stream, workspace)
    if workspace is None:
        size = _gemm_mxfp4_workspace_size(dev, M, N, K)
        if size > 0:
            workspace = _alloc_workspace(size, a.device, stream)
    sa_sm, sa_sk = sa.stride()
    sb_sn, sb_sk = sb.stride()
    _check(load_library().fp8q_gemm_mxfp4(a.data_ptr(), lda, sa.data_ptr(), fa, sa_sm, sa_sk, b.data_ptr(), ldb, sb.data_ptr(), fb, sb_sn,
                               sb_sk, y.data_ptr(), ldy, M, N, K, None if workspace is None else workspace.data_ptr(),
                               0 if workspace is None else workspace.numel() * workspace.element_size(), handle))


# ------------------------------------------------------------------------------ norm
def fp8q_rms_norm_group_quant(x: torch.Tensor, weight: torch.Tensor, q: torch.Tensor, s: torch.Tensor,
                              group_size: int = 128, eps: float = 1e-6, residual: torch.Tensor | None = None,
                              residual_out: torch.Tensor | None = None, stream=None) -> None:
    """h = x (+ residual); y = h / sqrt(mean(h^2) + eps) * weight; y quantized as by
    fp8q_group_quant into q (uint8 or float8_e4m3fn) and s (a [M, K/G] view, whose type and strides
    choose the format and layout). x, residual, residual_out [M, K] and weight [K] have one type;
    residual_out receives h rounded to it (it may be the residual's or x's own tensor)."""
    # written for few interpreter steps: with one token the checks are most of the call's time
    dt = _DTYPES.get(x.dtype)
    if dt is None or x.dim() != 2:
        raise ValueError("x must be a 2-D bf16, fp16 or fp32 tensor")
    shape = x.shape
    M, K = shape
    xs, qs, ss = x.stride(), q.stride(), s.stride()
    inner = K <= 1 or (xs[1] == 1 and qs[-1] == 1)
    r_ptr = ro_ptr = None
    r_sm = ro_sm = 0
    for t in (residual, residual_out):
        if t is not None and (t.dtype != x.dtype or t.shape != shape):
            raise ValueError("residual and residual_out must have x's shape and type")
    if residual is not None:
        r_ptr, (r_sm, r_sk) = residual.data_ptr(), residual.stride()
        inner = inner and (K <= 1 or r_sk == 1)
    if residual_out is not None:
        ro_ptr, (ro_sm, ro_sk) = residual_out.data_ptr(), residual_out.stride()
        inner = inner and (K <= 1 or ro_sk == 1)
    if weight.dtype != x.dtype or weight.dim() != 1 or weight.numel() != K or (K > 1 and weight.stride(0) != 1):
        raise ValueError("weight must be a contiguous [K] tensor of x's type")
    if q.element_size() != 1 or q.shape != shape:
        raise ValueError(f"q has shape {tuple(q.shape)} of {q.dtype}, expected e4m3 bytes of {(M, K)}")
    if not inner:
        raise ValueError("innermost dimensions must be contiguous")
    fmt = _scale_fmt_of(s)
    ng = K // group_size // (4 if fmt == SCALE_UE8M0_PACKED else 1) if group_size > 0 else 0
    if s.shape != (M, ng):
        raise ValueError(f"s has shape {tuple(s.shape)}, expected {(M, ng)}")
    if not 0 <= x.get_device() == weight.get_device() == q.get_device() == s.get_device() \
            or (residual is not None and residual.get_device() != x.get_device()) \
            or (residual_out is not None and residual_out.get_device() != x.get_device()):
        raise ValueError(_ELSEWHERE)
    _check(load_library().fp8q_rms_norm_group_quant(
        x.data_ptr(), dt, M, K, xs[0], r_ptr, r_sm, ro_ptr, ro_sm, weight.data_ptr(), eps, q.data_ptr(), qs[0],
        s.data_ptr(), fmt, ss[0], ss[1], group_size, _stream(stream)))


def rms_norm_group_quant(x: torch.Tensor, weight: torch.Tensor, group_size: int = 128, scale_fmt: str = "ue8m0",
                         layout: str = "col", eps: float = 1e-6, residual: torch.Tensor | None = None,
                         stream=None) -> tuple[torch.Tensor, torch.Tensor, torch.Tensor | None]:
    """Allocating form: (q uint8 [M, K] of e4m3 bytes, scales viewed as [M, K/G], x + residual
    or None without a residual)."""
    M, K = x.shape
    with _allocating_on(stream, x.device):
        q = torch.empty(M, K, dtype=torch.uint8, device=x.device)
        s = alloc_scales(None, M, K // group_size, scale_fmt, layout, x.device)
        h = None if residual is None else torch.empty(M, K, dtype=x.dtype, device=x.device)
    fp8q_rms_norm_group_quant(x, weight, q, s, group_size, eps, residual, h, stream)
    return q, s, h


# ------------------------------------------------------------------------------ 4-bit cache
class Kv4Cache(NamedTuple):
    """A paged cache of 4-bit keys and values: uint8 codes k, v viewed as [pages, page_size,
    heads, D/2] and uint8 UE8M0 scales k_scales, v_scales viewed as [pages, page_size, heads, D/32]. The
    strides carry the layout; k and v have the same, and so have their scales."""
    k: torch.Tensor
    k_scales: torch.Tensor
    v: torch.Tensor
    v_scales: torch.Tensor


def alloc_kv4_cache(pages: int, page_size: int, heads: int, head_dim: int, layout: str = "head",
                    device="cuda") -> Kv4Cache:
    """A cache of zeros. layout "head": a head's tokens of one page are adjacent (the order that
    attention reads); "token": a token's heads are."""
    def rows(width):
        if layout == "head":
            return torch.zeros(pages, heads, page_size, width, dtype=torch.uint8, device=device).transpose(1, 2)
        if layout == "token":
            return torch.zeros(pages, page_size, heads, width, dtype=torch.uint8, device=device)
        raise ValueError("layout must be 'head' or 'token'")
    return Kv4Cache(rows(head_dim // 2), rows(head_dim // 32), rows(head_dim // 2), rows(head_dim // 32))


def _kv4_args(cache: Kv4Cache, heads: int, head_dim: int) -> tuple:
    """The cache's C arguments: pointers, sizes and strides."""
    k, ks, v, vs = cache
    codes, scales = k.shape, ks.shape
    if codes != v.shape or scales != vs.shape or len(codes) != 4 or codes[2:] != (heads, head_dim // 2) \
            or scales != codes[:3] + (head_dim // 32,):
        raise ValueError(f"cached tensors do not fit {heads} heads of {head_dim}: codes {tuple(codes)}, "
                         f"scales {tuple(scales)}")
    c_sp, c_st, c_sh, c_in = cs = k.stride()
    s_sp, s_st, s_sh, s_in = ss = ks.stride()
    if cs != v.stride() or ss != vs.stride():
        raise ValueError("keys and values must have the same strides")
    if c_in != 1 or s_in != 1:
        raise ValueError("innermost dimensions must be contiguous")
    if not (k.dtype == ks.dtype == v.dtype == vs.dtype == torch.uint8):
        raise ValueError("cached tensors must be uint8")
    if not k.get_device() == ks.get_device() == v.get_device() == vs.get_device():
        raise ValueError(_ELSEWHERE)
    return (k.data_ptr(), ks.data_ptr(), v.data_ptr(), vs.data_ptr(), codes[0], codes[1], c_sp, c_st, c_sh, s_sp, s_st, s_sh)


def _kv4_rows(entry: str, k, v, slots, cache, stream) -> None:
    shape, dt = k.shape, _DTYPES.get(k.dtype)
    if len(shape) != 3 or shape != v.shape or k.dtype != v.dtype or dt is None:
        raise ValueError("k and v must be [T, heads, D] tensors of one type (bf16, fp16 or fp32)")
    T, H, D = shape
    k_st, k_sh, k_in = k.stride()
    v_st, v_sh, v_in = v.stride()
    if (k_in != 1 or v_in != 1) and k.numel() > 0:
        raise ValueError("innermost dimensions must be contiguous")
    if _dev_i32(slots, "slots").numel() != T:
        raise ValueError("slots needs one entry per token")
    if not k.get_device() == v.get_device() == slots.get_device() == cache.k.get_device():
        raise ValueError(_ELSEWHERE)
    _check(getattr(load_library(), entry)(
        k.data_ptr(), k_st, k_sh, v.data_ptr(), v_st, v_sh, dt, T, H, D, slots.data_ptr(),
        *_kv4_args(cache, H, D), _stream(stream)))


def fp8q_kv4_write(k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, cache: Kv4Cache, stream=None) -> None:
    """Quantizes token t's keys and values (k, v [T, heads, D]) into slot slots[t] of the cache
    (int32; slot n is token n % page_size of page n // page_size, negative or past the end: skipped)."""
    _kv4_rows("fp8q_kv4_write", k, v, slots, cache, stream)


def fp8q_kv4_read(k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, cache: Kv4Cache, stream=None) -> None:
    """Reads slot slots[t] of the cache into k[t] and v[t] [T, heads, D] (zeros for a slot outside
    the cache)."""
    _kv4_rows("fp8q_kv4_read", k, v, slots, cache, stream)


def kv4_read(cache: Kv4Cache, slots: torch.Tensor, dtype: torch.dtype = torch.bfloat16,
             stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """Allocating form of fp8q_kv4_read: (k, v) as [T, heads, D] of dtype."""
    shape = (slots.numel(), cache.k.shape[2], 2 * cache.k.shape[3])
    with _allocating_on(stream, slots.device):
        k, v = (torch.empty(shape, dtype=dtype, device=slots.device) for _ in range(2))
    fp8q_kv4_read(k, v, slots, cache, stream)
    return k, v


def fp8q_kv4_attention_workspace_size(dtype: torch.dtype, seqs: int, tokens: int, heads: int, kv_heads: int,
                                      head_dim: int, max_kv_tokens: int) -> int:
    """Bytes of workspace with which fp8q_kv4_attention splits long caches over more of the
    current device (0: it needs none). max_kv_tokens is the page table's width times page_size."""
    return int(load_library().fp8q_kv4_attention_workspace_size(_DTYPES[dtype], seqs, tokens, heads, kv_heads,
                                                                head_dim, max_kv_tokens))


def _kv4_attend(entry: str, sizes: tuple, extra: tuple, q, cache, block_table, kv_lens, out, sm_scale, q_indptr, lse,
                stream, workspace) -> None:
    """Checks and call of the attention entries: `extra` are the C arguments after sm_scale, `sizes` what the size of
    the workspace depends on besides the shape."""
    shape, dt = q.shape, _DTYPES.get(q.dtype, DTYPE_F32)
    if len(shape) != 3 or dt == DTYPE_F32:
        raise ValueError("q must be a [T, heads, D] bf16 or fp16 tensor")
    T, H, D = shape
    if out.dtype != q.dtype or out.shape != shape:
        raise ValueError("out must have q's shape and type")
    q_st, q_sh, q_in = q.stride()
    o_st, o_sh, o_in = out.stride()
    if (q_in != 1 or o_in != 1) and q.numel() > 0:
        raise ValueError("innermost dimensions must be contiguous")
    B = _dev_i32(kv_lens, "kv_lens").numel()
    if block_table.dtype != torch.int32 or not block_table.is_cuda or block_table.dim() != 2:
        raise ValueError("block_table must be a device int32 [B, max_pages] tensor")
    rows, max_pages = block_table.shape
    table_sb, table_in = block_table.stride()
    if rows != B or (table_in != 1 and max_pages > 1):
        raise ValueError("block_table must have contiguous rows, one per sequence")
    ip_ptr = lse_ptr = None
    l_st = 0
    if q_indptr is not None:
        if _dev_i32(q_indptr, "q_indptr").numel() != B + 1:
            raise ValueError("q_indptr needs B + 1 entries")
        ip_ptr = q_indptr.data_ptr()
    if lse is not None:
        if lse.dtype != torch.float32 or lse.shape != (T, H) or (H > 1 and lse.stride(1) != 1):
            raise ValueError("lse must be a float32 [T, heads] tensor with contiguous rows")
        lse_ptr, l_st = lse.data_ptr(), lse.stride(0)
    page, kv_heads = cache.k.shape[1:3]
    args = _kv4_args(cache, kv_heads, D)
    dev = q.get_device()
    if not kv_lens.get_device() == dev == out.get_device() == block_table.get_device() == cache.k.get_device() \
            or (q_indptr is not None and q_indptr.get_device() != dev) \
            or (lse is not None and lse.get_device() != dev) \
            or (workspace is not None and workspace.get_device() != dev):
        raise ValueError(_ELSEWHERE)
    handle = _stream_here(stream, dev)
    if handle is None:
        with torch.cuda.device(dev):
            return _kv4_attend(entry, sizes, extra, q, cache, block_table, kv_lens, out, sm_scale, q_indptr, lse, stream,
                               workspace)
    lib = load_library()
    ws_ptr, ws_bytes = None, 0
    if workspace is None:
        size = getattr(lib, entry + "_workspace_size")(dt, B, T, H, kv_heads, D, max_pages * page, *sizes)
        if size > 0:
            workspace = _alloc_workspace(size, q.device, stream)
    if workspace is not None:
        ws_ptr, ws_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    _check(getattr(lib, entry)(
        q.data_ptr(), dt, q_st, q_sh, *args, block_table.data_ptr(), table_sb, max_pages, kv_lens.data_ptr(), ip_ptr,
        out.data_ptr(), o_st, o_sh, lse_ptr, l_st, B, T, H, kv_heads, D, sm_scale, *extra, ws_ptr, ws_bytes, handle))


def fp8q_kv4_attention(q: torch.Tensor, cache: Kv4Cache, block_table: torch.Tensor, kv_lens: torch.Tensor,
                       out: torch.Tensor, sm_scale: float, causal: bool = True,
                       q_indptr: torch.Tensor | None = None, lse: torch.Tensor | None = None, stream=None,
                       workspace: torch.Tensor | None = None) -> None:
    """out[t, h] = softmax(sm_scale * q[t, h] k^T) v over the cached tokens that the query sees.
    q, out [T, heads, D] (bf16 or fp16); block_table int32 [B, max_pages]; kv_lens int32 [B];
    q_indptr int32 [B + 1]: sequence b's queries are rows q_indptr[b] .. q_indptr[b + 1] - 1 (None: row
    b, T == B). causal: the last query of a sequence sees all its cached tokens, the one before it
    one less, ... lse [T, heads] fp32 receives the logarithm of each row's softmax sum. The probabilities
    multiply the values in 16 bits for fp16 outputs and in bf16 for bf16 ones.
    When the shape can use a workspace and none is given, one is taken from torch's allocator."""
    _kv4_attend("fp8q_kv4_attention", (), (causal,), q, cache, block_table, kv_lens, out, sm_scale, q_indptr, lse, stream,
                workspace)


def kv4_attention(q: torch.Tensor, cache: Kv4Cache, block_table: torch.Tensor, kv_lens: torch.Tensor,
                  sm_scale: float, causal: bool = True, q_indptr: torch.Tensor | None = None,
                  stream=None) -> torch.Tensor:
    """Allocating form of fp8q_kv4_attention (rows of q in no sequence are left unset)."""
    with _allocating_on(stream, q.device):
        out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    fp8q_kv4_attention(q, cache, block_table, kv_lens, out, sm_scale, causal, q_indptr, None, stream)
    return out


def fp8q_kv4_window_attention_workspace_size(dtype: torch.dtype, seqs: int, tokens: int, heads: int, kv_heads: int,
                                             head_dim: int, max_kv_tokens: int, window: int, sinks: int = 0) -> int:
    """Bytes of workspace with which fp8q_kv4_window_attention splits long windows over more of the current device
    (0: it needs none)."""
    return int(load_library().fp8q_kv4_window_attention_workspace_size(_DTYPES[dtype], seqs, tokens, heads, kv_heads,
                                                                       head_dim, max_kv_tokens, window, sinks))


def fp8q_kv4_window_attention(q: torch.Tensor, cache: Kv4Cache, block_table: torch.Tensor, kv_lens: torch.Tensor,
                              out: torch.Tensor, sm_scale: float, window: int, sinks: int = 0,
                              q_indptr: torch.Tensor | None = None, lse: torch.Tensor | None = None, stream=None,
                              workspace: torch.Tensor | None = None) -> None:
    """fp8q_kv4_attention (causal) in which a query sees the last `window` tokens up to and with its own, and the
    first `sinks` of its sequence. The probabilities have 16 bits for both types."""
    _kv4_attend("fp8q_kv4_window_attention", (window, sinks), (window, sinks), q, cache, block_table, kv_lens, out, sm_scale,
                q_indptr, lse, stream, workspace)


def kv4_window_attention(q: torch.Tensor, cache: Kv4Cache, block_table: torch.Tensor, kv_lens: torch.Tensor,
                         sm_scale: float, window: int, sinks: int = 0, q_indptr: torch.Tensor | None = None,
                         stream=None) -> torch.Tensor:
    """Allocating form of fp8q_kv4_window_attention (rows of q in no sequence are left unset)."""
    with _allocating_on(stream, q.device):
        out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    fp8q_kv4_window_attention(q, cache, block_table, kv_lens, out, sm_scale, window, sinks, q_indptr, None, stream)
    return out


def fp8q_kv4_tree_attention_workspace_size(dtype: torch.dtype, seqs: int, tokens: int, heads: int, kv_heads: int,
                                           head_dim: int, max_kv_tokens: int) -> int:
    """Bytes of workspace with which fp8q_kv4_tree_attention splits long caches over more of the current device (0: it
    needs none)."""
    return int(load_library().fp8q_kv4_tree_attention_workspace_size(_DTYPES[dtype], seqs, tokens, heads, kv_heads,
                                                                     head_dim, max_kv_tokens))


def fp8q_kv4_tree_attention(q: torch.Tensor, cache: Kv4Cache, block_table: torch.Tensor, kv_lens: torch.Tensor,
                            out: torch.Tensor, sm_scale: float, tree_mask: torch.Tensor,
                            q_indptr: torch.Tensor | None = None, lse: torch.Tensor | None = None, stream=None,
                            workspace: torch.Tensor | None = None) -> None:
    """fp8q_kv4_attention for drafted tokens that form a tree: a sequence's n rows of q are held at its last n cached
    places; each sees every token before them, and drafted token j if bit j % 32 of word j // 32 of its row of
    tree_mask (int32 [T, words]) is set. The probabilities have 16 bits for both types."""
    if tree_mask.dtype != torch.int32 or tree_mask.dim() != 2 or tree_mask.shape[0] != q.shape[0] \
            or (tree_mask.shape[1] > 1 and tree_mask.stride(1) != 1):
        raise ValueError("tree_mask must be an int32 [T, words] tensor with contiguous rows")
    if tree_mask.get_device() != q.get_device():
        raise ValueError(_ELSEWHERE)
    _kv4_attend("fp8q_kv4_tree_attention", (), (tree_mask.data_ptr(), tree_mask.stride(0), tree_mask.shape[1]), q, cache,
                block_table, kv_lens, out, sm_scale, q_indptr, lse, stream, workspace)


def kv4_tree_attention(q: torch.Tensor, cache: Kv4Cache, block_table: torch.Tensor, kv_lens: torch.Tensor,
                       sm_scale: float, tree_mask: torch.Tensor, q_indptr: torch.Tensor | None = None,
                       stream=None) -> torch.Tensor:
    """Allocating form of fp8q_kv4_tree_attention (rows of q in no sequence are left unset)."""
    with _allocating_on(stream, q.device):
        out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    fp8q_kv4_tree_attention(q, cache, block_table, kv_lens, out, sm_scale, tree_mask, q_indptr, None, stream)
    return out


def fp8q_kv4_plan(kv_lens: torch.Tensor, q_lens: torch.Tensor, free_pages: torch.Tensor, block_table: torch.Tensor,
                  pages: int, page_size: int, new_lens: torch.Tensor, q_indptr: torch.Tensor, slots: torch.Tensor,
                  pages_taken: torch.Tensor, positions: torch.Tensor | None = None, stream=None) -> None:
    """One serving step's page bookkeeping for a cache of `pages` pages: sequence b holds kv_lens[b] tokens and gets
    q_lens[b] new ones. Writes the entries of block_table [B, max_pages] for the pages that are new, taken in order from
    free_pages; new_lens [B]; q_indptr [B + 1]; the slot (and position) of every new token [T], -1 past the last
    one; and pages_taken [1], how many pages were needed (more than free_pages holds: the missing ones are
    -1). All int32 on one GPU; no written tensor may share memory with another."""
    # written for few interpreter steps: at a decode step the checks are most of the call's time
    i32 = torch.int32
    if not (kv_lens.dtype == q_lens.dtype == free_pages.dtype == block_table.dtype == new_lens.dtype == q_indptr.dtype
            == slots.dtype == pages_taken.dtype == i32) or (positions is not None and positions.dtype != i32):
        raise ValueError("every tensor must be int32")
    dev = kv_lens.get_device()
    if not 0 <= dev == q_lens.get_device() == free_pages.get_device() == block_table.get_device() == new_lens.get_device() \
            == q_indptr.get_device() == slots.get_device() == pages_taken.get_device() \
            or (positions is not None and positions.get_device() != dev):
        raise ValueError(_ELSEWHERE)
    handle = _stream_here(stream, dev)
    if handle is None:
        with torch.cuda.device(dev):
            return fp8q_kv4_plan(kv_lens, q_lens, free_pages, block_table, pages, page_size, new_lens, q_indptr, slots,
                                 pages_taken, positions, stream)
    shape = kv_lens.shape
    if len(shape) != 1 or block_table.dim() != 2 or slots.dim() != 1 or free_pages.dim() != 1:
        raise ValueError("kv_lens, slots and free_pages must be 1-D, block_table 2-D")
    B, T, F = shape[0], slots.shape[0], free_pages.shape[0]
    rows, max_pages = block_table.shape
    if q_lens.shape != shape or new_lens.shape != shape or rows != B or q_indptr.shape != (B + 1,) \
            or pages_taken.numel() != 1 or (positions is not None and positions.shape != slots.shape):
        raise ValueError("expected q_lens and new_lens [B], block_table [B, max_pages], q_indptr [B + 1], positions [T] "
                         "and pages_taken [1]")
    table_sb, table_in = block_table.stride()
    if (table_in != 1 and max_pages > 1) or not (
            kv_lens.is_contiguous() and q_lens.is_contiguous() and new_lens.is_contiguous() and q_indptr.is_contiguous()
            and slots.is_contiguous() and free_pages.is_contiguous()
            and (positions is None or positions.is_contiguous())):
        raise ValueError("every tensor must be contiguous (block_table: its rows)")
    _check(load_library().fp8q_kv4_plan(
        kv_lens.data_ptr(), q_lens.data_ptr(), B, free_pages.data_ptr(), F, block_table.data_ptr(), table_sb, max_pages, pages,
        page_size, new_lens.data_ptr(), q_indptr.data_ptr(), slots.data_ptr(),
        None if positions is None else positions.data_ptr(), T, pages_taken.data_ptr(), handle))


class Kv4Plan(NamedTuple):
    """What fp8q_kv4_plan writes besides the block table."""
    kv_lens: torch.Tensor
    q_indptr: torch.Tensor
    slots: torch.Tensor
    positions: torch.Tensor
    pages_taken: torch.Tensor


def kv4_plan(cache: Kv4Cache, kv_lens: torch.Tensor, q_lens: torch.Tensor, free_pages: torch.Tensor,
             block_table: torch.Tensor, tokens: int, stream=None) -> Kv4Plan:
    """Allocating form of fp8q_kv4_plan for a cache and at most `tokens` new tokens."""
    B = kv_lens.numel()
    with _allocating_on(stream, kv_lens.device):
        new, ends, slots, positions, taken = (torch.empty(n, dtype=torch.int32, device=kv_lens.device)
                                              for n in (B, B + 1, tokens, tokens, 1))
    fp8q_kv4_plan(kv_lens, q_lens, free_pages, block_table, cache.k.shape[0], cache.k.shape[1], new, ends, slots, taken,
                  positions, stream)
    return Kv4Plan(new, ends, slots, positions, taken)


def fp8q_device_check(device: int = 0) -> int:
    return load_library().fp8q_device_check(device)


def fp8q_status_string(status: int) -> str:
    return _status_string(status)


def fp8q_last_error() -> str:
    return load_library().fp8q_last_error().decode()
