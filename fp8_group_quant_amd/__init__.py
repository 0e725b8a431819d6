"""Python binding of libfp8q.so: per-token-group FP8 quantization, block-scaled FP8 GEMMs,
and the operators between them in a serving layer (quantizing norm, 4-bit key/value cache,
attention over it) for AMD Instinct MI355X (gfx950).

This module only marshals torch tensors (device memory, strides, the current HIP
stream) into the C ABI declared in include/fp8q.h; every step of the computation runs
in the library's HIP kernels. The functions named fp8q_* mirror the C entry points one
to one and write into caller-allocated tensors; group_quant() additionally allocates
its outputs (the role of _allocate_outputs in the sglang PR #30924 design, prhub
report section "实现拆解" item 2), as do rms_norm_group_quant(), kv4_read() and
kv4_attention(); alloc_kv4_cache() allocates a cache.

There is no fallback: if libfp8q.so is missing or the device is not a gfx950, calls
raise.
"""
from __future__ import annotations

import contextlib
import ctypes
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


_WS_SIZES: dict = {}


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
    key = (torch.cuda.current_device(), M, N, K, mode)
    if key not in _WS_SIZES:
        _WS_SIZES[key] = int(load_library().fp8q_gemm_workspace_size(M, N, K, mode))
    return _WS_SIZES[key]


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


def fp8q_kv4_attention(q: torch.Tensor, cache: Kv4Cache, block_table: torch.Tensor, kv_lens: torch.Tensor,
                       out: torch.Tensor, sm_scale: float, causal: bool = True,
                       q_indptr: torch.Tensor | None = None, lse: torch.Tensor | None = None, stream=None,
                       workspace: torch.Tensor | None = None) -> None:
    """out[t, h] = softmax(sm_scale * q[t, h] k^T) v over the cached tokens that the query sees.
    q, out [T, heads, D] (bf16 or fp16); block_table int32 [B, max_pages]; kv_lens int32 [B];
    q_indptr int32 [B + 1]: sequence b's queries are rows q_indptr[b] .. q_indptr[b + 1] - 1 (None: row
    b, T == B). causal: the last query of a sequence sees all its cached tokens, the one before it
    one less, ... lse [T, heads] fp32 receives the logarithm of each row's softmax sum.
    When the shape can use a workspace and none is given, one is taken from torch's allocator."""
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
    if not kv_lens.get_device() == q.get_device() == out.get_device() == block_table.get_device() == cache.k.get_device() \
            or (q_indptr is not None and q_indptr.get_device() != q.get_device()) \
            or (lse is not None and lse.get_device() != q.get_device()) \
            or (workspace is not None and workspace.get_device() != q.get_device()):
        raise ValueError(_ELSEWHERE)
    lib = load_library()
    if workspace is None:
        workspace = _alloc_workspace(
            lib.fp8q_kv4_attention_workspace_size(dt, B, T, H, kv_heads, D, max_pages * page), q.device, stream)
    _check(lib.fp8q_kv4_attention(
        q.data_ptr(), dt, q_st, q_sh, *args, block_table.data_ptr(), table_sb, max_pages, kv_lens.data_ptr(), ip_ptr,
        out.data_ptr(), o_st, o_sh, lse_ptr, l_st, B, T, H, kv_heads, D, sm_scale, causal,
        None if workspace is None else workspace.data_ptr(),
        0 if workspace is None else workspace.numel() * workspace.element_size(), _stream(stream)))


def kv4_attention(q: torch.Tensor, cache: Kv4Cache, block_table: torch.Tensor, kv_lens: torch.Tensor,
                  sm_scale: float, causal: bool = True, q_indptr: torch.Tensor | None = None,
                  stream=None) -> torch.Tensor:
    """Allocating form of fp8q_kv4_attention (rows of q in no sequence are left unset)."""
    with _allocating_on(stream, q.device):
        out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    fp8q_kv4_attention(q, cache, block_table, kv_lens, out, sm_scale, causal, q_indptr, None, stream)
    return out


def fp8q_device_check(device: int = 0) -> int:
    return load_library().fp8q_device_check(device)


def fp8q_status_string(status: int) -> str:
    return _status_string(status)


def fp8q_last_error() -> str:
    return load_library().fp8q_last_error().decode()
