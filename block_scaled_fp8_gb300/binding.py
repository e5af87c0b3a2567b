"""Thin Python binding of the C ABI in include/dg.h (argument marshalling only).

Every function takes torch tensors that already live on the current CUDA
device, passes their data pointers and the current torch stream to the
library, and raises DGError on a non-OK status.  All arithmetic happens in
the library's CUDA kernels; nothing here computes.  The library must have
been built (block_scaled_fp8_gb300.build) -- there is no fallback.
"""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import os
import threading

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_build", "libdg_gb300.so")

DG_SF_FP32 = 0
DG_SF_UE8M0_PACKED = 1
DG_DEV_TIMEOUT = 1
DG_DEV_INEXACT_SCALE = 2
DG_DEV_BAD_GROUP = 4
DG_DEBUG_DROP_ONE_LOAD = 1
DG_DEBUG_PRINT_CONFIGS = 2
DG_DEBUG_SINGLE_CTA = 4
DG_DEBUG_WIDE_PAIR = 8
DG_LOGITS_F32 = 0
DG_LOGITS_BF16 = 1
DG_VALUES_F32 = 0
DG_VALUES_BF16 = 1
DG_SCORE_SOFTMAX = 0
DG_SCORE_SIGMOID = 1

# Every symbol include/dg.h declares.
EXPORTS = (
    "dg_fp8_gemm_nt", "dg_fp8_gemm_nt_f32", "dg_fp8_gemm_nn", "dg_fp8_gemm_tn", "dg_fp8_gemm_tt",
    "dg_fp8_fp4_gemm_nt", "dg_m_grouped_fp8_fp4_gemm_nt_contiguous", "dg_m_grouped_fp8_fp4_gemm_nt_masked",
    "dg_transform_sf", "dg_m_grouped_fp8_gemm_nt_contiguous", "dg_m_grouped_fp8_gemm_nt_contiguous_psum",
    "dg_k_grouped_fp8_gemm_tn_contiguous", "dg_transform_sf_k_grouped", "dg_k_grouped_packed_sf_rows",
    "dg_k_grouped_fp8_gemm_tn_contiguous_k32", "dg_transform_sf_k_grouped_k32",
    "dg_m_grouped_fp8_gemm_nt_masked", "dg_get_mk_alignment_for_contiguous_layout",
    "dg_get_tma_aligned_size", "dg_packed_sf_words", "dg_set_num_sms", "dg_get_num_sms",
    "dg_set_wait_timeout_ms", "dg_set_debug_flags", "dg_status_string", "dg_get_last_config",
    "dg_bf16_fp4_gemv_nt", "dg_bf16_fp8_gemv_nt", "dg_bf16_fp4_gemv_nt_f32", "dg_bf16_fp8_gemv_nt_f32",
    "dg_bf16_gemv_workspace_bytes", "dg_moe_route", "dg_moe_layer_workspace_bytes", "dg_moe_fp4_layer", "dg_moe_fp8_layer",
    "dg_fp8_gated_gemm_nt", "dg_m_grouped_fp8_gated_gemm_nt_contiguous", "dg_fp8_gated_gemm_nn_backward",
    "dg_m_grouped_fp8_gated_gemm_nn_backward_contiguous", "dg_quantize_fp8", "dg_quantize_fp8_blocks",
    "dg_newton_schulz", "dg_newton_schulz_workspace_bytes",
)


class DGError(RuntimeError):
    def __init__(self, fn: str, status: int, name: str):
        super().__init__(f"{fn} failed: {name} ({status})")
        self.status = status
        self.name = name


_lock = threading.Lock()
_lib = None


def lib():
    """Load the CUDA library (raises if it has not been built)."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(
                    f"CUDA library not built: {LIB_PATH} is missing "
                    "(run block_scaled_fp8_gb300.build.build())")
            L = ctypes.CDLL(LIB_PATH)
            P, i32, i64, u32 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_uint32
            L.dg_fp8_gemm_nt.argtypes = [P, i64, P, i32, P, i64, P, i32, P, i64, P, i64, i32, i32,
                                         i32, P, P]
            for f in ("dg_fp8_gemm_nt_f32", "dg_fp8_gemm_nn", "dg_fp8_gemm_tn", "dg_fp8_gemm_tt"):
                getattr(L, f).argtypes = L.dg_fp8_gemm_nt.argtypes
            L.dg_transform_sf.argtypes = [P, i32, i32, i32, i32, i32, i32, P, P, P]
            L.dg_m_grouped_fp8_gemm_nt_contiguous.argtypes = [P, i64, P, i32, P, i64, P, i32, P,
                                                              i64, P, i32, i32, i32, i32, P, P]
            L.dg_m_grouped_fp8_gemm_nt_contiguous_psum.argtypes = \
                L.dg_m_grouped_fp8_gemm_nt_contiguous.argtypes
            L.dg_m_grouped_fp8_gemm_nt_masked.argtypes = [P, P, i32, P, P, i32, P, P, i32, i32,
                                                          i32, i32, i32, P, P]
            L.dg_fp8_fp4_gemm_nt.argtypes = [P, i64, P, P, i64, P, P, i64, P, i64, i32, i32, i32, P, P]
            L.dg_fp8_fp4_gemm_nt.restype = i32
            L.dg_m_grouped_fp8_fp4_gemm_nt_contiguous.argtypes = [P, i64, P, P, i64, P, P, i64, P, i32, i32, i32,
                                                                  i32, P, P]
            L.dg_m_grouped_fp8_fp4_gemm_nt_masked.argtypes = [P, P, P, P, P, P, i32, i32, i32, i32, i32, P, P]
            for f in ("dg_m_grouped_fp8_fp4_gemm_nt_contiguous", "dg_m_grouped_fp8_fp4_gemm_nt_masked"):
                getattr(L, f).restype = i32
            L.dg_k_grouped_fp8_gemm_tn_contiguous.argtypes = [P, i64, P, P, i64, P, P, P, i32, i32, P, P, i32,
                                                              P, P]
            L.dg_transform_sf_k_grouped.argtypes = [P, i32, P, i32, P, P, P]
            L.dg_k_grouped_fp8_gemm_tn_contiguous_k32.argtypes = L.dg_k_grouped_fp8_gemm_tn_contiguous.argtypes
            L.dg_transform_sf_k_grouped_k32.argtypes = L.dg_transform_sf_k_grouped.argtypes
            L.dg_k_grouped_packed_sf_rows.restype = i64
            L.dg_k_grouped_packed_sf_rows.argtypes = [P, i32]
            for f in ("dg_k_grouped_fp8_gemm_tn_contiguous", "dg_transform_sf_k_grouped",
                      "dg_k_grouped_fp8_gemm_tn_contiguous_k32", "dg_transform_sf_k_grouped_k32"):
                getattr(L, f).restype = i32
            for f in ("dg_fp8_gemm_nt", "dg_fp8_gemm_nt_f32", "dg_fp8_gemm_nn", "dg_fp8_gemm_tn",
                      "dg_fp8_gemm_tt", "dg_transform_sf",
                      "dg_m_grouped_fp8_gemm_nt_contiguous",
                      "dg_m_grouped_fp8_gemm_nt_contiguous_psum", "dg_m_grouped_fp8_gemm_nt_masked"):
                getattr(L, f).restype = i32
            f32 = ctypes.c_float
            for f in ("dg_bf16_fp4_gemv_nt", "dg_bf16_fp8_gemv_nt", "dg_bf16_fp4_gemv_nt_f32",
                      "dg_bf16_fp8_gemv_nt_f32"):
                getattr(L, f).argtypes = [P, i64, P, i64, P, P, i64, P, i64, i32, i32, i32, P, i64, P, P]
                getattr(L, f).restype = i32
            L.dg_bf16_gemv_workspace_bytes.argtypes = [i32, i32, i32]
            L.dg_bf16_gemv_workspace_bytes.restype = i64
            L.dg_moe_route.argtypes = [P, i64, i32, P, P, P, i32, i32, i32, i32, i32, f32, P]
            L.dg_moe_route.restype = i32
            L.dg_moe_layer_workspace_bytes.argtypes = [i32, i32, i32, i32, i32]
            L.dg_moe_layer_workspace_bytes.restype = i64
            for f in ("dg_moe_fp4_layer", "dg_moe_fp8_layer"):
                getattr(L, f).argtypes = [P, i64, P, P, P, P, P, P, P, i64, P, i64, i32, i32, i32, i32, i32, P, i64,
                                          P, P]
                getattr(L, f).restype = i32
            gated = [P, i64, P, P, i64, P, P, i64, P, i64, P, i64, P]
            L.dg_fp8_gated_gemm_nt.argtypes = gated + [i32, i32, i32, P, P]
            L.dg_m_grouped_fp8_gated_gemm_nt_contiguous.argtypes = gated + [P, i32, i32, i32, i32, P, P]
            gated = [P, i64, P, P, i64, P, P, i64, P, i64, P, i64]
            L.dg_fp8_gated_gemm_nn_backward.argtypes = gated + [i32, i32, i32, P, P]
            L.dg_m_grouped_fp8_gated_gemm_nn_backward_contiguous.argtypes = gated + [P, i32, i32, i32, i32, P, P]
            L.dg_quantize_fp8.argtypes = [P, i32, i64, P, i64, P, P, i64, P, i32, i32, P, i32, P]
            L.dg_quantize_fp8_blocks.argtypes = [P, i32, i64, i64, P, i64, i64, P, P, i32, i32, i32, P]
            L.dg_newton_schulz.argtypes = [P, i32, i64, i64, P, i64, i64, i32, i32, i32, i32, f32, f32, f32, f32, P, i64,
                                           P, P]
            L.dg_newton_schulz.restype = i32
            L.dg_newton_schulz_workspace_bytes.argtypes = [i32, i32, i32]
            L.dg_newton_schulz_workspace_bytes.restype = i64
            L.dg_quantize_fp8.restype = L.dg_quantize_fp8_blocks.restype = i32
            for f in ("dg_fp8_gated_gemm_nt", "dg_m_grouped_fp8_gated_gemm_nt_contiguous",
                      "dg_fp8_gated_gemm_nn_backward", "dg_m_grouped_fp8_gated_gemm_nn_backward_contiguous"):
                getattr(L, f).restype = i32
            L.dg_get_mk_alignment_for_contiguous_layout.restype = i32
            L.dg_get_mk_alignment_for_contiguous_layout.argtypes = []
            L.dg_get_tma_aligned_size.restype = i64
            L.dg_get_tma_aligned_size.argtypes = [i64, i32]
            L.dg_packed_sf_words.restype = i64
            L.dg_packed_sf_words.argtypes = [i32, i32, i32]
            L.dg_set_num_sms.restype = None
            L.dg_set_num_sms.argtypes = [i32]
            L.dg_get_num_sms.restype = i32
            L.dg_get_num_sms.argtypes = []
            L.dg_set_wait_timeout_ms.restype = None
            L.dg_set_wait_timeout_ms.argtypes = [i32]
            L.dg_set_debug_flags.restype = None
            L.dg_set_debug_flags.argtypes = [u32]
            L.dg_status_string.restype = ctypes.c_char_p
            L.dg_status_string.argtypes = [i32]
            L.dg_get_last_config.restype = None
            L.dg_get_last_config.argtypes = [ctypes.POINTER(ctypes.c_int)]
            _lib = L
    return _lib


def _check(fn: str, status: int):
    if status != 0:
        raise DGError(fn, status, lib().dg_status_string(status).decode())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _p(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _sf_fmt(t):
    return DG_SF_FP32 if t.dtype == torch.float32 else DG_SF_UE8M0_PACKED


# --------------------------------------------------------------------- utilities

def get_mk_alignment_for_contiguous_layout() -> int:
    return int(lib().dg_get_mk_alignment_for_contiguous_layout())


def get_tma_aligned_size(mn: int, elem_size: int) -> int:
    return int(lib().dg_get_tma_aligned_size(mn, elem_size))


def packed_sf_words(batch: int, mn: int, k: int) -> int:
    return int(lib().dg_packed_sf_words(batch, mn, k))


def set_num_sms(n: int):
    lib().dg_set_num_sms(n)


def get_num_sms() -> int:
    return int(lib().dg_get_num_sms())


def set_wait_timeout_ms(ms: int):
    lib().dg_set_wait_timeout_ms(ms)


def set_debug_flags(flags: int):
    lib().dg_set_debug_flags(flags)


def last_config() -> dict:
    arr = (ctypes.c_int * 6)()
    lib().dg_get_last_config(arr)
    return {"block_m": arr[0], "block_n": arr[1], "stages": arr[2], "grid": arr[3],
            "kind": arr[4], "launches": arr[5]}


# --------------------------------------------------------------------- entry points

def dg_transform_sf(sf: torch.Tensor, gran_mn: int, mn: int, out: torch.Tensor,
                    packed: bool = True, status: torch.Tensor | None = None, stream=None):
    """sf: float32 [batch?, mn_rows, sf_k] -> out (int32 packed [batch?, psf_k, align4(mn)]
    or float32 [batch?, sf_k, align4(mn)])."""
    assert sf.dtype == torch.float32 and sf.is_contiguous() and out.is_contiguous()
    s = sf if sf.dim() == 3 else sf.unsqueeze(0)
    batch, mn_rows, sf_k = s.shape
    _check("dg_transform_sf", lib().dg_transform_sf(
        _p(s), batch, mn_rows, sf_k, gran_mn, mn, DG_SF_UE8M0_PACKED if packed else DG_SF_FP32,
        _p(out), _p(status), _stream(stream)))
    return out


def transform_sf(sf: torch.Tensor, gran_mn: int, mn: int, packed: bool = True,
                 status: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Allocates the output with torch and calls dg_transform_sf."""
    batch = () if sf.dim() == 2 else (sf.shape[0],)
    sf_k = sf.shape[-1]
    stride = (mn + 3) // 4 * 4
    if packed:
        out = torch.empty(*batch, (sf_k + 3) // 4, stride, dtype=torch.int32, device=sf.device)
    else:
        out = torch.empty(*batch, sf_k, stride, dtype=torch.float32, device=sf.device)
    return dg_transform_sf(sf, gran_mn, mn, out, packed=packed, status=status, stream=stream)


def dg_fp8_gemm_nt(a: torch.Tensor, sfa: torch.Tensor, b: torch.Tensor, sfb: torch.Tensor,
                   d: torch.Tensor, c: torch.Tensor | None = None,
                   status: torch.Tensor | None = None, stream=None):
    """D = C + A @ B^T.  a [M, K] and b [N, K] float8_e4m3fn (row stride = stride(0));
    sfa/sfb packed int32 (MN-major) or float32 ([M, sf_k] / [ceil(N/128), sf_k]);
    d (and c) bf16 [M, N] with unit column stride."""
    M, K = a.shape
    N = b.shape[0]
    assert a.stride(1) == 1 and b.stride(1) == 1 and d.stride(1) == 1
    assert d.dtype == torch.bfloat16 and (c is None or (c.dtype == torch.bfloat16 and c.stride(1) == 1))
    _check("dg_fp8_gemm_nt", lib().dg_fp8_gemm_nt(
        _p(a), a.stride(0), _p(sfa), _sf_fmt(sfa), _p(b), b.stride(0), _p(sfb), _sf_fmt(sfb),
        _p(c), 0 if c is None else c.stride(0), _p(d), d.stride(0), M, N, K, _p(status),
        _stream(stream)))
    return d


def dg_fp8_gemm_nt_f32(a: torch.Tensor, sfa: torch.Tensor, b: torch.Tensor, sfb: torch.Tensor,
                       d: torch.Tensor, c: torch.Tensor | None = None,
                       status: torch.Tensor | None = None, stream=None):
    """D = C + A @ B^T with FP32 d (and c) [M, N], unit column stride; scales packed."""
    M, K = a.shape
    N = b.shape[0]
    assert a.stride(1) == 1 and b.stride(1) == 1 and d.stride(1) == 1
    assert d.dtype == torch.float32 and (c is None or (c.dtype == torch.float32 and c.stride(1) == 1))
    _check("dg_fp8_gemm_nt_f32", lib().dg_fp8_gemm_nt_f32(
        _p(a), a.stride(0), _p(sfa), _sf_fmt(sfa), _p(b), b.stride(0), _p(sfb), _sf_fmt(sfb),
        _p(c), 0 if c is None else c.stride(0), _p(d), d.stride(0), M, N, K, _p(status),
        _stream(stream)))
    return d


def _gemm_layout(fn: str, a_mn: bool, b_mn: bool, a, sfa, b, sfb, d, c, status, stream):
    # a is [M, K] (K-contiguous) or [K, M] (M-contiguous); b is [N, K] or [K, N]
    M = a.shape[1] if a_mn else a.shape[0]
    K = a.shape[0] if a_mn else a.shape[1]
    N = b.shape[1] if b_mn else b.shape[0]
    assert (b.shape[0] if b_mn else b.shape[1]) == K
    assert a.stride(1) == 1 and b.stride(1) == 1 and d.stride(1) == 1
    assert d.dtype == torch.bfloat16 and (c is None or (c.dtype == torch.bfloat16 and c.stride(1) == 1))
    _check(fn, getattr(lib(), fn)(
        _p(a), a.stride(0), _p(sfa), _sf_fmt(sfa), _p(b), b.stride(0), _p(sfb), _sf_fmt(sfb),
        _p(c), 0 if c is None else c.stride(0), _p(d), d.stride(0), M, N, K, _p(status),
        _stream(stream)))
    return d


def dg_fp8_gemm_nn(a, sfa, b, sfb, d, c=None, status=None, stream=None):
    """D = C + A @ B: a [M, K], b [K, N] (N contiguous); packed scales as for the NT call."""
    return _gemm_layout("dg_fp8_gemm_nn", False, True, a, sfa, b, sfb, d, c, status, stream)


def dg_fp8_gemm_tn(a, sfa, b, sfb, d, c=None, status=None, stream=None):
    """D = C + A^T @ B: a [K, M] (M contiguous), b [K, N] (N contiguous)."""
    return _gemm_layout("dg_fp8_gemm_tn", True, True, a, sfa, b, sfb, d, c, status, stream)


def dg_fp8_gemm_tt(a, sfa, b, sfb, d, c=None, status=None, stream=None):
    """D = C + A^T @ B^T: a [K, M] (M contiguous), b [N, K] (K contiguous)."""
    return _gemm_layout("dg_fp8_gemm_tt", True, False, a, sfa, b, sfb, d, c, status, stream)


def dg_fp8_fp4_gemm_nt(a, sfa, b, sfb, d, c=None, status=None, stream=None):
    """D = C + A @ B^T with FP8 A [M, K] (packed 1x128 scales) and FP4 B: b uint8
    [N, K/2], two E2M1 codes per byte (even k in the low nibble), row stride =
    stride(0) bytes; sfb packed int32 [K/128, align4(N)] (4 x 32 K per word)."""
    M, K = a.shape
    N = b.shape[0]
    assert b.dtype == torch.uint8 and b.shape[1] * 2 == K and b.stride(1) == 1
    assert a.stride(1) == 1 and d.stride(1) == 1 and d.dtype == torch.bfloat16
    assert c is None or (c.dtype == torch.bfloat16 and c.stride(1) == 1)
    _check("dg_fp8_fp4_gemm_nt", lib().dg_fp8_fp4_gemm_nt(
        _p(a), a.stride(0), _p(sfa), _p(b), b.stride(0), _p(sfb), _p(c), 0 if c is None else c.stride(0), _p(d),
        d.stride(0), M, N, K, _p(status), _stream(stream)))
    return d


def dg_m_grouped_fp8_fp4_gemm_nt_contiguous(a, sfa, b, sfb, d, grouped_layout, status=None, stream=None):
    """a [M_total, K] E4M3; b uint8 [E, N, K/2] packed E2M1 (row stride = stride(1)
    bytes, expert stride N * stride(1)); sfa packed [ceil(K/512), align4(M_total)];
    sfb packed [E, K/128, align4(N)]; d bf16 [M_total, N]; grouped_layout int32 [M_total]."""
    M, K = a.shape
    E, N, _ = b.shape
    assert b.dtype == torch.uint8 and b.stride(0) == N * b.stride(1) and b.stride(2) == 1
    assert a.stride(1) == 1 and d.stride(1) == 1
    _check("dg_m_grouped_fp8_fp4_gemm_nt_contiguous", lib().dg_m_grouped_fp8_fp4_gemm_nt_contiguous(
        _p(a), a.stride(0), _p(sfa), _p(b), b.stride(1), _p(sfb), _p(d), d.stride(0), _p(grouped_layout), M, N, K,
        E, _p(status), _stream(stream)))
    return d


def dg_m_grouped_fp8_fp4_gemm_nt_masked(a, sfa, b, sfb, d, masked_m, expected_m, status=None, stream=None):
    """a [E, max_m, K] E4M3 contiguous; b uint8 [E, N, K/2] contiguous; sfa packed
    [E, ceil(K/512), align4(max_m)]; sfb packed [E, K/128, align4(N)]; d bf16 [E, max_m, N]."""
    E, max_m, K = a.shape
    N = b.shape[1]
    assert a.is_contiguous() and b.is_contiguous() and d.is_contiguous() and b.dtype == torch.uint8
    _check("dg_m_grouped_fp8_fp4_gemm_nt_masked", lib().dg_m_grouped_fp8_fp4_gemm_nt_masked(
        _p(a), _p(sfa), _p(b), _p(sfb), _p(d), _p(masked_m), E, max_m, int(expected_m), N, K, _p(status),
        _stream(stream)))
    return d


def _ks_host(ks):
    arr = (ctypes.c_int * max(1, len(ks)))(*[int(k) for k in ks])
    return arr


def k_grouped_packed_sf_rows(ks) -> int:
    """Packed scale rows of the K-grouped layout for group sizes ks (-1 if invalid)."""
    return int(lib().dg_k_grouped_packed_sf_rows(_ks_host(ks), len(ks)))


def dg_transform_sf_k_grouped(sf: torch.Tensor, ks, out: torch.Tensor | None = None,
                              status: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """sf FP32 [sum(ks)/128, mn] -> packed int32 [k_grouped_packed_sf_rows(ks), mn]."""
    assert sf.dtype == torch.float32 and sf.is_contiguous()
    mn = sf.shape[1]
    if out is None:
        out = torch.empty(max(0, k_grouped_packed_sf_rows(ks)), mn, dtype=torch.int32, device=sf.device)
    _check("dg_transform_sf_k_grouped", lib().dg_transform_sf_k_grouped(
        _p(sf), mn, _ks_host(ks), len(ks), _p(out), _p(status), _stream(stream)))
    return out


def dg_transform_sf_k_grouped_k32(sf: torch.Tensor, ks, out: torch.Tensor | None = None,
                                  status: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """sf FP32 [sum(ks)/32, mn] (one scale row per 32 rows of K) -> packed int32
    [sum(ks)/128, mn]."""
    assert sf.dtype == torch.float32 and sf.is_contiguous()
    mn = sf.shape[1]
    if out is None:
        out = torch.empty(sum(ks) // 128, mn, dtype=torch.int32, device=sf.device)
    _check("dg_transform_sf_k_grouped_k32", lib().dg_transform_sf_k_grouped_k32(
        _p(sf), mn, _ks_host(ks), len(ks), _p(out), _p(status), _stream(stream)))
    return out


def dg_k_grouped_fp8_gemm_tn_contiguous_k32(a, sfa, b, sfb, d, ks, ks_dev=None, c=None,
                                            status: torch.Tensor | None = None, stream=None):
    """As dg_k_grouped_fp8_gemm_tn_contiguous with scales every 32 rows of K:
    sfa/sfb packed int32 [sum(ks)/128, M] / [sum(ks)/128, N]."""
    K, M = a.shape
    N = b.shape[1]
    assert a.stride(1) == 1 and b.stride(1) == 1 and d.is_contiguous() and d.dtype == torch.float32
    assert c is not None and c.is_contiguous() and c.dtype == torch.float32
    if ks_dev is None:
        ks_dev = torch.tensor(list(ks), dtype=torch.int32, device=d.device)
    _check("dg_k_grouped_fp8_gemm_tn_contiguous_k32", lib().dg_k_grouped_fp8_gemm_tn_contiguous_k32(
        _p(a), a.stride(0), _p(sfa), _p(b), b.stride(0), _p(sfb), _p(c), _p(d), M, N, _ks_host(ks),
        _p(ks_dev), len(ks), _p(status), _stream(stream)))
    return d


def dg_k_grouped_fp8_gemm_tn_contiguous(a, sfa, b, sfb, d, ks, ks_dev=None, c=None,
                                        status: torch.Tensor | None = None, stream=None):
    """D[e] = C[e] + A_e^T B_e.  a [K_total, M] and b [K_total, N] float8_e4m3fn
    (unit column stride, row stride = stride(0)); sfa/sfb packed int32
    [P, M] / [P, N]; c (required, may be d) and d FP32 [E, M, N] contiguous;
    ks host list of group sizes (multiples of 128); ks_dev the same as a
    device int32 tensor (made here if not given)."""
    K, M = a.shape
    N = b.shape[1]
    assert a.stride(1) == 1 and b.stride(1) == 1 and d.is_contiguous() and d.dtype == torch.float32
    assert c is not None and c.is_contiguous() and c.dtype == torch.float32
    if ks_dev is None:
        ks_dev = torch.tensor(list(ks), dtype=torch.int32, device=d.device)
    _check("dg_k_grouped_fp8_gemm_tn_contiguous", lib().dg_k_grouped_fp8_gemm_tn_contiguous(
        _p(a), a.stride(0), _p(sfa), _p(b), b.stride(0), _p(sfb), _p(c), _p(d), M, N, _ks_host(ks),
        _p(ks_dev), len(ks), _p(status), _stream(stream)))
    return d


def dg_m_grouped_fp8_gemm_nt_contiguous(a, sfa, b, sfb, d, grouped_layout,
                                        status: torch.Tensor | None = None, stream=None):
    """a [M_total, K]; b [E, N, K]; sfa packed [psf_k, align4(M_total)];
    sfb packed [E, psf_k, align4(N)]; d bf16 [M_total, N]; grouped_layout int32 [M_total]."""
    M, K = a.shape
    E, N, _ = b.shape
    assert b.stride(0) == N * b.stride(1) and b.stride(2) == 1
    _check("dg_m_grouped_fp8_gemm_nt_contiguous", lib().dg_m_grouped_fp8_gemm_nt_contiguous(
        _p(a), a.stride(0), _p(sfa), _sf_fmt(sfa), _p(b), b.stride(1), _p(sfb), _sf_fmt(sfb),
        _p(d), d.stride(0), _p(grouped_layout), M, N, K, E, _p(status), _stream(stream)))
    return d


def dg_m_grouped_fp8_gemm_nt_contiguous_psum(a, sfa, b, sfb, d, psum,
                                             status: torch.Tensor | None = None, stream=None):
    """As dg_m_grouped_fp8_gemm_nt_contiguous, with psum int32 [E] (device):
    inclusive prefix sums of the experts' row counts; each expert's rows start
    on a multiple of 128 after the previous expert's; gap rows of D get 0."""
    M, K = a.shape
    E, N, _ = b.shape
    assert b.stride(0) == N * b.stride(1) and b.stride(2) == 1
    _check("dg_m_grouped_fp8_gemm_nt_contiguous_psum", lib().dg_m_grouped_fp8_gemm_nt_contiguous_psum(
        _p(a), a.stride(0), _p(sfa), _sf_fmt(sfa), _p(b), b.stride(1), _p(sfb), _sf_fmt(sfb),
        _p(d), d.stride(0), _p(psum), M, N, K, E, _p(status), _stream(stream)))
    return d


def dg_m_grouped_fp8_gemm_nt_masked(a, sfa, b, sfb, d, masked_m, expected_m: int,
                                    status: torch.Tensor | None = None, stream=None):
    """a [E, max_m, K]; b [E, N, K]; sfa packed [E, psf_k, align4(max_m)];
    sfb packed [E, psf_k, align4(N)]; d bf16 [E, max_m, N]; masked_m int32 [E] (device)."""
    E, max_m, K = a.shape
    N = b.shape[1]
    assert a.is_contiguous() and b.is_contiguous() and d.is_contiguous()
    _check("dg_m_grouped_fp8_gemm_nt_masked", lib().dg_m_grouped_fp8_gemm_nt_masked(
        _p(a), _p(sfa), _sf_fmt(sfa), _p(b), _p(sfb), _sf_fmt(sfb), _p(d), _p(masked_m), E, max_m,
        expected_m, N, K, _p(status), _stream(stream)))
    return d


# --------------------------------------------------------------------- decode: few rows, routing, the MoE layer
#
# Calls of a few microseconds: their arguments are checked and marshalled in C
# (csrc/marshal.c), through the tensors' own methods.  A wrong dtype, shape or layout raises
# AssertionError, what the library refuses DGError.

_marshal = None


def _load_marshal():
    global _marshal
    L = lib()
    with _lock:
        if _marshal is None:
            from .build import MARSHAL
            if not os.path.exists(MARSHAL):
                raise RuntimeError(f"{MARSHAL} is missing (run block_scaled_fp8_gb300.build.build(), with "
                                   "Python's headers installed)")
            loader = importlib.machinery.ExtensionFileLoader("dg_marshal", MARSHAL)
            m = importlib.util.module_from_spec(importlib.util.spec_from_file_location("dg_marshal", MARSHAL, loader=loader))
            loader.exec_module(m)
            fns = ("dg_bf16_fp4_gemv_nt", "dg_bf16_fp8_gemv_nt", "dg_bf16_fp4_gemv_nt_f32", "dg_bf16_fp8_gemv_nt_f32",
                   "dg_moe_route", "dg_moe_fp4_layer", "dg_moe_fp8_layer", "dg_bf16_gemv_workspace_bytes",
                   "dg_moe_layer_workspace_bytes", "dg_fp8_gated_gemm_nt", "dg_m_grouped_fp8_gated_gemm_nt_contiguous",
                   "dg_fp8_gated_gemm_nn_backward", "dg_m_grouped_fp8_gated_gemm_nn_backward_contiguous", "dg_quantize_fp8",
                   "dg_quantize_fp8_blocks", "dg_newton_schulz", "dg_newton_schulz_workspace_bytes",
                   "dg_k_grouped_packed_sf_rows")
            m.setup(tuple(ctypes.cast(getattr(L, f), ctypes.c_void_p).value for f in fns),
                    (torch.bfloat16, torch.float32, torch.float8_e4m3fn, torch.uint8, torch.int32),
                    torch._C._cuda_getCurrentRawStream,
                    torch._C._cuda_getDevice if torch.cuda.is_available() else lambda: -2,   # (no tensor is there)
                    _workspace)
            _marshal = m
    return _marshal


def _fail(fn: str, status: int):
    raise DGError(fn, status, lib().dg_status_string(status).decode())


_kept = threading.local()   # .workspaces: {(device, stream): buffer}
_MAX_KEPT = 8
_MAX_KEPT_BYTES = 128 << 20   # of one buffer: 64 tokens, 16 of 1024 experts, 7168 x 2048 take 120 MB


def _workspace(nbytes: int, t, stream):
    """Device memory for a call whose caller gave none.  On the current stream: a buffer kept
    for this stream by this host thread (calls there run one after another), as long as the thread
    lives and uses no more than _MAX_KEPT streams after it; of more than _MAX_KEPT_BYTES, one that goes back
    to the allocator with the call (which gives it to nothing but later work on this stream).  In a graph
    capture: one of its own, which the allocator keeps from other use as long as the capture needs it.
    On a stream that the caller names: the same there, so that the call waits for nothing on the
    current stream."""
    if stream is not None:
        if not isinstance(stream, torch.cuda.Stream):
            stream = torch.cuda.ExternalStream(stream.cuda_stream, device=t.device)
        with torch.cuda.stream(stream):
            return _workspace(nbytes, t, None)
    if nbytes > _MAX_KEPT_BYTES or torch._C._cuda_isCurrentStreamCapturing():
        return torch.empty(nbytes, dtype=torch.uint8, device=t.device)
    i = t.get_device()
    key = (i, torch._C._cuda_getCurrentRawStream(i))
    try:
        kept = _kept.workspaces
    except AttributeError:
        kept = _kept.workspaces = {}
    ws = kept.get(key)
    if ws is None or ws.numel() < nbytes:
        kept.pop(key, None)
        while len(kept) >= _MAX_KEPT:
            del kept[next(iter(kept))]   # the longest there
        ws = kept[key] = torch.empty(max(nbytes, 1 << 20), dtype=torch.uint8, device=t.device)
    return ws


def gemv_workspace_bytes(m: int, n: int, k: int) -> int:
    return int(lib().dg_bf16_gemv_workspace_bytes(m, n, k))


def dg_bf16_fp4_gemv_nt(a, b, sfb, d, c=None, workspace=None, status=None, stream=None):
    """D = C + A @ B^T for 1..64 rows: a bf16 [M, K]; b uint8 [N, K/2], two E2M1 codes
    per byte (even k in the low nibble); sfb packed int32 [K/128, align4(N)] (4 x 32
    K per word); d (and c) bf16 [M, N].  workspace: a device buffer of
    gemv_workspace_bytes(M, N, K) bytes (made here if not given)."""
    st = (_marshal or _load_marshal()).gemv(0, a, b, sfb, d, c, workspace, status, stream)
    if st:
        _fail("dg_bf16_fp4_gemv_nt", st)
    return d


def dg_bf16_fp8_gemv_nt(a, b, sfb, d, c=None, workspace=None, status=None, stream=None):
    """As dg_bf16_fp4_gemv_nt with b float8_e4m3fn [N, K] and sfb packed int32
    [ceil(K/512), align4(N)] (4 x 128 K per word)."""
    st = (_marshal or _load_marshal()).gemv(1, a, b, sfb, d, c, workspace, status, stream)
    if st:
        _fail("dg_bf16_fp8_gemv_nt", st)
    return d


def dg_bf16_fp4_gemv_nt_f32(a, b, sfb, d, c=None, workspace=None, status=None, stream=None):
    """dg_bf16_fp4_gemv_nt with FP32 d (and c)."""
    st = (_marshal or _load_marshal()).gemv(2, a, b, sfb, d, c, workspace, status, stream)
    if st:
        _fail("dg_bf16_fp4_gemv_nt_f32", st)
    return d


def dg_bf16_fp8_gemv_nt_f32(a, b, sfb, d, c=None, workspace=None, status=None, stream=None):
    """dg_bf16_fp8_gemv_nt with FP32 d (and c)."""
    st = (_marshal or _load_marshal()).gemv(3, a, b, sfb, d, c, workspace, status, stream)
    if st:
        _fail("dg_bf16_fp8_gemv_nt_f32", st)
    return d


def dg_moe_route(logits, ids, weights, bias=None, scoring: str = "softmax", renormalize: bool = True,
                 scale: float = 1.0, stream=None):
    """Top-k routing: logits [T, E] float32 or bfloat16 (unit column stride) -> ids int32
    [T, topk] and weights float32 [T, topk] (both contiguous); bias float32 [E]
    shifts the choice only.  scoring "softmax" or "sigmoid"."""
    assert scoring == "softmax" or scoring == "sigmoid"
    st = (_marshal or _load_marshal()).route(logits, ids, weights, bias, scoring == "sigmoid", renormalize, scale, stream)
    if st:
        _fail("dg_moe_route", st)
    return ids, weights


def moe_layer_workspace_bytes(t: int, topk: int, h: int, i: int, experts: int) -> int:
    return int(lib().dg_moe_layer_workspace_bytes(t, topk, h, i, experts))


def dg_moe_fp4_layer(x, ids, weights, w1, sf1, w2, sf2, y, c=None, workspace=None, status=None, stream=None):
    """y = c + sum_j weights[:, j] * W2[e] (silu(W1g[e] x) * (W1u[e] x)), e = ids[:, j] (negative:
    empty slot), for 1..64 tokens.  x bf16 [T, H]; ids int32 and weights float32 [T, topk];
    w1 uint8 [E, 2I, H/2] (gate rows, then up rows) and w2 uint8 [E, H, I/2], packed E2M1;
    sf1 packed int32 [E, H/128, 2I], sf2 [E, I/128, H]; y (and c) bf16 [T, H].  workspace:
    a device buffer of moe_layer_workspace_bytes(T, topk, H, I, E) bytes (made here if not given)."""
    st = (_marshal or _load_marshal()).layer(True, x, ids, weights, w1, sf1, w2, sf2, y, c, workspace, status, stream)
    if st:
        _fail("dg_moe_fp4_layer", st)
    return y


def dg_moe_fp8_layer(x, ids, weights, w1, sf1, w2, sf2, y, c=None, workspace=None, status=None, stream=None):
    """As dg_moe_fp4_layer with float8_e4m3fn w1 [E, 2I, H] and w2 [E, H, I], and scales packed
    4 x 128 K per word: sf1 [E, ceil(H/512), 2I], sf2 [E, ceil(I/512), H]."""
    st = (_marshal or _load_marshal()).layer(False, x, ids, weights, w1, sf1, w2, sf2, y, c, workspace, status, stream)
    if st:
        _fail("dg_moe_fp8_layer", st)
    return y


# --------------------------------------------------------------------- feed-forward training: gated block, quantiser, update
#
# Marshalled in C as the decode calls are: a wrong dtype, shape, layout or device raises
# AssertionError, what the library refuses DGError.

def dg_fp8_gated_gemm_nt(a, sfa, b, sfb, h=None, hq=None, sfh=None, gu=None, status=None, stream=None):
    """silu(A Wg^T) * (A Wu^T) with Wg, Wu the first and second half of b's rows.  a
    float8_e4m3fn [M, K], sfa packed int32 [ceil(K/512), align4(M)]; b float8_e4m3fn
    [2I, K], sfb [ceil(K/512), align4(2I)].  The result goes to h bf16 [M, I], or,
    quantised, to hq float8_e4m3fn [M, I] with sfh packed int32 [ceil(I/512), align4(M)]
    (the down product's A).  gu bf16 [M, 2I], if given, gets gate and up for the
    backward pass.  Returns h or hq."""
    st = (_marshal or _load_marshal()).gated(a, sfa, b, sfb, None, h, hq, sfh, gu, status, stream)
    if st:
        _fail("dg_fp8_gated_gemm_nt", st)
    return h if hq is None else hq


def dg_m_grouped_fp8_gated_gemm_nt_contiguous(a, sfa, b, sfb, grouped_layout, h=None, hq=None, sfh=None, gu=None,
                                              status=None, stream=None):
    """As dg_fp8_gated_gemm_nt with an expert for each 128 rows: b [E, 2I, K], sfb
    [E, ceil(K/512), align4(2I)], grouped_layout int32 [M] (-1: not computed)."""
    assert grouped_layout is not None
    st = (_marshal or _load_marshal()).gated(a, sfa, b, sfb, grouped_layout, h, hq, sfh, gu, status, stream)
    if st:
        _fail("dg_m_grouped_fp8_gated_gemm_nt_contiguous", st)
    return h if hq is None else hq


def dg_fp8_gated_gemm_nn_backward(dy, sfdy, w2, sfw2, gu, dgu, h=None, status=None, stream=None):
    """Gradient of gate and up: dh = dY @ W2, dgu = [dh * up * silu'(gate), dh * silu(gate)].
    dy float8_e4m3fn [M, K], sfdy packed int32 [ceil(K/512), align4(M)]; w2 float8_e4m3fn
    [K, I] (I contiguous), sfw2 [ceil(K/512), align4(I)]; gu and dgu bf16 [M, 2I] (may be one
    buffer); h bf16 [M, I], if given, gets silu(gate) * up again.  Returns dgu."""
    st = (_marshal or _load_marshal()).gated_backward(dy, sfdy, w2, sfw2, None, gu, dgu, h, status, stream)
    if st:
        _fail("dg_fp8_gated_gemm_nn_backward", st)
    return dgu


def dg_m_grouped_fp8_gated_gemm_nn_backward_contiguous(dy, sfdy, w2, sfw2, grouped_layout, gu, dgu, h=None,
                                                       status=None, stream=None):
    """As dg_fp8_gated_gemm_nn_backward with an expert for each 128 rows: w2 [E, K, I], sfw2
    [E, ceil(K/512), align4(I)], grouped_layout int32 [M] (-1: not computed)."""
    assert grouped_layout is not None
    st = (_marshal or _load_marshal()).gated_backward(dy, sfdy, w2, sfw2, grouped_layout, gu, dgu, h, status, stream)
    if st:
        _fail("dg_m_grouped_fp8_gated_gemm_nn_backward_contiguous", st)
    return dgu


def dg_quantize_fp8(x, q=None, sf=None, qk=None, sfk=None, ks=None, stream=None):
    """E4M3 codes and packed scales of x [R, C] (float32 or bfloat16): q float8_e4m3fn [R, C]
    and sf int32 [ceil(C/512), align4(R)] with a scale for each 1x128, qk [R, C] and sfk with one
    for each 128x1 (either pair may be left out).  sfk is int32 [ceil(R/512), align4(C)], or with
    group sizes ks (host list, multiples of 128, in sum R) [k_grouped_packed_sf_rows(ks), C], as
    the K-grouped call takes it.  Returns (q, sf, qk, sfk)."""
    st = (_marshal or _load_marshal()).quantize(x, q, sf, qk, sfk, ks, stream)
    if st:
        _fail("dg_quantize_fp8", st)
    return q, sf, qk, sfk


def dg_quantize_fp8_blocks(x, q, sf=None, sft=None, stream=None):
    """E4M3 codes q and packed scales of x [R, C] or [B, R, C] (float32 or bfloat16) with a scale for
    each 128x128: sf int32 [B, ceil(C/512), align4(R)] for x as B of the NT calls, sft
    [B, ceil(R/512), align4(C)] for x as B of the NN calls (one may be left out).  Returns (q, sf, sft)."""
    st = (_marshal or _load_marshal()).quantize_blocks(x, q, sf, sft, stream)
    if st:
        _fail("dg_quantize_fp8_blocks", st)
    return q, sf, sft


def newton_schulz_workspace_bytes(batch: int, rows: int, cols: int) -> int:
    return int(lib().dg_newton_schulz_workspace_bytes(batch, rows, cols))


def dg_newton_schulz(g, out, steps: int = 5, coef=(3.4445, -4.7750, 2.0315), eps: float = 1e-7, workspace=None,
                     status=None, stream=None):
    """Orthogonalises g [R, C] or [B, R, C] (float32 or bfloat16) into out (bfloat16, same shape): X = g /
    (|g| + eps), then `steps` times X <- a X + (b A + c A A) X with A = X X^T and (a, b, c) = coef
    (X^T X on the right where R > C).  workspace: a device buffer of
    newton_schulz_workspace_bytes(B, R, C) bytes (made here if not given).  Returns out."""
    a, b, c = coef
    st = (_marshal or _load_marshal()).newton_schulz(g, out, steps, a, b, c, eps, workspace, status, stream)
    if st:
        _fail("dg_newton_schulz", st)
    return out
