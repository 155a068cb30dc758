"""ctypes binding of libw4a8moe.so: argument marshalling only.

Every step runs in the library's CUDA kernels; this module allocates outputs
with torch (device memory), passes raw pointers, sizes and the current CUDA
stream, and raises on a non-OK status.  There is no fallback: without the
built library every call raises.
"""
from __future__ import annotations

import ctypes
import importlib.util
import math
import os

import torch

from .build import EXT, LIB

_c_i64 = ctypes.c_int64
_c_int = ctypes.c_int
_c_f32 = ctypes.c_float
_c_vp = ctypes.c_void_p
_c_sz = ctypes.c_size_t

_SIGS = {
    "w4a8_status_string": (ctypes.c_char_p, [_c_int]),
    "w4a8_last_error": (ctypes.c_char_p, []),
    "w4a8_abi_version": (_c_int, []),
    "w4a8_device_error": (_c_int, []),
    "moe_route_topk": (_c_int, [_c_vp, _c_i64, _c_i64, _c_int, _c_int, _c_vp, _c_vp, _c_vp]),
    "moe_permute": (_c_int, [_c_vp, _c_i64, _c_int, _c_i64, _c_vp, _c_vp, _c_vp, _c_vp, _c_sz, _c_vp]),
    "moe_permute_ep": (_c_int, [_c_vp, _c_i64, _c_int, _c_i64, _c_vp, _c_i64, _c_vp, _c_vp, _c_vp, _c_vp, _c_sz,
                                _c_vp]),
    "fp8_quant_per_token_group": (_c_int, [_c_vp, _c_i64, _c_i64, _c_vp, _c_i64, _c_i64, _c_vp, _c_vp, _c_vp,
                                           _c_i64, _c_vp]),
    "fp8_quant_scatter_per_token_group": (_c_int, [_c_vp, _c_i64, _c_i64, _c_vp, _c_int, _c_i64, _c_vp, _c_vp,
                                                   _c_vp, _c_i64, _c_vp]),
    "w4a8_grouped_gemm": (_c_int, [_c_vp, _c_vp, _c_vp, _c_i64, _c_vp, _c_vp, _c_vp, _c_i64, _c_i64, _c_i64,
                                   _c_i64, _c_vp, _c_vp, _c_sz, _c_vp]),
    "w4a8_prepack_weights": (_c_int, [_c_vp, _c_i64, _c_i64, _c_vp, _c_vp]),
    "w4a8_grouped_gemm_silu": (_c_int, [_c_vp, _c_vp, _c_vp, _c_i64, _c_vp, _c_vp, _c_vp, _c_i64, _c_i64, _c_i64,
                                        _c_i64, _c_vp, _c_vp, _c_vp, _c_i64, _c_vp, _c_sz, _c_vp]),
    "w4a8_grouped_gemm_silu_unfused": (_c_int, [_c_vp, _c_vp, _c_vp, _c_i64, _c_vp, _c_vp, _c_vp, _c_i64, _c_i64,
                                                _c_i64, _c_i64, _c_vp, _c_vp, _c_vp, _c_i64, _c_vp, _c_sz, _c_vp]),
    "silu_mul_requant": (_c_int, [_c_vp, _c_i64, _c_i64, _c_vp, _c_vp, _c_vp, _c_i64, _c_vp]),
    "silu_mul_requant_rows": (_c_int, [_c_vp, _c_i64, _c_vp, _c_i64, _c_vp, _c_vp, _c_vp, _c_i64, _c_vp]),
    "moe_unpermute_combine": (_c_int, [_c_vp, _c_vp, _c_vp, _c_i64, _c_int, _c_i64, _c_vp, _c_vp]),
    "w4a8_linear": (_c_int, [_c_vp, _c_vp, _c_vp, _c_i64, _c_vp, _c_vp, _c_i64, _c_i64, _c_i64, _c_vp, _c_vp,
                             _c_sz, _c_vp]),
    "w4a8_workspace_bytes": (_c_sz, [_c_int, _c_i64, _c_i64, _c_i64, _c_i64]),
    "w4a8_linear_split_k": (_c_int, [_c_i64, _c_i64, _c_i64]),
    "w4a8_test_wait_timeout": (_c_int, [ctypes.c_uint64, _c_vp, _c_vp]),
    "w4a8_test_tile_list_limit": (_c_int, [_c_int]),
    "w4a8_grouped_gemm_plan": (_c_int, [_c_i64, _c_i64, _c_i64, ctypes.POINTER(_c_int)]),
    "w4a8_tile_cost": (ctypes.c_double, [_c_int, _c_i64]),
    "w4a8_expected_tile_cost": (ctypes.c_double, [_c_int, ctypes.c_double]),
    "w4a8_moe_forward": (_c_int, [_c_vp, _c_vp, _c_i64, _c_i64, _c_i64, _c_i64, _c_int, _c_int, _c_vp,
                                  _c_vp, _c_vp, _c_vp, _c_vp, _c_vp, _c_sz, _c_vp]),
    "w4a8_moe_workspace_bytes": (_c_sz, [_c_i64, _c_i64, _c_i64, _c_i64, _c_int]),
    "w4a8_moe_forward_ep": (_c_int, [_c_vp, _c_vp, _c_i64, _c_i64, _c_i64, _c_i64, _c_int, _c_int, _c_vp, _c_i64,
                                     _c_vp, _c_vp, _c_vp, _c_vp, _c_vp, _c_vp, _c_sz, _c_vp]),
    "w4a8_moe_forward_noalloc": (_c_int, [_c_vp, _c_vp, _c_i64, _c_i64, _c_i64, _c_i64, _c_int, _c_int, _c_vp,
                                          _c_vp, _c_vp, _c_vp, _c_vp, _c_vp]),
    "w4a8_moe_noalloc_scratch_bytes": (_c_sz, []),
    "w4a8_moe_forward_routed": (_c_int, [_c_vp, _c_vp, _c_vp, _c_i64, _c_i64, _c_i64, _c_i64, _c_int, _c_vp, _c_vp,
                                         _c_vp, _c_vp, _c_vp, _c_vp, _c_sz, _c_vp]),
    "moe_route_grouped_topk": (_c_int, [_c_vp, _c_int, _c_i64, _c_i64, _c_i64, _c_int, _c_int, _c_vp, _c_int, _c_int,
                                        _c_int, _c_int, _c_f32, _c_vp, _c_vp, _c_vp]),
    "block_norm": (_c_int, [_c_vp, _c_i64, _c_int, _c_vp, _c_i64, _c_int, _c_int, _c_vp, _c_vp, _c_vp, _c_i64,
                            _c_i64, _c_i64, _c_int, _c_f32, _c_f32, _c_int, _c_vp, _c_vp, _c_int, _c_f32, _c_i64,
                            _c_i64, _c_vp, _c_i64, _c_vp, _c_i64, _c_vp]),
    "dense_linear": (_c_int, [_c_vp, _c_i64, _c_vp, _c_i64, _c_int, _c_vp, _c_int, _c_int, _c_int, _c_vp, _c_i64,
                              _c_vp, _c_i64, _c_int, _c_i64, _c_i64, _c_i64, _c_vp, _c_sz, _c_vp]),
    "dense_linear_workspace_bytes": (_c_sz, [_c_i64, _c_i64, _c_i64]),
    "rotary_embedding": (_c_int, [_c_vp, _c_i64, _c_i64, _c_int, _c_i64, _c_i64, _c_i64, _c_vp, _c_vp, _c_i64, _c_i64,
                                  _c_vp]),
    "paged_kv_append": (_c_int, [_c_vp, _c_i64, _c_i64, _c_vp, _c_i64, _c_i64, _c_int, _c_i64, _c_vp, _c_vp, _c_vp,
                                 _c_vp, _c_i64, _c_i64, _c_i64, _c_vp, _c_i64, _c_i64, _c_vp]),
    "paged_kv_append_whole": (_c_int, [_c_vp, _c_i64, _c_i64, _c_vp, _c_i64, _c_i64, _c_int, _c_i64, _c_vp, _c_vp, _c_vp,
                                       _c_vp, _c_i64, _c_i64, _c_i64, _c_vp, _c_i64, _c_i64, _c_vp]),
    "paged_attention_decode": (_c_int, [_c_vp, _c_i64, _c_i64, _c_int, _c_i64, _c_vp, _c_f32, _c_i64, _c_vp, _c_i64,
                                        _c_i64, _c_vp, _c_vp, _c_sz, _c_vp]),
    "paged_attention_workspace_bytes": (_c_sz, [_c_i64, _c_i64, _c_i64, _c_i64, _c_int, _c_i64]),
    "fp8_block_linear": (_c_int, [_c_vp, _c_vp, _c_i64, _c_vp, _c_vp, _c_i64, _c_i64, _c_i64, _c_vp, _c_i64, _c_int,
                                  _c_vp]),
    "w4a8_test_paged_attention_way": (_c_int, [_c_int]),
    "w4a8_test_fp8_linear_config": (_c_int, [_c_int, _c_int]),
    "w4a8_test_fp8_linear_without": (_c_int, [_c_int]),
    "w4a8_test_linear_config": (_c_int, [_c_int, _c_int]),
    "w4a8_test_linear_wait": (_c_int, [_c_int, ctypes.c_uint64, _c_vp, _c_vp]),
}


class MoeLayout(ctypes.Structure):
    _fields_ = [(n, ctypes.c_size_t) for n in ("topk_ids", "topk_w", "seg_indptr", "src2dst", "dst2src",
                                               "xq", "xs", "xc", "y13", "hq", "hs", "hc", "y2",
                                               "permute_ws")] + \
               [("scale_ld", ctypes.c_int64), ("total", ctypes.c_size_t)]


class Rotary(ctypes.Structure):
    """w4a8_rotary of the C ABI."""
    _fields_ = [("freqs", _c_vp), ("R", _c_i64), ("start", _c_i64), ("interleaved", _c_int), ("inverse", _c_int),
                ("scale", _c_f32), ("positions", _c_vp), ("positions64", _c_int)]


class PagedCache(ctypes.Structure):
    """w4a8_paged_cache of the C ABI."""
    _fields_ = [("k", _c_vp), ("v", _c_vp)] + \
               [(n, _c_i64) for n in ("k_page", "k_slot", "k_head", "v_page", "v_slot", "v_head")] + \
               [("dtype", _c_int)] + [(n, _c_i64) for n in ("pages", "page_size", "heads", "D")] + \
               [("page_table", _c_vp), ("table_ld", _c_i64), ("table_pages", _c_i64), ("seq_lens", _c_vp),
                ("B", _c_i64), ("k_scale", _c_vp), ("v_scale", _c_vp)]


_lib = None


def load(path: str | None = None):
    """Load the CUDA library (once).  Raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    path = path or LIB
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with w4afp8_mixture_experts_gb300.build.build()")
    lib = ctypes.CDLL(path)
    for name, (res, args) in _SIGS.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    lib.w4a8_moe_workspace_layout.restype = _c_int
    lib.w4a8_moe_workspace_layout.argtypes = [_c_i64, _c_i64, _c_i64, _c_i64, _c_int, ctypes.POINTER(MoeLayout)]
    _lib = lib
    return lib


class W4A8Error(RuntimeError):
    def __init__(self, status, msg):
        super().__init__(f"{msg} ({status})")
        self.status = status


def _check(status: int):
    if status != 0:
        lib = load()
        raise W4A8Error(status, lib.w4a8_last_error().decode())


def _p(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(device=None):
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def scale_ld(m: int) -> int:
    """Leading dimension of an activation-scale tensor [K/128][ld] for m rows."""
    return max(4, (m + 3) // 4 * 4)


def _req(t, dtype, name, ndim=None):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dimensions")


# ---------------------------------------------------------------------------

def moe_route_topk(logits, k: int, renormalize: bool = True):
    _req(logits, torch.float32, "logits", 2)
    T, E = logits.shape
    ids = torch.empty((T, k), dtype=torch.int32, device=logits.device)
    w = torch.empty((T, k), dtype=torch.float32, device=logits.device)
    _check(load().moe_route_topk(_p(logits), T, E, k, int(bool(renormalize)), _p(ids), _p(w), _stream()))
    return ids, w


def moe_permute(topk_ids, E: int):
    _req(topk_ids, torch.int32, "topk_ids", 2)
    T, k = topk_ids.shape
    dev = topk_ids.device
    seg = torch.empty(E + 1, dtype=torch.int64, device=dev)
    s2d = torch.empty(T * k, dtype=torch.int32, device=dev)
    d2s = torch.empty(T * k, dtype=torch.int32, device=dev)
    need = int(load().w4a8_workspace_bytes(1, T * k, 0, 0, E))
    ws = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
    _check(load().moe_permute(_p(topk_ids), T, k, E, _p(seg), _p(s2d), _p(d2s), _p(ws), need, _stream()))
    return seg, s2d, d2s


def moe_permute_ep(topk_ids, E: int, expert_map, E_local: int):
    """One expert-parallel shard's permutation: expert_map int32 [E] (local id or -1).
    Returns (seg_indptr int64 [E_local+1], src2dst int32 [T*k], dst2src int32 [T*k])."""
    _req(topk_ids, torch.int32, "topk_ids", 2)
    _req(expert_map, torch.int32, "expert_map", 1)
    T, k = topk_ids.shape
    dev = topk_ids.device
    seg = torch.empty(E_local + 1, dtype=torch.int64, device=dev)
    s2d = torch.empty(T * k, dtype=torch.int32, device=dev)
    d2s = torch.empty(T * k, dtype=torch.int32, device=dev)
    need = int(load().w4a8_workspace_bytes(1, T * k, 0, 0, E_local))
    ws = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
    _check(load().moe_permute_ep(_p(topk_ids), T, k, E, _p(expert_map), E_local, _p(seg), _p(s2d), _p(d2s), _p(ws),
                                 need, _stream()))
    return seg, s2d, d2s


def fp8_quant_scatter_per_token_group(x, src2dst, k: int, m_out: int):
    """bf16 [T, K] -> codes uint8 [m_out, K], scales and gcorr fp32 [K/128, ld]: row t quantised once and
    written to rows src2dst[t*k + j] (-1 skipped; rows nothing maps to are left zero here)."""
    _req(x, torch.bfloat16, "x", 2)
    _req(src2dst, torch.int32, "src2dst", 1)
    T, K = x.shape
    ld = scale_ld(m_out)
    q = torch.zeros((m_out, K), dtype=torch.uint8, device=x.device)
    s = torch.zeros((max(1, K // 128), ld), dtype=torch.float32, device=x.device)
    c = torch.zeros((max(1, K // 128), ld), dtype=torch.float32, device=x.device)
    _check(load().fp8_quant_scatter_per_token_group(_p(x), T, K, _p(src2dst), k, m_out, _p(q), _p(s), _p(c), ld,
                                                    _stream()))
    return q, s, c


def fp8_quant_per_token_group(x, row_index=None, row_div: int = 1, m_out: int | None = None):
    """bf16 [M, K] -> (E4M3 codes uint8 [M_out, K], scales fp32 [K/128, ld], gcorr fp32 [K/128, ld])."""
    _req(x, torch.bfloat16, "x", 2)
    M, K = x.shape
    if row_index is not None:
        _req(row_index, torch.int32, "row_index", 1)
        m_out = row_index.numel() if m_out is None else m_out
    else:
        m_out = M
    ld = scale_ld(m_out)
    G = K // 128 if K % 128 == 0 else 1
    q = torch.empty((m_out, K), dtype=torch.uint8, device=x.device)
    s = torch.empty((G, ld), dtype=torch.float32, device=x.device)
    c = torch.empty((G, ld), dtype=torch.float32, device=x.device)
    _check(load().fp8_quant_per_token_group(_p(x), M, K, _p(row_index), row_div, m_out, _p(q), _p(s), _p(c), ld,
                                            _stream()))
    return q, s, c


def w4a8_prepack_weights(w):
    """Canonical packed int4 uint8 [..., K/2] -> the GEMMs' prepacked layout (same shape)."""
    _req(w, torch.uint8, "w")
    out = torch.empty_like(w)
    K = w.shape[-1] * 2
    _check(load().w4a8_prepack_weights(_p(w), w.numel() // (K // 2), K, _p(out), _stream()))
    return out


def w4a8_grouped_gemm(A, a_scales, a_gcorr, B_prepacked, b_scales, seg_indptr):
    """A uint8 [M, K], a_scales [K/128, ld], a_gcorr [K/128, ld] or None (the library then computes the
    corrections from A in a workspace), B prepacked uint8 [E, N, K/2], b_scales [E, K/128, N] -> bf16 [M, N]."""
    _req(A, torch.uint8, "A", 2)
    _req(a_scales, torch.float32, "a_scales", 2)
    if a_gcorr is not None:
        _req(a_gcorr, torch.float32, "a_gcorr", 2)
    _req(B_prepacked, torch.uint8, "B_prepacked", 3)
    _req(b_scales, torch.float32, "b_scales", 3)
    _req(seg_indptr, torch.int64, "seg_indptr", 1)
    M, K = A.shape
    E, N, Kh = B_prepacked.shape
    if Kh * 2 != K or seg_indptr.numel() != E + 1 or (a_gcorr is not None and a_gcorr.shape != a_scales.shape):
        raise ValueError("shape mismatch")
    ws = None
    if a_gcorr is None:  # room for the corrections at this call's scale leading dimension
        ws = torch.empty((K // 128) * a_scales.shape[1] * 4, dtype=torch.uint8, device=A.device)
    C = torch.empty((M, N), dtype=torch.bfloat16, device=A.device)
    _check(load().w4a8_grouped_gemm(_p(A), _p(a_scales), _p(a_gcorr), a_scales.shape[1], _p(B_prepacked),
                                    _p(b_scales), _p(seg_indptr), E, N, K, M, _p(C), _p(ws),
                                    0 if ws is None else ws.numel(), _stream()))
    return C


def w4a8_grouped_gemm_silu(A, a_scales, a_gcorr, B_prepacked, b_scales, seg_indptr, fused: bool = True):
    """The w13 grouped GEMM (B_prepacked [E, 2I, K/2]: gate rows then up rows) followed by SiLU-and-Mul
    requantisation -> (codes uint8 [M, I], scales fp32 [I/128, ld], gcorr fp32 [I/128, ld]).  With
    fused=True the requantisation runs in the GEMM's epilogue when the tile plan allows (same bits)."""
    _req(A, torch.uint8, "A", 2)
    _req(a_scales, torch.float32, "a_scales", 2)
    if a_gcorr is not None:
        _req(a_gcorr, torch.float32, "a_gcorr", 2)
    _req(B_prepacked, torch.uint8, "B_prepacked", 3)
    _req(b_scales, torch.float32, "b_scales", 3)
    _req(seg_indptr, torch.int64, "seg_indptr", 1)
    M, K = A.shape
    E, N, Kh = B_prepacked.shape
    if Kh * 2 != K or seg_indptr.numel() != E + 1 or N % 256:
        raise ValueError("shape mismatch")
    I = N // 2
    ld = scale_ld(M)
    need = int(load().w4a8_workspace_bytes(4, M, N, K, E))
    if a_gcorr is None:
        need += (K // 128) * (a_scales.shape[1] - scale_ld(M)) * 4
    ws = torch.empty(max(need, 16), dtype=torch.uint8, device=A.device)
    q = torch.empty((M, I), dtype=torch.uint8, device=A.device)
    s = torch.empty((I // 128, ld), dtype=torch.float32, device=A.device)
    c = torch.empty((I // 128, ld), dtype=torch.float32, device=A.device)
    fn = load().w4a8_grouped_gemm_silu if fused else load().w4a8_grouped_gemm_silu_unfused
    _check(fn(_p(A), _p(a_scales), _p(a_gcorr), a_scales.shape[1], _p(B_prepacked), _p(b_scales), _p(seg_indptr), E,
              I, K, M, _p(q), _p(s), _p(c), ld, _p(ws), ws.numel(), _stream()))
    return q, s, c


def silu_mul_requant(gate_up):
    _req(gate_up, torch.bfloat16, "gate_up", 2)
    M, I2 = gate_up.shape
    I = I2 // 2
    ld = scale_ld(M)
    q = torch.empty((M, I), dtype=torch.uint8, device=gate_up.device)
    s = torch.empty((max(1, I // 128), ld), dtype=torch.float32, device=gate_up.device)
    c = torch.empty((max(1, I // 128), ld), dtype=torch.float32, device=gate_up.device)
    _check(load().silu_mul_requant(_p(gate_up), M, I, _p(q), _p(s), _p(c), ld, _stream()))
    return q, s, c


def moe_unpermute_combine(Y, src2dst, topk_w):
    _req(Y, torch.bfloat16, "Y", 2)
    _req(src2dst, torch.int32, "src2dst", 1)
    _req(topk_w, torch.float32, "topk_w", 2)
    T, k = topk_w.shape
    H = Y.shape[1]
    out = torch.empty((T, H), dtype=torch.bfloat16, device=Y.device)
    _check(load().moe_unpermute_combine(_p(Y), _p(src2dst), _p(topk_w), T, k, H, _p(out), _stream()))
    return out


def linear_workspace_bytes(M: int, N: int, K: int) -> int:
    """Workspace of w4a8_linear (split-K partial sums, and room for the corrections when a_gcorr is None)."""
    return int(load().w4a8_workspace_bytes(3, M, N, K, 1))


def linear_split_k(M: int, N: int, K: int) -> int:
    """K splits w4a8_linear uses for this shape on the current device (1: none)."""
    return int(load().w4a8_linear_split_k(M, N, K))


def w4a8_linear(A, a_scales, a_gcorr, B_prepacked, b_scales, ws=None):
    """A uint8 [M, K], a_scales [K/128, ld], a_gcorr [K/128, ld] or None (computed by the library),
    B prepacked uint8 [N, K/2], b_scales [K/128, N] -> bf16 [M, N]."""
    _req(A, torch.uint8, "A", 2)
    _req(a_scales, torch.float32, "a_scales", 2)
    if a_gcorr is not None:
        _req(a_gcorr, torch.float32, "a_gcorr", 2)
    _req(B_prepacked, torch.uint8, "B_prepacked", 2)
    _req(b_scales, torch.float32, "b_scales", 2)
    M, K = A.shape
    N = B_prepacked.shape[0]
    if ws is None:
        need = linear_workspace_bytes(M, N, K)
        if a_gcorr is None:  # the corrections at this call's scale leading dimension
            need += (K // 128) * (a_scales.shape[1] - scale_ld(M)) * 4
        ws = torch.empty(need, dtype=torch.uint8, device=A.device) if need else None
    C = torch.empty((M, N), dtype=torch.bfloat16, device=A.device)
    _check(load().w4a8_linear(_p(A), _p(a_scales), _p(a_gcorr), a_scales.shape[1], _p(B_prepacked), _p(b_scales),
                              M, N, K, _p(C), _p(ws), 0 if ws is None else ws.numel(), _stream()))
    return C


def moe_workspace_layout(T: int, H: int, I: int, E: int, k: int) -> MoeLayout:
    L = MoeLayout()
    _check(load().w4a8_moe_workspace_layout(T, H, I, E, k, ctypes.byref(L)))
    return L


def w4a8_moe_forward(x, logits, k: int, w13, w13_s, w2, w2_s, renormalize: bool = True, ws=None, out=None):
    """The whole layer.  x bf16 [T, H], logits fp32 [T, E], w13 prepacked uint8 [E, 2I, H/2],
    w13_s fp32 [E, H/128, 2I], w2 prepacked uint8 [E, H, I/2], w2_s fp32 [E, I/128, H] -> bf16 [T, H]."""
    _req(x, torch.bfloat16, "x", 2)
    _req(logits, torch.float32, "logits", 2)
    _req(w13, torch.uint8, "w13", 3)
    _req(w2, torch.uint8, "w2", 3)
    _req(w13_s, torch.float32, "w13_s", 3)
    _req(w2_s, torch.float32, "w2_s", 3)
    T, H = x.shape
    E = logits.shape[1]
    I = w13.shape[1] // 2
    need = int(load().w4a8_moe_workspace_bytes(T, H, I, E, k))
    if ws is None:
        ws = torch.empty(need, dtype=torch.uint8, device=x.device)
    if out is None:
        out = torch.empty((T, H), dtype=torch.bfloat16, device=x.device)
    _check(load().w4a8_moe_forward(_p(x), _p(logits), T, H, I, E, k, int(bool(renormalize)), _p(w13), _p(w13_s),
                                   _p(w2), _p(w2_s), _p(out), _p(ws), ws.numel(), _stream()))
    return out


def w4a8_moe_forward_routed(x, topk_ids, topk_w, w13, w13_s, w2, w2_s, ws=None, out=None):
    """The layer with its routing given (topk_ids int32 [T, k], topk_w fp32 [T, k], as moe_route_grouped_topk returns
    them); everything else as in w4a8_moe_forward.  Every tensor is contiguous and on x's device; ws is a uint8
    workspace of moe_workspace_layout(T, H, I, E, k).total bytes, out bf16 [T, H]."""
    _req(x, torch.bfloat16, "x", 2)
    _req(topk_ids, torch.int32, "topk_ids", 2)
    _req(topk_w, torch.float32, "topk_w", 2)
    _req(w13, torch.uint8, "w13", 3)
    T, H = x.shape
    k = topk_ids.shape[1]
    E, I = w13.shape[0], w13.shape[1] // 2
    if topk_ids.shape[0] != T or topk_w.shape != topk_ids.shape:
        raise ValueError(f"topk_ids and topk_w must have {T} rows and the same shape")
    dev = x.device
    for t, dtype, name, shape in ((topk_ids, torch.int32, "topk_ids", (T, k)), (topk_w, torch.float32, "topk_w", (T, k)),
                                  (w13, torch.uint8, "w13", (E, 2 * I, H // 2)),
                                  (w13_s, torch.float32, "w13_s", (E, H // 128, 2 * I)),
                                  (w2, torch.uint8, "w2", (E, H, I // 2)),
                                  (w2_s, torch.float32, "w2_s", (E, I // 128, H)),
                                  (ws, torch.uint8, "ws", None), (out, torch.bfloat16, "out", (T, H))):
        if t is None and name in ("ws", "out"):
            continue
        _req(t, dtype, name)
        if t.device != dev:
            raise ValueError(f"{name} must be on {dev}, got {t.device}")
        if shape is not None and tuple(t.shape) != shape:
            raise ValueError(f"{name} must have shape {shape}, got {tuple(t.shape)}")
    with torch.cuda.device(dev):
        if ws is None:
            ws = torch.empty(int(load().w4a8_moe_workspace_bytes(T, H, I, E, k)), dtype=torch.uint8, device=dev)
        if out is None:
            out = torch.empty((T, H), dtype=torch.bfloat16, device=dev)
        _check(load().w4a8_moe_forward_routed(_p(x), _p(topk_ids), _p(topk_w), T, H, I, E, k, _p(w13), _p(w13_s),
                                              _p(w2), _p(w2_s), _p(out), _p(ws), ws.numel(), _stream(dev)))
    return out


def w4a8_moe_forward_ep(x, logits, k: int, expert_map, w13, w13_s, w2, w2_s, renormalize: bool = True, ws=None,
                        out=None):
    """One expert-parallel shard of the layer: routing over the E = logits.shape[1] experts, the rest over
    the E_local = w13.shape[0] local experts named by expert_map (int32 [E], local id or -1).  Returns
    this shard's share of the layer output, bf16 [T, H]."""
    _req(x, torch.bfloat16, "x", 2)
    _req(logits, torch.float32, "logits", 2)
    _req(expert_map, torch.int32, "expert_map", 1)
    _req(w13, torch.uint8, "w13", 3)
    _req(w2, torch.uint8, "w2", 3)
    _req(w13_s, torch.float32, "w13_s", 3)
    _req(w2_s, torch.float32, "w2_s", 3)
    T, H = x.shape
    E = logits.shape[1]
    E_local = w13.shape[0]
    I = w13.shape[1] // 2
    need = int(load().w4a8_moe_workspace_bytes(T, H, I, E, k))
    if ws is None:
        ws = torch.empty(need, dtype=torch.uint8, device=x.device)
    if out is None:
        out = torch.empty((T, H), dtype=torch.bfloat16, device=x.device)
    _check(load().w4a8_moe_forward_ep(_p(x), _p(logits), T, H, I, E, k, int(bool(renormalize)), _p(expert_map),
                                      E_local, _p(w13), _p(w13_s), _p(w2), _p(w2_s), _p(out), _p(ws), ws.numel(),
                                      _stream()))
    return out


def w4a8_moe_forward_noalloc(x, logits, k: int, w13, w13_s, w2, w2_s, out, renormalize: bool = True):
    """The whole layer into a caller-given `out`, with the intermediates kept in the
    library's fixed device array instead of a workspace (for callers that cannot
    allocate device memory).  Calls that overlap on the GPU race on that array."""
    _req(x, torch.bfloat16, "x", 2)
    _req(logits, torch.float32, "logits", 2)
    _req(out, torch.bfloat16, "out", 2)
    T, H = x.shape
    E = logits.shape[1]
    I = w13.shape[1] // 2
    _check(load().w4a8_moe_forward_noalloc(_p(x), _p(logits), T, H, I, E, k, int(bool(renormalize)), _p(w13),
                                           _p(w13_s), _p(w2), _p(w2_s), _p(out), _stream()))
    return out


# --- operators around the routed experts -----------------------------------------------------------------------
# Their tensors are marshalled by the extension beside the library (csrc/torch_ops.cpp): the checks, the output
# tensors and the stream lookup cost several times the smallest device times when done here.

_SCORES = {"softmax": 0, "sigmoid": 1}
_NORMS = {"none": 0, "rms": 1, "layer": 2}
_ACTS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4}

_ops = None


def _load_ops():
    """The extension module (once), after the library.  Raises if it has not been built."""
    global _ops
    if _ops is None:
        load()
        if not os.path.exists(EXT):
            raise RuntimeError(f"{EXT} is missing: build it with w4afp8_mixture_experts_gb300.build.build()")
        spec = importlib.util.spec_from_file_location("w4a8_torch_ops", EXT)
        mod = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(mod)
        mod.init(_check)
        _ops = mod
    return _ops


def _one_of(table, value, name):
    got = table.get(value)
    if got is None:
        raise ValueError(f"{name} must be one of {sorted(table)}, got {value!r}")
    return got


def moe_route_grouped_topk(logits, k: int, bias=None, score: str = "sigmoid", n_group: int = 1, topk_group: int = 1,
                           group_top: int = 1, renormalize: bool = True, scale: float = 1.0):
    """Grouped routing.  logits [T, E] fp32, bf16 or f16 (any row stride), bias fp32 [E] or None (choice only) ->
    (ids int32 [T, k], weights fp32 [T, k]).  A logit of -inf (or its type's lowest value, or NaN) takes its expert
    out; see moe_route_grouped_topk in include/w4a8moe.h for the rules."""
    return (_ops or _load_ops()).route(logits, k, bias, _one_of(_SCORES, score, "score"), n_group, topk_group,
                                       group_top, renormalize, scale)


def block_norm(f, residual=None, *, post: str = "none", w_post=None, b_post=None, gate=None, branch_scale: float = 1.0,
               residual_scale: float = 1.0, pre: str = "rms", w_pre=None, b_pre=None, eps: float = 1e-6,
               residual_dtype=None, want_h: bool = True, want_y: bool = True, h=None, y=None):
    """The norms after and before a block with its gate and residual, in one pass:
    u = norm_post(f), h = residual_scale * residual + branch_scale * gate * u, y = norm_pre(h).

    f [T, H] bf16, f16 or fp32; residual [T, H] of f's dtype or fp32 (None: none; h then has residual_dtype, by
    default f's); gate [1 or B or T, H or 1] of f's dtype or fp32, B dividing T; w_*, b_* [H], all of f's dtype or all
    fp32.  post and pre are "none", "rms" or "layer".  Returns (h, y); h or y may be given as outputs (h may be
    residual and y may be f itself), and is None where want_h or want_y is false."""
    return (_ops or _load_ops()).norm(f, residual, _one_of(_NORMS, post, "post"), w_post, b_post, gate, branch_scale,
                                      residual_scale, _one_of(_NORMS, pre, "pre"), w_pre, b_pre, eps, residual_dtype,
                                      want_h, want_y, h, y)


def dense_linear(x, w, bias=None, act: str = "none", gated: bool = False, residual=None, out_dtype=None, out=None,
                 ws=None):
    """act(x w^T + bias) + residual, or with gated act(z[:, :N/2]) * z[:, N/2:] + residual for z = x w^T + bias.

    x [M, K], w [N, K] bf16 or f16 (one dtype, any row strides); bias [N] of that dtype or fp32; residual and the
    result [M, N] ([M, N/2] when gated) of out_dtype: x's dtype (default) or fp32.  act is "none", "relu", "silu",
    "gelu" or "gelu_tanh".  out may be given, also as the residual itself; ws is a uint8 workspace of
    dense_linear_workspace_bytes(M, N, K) bytes, used where x or w is not 16-byte aligned (made here when needed)."""
    return (_ops or _load_ops()).linear(x, w, bias, _one_of(_ACTS, act, "act"), gated, residual, out_dtype, out, ws)


def dense_linear_workspace_bytes(M: int, N: int, K: int) -> int:
    """Workspace of dense_linear where x or w is not 16-byte aligned (0: none)."""
    return int(load().dense_linear_workspace_bytes(M, N, K))


# --- the attention half of a block ------------------------------------------------------------------------------

_SCALINGS = ("none", "linear", "ntk", "yarn")


def rotary_frequencies(dim: int, base: float = 10000.0, *, scaling: str = "none", factor: float = 1.0,
                       length: int = 4096, beta_fast: float = 32.0, beta_slow: float = 1.0, inv_freq=None, device=None):
    """The frequencies that rotary_embedding and paged_kv_append take, int64 [dim / 2]: turns per position in units of
    2^-64, made once per model.

    f_i = base^(-2 i / dim) radians per position (or inv_freq, a sequence of dim / 2 numbers), scaled for contexts
    `factor` times longer than the `length` that a model was trained on: "linear" divides all by factor, "ntk" takes
    base * factor^(dim / (dim - 2)), that is f_i * factor^(-2 i / (dim - 2)), "yarn" divides those with fewer than
    beta_slow turns over `length`, keeps those with more than beta_fast, and blends in between (its factor on the
    rotated values is rotary_yarn_scale).  The blend is linear in a frequency's place among those of `base`, from and to a
    whole place; a given frequency's place follows from its own turns."""
    if dim < 2 or dim % 2:
        raise ValueError(f"dim must be even and positive, got {dim}")
    if scaling not in _SCALINGS:
        raise ValueError(f"scaling must be one of {sorted(_SCALINGS)}, got {scaling!r}")
    if not (factor > 0 and math.isfinite(factor)) or not (base > 1 and math.isfinite(base)) or length < 1:
        raise ValueError("factor and length must be positive and base above 1")
    half = dim // 2
    if inv_freq is not None:
        f = [float(v) for v in inv_freq]
        if len(f) != half or not all(math.isfinite(v) for v in f):
            raise ValueError(f"inv_freq must have {half} finite numbers")
    if scaling == "ntk" and dim == 2:
        raise ValueError("ntk scaling needs dim above 2")
    if inv_freq is None:
        if scaling == "ntk":
            base = base * factor ** (dim / (dim - 2))
        f = [base ** (-2.0 * i / dim) for i in range(half)]
    elif scaling == "ntk":  # the same change of the base, a power for each pair
        f = [v * factor ** (-2.0 * i / (dim - 2)) for i, v in enumerate(f)]
    if scaling == "linear":
        f = [v / factor for v in f]
    elif scaling == "yarn":
        def pair_of(turns):  # the pair that makes this many turns over `length`
            return dim * math.log(length / (turns * 2 * math.pi)) / (2 * math.log(base))
        lo, hi = max(math.floor(pair_of(beta_fast)), 0), min(math.ceil(pair_of(beta_slow)), dim - 1)
        at = range(half)
        if inv_freq is not None:  # which pair of `base` each would be, by its own turns over `length`
            at = [pair_of(abs(v) * length / (2 * math.pi)) if v else math.inf for v in f]
        keep = [1.0 - min(max((i - lo) / max(hi - lo, 0.001), 0.0), 1.0) for i in at]
        f = [v / factor * (1.0 - k) + v * k for v, k in zip(f, keep)]
    turns = [int(math.fmod(v / (2 * math.pi), 1.0) * 2.0 ** 64) for v in f]
    turns = [(t + 2 ** 63) % 2 ** 64 - 2 ** 63 for t in turns]
    return torch.tensor(turns, dtype=torch.int64, device="cuda" if device is None else device)


def rotary_yarn_scale(factor: float, mscale: float = 1.0) -> float:
    """The factor on rotated queries and keys that goes with yarn frequencies: 0.1 mscale ln(factor) + 1."""
    return 1.0 if factor <= 1 else 0.1 * mscale * math.log(factor) + 1.0


def rotary_embedding(x, positions, freqs, *, interleaved: bool = False, start: int = 0, scale: float = 1.0,
                     inverse: bool = False, out=None):
    """x [T, H, D] bf16, f16 or fp32 (any strides, D contiguous) rotated at positions [T] (int32 or int64): elements
    start ... start + 2 len(freqs) of each head in pairs (i, i + len(freqs)), or neighbours when interleaved, by the
    angle position * f_i, times scale; the others as they are.  freqs from rotary_frequencies.  inverse turns back (the
    transpose: the gradient with respect to x of a result's gradient).  out may be x."""
    return (_ops or _load_ops()).rotary(x, positions, freqs, interleaved, start, scale, inverse, out)


def paged_kv_append(k, v, k_cache, v_cache, page_table, seq_lens, indptr=None, *, freqs=None, positions=None,
                    interleaved: bool = False, start: int = 0, scale: float = 1.0, k_scale=None, v_scale=None, q=None,
                    q_out=None):
    """Writes k, v [T, Hkv, D] (bf16 or f16) into the caches [pages, page_size, Hkv, D] (that type or float8_e4m3fn, any
    strides, D contiguous), keys rotated as in rotary_embedding when freqs is given, at the cache position or at
    positions [T].  Rows indptr[b] ... indptr[b + 1] are the last tokens of sequence b, whose length seq_lens[b] (int32
    [B]) counts them; indptr None: one token each.  page_table int32 [B, n].  Rows behind the last sequence, or of one of
    length 0, are left out.  k_scale, v_scale fp32 [Hkv]: an 8-bit cache holds x / scale.
    q [T, Hq, D] is rotated like the keys into q_out (made when None; may be q) and returned; rows that are left out are
    zeros in a q_out made here and stay as they were in a given one."""
    return (_ops or _load_ops()).append(k, v, k_cache, v_cache, page_table, seq_lens, indptr, freqs, positions,
                                        interleaved, start, scale, k_scale, v_scale, q, q_out)


def paged_attention_decode(q, k_cache, v_cache, page_table, seq_lens, *, scale=None, window: int = 0, k_scale=None,
                           v_scale=None, return_lse: bool = False, out=None, ws=None):
    """Attention of one new token per sequence, q [B, Hq, D] (bf16 or f16), over its seq_lens[b] tokens in a paged cache
    (see paged_kv_append; Hq a multiple of Hkv, D a multiple of 8 up to 256, of 16 with 8-bit caches).  scale defaults
    to D^-0.5; window > 0 sees the last `window` tokens only; tokens that page_table has no place for are left out, and
    reported (device_error).  Returns out [B, Hq, D] of q's type, with return_lse (out, fp32 [B, Hq] log-sums of the
    exponentials); an empty sequence gives zeros and -inf.  out may be q.  ws is a uint8 workspace of
    paged_attention_workspace_bytes(B, Hq, Hkv, D) bytes (made when None)."""
    return (_ops or _load_ops()).attend(q, k_cache, v_cache, page_table, seq_lens, scale, window, k_scale, v_scale,
                                        return_lse, out, ws)


def paged_attention_workspace_bytes(B: int, Hq: int, Hkv: int, D: int) -> int:
    """Workspace of paged_attention_decode on the current device, enough for sequences of any length."""
    return int(load().paged_attention_workspace_bytes(B, Hq, Hkv, D, 0, -1))


def fp8_block_linear(A, a_scales, B, b_scales, *, out_dtype=None, out=None):
    """A [M, K] times B [N, K]^T in E4M3 (uint8 codes or float8_e4m3fn), K a multiple of 128: a_scales fp32 [K/128, ld]
    per token and 128 columns, as fp8_quant_per_token_group writes them, b_scales fp32 [ceil(N/128), K/128] per 128 x
    128 weights -> [M, N] of out_dtype (bf16 by default, f16 or fp32), which a given out has too."""
    return (_ops or _load_ops()).fp8_linear(A, a_scales, B, b_scales, out_dtype, out)


def device_error() -> int:
    return int(load().w4a8_device_error())
