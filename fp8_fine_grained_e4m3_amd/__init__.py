"""Python binding of libdg.so, the MI355X (gfx950) fine-grained FP8 e4m3 GEMM.

Argument marshalling only: every step of every GEMM, and of the FP8 casting
that prepares its operands, runs in the HIP kernels behind the C ABI declared
in include/dg.h.  PyTorch supplies device memory and
the current stream.  There is no fallback path: if libdg.so is missing or a
call fails, an exception is raised.

FP8 operands are passed as (data, scale) pairs, data being uint8 (raw e4m3
bytes) or torch.float8_e4m3fn, scales fp32 (the operand convention of the
"DeepGEMM" README, yuguo-Jack fork, section "Interfaces").  For the three NT
forms the scales may instead be packed UE8M0 words (int32, four power-of-two
exponents per word, the README's newer-path format): the dtype of the scale
tensors picks the C entry point.  The caller allocates the output and passes
it in.

For steps of a few tokens there are the paged FP8 key/value cache
(make_fp8_kv_cache, fp8_kv_cache_write, fp8_kv_cache_read), attention of drafted
trees or single tokens over it (fp8_tree_attention) and a whole
mixture-of-experts layer (fp8_moe_few_tokens).  Around a cache of either kind
there are the plan that gives requests their pages and tokens their slots
(make_kv_page_pool, kv_cache_plan), the norms of queries and keys with their
rotation (qk_norm_rope, and qk_norm_rope_backward for training), and the cache in
4 bits with its attention (make_fp4_kv_cache, fp4_kv_cache_write,
fp4_kv_cache_read, fp4_tree_attention).  All these allocate what they return
unless it is passed in, and take their workspace from torch's allocator unless
one is given (make_*_workspace).
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional, Sequence, Tuple

import numpy as np
import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libdg.so")

DG_OK, DG_ERR_INVALID_ARG, DG_ERR_UNSUPPORTED, DG_ERR_HIP = 0, 1, 2, 3
DG_BF16, DG_F32 = 1, 2

# Every symbol include/dg.h declares (the CPU tests check the library exports them).
EXPORTED = (
    "dg_fp8_gemm_nt",
    "dg_m_grouped_fp8_gemm_nt_contiguous",
    "dg_m_grouped_fp8_gemm_nt_masked",
    "dg_k_grouped_fp8_gemm_tn_contiguous",
    "dg_last_error",
    "dg_get_num_cus",
    "dg_set_num_cus",
    "dg_get_mk_alignment_for_contiguous_layout",
    "dg_kernel_config_name",
    "dg_per_token_cast_to_fp8",
    "dg_per_block_cast_to_fp8",
    "dg_fp8_gemm_nt_ue8m0",
    "dg_m_grouped_fp8_gemm_nt_contiguous_ue8m0",
    "dg_m_grouped_fp8_gemm_nt_masked_ue8m0",
    "dg_pack_ue8m0_scales",
    "dg_fp8_gemm_nn",
    "dg_fp8_gemm_tn",
    "dg_fp8_gemm_tt",
    "dg_m_grouped_fp8_gemm_nn_contiguous",
    "dg_fp8_mqa_logits",
    "dg_k_grouped_fp8_gemm_tn_contiguous_ue8m0",
    "dg_pack_ue8m0_scales_k_grouped",
    "dg_fp8_gemm_nt_workspace_bytes",
    "dg_fp8_gemm_nt_noalloc",
    "dg_fp8_kv_cache_write",
    "dg_fp8_kv_cache_read",
    "dg_fp8_tree_attention",
    "dg_fp8_tree_attention_workspace_bytes",
    "dg_fp8_moe_few_tokens",
    "dg_fp8_moe_few_tokens_workspace_bytes",
    "dg_kv_cache_plan",
    "dg_qk_norm_rope",
    "dg_qk_norm_rope_backward",
    "dg_qk_norm_rope_backward_workspace_bytes",
    "dg_fp4_kv_cache_write",
    "dg_fp4_kv_cache_read",
    "dg_fp4_tree_attention",
    "dg_fp4_tree_attention_workspace_bytes",
)
DG_CAST_POW2_SCALE = 1

_lib = None


class DGError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"dg status {status}: {message}")
        self.status = status


def load_library(path: Optional[str] = None):
    """Load libdg.so (raises if it has not been built)."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise ImportError(f"{p} is missing: build it with `python -m fp8_fine_grained_e4m3_amd.build` "
                          "(or __graft_entry__.build())")
    lib = ctypes.CDLL(p)
    P, I64, I = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
    lib.dg_fp8_gemm_nt.argtypes = [P, P, P, P, P, P, I, I64, I64, I64, P, I64, P]
    lib.dg_fp8_gemm_nt_noalloc.argtypes = [P, P, P, P, P, P, I, I64, I64, I64, P]
    lib.dg_fp8_gemm_nt_noalloc.restype = I
    lib.dg_fp8_gemm_nt_workspace_bytes.argtypes = [I64, I64, I64]
    lib.dg_fp8_gemm_nt_workspace_bytes.restype = I64
    lib.dg_m_grouped_fp8_gemm_nt_contiguous.argtypes = [P, P, P, P, P, P, I64, I64, I64, I64, P]
    lib.dg_m_grouped_fp8_gemm_nt_masked.argtypes = [P, P, P, P, P, P, I64, I64, I64, I64, P]
    lib.dg_k_grouped_fp8_gemm_tn_contiguous.argtypes = [P, P, P, P, P, P, P, I64, I64, I64, I64, P]
    for name in EXPORTED[:4]:
        getattr(lib, name).restype = I
    lib.dg_last_error.argtypes = []
    lib.dg_last_error.restype = ctypes.c_char_p
    lib.dg_get_num_cus.argtypes = []
    lib.dg_get_num_cus.restype = I
    lib.dg_set_num_cus.argtypes = [I]
    lib.dg_set_num_cus.restype = I
    lib.dg_get_mk_alignment_for_contiguous_layout.argtypes = []
    lib.dg_get_mk_alignment_for_contiguous_layout.restype = I
    lib.dg_kernel_config_name.argtypes = [I, I64, I64, I64, I]
    lib.dg_kernel_config_name.restype = ctypes.c_char_p
    for name in ("dg_per_token_cast_to_fp8", "dg_per_block_cast_to_fp8"):
        getattr(lib, name).argtypes = [P, I, P, P, I64, I64, I64, I, P]
        getattr(lib, name).restype = I
    lib.dg_fp8_gemm_nt_ue8m0.argtypes = [P, P, P, P, P, P, I, I64, I64, I64, P, I64, P]
    lib.dg_m_grouped_fp8_gemm_nt_contiguous_ue8m0.argtypes = [P, P, P, P, P, P, I64, I64, I64,
                                                              I64, P]
    lib.dg_m_grouped_fp8_gemm_nt_masked_ue8m0.argtypes = [P, P, P, P, P, P, I64, I64, I64, I64, P]
    lib.dg_pack_ue8m0_scales.argtypes = [P, I, P, I64, I64, I64, P]
    for name in ("dg_fp8_gemm_nn", "dg_fp8_gemm_tn", "dg_fp8_gemm_tt"):
        getattr(lib, name).argtypes = [P, P, P, P, P, P, I, I64, I64, I64, P]
        getattr(lib, name).restype = I
    lib.dg_m_grouped_fp8_gemm_nn_contiguous.argtypes = [P, P, P, P, P, P, I64, I64, I64, I64, P]
    lib.dg_m_grouped_fp8_gemm_nn_contiguous.restype = I
    lib.dg_fp8_mqa_logits.argtypes = [P, P, P, P, P, P, P, I64, I64, I64, I64, I, P]
    lib.dg_fp8_mqa_logits.restype = I
    lib.dg_k_grouped_fp8_gemm_tn_contiguous_ue8m0.argtypes = [P, P, P, P, P, P, P, I64, I64, I64,
                                                              I64, P]
    lib.dg_k_grouped_fp8_gemm_tn_contiguous_ue8m0.restype = I
    lib.dg_pack_ue8m0_scales_k_grouped.argtypes = [P, P, P, I64, I64, I64, P]
    lib.dg_pack_ue8m0_scales_k_grouped.restype = I
    for name in ("dg_fp8_gemm_nt_ue8m0", "dg_m_grouped_fp8_gemm_nt_contiguous_ue8m0",
                 "dg_m_grouped_fp8_gemm_nt_masked_ue8m0", "dg_pack_ue8m0_scales"):
        getattr(lib, name).restype = I
    F = ctypes.c_float
    lib.dg_qk_norm_rope.argtypes = [P, P, I, I64, I64, P, P, I, P, P, P, P, I64, I64, F, I, I64, I64, I64, I64, I64, P]
    lib.dg_qk_norm_rope.restype = I
    lib.dg_qk_norm_rope_backward.argtypes = ([P, P, P, P, I, I64, I64, I64, I64, P, P, I, P, P, P, P, I64, I64, P, P, F, I]
                                             + [I64] * 5 + [P, I64, P])
    lib.dg_qk_norm_rope_backward.restype = I
    lib.dg_qk_norm_rope_backward_workspace_bytes.argtypes = [I64] * 4
    lib.dg_qk_norm_rope_backward_workspace_bytes.restype = I64
    lib.dg_kv_cache_plan.argtypes = [P] * 9 + [I64, I64, I, I64, I64, I64, P]
    lib.dg_kv_cache_plan.restype = I
    for bits in ("fp8", "fp4"):
        write, read, attention, need = (getattr(lib, f"dg_{bits}_{name}") for name in (
            "kv_cache_write", "kv_cache_read", "tree_attention", "tree_attention_workspace_bytes"))
        write.argtypes = [P, P, I, I64, I64, P, P, P, P, P, I64, I64, I64, I64, I64, P]
        read.argtypes = [P, P, P, P, P, P, P, I, I64, I64, I64, I64, I64, P]
        attention.argtypes = [P, I64, P, P, P, P, P, P, P, P, P, P, F, I64, I64, I64, I64, I64, I64, I64, I64, P, I64, P]
        need.argtypes, need.restype = [I64] * 7, I64
        for f in (write, read, attention):
            f.restype = I
    lib.dg_fp8_moe_few_tokens.argtypes = [P, P, P, P, P, P, P, P, I, I64, I64, I64, I64, I64, P, I64, P]
    lib.dg_fp8_moe_few_tokens.restype = I
    lib.dg_fp8_moe_few_tokens_workspace_bytes.argtypes = [I64] * 5
    lib.dg_fp8_moe_few_tokens_workspace_bytes.restype = I64
    if path is None:
        _lib = lib
    return lib


def _check(status: int):
    if status != DG_OK:
        raise DGError(status, load_library().dg_last_error().decode())


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _fp8(t: torch.Tensor, name: str) -> torch.Tensor:
    if t.dtype == torch.float8_e4m3fn:
        t = t.view(torch.uint8)
    if t.dtype != torch.uint8:
        raise TypeError(f"{name} must be uint8 or float8_e4m3fn, got {t.dtype}")
    return _dev(t, name)


def _dev(t: torch.Tensor, name: str) -> torch.Tensor:
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _f32(t: torch.Tensor, name: str) -> torch.Tensor:
    if t.dtype != torch.float32:
        raise TypeError(f"{name} must be float32, got {t.dtype}")
    return _dev(t, name)


def _i32(t: torch.Tensor, name: str) -> torch.Tensor:
    if t.dtype != torch.int32:
        raise TypeError(f"{name} must be int32, got {t.dtype}")
    return _dev(t, name)


def _scales(sa: torch.Tensor, sb: torch.Tensor):
    """Both fp32 (-> False) or both packed UE8M0 int32 words (-> True)."""
    if sa.dtype == torch.int32 and sb.dtype == torch.int32:
        return _dev(sa, "SFA"), _dev(sb, "SFB"), True
    return _f32(sa, "SFA"), _f32(sb, "SFB"), False


def _k4(K: int) -> int:
    """Packed UE8M0 words per row: ceil(K / 512)."""
    return (K // 128 + 3) // 4


def _stream(t: torch.Tensor):
    return ctypes.c_void_p(torch.cuda.current_stream(t.device).cuda_stream)


def get_fp8_gemm_nt_workspace_bytes(M: int, N: int, K: int) -> int:
    """Split-K workspace bytes a dense NT call of this shape needs (0: none)."""
    return int(load_library().dg_fp8_gemm_nt_workspace_bytes(M, N, K))


def make_fp8_gemm_nt_workspace(M: int, N: int, K: int, device=None) -> Optional[torch.Tensor]:
    """A zero-filled workspace for dense NT calls of this shape (None when the
    shape needs none).  Stream-ordered calls may reuse it: every call leaves
    its counters zero again."""
    n = get_fp8_gemm_nt_workspace_bytes(M, N, K)
    if n == 0:
        return None
    return torch.zeros(n, dtype=torch.uint8, device=device or torch.cuda.current_device())


def fp8_gemm_nt(a: Tuple[torch.Tensor, torch.Tensor], b: Tuple[torch.Tensor, torch.Tensor],
                d: torch.Tensor, c: Optional[torch.Tensor] = None,
                workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """d[M,N] = c + a @ b^T.  a = (A [M,K], SFA [K/128, M]), b = (B [N,K],
    SFB [ceil(N/128), K/128]); d bf16 or fp32; c None or like d (may be d).
    Packed UE8M0 scales (int32): SFA [ceil(K/512), M], SFB [ceil(K/512), N].
    workspace: a uint8 device buffer of at least
    get_fp8_gemm_nt_workspace_bytes(M, N, K) bytes whose counters are zero
    (make_fp8_gemm_nt_workspace); when None and the shape splits K, a
    zero-filled one is allocated for this call from torch's allocator."""
    A, B = _fp8(a[0], "A"), _fp8(b[0], "B")
    SA, SB, ue8m0 = _scales(a[1], b[1])
    d = _dev(d, "d")
    if d.dtype not in (torch.bfloat16, torch.float32):
        raise TypeError("d must be bfloat16 or float32")
    if c is not None:
        c = _dev(c, "c")
        if c.dtype != d.dtype or c.shape != d.shape:
            raise ValueError("c must match d in dtype and shape")
    M, K = A.shape
    N = B.shape[0]
    if B.shape[1] != K or tuple(d.shape) != (M, N):
        raise ValueError(f"shape mismatch: A {tuple(A.shape)} B {tuple(B.shape)} d {tuple(d.shape)}")
    want = (((_k4(K), M), (_k4(K), N)) if ue8m0
            else ((K // 128, M), ((N + 127) // 128, K // 128)))
    if (tuple(SA.shape), tuple(SB.shape)) != want:
        raise ValueError(f"scale shapes: SFA {tuple(SA.shape)} SFB {tuple(SB.shape)}, want {want}")
    fn = "dg_fp8_gemm_nt_ue8m0" if ue8m0 else "dg_fp8_gemm_nt"
    with torch.cuda.device(d.device):
        need = get_fp8_gemm_nt_workspace_bytes(M, N, K)
        if workspace is None and need > 0:
            workspace = torch.zeros(need, dtype=torch.uint8, device=d.device)
        ws_bytes = 0
        if workspace is not None:
            workspace = _dev(workspace, "workspace")
            if workspace.dtype != torch.uint8:
                raise TypeError("workspace must be uint8")
            ws_bytes = workspace.numel()
        _check(getattr(load_library(), fn)(
            _ptr(A), _ptr(SA), _ptr(B), _ptr(SB), _ptr(c), _ptr(d),
            DG_F32 if d.dtype == torch.float32 else DG_BF16, M, N, K,
            _ptr(workspace), ws_bytes, _stream(d)))
    return d


def fp8_gemm_nt_noalloc(a: Tuple[torch.Tensor, torch.Tensor], b: Tuple[torch.Tensor, torch.Tensor],
                        d: torch.Tensor, c: Optional[torch.Tensor] = None) -> torch.Tensor:
    """fp8_gemm_nt (fp32 scales) with the split-K workspace taken from the
    library's static per-GPU scratch: nothing is allocated on any call.
    Calls that may overlap on one GPU race on that scratch."""
    A, B = _fp8(a[0], "A"), _fp8(b[0], "B")
    SA, SB = _f32(a[1], "SFA"), _f32(b[1], "SFB")
    d = _dev(d, "d")
    if d.dtype not in (torch.bfloat16, torch.float32):
        raise TypeError("d must be bfloat16 or float32")
    if c is not None:
        c = _dev(c, "c")
        if c.dtype != d.dtype or c.shape != d.shape:
            raise ValueError("c must match d in dtype and shape")
    M, K = A.shape
    N = B.shape[0]
    if B.shape[1] != K or tuple(d.shape) != (M, N):
        raise ValueError(f"shape mismatch: A {tuple(A.shape)} B {tuple(B.shape)} d {tuple(d.shape)}")
    want = ((K // 128, M), ((N + 127) // 128, K // 128))
    if (tuple(SA.shape), tuple(SB.shape)) != want:
        raise ValueError(f"scale shapes: SFA {tuple(SA.shape)} SFB {tuple(SB.shape)}, want {want}")
    with torch.cuda.device(d.device):
        _check(load_library().dg_fp8_gemm_nt_noalloc(
            _ptr(A), _ptr(SA), _ptr(B), _ptr(SB), _ptr(c), _ptr(d),
            DG_F32 if d.dtype == torch.float32 else DG_BF16, M, N, K, _stream(d)))
    return d


def m_grouped_fp8_gemm_nt_contiguous(a: Tuple[torch.Tensor, torch.Tensor],
                                     b: Tuple[torch.Tensor, torch.Tensor],
                                     d: torch.Tensor, m_indices: torch.Tensor) -> torch.Tensor:
    """d[r] = a[r] @ b[m_indices[r]]^T; a = (A [M_tot,K], SFA [K/128, M_tot]),
    b = (B [G,N,K], SFB [G, ceil(N/128), K/128]); d bf16 [M_tot, N].
    Packed UE8M0 scales (int32): SFA [ceil(K/512), M_tot], SFB [G, ceil(K/512), N]."""
    A, B = _fp8(a[0], "A"), _fp8(b[0], "B")
    SA, SB, ue8m0 = _scales(a[1], b[1])
    d, mi = _dev(d, "d"), _i32(m_indices, "m_indices")
    if d.dtype != torch.bfloat16:
        raise TypeError("d must be bfloat16")
    M_tot, K = A.shape
    G, N, Kb = B.shape
    if Kb != K or tuple(d.shape) != (M_tot, N) or tuple(mi.shape) != (M_tot,):
        raise ValueError("shape mismatch")
    want = (((_k4(K), M_tot), (G, _k4(K), N)) if ue8m0
            else ((K // 128, M_tot), (G, (N + 127) // 128, K // 128)))
    if (tuple(SA.shape), tuple(SB.shape)) != want:
        raise ValueError(f"scale shapes: SFA {tuple(SA.shape)} SFB {tuple(SB.shape)}, want {want}")
    fn = ("dg_m_grouped_fp8_gemm_nt_contiguous_ue8m0" if ue8m0
          else "dg_m_grouped_fp8_gemm_nt_contiguous")
    with torch.cuda.device(d.device):
        _check(getattr(load_library(), fn)(
            _ptr(A), _ptr(SA), _ptr(B), _ptr(SB), _ptr(mi), _ptr(d), M_tot, N, K, G, _stream(d)))
    return d


def m_grouped_fp8_gemm_nt_masked(a: Tuple[torch.Tensor, torch.Tensor],
                                 b: Tuple[torch.Tensor, torch.Tensor],
                                 d: torch.Tensor, masked_m: torch.Tensor) -> torch.Tensor:
    """d[g, r] = a[g, r] @ b[g]^T for r < masked_m[g]; other rows untouched.
    a = (A [G,M_max,K], SFA [G, K/128, M_max]), b = (B [G,N,K], SFB [G,NB,KB]).
    Packed UE8M0 scales (int32): SFA [G, ceil(K/512), M_max], SFB [G, ceil(K/512), N]."""
    A, B = _fp8(a[0], "A"), _fp8(b[0], "B")
    SA, SB, ue8m0 = _scales(a[1], b[1])
    d, mm = _dev(d, "d"), _i32(masked_m, "masked_m")
    if d.dtype != torch.bfloat16:
        raise TypeError("d must be bfloat16")
    G, M_max, K = A.shape
    N = B.shape[1]
    if tuple(B.shape) != (G, N, K) or tuple(d.shape) != (G, M_max, N) or tuple(mm.shape) != (G,):
        raise ValueError("shape mismatch")
    want = (((G, _k4(K), M_max), (G, _k4(K), N)) if ue8m0
            else ((G, K // 128, M_max), (G, (N + 127) // 128, K // 128)))
    if (tuple(SA.shape), tuple(SB.shape)) != want:
        raise ValueError(f"scale shapes: SFA {tuple(SA.shape)} SFB {tuple(SB.shape)}, want {want}")
    fn = "dg_m_grouped_fp8_gemm_nt_masked_ue8m0" if ue8m0 else "dg_m_grouped_fp8_gemm_nt_masked"
    with torch.cuda.device(d.device):
        _check(getattr(load_library(), fn)(
            _ptr(A), _ptr(SA), _ptr(B), _ptr(SB), _ptr(mm), _ptr(d), G, M_max, N, K, _stream(d)))
    return d


def k_grouped_fp8_gemm_tn_contiguous(a: Tuple[torch.Tensor, torch.Tensor],
                                     b: Tuple[torch.Tensor, torch.Tensor],
                                     d: torch.Tensor, k_sizes: Sequence[int],
                                     c: Optional[torch.Tensor] = None) -> torch.Tensor:
    """d[g] = c[g] + a_g^T @ b_g over group g's K rows.  a = (A [K_tot, M],
    SFA [K_tot/128, M]), b = (B [K_tot, N], SFB [K_tot/128, N]); k_sizes is a
    host sequence; d (and c) fp32 [G, M, N].  Packed UE8M0 scales (int32):
    SFA [W, M], SFB [W, N], each group on its own ceil(K_g / 512) word rows."""
    A, B = _fp8(a[0], "A"), _fp8(b[0], "B")
    SA, SB, ue8m0 = _scales(a[1], b[1])
    d = _f32(d, "d")
    if c is not None:
        c = _f32(c, "c")
        if c.shape != d.shape:
            raise ValueError("c must match d")
    ks = np.ascontiguousarray(np.asarray(k_sizes, dtype=np.int64))
    if ks.ndim != 1 or np.any(ks > np.iinfo(np.int32).max) or np.any(ks < np.iinfo(np.int32).min):
        raise ValueError("k_sizes must be a 1-D sequence of int32 values")
    ks = ks.astype(np.int32)
    K_tot, M = A.shape
    N = B.shape[1]
    G = len(ks)
    if B.shape[0] != K_tot or tuple(d.shape) != (G, M, N):
        raise ValueError("shape mismatch")
    rows = _k_grouped_words(ks) if ue8m0 else K_tot // 128
    if tuple(SA.shape) != (rows, M) or tuple(SB.shape) != (rows, N):
        raise ValueError("scale shape mismatch")
    fn = ("dg_k_grouped_fp8_gemm_tn_contiguous_ue8m0" if ue8m0
          else "dg_k_grouped_fp8_gemm_tn_contiguous")
    with torch.cuda.device(d.device):
        _check(getattr(load_library(), fn)(
            _ptr(A), _ptr(SA), _ptr(B), _ptr(SB), ks.ctypes.data_as(ctypes.c_void_p), _ptr(c),
            _ptr(d), G, M, N, K_tot, _stream(d)))
    return d


def get_num_cus() -> int:
    return load_library().dg_get_num_cus()


def set_num_cus(n: int) -> None:
    _check(load_library().dg_set_num_cus(int(n)))


def get_mk_alignment_for_contiguous_layout() -> int:
    return load_library().dg_get_mk_alignment_for_contiguous_layout()


FORM_DENSE, FORM_CONTIGUOUS, FORM_MASKED, FORM_K_GROUPED = 0, 1, 2, 3
FORM_NN, FORM_TN, FORM_TT, FORM_NN_CONTIGUOUS = 4, 5, 6, 7


def kernel_config_name(form: int, rows: int, N: int, K: int, out_f32: bool = False) -> str:
    """Kernel instance (tile configuration) a call with these sizes launches."""
    return load_library().dg_kernel_config_name(form, rows, N, K, int(out_f32)).decode()


def to_mn_major_sf(sf: torch.Tensor) -> torch.Tensor:
    """[rows, K/128] per-row scales -> the MN-major [K/128, rows] layout the
    A-side scale factors use (a transpose + copy; layout only)."""
    return sf.transpose(-1, -2).contiguous()


def _cast(fn: str, x: torch.Tensor, block_scale: bool, pow2_scale: bool,
          out: Optional[Tuple[torch.Tensor, torch.Tensor]]):
    x = _dev(x, "x")
    if x.dtype not in (torch.bfloat16, torch.float32):
        raise TypeError(f"x must be bfloat16 or float32, got {x.dtype}")
    if x.dim() not in (2, 3):
        raise ValueError("x must be [rows, K] or [G, rows, K]")
    batched = x.dim() == 3
    G, R, K = x.shape if batched else (1,) + tuple(x.shape)
    if K % 128:
        raise ValueError(f"K={K} is not a multiple of 128")
    sf_shape = (G, (R + 127) // 128, K // 128) if block_scale else (G, K // 128, R)
    if not batched:
        sf_shape = sf_shape[1:]
    if out is None:
        codes = torch.empty(x.shape, dtype=torch.uint8, device=x.device)
        sf = torch.empty(sf_shape, dtype=torch.float32, device=x.device)
    else:
        codes, sf = _fp8(out[0], "codes"), _f32(out[1], "sf")
        if tuple(codes.shape) != tuple(x.shape) or tuple(sf.shape) != sf_shape:
            raise ValueError(f"out shapes: codes {tuple(codes.shape)} sf {tuple(sf.shape)}, "
                             f"want {tuple(x.shape)} and {sf_shape}")
    with torch.cuda.device(x.device):
        _check(getattr(load_library(), fn)(
            _ptr(x), DG_F32 if x.dtype == torch.float32 else DG_BF16, _ptr(codes), _ptr(sf),
            G, R, K, DG_CAST_POW2_SCALE if pow2_scale else 0, _stream(x)))
    return codes, sf


def per_token_cast_to_fp8(x: torch.Tensor, pow2_scale: bool = False,
                          out: Optional[Tuple[torch.Tensor, torch.Tensor]] = None):
    """1 x 128 casting of activations x [R, K] or [G, R, K] (bf16 or fp32).
    Returns (codes uint8 like x, sf fp32 [K/128, R] or [G, K/128, R]): the A
    operand and its MN-major scales for the GEMM calls above."""
    return _cast("dg_per_token_cast_to_fp8", x, False, pow2_scale, out)


def per_block_cast_to_fp8(w: torch.Tensor, pow2_scale: bool = False,
                          out: Optional[Tuple[torch.Tensor, torch.Tensor]] = None):
    """128 x 128 casting of weights w [N, K] or [G, N, K] (bf16 or fp32).
    Returns (codes uint8 like w, sf fp32 [ceil(N/128), K/128] or
    [G, ceil(N/128), K/128]): the B operand and its scales."""
    return _cast("dg_per_block_cast_to_fp8", w, True, pow2_scale, out)


def pack_ue8m0_scales(sf: torch.Tensor, mn: Optional[int] = None,
                      per_block: bool = False) -> torch.Tensor:
    """fp32 power-of-two scales -> packed UE8M0 int32 words [.., ceil(K/512), MN].

    per_block False: sf [K/128, MN] or [G, K/128, MN] (A-side, MN-major);
    per_block True: sf [ceil(MN/128), K/128] or [G, ..] (128 x 128 weight
    blocks, each given to its rows; pass mn = N).  Byte i of word k4 holds
    the exponent of K block 4 k4 + i (the layout the *_ue8m0 GEMMs take)."""
    sf = _f32(sf, "sf")
    if sf.dim() not in (2, 3):
        raise ValueError("sf must be 2-D or 3-D")
    batched = sf.dim() == 3
    sf3 = sf if batched else sf.unsqueeze(0)
    G = sf3.shape[0]
    if per_block:
        if mn is None:
            raise ValueError("per_block packing needs mn (the row count N)")
        KB = sf3.shape[2]
        if sf3.shape[1] != (mn + 127) // 128:
            raise ValueError(f"sf {tuple(sf.shape)} does not cover {mn} rows")
    else:
        KB, MN = sf3.shape[1], sf3.shape[2]
        if mn is not None and mn != MN:
            raise ValueError(f"mn={mn} but sf has {MN} rows")
        mn = MN
    out = torch.empty((G, (KB + 3) // 4, mn), dtype=torch.int32, device=sf.device)
    with torch.cuda.device(sf.device):
        _check(load_library().dg_pack_ue8m0_scales(_ptr(sf3), int(per_block), _ptr(out), G, mn,
                                                   KB * 128, _stream(sf)))
    return out if batched else out[0]


def _gemm_layout(layout: str, a, b, d, c):
    """Dense NN / TN / TT: A stored [M, K] ("n") or [K, M] ("t"); B stored
    [K, N] ("n") or [N, K] ("t"); SFA fp32 [K/128, M], SFB fp32 [K/128, N]."""
    A, SA = _fp8(a[0], "A"), _f32(a[1], "SFA")
    B, SB = _fp8(b[0], "B"), _f32(b[1], "SFB")
    d = _dev(d, "d")
    if d.dtype not in (torch.bfloat16, torch.float32):
        raise TypeError("d must be bfloat16 or float32")
    if c is not None:
        c = _dev(c, "c")
        if c.dtype != d.dtype or c.shape != d.shape:
            raise ValueError("c must match d in dtype and shape")
    M, K = A.shape if layout[0] == "n" else A.shape[::-1]
    N, Kb = B.shape if layout[1] == "t" else B.shape[::-1]
    if Kb != K or tuple(d.shape) != (M, N):
        raise ValueError(f"shape mismatch: A {tuple(A.shape)} B {tuple(B.shape)} d {tuple(d.shape)}")
    if tuple(SA.shape) != (K // 128, M) or tuple(SB.shape) != (K // 128, N):
        raise ValueError(f"scale shapes: SFA {tuple(SA.shape)} SFB {tuple(SB.shape)}, "
                         f"want {(K // 128, M)} and {(K // 128, N)}")
    with torch.cuda.device(d.device):
        _check(getattr(load_library(), f"dg_fp8_gemm_{layout}")(
            _ptr(A), _ptr(SA), _ptr(B), _ptr(SB), _ptr(c), _ptr(d),
            DG_F32 if d.dtype == torch.float32 else DG_BF16, M, N, K, _stream(d)))
    return d


def fp8_gemm_nn(a, b, d, c=None):
    """d[M,N] = c + A @ B; a = (A [M,K], SFA [K/128, M]), b = (B [K,N], SFB [K/128, N])."""
    return _gemm_layout("nn", a, b, d, c)


def fp8_gemm_tn(a, b, d, c=None):
    """d[M,N] = c + A^T @ B; a = (A [K,M], SFA [K/128, M]), b = (B [K,N], SFB [K/128, N])."""
    return _gemm_layout("tn", a, b, d, c)


def fp8_gemm_tt(a, b, d, c=None):
    """d[M,N] = c + A^T @ B^T; a = (A [K,M], SFA [K/128, M]), b = (B [N,K], SFB [K/128, N])."""
    return _gemm_layout("tt", a, b, d, c)


def m_grouped_fp8_gemm_nn_contiguous(a, b, d: torch.Tensor, m_indices: torch.Tensor) -> torch.Tensor:
    """d[r] = a[r] @ b[m_indices[r]]; a = (A [M_tot,K], SFA [K/128, M_tot]),
    b = (B [G,K,N], SFB [G, K/128, N]); d bf16 [M_tot, N]."""
    A, SA = _fp8(a[0], "A"), _f32(a[1], "SFA")
    B, SB = _fp8(b[0], "B"), _f32(b[1], "SFB")
    d, mi = _dev(d, "d"), _i32(m_indices, "m_indices")
    if d.dtype != torch.bfloat16:
        raise TypeError("d must be bfloat16")
    M_tot, K = A.shape
    G, Kb, N = B.shape
    if Kb != K or tuple(d.shape) != (M_tot, N) or tuple(mi.shape) != (M_tot,):
        raise ValueError("shape mismatch")
    if tuple(SA.shape) != (K // 128, M_tot) or tuple(SB.shape) != (G, K // 128, N):
        raise ValueError("scale shape mismatch")
    with torch.cuda.device(d.device):
        _check(load_library().dg_m_grouped_fp8_gemm_nn_contiguous(
            _ptr(A), _ptr(SA), _ptr(B), _ptr(SB), _ptr(mi), _ptr(d), M_tot, N, K, G, _stream(d)))
    return d


def fp8_mqa_logits(q: torch.Tensor, kv: Tuple[torch.Tensor, torch.Tensor], weights: torch.Tensor,
                   cu_seq_len_k_start: torch.Tensor, cu_seq_len_k_end: torch.Tensor,
                   clean_logits: bool = True, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """logits[i, j] = sum_h relu(q[i, h] . kv[j] * sf[j]) * weights[i, h] for j in
    [start[i], end[i]) (-inf elsewhere when clean_logits).  q e4m3 [S, H, 128],
    kv = (e4m3 [S_kv, 128], fp32 [S_kv]), weights fp32 [S, H], ranges int32 [S];
    returns fp32 [S, S_kv] (or fills `out`)."""
    Q = _fp8(q, "q")
    KV, SF = _fp8(kv[0], "kv"), _f32(kv[1], "kv_sf")
    W = _f32(weights, "weights")
    ks, ke = _i32(cu_seq_len_k_start, "cu_seq_len_k_start"), _i32(cu_seq_len_k_end, "cu_seq_len_k_end")
    if Q.dim() != 3:
        raise ValueError("q must be [seq_len, num_heads, head_dim]")
    S, H, D = Q.shape
    S_kv = KV.shape[0]
    if tuple(KV.shape) != (S_kv, D) or tuple(SF.shape) != (S_kv,) or tuple(W.shape) != (S, H):
        raise ValueError("shape mismatch")
    if tuple(ks.shape) != (S,) or tuple(ke.shape) != (S,):
        raise ValueError("range shape mismatch")
    if out is None:
        out = torch.empty(S, S_kv, dtype=torch.float32, device=Q.device)
    else:
        out = _f32(out, "out")
        if tuple(out.shape) != (S, S_kv):
            raise ValueError("out shape mismatch")
    with torch.cuda.device(Q.device):
        _check(load_library().dg_fp8_mqa_logits(
            _ptr(Q), _ptr(KV), _ptr(SF), _ptr(W), _ptr(ks), _ptr(ke), _ptr(out), S, S_kv, H, D,
            int(bool(clean_logits)), _stream(out)))
    return out


def _k_grouped_words(k_sizes) -> int:
    return int(sum((int(k) // 128 + 3) // 4 for k in k_sizes))


def pack_ue8m0_scales_k_grouped(sf: torch.Tensor, k_sizes: Sequence[int]) -> torch.Tensor:
    """fp32 power-of-two scales [K_tot/128, MN] of a K-grouped operand ->
    packed UE8M0 words [sum_g ceil(K_g / 512), MN], each group on its own rows."""
    sf = _f32(sf, "sf")
    ks = np.ascontiguousarray(np.asarray(k_sizes, dtype=np.int32))
    KB, MN = sf.shape
    out = torch.empty((_k_grouped_words(ks), MN), dtype=torch.int32, device=sf.device)
    with torch.cuda.device(sf.device):
        _check(load_library().dg_pack_ue8m0_scales_k_grouped(
            _ptr(sf), ks.ctypes.data_as(ctypes.c_void_p), _ptr(out), len(ks), MN, KB * 128,
            _stream(sf)))
    return out


# ---- few tokens at a time: FP8 cache, tree attention, mixture of experts ---------------------

def make_fp8_kv_cache(num_pages: int, num_kv_heads: int, page_size: int, head_dim: int, device=None):
    """An empty paged FP8 cache: ((k codes, k scales), (v codes, v scales)),
    codes uint8 [num_pages, num_kv_heads, page_size, head_dim], scales fp32
    [num_pages, num_kv_heads, page_size].  page_size is a power of two from 16
    to 4096, head_dim 64, 128 or 256."""
    shape = (num_pages, num_kv_heads, page_size, head_dim)
    device = torch.cuda.current_device() if device is None else device
    return tuple((torch.zeros(shape, dtype=torch.uint8, device=device),
                  torch.ones(shape[:3], dtype=torch.float32, device=device)) for _ in range(2))


# The few-token calls take microseconds on the device, so their checks are one
# test of everything first; what is wrong is looked for only when it fails.
_U8, _I32, _I64, _F32, _BF16 = torch.uint8, torch.int32, torch.int64, torch.float32, torch.bfloat16
_ROW_TYPES = {_BF16: DG_BF16, _F32: DG_F32}


def _cache(cache):
    """The cache's four tensors, checked, its sizes and its device's index."""
    (kc, ks), (vc, vs) = cache
    shape, sf_shape, on = kc.shape, ks.shape, kc.get_device()
    if not (kc.dtype is _U8 and vc.dtype is _U8 and ks.dtype is _F32 and vs.dtype is _F32 and on >= 0
            and vc.shape == shape and len(shape) == 4 and shape[:3] == sf_shape and vs.shape == sf_shape
            and kc.is_contiguous() and vc.is_contiguous() and ks.is_contiguous() and vs.is_contiguous()
            and ks.get_device() == on and vc.get_device() == on and vs.get_device() == on):
        kc, vc, ks, vs = _fp8(kc, "k codes"), _fp8(vc, "v codes"), _f32(ks, "k scales"), _f32(vs, "v scales")
        if kc.dim() != 4 or kc.shape != vc.shape or ks.shape != kc.shape[:3] or vs.shape != kc.shape[:3]:
            raise ValueError(f"cache shapes: codes {tuple(kc.shape)} {tuple(vc.shape)}, scales {tuple(ks.shape)} "
                             f"{tuple(vs.shape)}, want [pages, heads, page_size, head_dim] and its first three")
        _same_device(kc, ks, vc, vs)
        shape, on = kc.shape, kc.get_device()
    return kc, ks, vc, vs, shape, on


def _rows(t: torch.Tensor, name: str) -> int:
    """Elements between the tokens of device rows [..., tokens, heads, D] whose
    last two dimensions are dense; what a single token has there says nothing."""
    shape, strides = t.shape, t.stride()
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    dense = shape[-1] * shape[-2]
    if dense and (strides[-1] != 1 or (shape[-2] > 1 and strides[-2] != shape[-1])):
        raise ValueError(f"{name}: heads and head_dim must be dense, strides are {strides}")
    return strides[-3] if shape[-3] > 1 else dense


def _same_device(first: torch.Tensor, *others):
    for t in others:
        if t is not None and t.device != first.device:
            raise ValueError(f"tensors on {first.device} and {t.device}")


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _call(fn: str, device: int, *args):
    """An entry point on the device's current stream."""
    f = getattr(load_library(), fn)
    if _current_device() == device:
        status = f(*args, _raw_stream(device))
    else:
        with torch.cuda.device(device):
            status = f(*args, _raw_stream(device))
    if status != DG_OK:
        _check(status)


def _write(fn: str, parts, k: torch.Tensor, v: torch.Tensor, cache, slots: torch.Tensor):
    """A write into a cache, given its checked parts (_cache, _cache4)."""
    kc, ks, vc, vs, (P, H, page, D), on = parts
    T = slots.shape[0] if slots.dim() == 1 else -1
    if not (k.dtype in _ROW_TYPES and v.dtype is k.dtype and k.shape == (T, H, D) and v.shape == k.shape
            and slots.dtype is _I32 and slots.is_contiguous()
            and k.get_device() == on and v.get_device() == on and slots.get_device() == on):
        _i32(slots, "slots")
        if k.dtype not in _ROW_TYPES or v.dtype != k.dtype:
            raise TypeError(f"k and v must both be bfloat16 or float32, got {k.dtype} and {v.dtype}")
        if tuple(k.shape) != (T, H, D) or v.shape != k.shape:
            raise ValueError(f"shape mismatch: k {tuple(k.shape)} v {tuple(v.shape)} slots {tuple(slots.shape)}, "
                             f"the cache has {H} heads of {D}")
        _dev(slots, "slots"), _rows(k, "k"), _rows(v, "v")
        _same_device(kc, k, v, slots)
    _call(fn, on, k.data_ptr(), v.data_ptr(), _ROW_TYPES[k.dtype], _rows(k, "k"), _rows(v, "v"),
          slots.data_ptr(), kc.data_ptr(), ks.data_ptr(), vc.data_ptr(), vs.data_ptr(), T, H, D, P, page)
    return cache


def fp8_kv_cache_write(k: torch.Tensor, v: torch.Tensor, cache, slots: torch.Tensor):
    """Quantises k, v [T, H, D] (bf16 or fp32; tokens may be strided, as in a
    slice of a fused projection) into the cache's slots (int32 [T], page *
    page_size + offset; a slot outside the cache stores nothing, one given twice
    is left with either token's codes and either one's scale).  One fp32 scale
    per token and head.  Changes and returns the cache
    (make_fp8_kv_cache)."""
    return _write("dg_fp8_kv_cache_write", _cache(cache), k, v, cache, slots)


def _read(fn: str, parts, slots: torch.Tensor, dtype: torch.dtype, out):
    """A read of a cache, given its checked parts."""
    kc, ks, vc, vs, (P, H, page, D), on = parts
    if not (slots.dtype is _I32 and slots.dim() == 1 and slots.is_contiguous() and slots.get_device() == on):
        if _i32(slots, "slots").dim() != 1:
            raise ValueError(f"slots must be [T], got {tuple(slots.shape)}")
        _same_device(kc, slots)
    T = slots.shape[0]
    if out is None:
        if dtype not in _ROW_TYPES:
            raise TypeError(f"dtype must be bfloat16 or float32, got {dtype}")
        k = kc.new_empty((T, H, D), dtype=dtype)
        v = torch.empty_like(k)
    else:
        k, v = _dev(out[0], "out k"), _dev(out[1], "out v")
        if k.dtype not in _ROW_TYPES or v.dtype != k.dtype:
            raise TypeError(f"out must both be bfloat16 or float32, got {k.dtype} and {v.dtype}")
        if tuple(k.shape) != (T, H, D) or v.shape != k.shape:
            raise ValueError(f"out shapes {tuple(k.shape)} {tuple(v.shape)}, want {(T, H, D)}")
        _same_device(kc, k, v)
    _call(fn, on, kc.data_ptr(), ks.data_ptr(), vc.data_ptr(), vs.data_ptr(), slots.data_ptr(),
          k.data_ptr(), v.data_ptr(), _ROW_TYPES[k.dtype], T, H, D, P, page)
    return k, v


def fp8_kv_cache_read(cache, slots: torch.Tensor, dtype: torch.dtype = torch.bfloat16,
                      out: Optional[Tuple[torch.Tensor, torch.Tensor]] = None):
    """The keys and values at slots (int32 [T]) of the cache as (k, v) [T, H, D]
    of dtype (bfloat16 or float32), or into out; a slot outside the cache gives
    zeros."""
    return _read("dg_fp8_kv_cache_read", _cache(cache), slots, dtype, out)


def make_kv_page_pool(num_pages: int, device=None):
    """A pool in which all of a cache's pages are free: (pages int32 [num_pages], a
    ring, state int32 [2]: the place of the first free page, and how many are free)."""
    device = torch.cuda.current_device() if device is None else device
    return (torch.arange(num_pages, dtype=torch.int32, device=device),
            torch.tensor([0, num_pages], dtype=torch.int32, device=device))


def kv_cache_plan(page_table: torch.Tensor, context_lens: torch.Tensor, add_lens: torch.Tensor, pool, page_size: int,
                  rows: int, padded: bool = False, out=None):
    """Gives requests their pages and new tokens their slots.  Request b of
    context_lens[b] tokens (int32 [B]) gets add_lens[b] more (int32 [B]); where that
    is negative it loses tokens at its end.  pool = (pages, state), as
    make_kv_page_pool makes it.  New pages go from the pool into page_table (int32
    [B, max_pages]), pages behind a new end back into it; both are changed in place.  A
    page that several requests hold would come back from each.
    Returns (slots, positions, lens, state): int32 [B, rows] where padded, else
    [rows], the requests' tokens end to end (rows without a token, and tokens of
    requests that the pool or the table has no room for, have the slot -1); the lengths
    afterwards, int32 [B] (as before where there was no room); the pool's state
    afterwards, int32 [2].  out: these four, to be filled, other tensors than the
    arguments."""
    pages, state = pool
    table, ctx, add = page_table, context_lens, add_lens
    if table.dim() != 2 or pages.dim() != 1:
        raise ValueError(f"page_table {tuple(table.shape)} and the pool's pages {tuple(pages.shape)} must be "
                         "[B, max_pages] and [num_pages]")
    (B, most), P, on = table.shape, pages.shape[0], table.get_device()
    if not (table.dtype is _I32 and ctx.dtype is _I32 and add.dtype is _I32 and pages.dtype is _I32 and state.dtype is _I32
            and ctx.shape == (B,) and add.shape == (B,) and state.shape == (2,) and on >= 0
            and table.is_contiguous() and ctx.is_contiguous() and add.is_contiguous() and pages.is_contiguous()
            and state.is_contiguous() and ctx.get_device() == on and add.get_device() == on
            and pages.get_device() == on and state.get_device() == on):
        _i32(table, "page_table"), _i32(ctx, "context_lens"), _i32(add, "add_lens"), _i32(pages, "pool pages")
        _i32(state, "pool state")
        if tuple(ctx.shape) != (B,) or tuple(add.shape) != (B,) or tuple(state.shape) != (2,):
            raise ValueError(f"context_lens {tuple(ctx.shape)} and add_lens {tuple(add.shape)} must be [{B}], the "
                             f"pool's state {tuple(state.shape)} [2]")
        _same_device(table, ctx, add, pages, state)
    shape = (B, rows) if padded else (rows,)
    if out is None:
        if rows < 0:
            raise ValueError(f"rows={rows} must not be negative")
        slots = table.new_empty(shape)
        positions, lens, new_state = torch.empty_like(slots), torch.empty_like(ctx), torch.empty_like(state)
    else:
        slots, positions, lens, new_state = (_i32(t, f"out {name}") for t, name in zip(out, ("slots", "positions", "lens", "state")))
        if tuple(slots.shape) != shape or tuple(positions.shape) != shape or tuple(lens.shape) != (B,) or tuple(new_state.shape) != (2,):
            raise ValueError(f"out shapes {tuple(slots.shape)} {tuple(positions.shape)} {tuple(lens.shape)} "
                             f"{tuple(new_state.shape)}, want {shape} {shape} {(B,)} {(2,)}")
        _same_device(table, slots, positions, lens, new_state)
    _call("dg_kv_cache_plan", on, table.data_ptr(), ctx.data_ptr(), add.data_ptr(), pages.data_ptr(), state.data_ptr(),
          slots.data_ptr(), positions.data_ptr(), lens.data_ptr(), new_state.data_ptr(), B, rows, padded, most, P,
          page_size)
    return slots, positions, lens, new_state


def _workspace(given: Optional[torch.Tensor], on: int, need) -> Tuple[torch.Tensor, int, int]:
    """The caller's workspace, or one of torch's allocator for this call (need()
    says how large): itself, its address and its bytes."""
    if given is None:
        given = torch.empty(need(), dtype=_U8, device=on)
    elif not (given.dtype is _U8 and given.get_device() == on and given.is_contiguous()):
        if given.dtype != _U8:
            raise TypeError("workspace must be uint8")
        raise ValueError(f"workspace must be contiguous and on device {on}, is on {_dev(given, 'workspace').device}")
    return given, given.data_ptr(), given.numel()


def _check_norm_rope(given, q, k, weights, positions, inv_freq):
    """Finds what is wrong with the arguments of a norm and rotation: rows of both
    tensors, weights, positions and frequencies."""
    dtype, D = q.dtype, q.shape[2]
    if dtype not in _ROW_TYPES or any(t.dtype != dtype for t, _, _ in given):
        raise TypeError(f"{', '.join(name for _, _, name in given)} must all be bfloat16 or float32, got "
                        f"{[t.dtype for t, _, _ in given]}")
    for t, like, name in given:
        want = (q.shape[0], like.shape[1], D)
        if tuple(t.shape) != want:
            raise ValueError(f"shape mismatch: {name} {tuple(t.shape)} must be {want}")
        _rows(t, name)
    for w, name in zip(weights, ("q_weight", "k_weight")):
        if w is not None:
            if w.dtype not in _ROW_TYPES:
                raise TypeError(f"{name} must be bfloat16 or float32, got {w.dtype}")
            if tuple(_dev(w, name).shape) != (D,):
                raise ValueError(f"{name} {tuple(w.shape)} must be [{D}]")
    if weights[0] is not None and weights[1] is not None and weights[0].dtype != weights[1].dtype:
        raise TypeError(f"q_weight and k_weight must be of one type, got {weights[0].dtype} and {weights[1].dtype}")
    if tuple(_i32(positions, "positions").shape) != (q.shape[0],):
        raise ValueError(f"positions {tuple(positions.shape)} must be [{q.shape[0]}]")
    if _f32(inv_freq, "inv_freq").dim() != 1:
        raise ValueError(f"inv_freq {tuple(inv_freq.shape)} must be [R / 2]")
    _same_device(q, k, *(t for t, _, _ in given), *weights, positions, inv_freq)


def _norm_rope_right(q, k, wq, wk, positions, inv_freq, on) -> bool:
    """Whether what both directions of the norm and rotation share is as it should be."""
    T, _, D = q.shape
    w = wk if wq is None else wq
    return (on >= 0 and q.dtype in _ROW_TYPES and k.dtype is q.dtype and k.shape[0] == T and k.shape[2] == D
            and k.get_device() == on and positions.dtype is _I32 and positions.shape == (T,) and positions.is_contiguous()
            and positions.get_device() == on and inv_freq.dtype is _F32 and inv_freq.dim() == 1 and inv_freq.is_contiguous()
            and inv_freq.get_device() == on
            and (w is None or (w.dtype in _ROW_TYPES and w.shape == (D,) and w.is_contiguous() and w.get_device() == on))
            and (wq is None or wk is None or (wk.dtype is w.dtype and wk.shape == (D,) and wk.is_contiguous()
                                              and wk.get_device() == on)))


def qk_norm_rope(q: torch.Tensor, k: torch.Tensor, q_weight: Optional[torch.Tensor], k_weight: Optional[torch.Tensor],
                 positions: torch.Tensor, inv_freq: torch.Tensor, eps: float = 1e-6, interleaved: bool = False,
                 out: Optional[Tuple[torch.Tensor, torch.Tensor]] = None):
    """RMS norms of each head of q [T, Hq, D] and k [T, H, D] (bf16 or fp32; tokens may
    be strided, as in slices of a fused projection) with weights [D] (bf16 or fp32;
    None: ones), then the rotation of the first R = 2 * len(inv_freq) values by
    positions (int32 [T]) times inv_freq (fp32 [R / 2], R a multiple of 16): values i and
    i + R / 2 are a pair, or 2 i and 2 i + 1 where interleaved.  Returns (q, k) like
    those given but dense, or fills out, which may be q and k themselves.  As elsewhere
    here nothing is recorded for autograd: qk_norm_rope_backward has the gradients."""
    if q.dim() != 3 or k.dim() != 3:
        raise ValueError(f"q {tuple(q.shape)} and k {tuple(k.shape)} must be [T, heads, D]")
    (T, Hq, D), H, on, wq, wk = q.shape, k.shape[1], q.get_device(), q_weight, k_weight
    right = _norm_rope_right(q, k, wq, wk, positions, inv_freq, on)
    if out is not None:
        oq, ok = out
        right = (right and oq.dtype is q.dtype and ok.dtype is q.dtype and oq.shape == q.shape and ok.shape == k.shape
                 and oq.get_device() == on and ok.get_device() == on)
    if not right:
        _check_norm_rope([(q, q, "q"), (k, k, "k")] + ([] if out is None else [(out[0], q, "out q"), (out[1], k, "out k")]),
                         q, k, (wq, wk), positions, inv_freq)
    if out is None:
        oq, ok = q.new_empty((T, Hq, D)), k.new_empty((T, H, D))
        sq, sk = Hq * D, H * D
    else:
        sq, sk = _rows(oq, "out q"), _rows(ok, "out k")
    w = wk if wq is None else wq
    _call("dg_qk_norm_rope", on, q.data_ptr(), k.data_ptr(), _ROW_TYPES[q.dtype], _rows(q, "q"), _rows(k, "k"),
          0 if wq is None else wq.data_ptr(), 0 if wk is None else wk.data_ptr(), DG_F32 if w is None else _ROW_TYPES[w.dtype],
          positions.data_ptr(), inv_freq.data_ptr(), oq.data_ptr(), ok.data_ptr(), sq, sk, eps, interleaved, T, Hq, H, D,
          2 * inv_freq.shape[0])
    return oq, ok


def get_qk_norm_rope_backward_workspace_bytes(T: int, Hq: int, H: int, D: int) -> int:
    """Workspace bytes that the gradients of a norm and rotation of these sizes need."""
    return int(load_library().dg_qk_norm_rope_backward_workspace_bytes(T, Hq, H, D))


def make_qk_norm_rope_backward_workspace(q: torch.Tensor, k: torch.Tensor) -> torch.Tensor:
    """A workspace for qk_norm_rope_backward calls with arguments of these shapes.
    Stream-ordered calls may share it."""
    need = get_qk_norm_rope_backward_workspace_bytes(q.shape[0], q.shape[1], k.shape[1], q.shape[2])
    return torch.empty(need, dtype=torch.uint8, device=q.device)


def qk_norm_rope_backward(dq: torch.Tensor, dk: torch.Tensor, q: torch.Tensor, k: torch.Tensor,
                          q_weight: Optional[torch.Tensor], k_weight: Optional[torch.Tensor], positions: torch.Tensor,
                          inv_freq: torch.Tensor, eps: float = 1e-6, interleaved: bool = False,
                          out: Optional[Tuple[torch.Tensor, torch.Tensor]] = None,
                          workspace: Optional[torch.Tensor] = None):
    """The gradients of qk_norm_rope from those of its outputs, dq and dk, and its
    inputs: (dq_in, dk_in, dq_weight, dk_weight), the first two like q and k but dense
    (or out, other tensors than the arguments), the last two fp32 [D] (None where the
    weight is).  workspace: a uint8 buffer (make_qk_norm_rope_backward_workspace); when
    None, one is allocated for the call."""
    if q.dim() != 3 or k.dim() != 3:
        raise ValueError(f"q {tuple(q.shape)} and k {tuple(k.shape)} must be [T, heads, D]")
    (T, Hq, D), H, on, wq, wk = q.shape, k.shape[1], q.get_device(), q_weight, k_weight
    right = (_norm_rope_right(q, k, wq, wk, positions, inv_freq, on) and dq.dtype is q.dtype and dk.dtype is q.dtype
             and dq.shape == q.shape and dk.shape == k.shape and dq.get_device() == on and dk.get_device() == on)
    if out is not None:
        oq, ok = out
        right = (right and oq.dtype is q.dtype and ok.dtype is q.dtype and oq.shape == q.shape and ok.shape == k.shape
                 and oq.get_device() == on and ok.get_device() == on)
    if not right:
        _check_norm_rope([(q, q, "q"), (k, k, "k"), (dq, q, "dq"), (dk, k, "dk")]
                         + ([] if out is None else [(out[0], q, "out q"), (out[1], k, "out k")]), q, k, (wq, wk), positions, inv_freq)
    if out is None:
        oq, ok = q.new_empty((T, Hq, D)), k.new_empty((T, H, D))
        sq, sk = Hq * D, H * D
    else:
        sq, sk = _rows(oq, "out q"), _rows(ok, "out k")
    gq, gk = (None if x is None else x.new_empty(D, dtype=_F32) for x in (wq, wk))
    w, ws, ws_bytes = wk if wq is None else wq, 0, 0
    if w is not None:
        workspace, ws, ws_bytes = _workspace(workspace, on, lambda: get_qk_norm_rope_backward_workspace_bytes(T, Hq, H, D))
    _call("dg_qk_norm_rope_backward", on, dq.data_ptr(), dk.data_ptr(), q.data_ptr(), k.data_ptr(), _ROW_TYPES[q.dtype],
          _rows(dq, "dq"), _rows(dk, "dk"), _rows(q, "q"), _rows(k, "k"), 0 if wq is None else wq.data_ptr(),
          0 if wk is None else wk.data_ptr(), DG_F32 if w is None else _ROW_TYPES[w.dtype], positions.data_ptr(),
          inv_freq.data_ptr(), oq.data_ptr(), ok.data_ptr(), sq, sk, 0 if gq is None else gq.data_ptr(),
          0 if gk is None else gk.data_ptr(), eps, interleaved, T, Hq, H, D, 2 * inv_freq.shape[0], ws, ws_bytes)
    return oq, ok, gq, gk


def get_fp8_tree_attention_workspace_bytes(B: int, N: int, Hq: int, num_kv_heads: int, head_dim: int,
                                           page_size: int, max_pages: int) -> int:
    """Workspace bytes a tree attention call of these sizes needs (0: none)."""
    return int(load_library().dg_fp8_tree_attention_workspace_bytes(B, N, Hq, num_kv_heads, head_dim,
                                                                    page_size, max_pages))


def make_fp8_tree_attention_workspace(q: torch.Tensor, cache, page_table: torch.Tensor) -> torch.Tensor:
    """A workspace for fp8_tree_attention calls with arguments of these shapes.
    Stream-ordered calls may share it."""
    B, N, Hq, D = q.shape
    _, H, page, _ = cache[0][0].shape
    need = get_fp8_tree_attention_workspace_bytes(B, N, Hq, H, D, page, page_table.shape[1])
    return torch.empty(need, dtype=torch.uint8, device=q.device)


def _tree_attention(fn: str, need, parts, q, table, ctx, tree_lens, tree_mask, scale, out, workspace):
    """Attention over a cache, given its checked parts; need: workspace bytes of these sizes."""
    kc, ks, vc, vs, (P, H, page, D), on = parts
    if q.dim() != 4 or q.shape[3] != D:
        raise ValueError(f"q {tuple(q.shape)} must be [B, N, Hq, {D}]")
    B, N, Hq, _ = q.shape
    stride = _rows(q, "q")
    if N == 1 and B > 1:                          # a token a request: requests are the rows
        stride = q.stride(0)
    mask_shape = (B, N, (N + 63) // 64)
    if not (q.dtype is _BF16 and table.dtype is _I32 and ctx.dtype is _I32 and table.dim() == 2
            and table.shape[0] == B and ctx.shape == (B,) and table.is_contiguous() and ctx.is_contiguous()
            and q.get_device() == on and table.get_device() == on and ctx.get_device() == on
            and (B <= 1 or N == 0 or q.stride(0) == N * stride)
            and (tree_lens is None or (tree_lens.dtype is _I32 and tree_lens.shape == (B,)
                                       and tree_lens.is_contiguous() and tree_lens.get_device() == on))
            and (tree_mask is None or (tree_mask.dtype is _I64 and tree_mask.shape == mask_shape
                                       and tree_mask.is_contiguous() and tree_mask.get_device() == on))):
        if q.dtype != torch.bfloat16:
            raise TypeError(f"q must be bfloat16, got {q.dtype}")
        _rows(q, "q")
        if B > 1 and N > 0 and q.stride(0) != N * stride:
            raise ValueError(f"q: tokens must be evenly spaced over requests, strides are {q.stride()}")
        _i32(table, "page_table"), _i32(ctx, "context_lens")
        if table.dim() != 2 or table.shape[0] != B or tuple(ctx.shape) != (B,):
            raise ValueError(f"page_table {tuple(table.shape)} and context_lens {tuple(ctx.shape)} must be "
                             f"[{B}, max_pages] and [{B}]")
        if tree_lens is not None and tuple(_i32(tree_lens, "tree_lens").shape) != (B,):
            raise ValueError(f"tree_lens {tuple(tree_lens.shape)} must be [{B}]")
        if tree_mask is not None:
            if tree_mask.dtype != torch.int64:
                raise TypeError(f"tree_mask must be int64, got {tree_mask.dtype}")
            if tuple(_dev(tree_mask, "tree_mask").shape) != mask_shape:
                raise ValueError(f"tree_mask {tuple(tree_mask.shape)} must be {mask_shape}")
        _same_device(kc, q, table, ctx, tree_lens, tree_mask)
    if out is None:
        o = torch.empty_like(q) if q.is_contiguous() else q.new_empty(q.shape)
        lse = q.new_empty((B, N, Hq), dtype=_F32)
    else:
        o, lse = _dev(out[0], "out"), _f32(out[1], "lse")
        if o.dtype != torch.bfloat16:
            raise TypeError("out must be bfloat16")
        if o.shape != q.shape or tuple(lse.shape) != (B, N, Hq):
            raise ValueError(f"out shapes {tuple(o.shape)} {tuple(lse.shape)}, want {tuple(q.shape)} and {(B, N, Hq)}")
        _same_device(kc, o, lse)
    workspace, ws, ws_bytes = _workspace(workspace, on, lambda: need(B, N, Hq, H, D, page, table.shape[1]))
    _call(fn, on, q.data_ptr(), stride, kc.data_ptr(), ks.data_ptr(), vc.data_ptr(),
          vs.data_ptr(), table.data_ptr(), ctx.data_ptr(), 0 if tree_lens is None else tree_lens.data_ptr(),
          0 if tree_mask is None else tree_mask.data_ptr(), o.data_ptr(), lse.data_ptr(),
          D ** -0.5 if scale is None else scale, B, N, Hq, H, D, P, page, table.shape[1], ws, ws_bytes)
    return o, lse


def fp8_tree_attention(q: torch.Tensor, cache, page_table: torch.Tensor, context_lens: torch.Tensor,
                       tree_lens: Optional[torch.Tensor] = None, tree_mask: Optional[torch.Tensor] = None,
                       scale: Optional[float] = None,
                       out: Optional[Tuple[torch.Tensor, torch.Tensor]] = None,
                       workspace: Optional[torch.Tensor] = None):
    """Attention of drafted tokens q [B, N, Hq, D] (bf16; tokens may be strided)
    over the FP8 cache.  page_table int32 [B, max_pages]; request b has
    context_lens[b] tokens in the cache, then its tree_lens[b] (int32 [B], N
    when None) drafted ones.  tree_mask int64 [B, N, ceil(N/64)]: bit j % 64 of
    word j / 64 of token i lets it see drafted token j (None: a chain, j <= i);
    every context token is seen.  scale defaults to D ** -0.5.  Returns (o bf16
    like q, lse fp32 [B, N, Hq]), or fills out; rows past a tree's end, and rows
    that see nothing, are 0 and -inf.  workspace: a uint8 buffer
    (make_fp8_tree_attention_workspace); when None, one is allocated for the
    call."""
    return _tree_attention("dg_fp8_tree_attention", get_fp8_tree_attention_workspace_bytes, _cache(cache), q, page_table,
                           context_lens, tree_lens, tree_mask, scale, out, workspace)


# ---- the cache in 4 bits ---------------------------------------------------------------------

def make_fp4_kv_cache(num_pages: int, num_kv_heads: int, page_size: int, head_dim: int, device=None):
    """An empty paged FP4 cache: ((k codes, k scales), (v codes, v scales)), codes
    uint8 [num_pages, num_kv_heads, page_size, head_dim / 2], two e2m1 a byte, scales uint8
    [num_pages, num_kv_heads, page_size, head_dim / 32], exponents of powers of two, one for
    32 values.  page_size is a power of two from 16 to 4096, head_dim 64, 128 or 256."""
    shape = (num_pages, num_kv_heads, page_size)
    device = torch.cuda.current_device() if device is None else device
    return tuple((torch.zeros(shape + (head_dim // 2,), dtype=torch.uint8, device=device),
                  torch.full(shape + (head_dim // 32,), 127, dtype=torch.uint8, device=device)) for _ in range(2))


def _cache4(cache):
    """The FP4 cache's four tensors, checked, its sizes and its device's index."""
    (kc, ks), (vc, vs) = cache
    shape, sf_shape, on = kc.shape, ks.shape, kc.get_device()
    if not (kc.dtype is _U8 and vc.dtype is _U8 and ks.dtype is _U8 and vs.dtype is _U8 and on >= 0
            and vc.shape == shape and len(shape) == 4 and len(sf_shape) == 4 and shape[:3] == sf_shape[:3]
            and shape[3] == 16 * sf_shape[3] and vs.shape == sf_shape
            and kc.is_contiguous() and vc.is_contiguous() and ks.is_contiguous() and vs.is_contiguous()
            and ks.get_device() == on and vc.get_device() == on and vs.get_device() == on):
        for t, name in ((kc, "k codes"), (ks, "k scales"), (vc, "v codes"), (vs, "v scales")):
            if t.dtype != torch.uint8:
                raise TypeError(f"{name} must be uint8, got {t.dtype}")
            _dev(t, name)
        if (kc.dim() != 4 or kc.shape != vc.shape or ks.dim() != 4 or ks.shape[:3] != kc.shape[:3] or vs.shape != ks.shape
                or kc.shape[3] != 16 * ks.shape[3]):
            raise ValueError(f"cache shapes: codes {tuple(kc.shape)} {tuple(vc.shape)}, scales {tuple(ks.shape)} "
                             f"{tuple(vs.shape)}, want [pages, heads, page_size, head_dim / 2] and [..., head_dim / 32]")
        _same_device(kc, ks, vc, vs)
    return kc, ks, vc, vs, (shape[0], shape[1], shape[2], 2 * shape[3]), on


def fp4_kv_cache_write(k: torch.Tensor, v: torch.Tensor, cache, slots: torch.Tensor):
    """fp8_kv_cache_write for an FP4 cache (make_fp4_kv_cache): k, v [T, H, D] quantised
    into slots, e2m1 codes with the least power of two that brings each 32 values to 6 at
    most.  Changes and returns the cache."""
    return _write("dg_fp4_kv_cache_write", _cache4(cache), k, v, cache, slots)


def fp4_kv_cache_read(cache, slots: torch.Tensor, dtype: torch.dtype = torch.bfloat16,
                      out: Optional[Tuple[torch.Tensor, torch.Tensor]] = None):
    """The keys and values at slots (int32 [T]) of an FP4 cache as (k, v) [T, H, D] of
    dtype (bfloat16 or float32; both hold them exactly), or into out; a slot outside the
    cache gives zeros."""
    return _read("dg_fp4_kv_cache_read", _cache4(cache), slots, dtype, out)


def get_fp4_tree_attention_workspace_bytes(B: int, N: int, Hq: int, num_kv_heads: int, head_dim: int,
                                           page_size: int, max_pages: int) -> int:
    """Workspace bytes a tree attention call over an FP4 cache needs (0: none)."""
    return int(load_library().dg_fp4_tree_attention_workspace_bytes(B, N, Hq, num_kv_heads, head_dim,
                                                                    page_size, max_pages))


def make_fp4_tree_attention_workspace(q: torch.Tensor, cache, page_table: torch.Tensor) -> torch.Tensor:
    """A workspace for fp4_tree_attention calls with arguments of these shapes.
    Stream-ordered calls may share it."""
    B, N, Hq, D = q.shape
    _, H, page, _ = cache[0][0].shape
    need = get_fp4_tree_attention_workspace_bytes(B, N, Hq, H, D, page, page_table.shape[1])
    return torch.empty(need, dtype=torch.uint8, device=q.device)


def fp4_tree_attention(q: torch.Tensor, cache, page_table: torch.Tensor, context_lens: torch.Tensor,
                       tree_lens: Optional[torch.Tensor] = None, tree_mask: Optional[torch.Tensor] = None,
                       scale: Optional[float] = None,
                       out: Optional[Tuple[torch.Tensor, torch.Tensor]] = None,
                       workspace: Optional[torch.Tensor] = None):
    """fp8_tree_attention over an FP4 cache (make_fp4_kv_cache): the same arguments and
    results.  workspace: make_fp4_tree_attention_workspace."""
    return _tree_attention("dg_fp4_tree_attention", get_fp4_tree_attention_workspace_bytes, _cache4(cache), q, page_table,
                           context_lens, tree_lens, tree_mask, scale, out, workspace)


def get_fp8_moe_few_tokens_workspace_bytes(T: int, topk: int, E: int, H: int, I: int) -> int:
    """Workspace bytes a few-token mixture-of-experts call of these sizes needs."""
    return int(load_library().dg_fp8_moe_few_tokens_workspace_bytes(T, topk, E, H, I))


def make_fp8_moe_few_tokens_workspace(x: torch.Tensor, w2: Tuple[torch.Tensor, torch.Tensor],
                                      topk_ids: torch.Tensor) -> torch.Tensor:
    """A workspace for fp8_moe_few_tokens calls with arguments of these shapes.
    Stream-ordered calls may share it."""
    E, H, I = w2[0].shape
    need = get_fp8_moe_few_tokens_workspace_bytes(topk_ids.shape[0], topk_ids.shape[1], E, H, I)
    return torch.empty(need, dtype=torch.uint8, device=x.device)


def fp8_moe_few_tokens(x: torch.Tensor, w1: Tuple[torch.Tensor, torch.Tensor],
                       w2: Tuple[torch.Tensor, torch.Tensor], topk_ids: torch.Tensor,
                       topk_weights: torch.Tensor, out: Optional[torch.Tensor] = None,
                       dtype: torch.dtype = torch.bfloat16,
                       workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """A mixture-of-experts layer for x bf16 [T, H], T <= 256:
    y[t] = sum_j topk_weights[t, j] * W2_e (silu(W1_e[:I] x[t]) * (W1_e[I:] x[t])),
    e = topk_ids[t, j] (int32 [T, topk]; ids outside [0, E) take no part).
    w1 = (W1 e4m3 [E, 2I, H], fp32 [E, 2I/128, H/128]), w2 = (W2 e4m3 [E, H, I],
    fp32 [E, H/128, I/128]), as per_block_cast_to_fp8 makes them; H and I are
    multiples of 128.  Returns y [T, H] of dtype (bfloat16 or float32), or fills
    out.  workspace: a uint8 buffer (make_fp8_moe_few_tokens_workspace); when
    None, one is allocated for the call."""
    (W1, S1), (W2, S2), ids, weights, on = w1, w2, topk_ids, topk_weights, x.get_device()
    if x.dim() != 2 or W1.dim() != 3 or W2.dim() != 3 or ids.dim() != 2:
        raise ValueError("x and topk_ids must be 2-D, W1 and W2 3-D")
    T, H = x.shape
    E, H2, I = W2.shape
    topk = ids.shape[1]
    if not (x.dtype is _BF16 and W1.dtype is _U8 and W2.dtype is _U8 and S1.dtype is _F32 and S2.dtype is _F32
            and ids.dtype is _I32 and weights.dtype is _F32 and H2 == H and W1.shape == (E, 2 * I, H)
            and ids.shape[0] == T and weights.shape == ids.shape
            and S1.shape == (E, 2 * I // 128, H // 128) and S2.shape == (E, H // 128, I // 128)
            and x.is_contiguous() and W1.is_contiguous() and S1.is_contiguous() and W2.is_contiguous()
            and S2.is_contiguous() and ids.is_contiguous() and weights.is_contiguous()
            and on >= 0 and W1.get_device() == on and S1.get_device() == on and W2.get_device() == on
            and S2.get_device() == on and ids.get_device() == on and weights.get_device() == on):
        if _dev(x, "x").dtype != torch.bfloat16:
            raise TypeError(f"x must be bfloat16, got {x.dtype}")
        W1, S1, W2, S2 = _fp8(W1, "W1"), _f32(S1, "S1"), _fp8(W2, "W2"), _f32(S2, "S2")
        _i32(ids, "topk_ids"), _f32(weights, "topk_weights")
        if H2 != H or tuple(W1.shape) != (E, 2 * I, H) or ids.shape[0] != T or weights.shape != ids.shape:
            raise ValueError(f"shape mismatch: x {tuple(x.shape)} W1 {tuple(W1.shape)} W2 {tuple(W2.shape)} "
                             f"topk_ids {tuple(ids.shape)} topk_weights {tuple(weights.shape)}")
        if tuple(S1.shape) != (E, 2 * I // 128, H // 128) or tuple(S2.shape) != (E, H // 128, I // 128):
            raise ValueError(f"scale shapes: S1 {tuple(S1.shape)} S2 {tuple(S2.shape)}, want "
                             f"{(E, 2 * I // 128, H // 128)} and {(E, H // 128, I // 128)}")
        _same_device(x, W1, S1, W2, S2, ids, weights)
    if out is None:
        if dtype not in _ROW_TYPES:
            raise TypeError(f"dtype must be bfloat16 or float32, got {dtype}")
        out = torch.empty_like(x) if dtype is _BF16 else x.new_empty((T, H), dtype=dtype)
    else:
        out = _dev(out, "out")
        if out.dtype not in _ROW_TYPES:
            raise TypeError(f"out must be bfloat16 or float32, got {out.dtype}")
        if out.shape != x.shape:
            raise ValueError(f"out {tuple(out.shape)} must be {tuple(x.shape)}")
        _same_device(x, out)
    workspace, ws, ws_bytes = _workspace(workspace, on, lambda: get_fp8_moe_few_tokens_workspace_bytes(
        T, topk, E, H, I))
    _call("dg_fp8_moe_few_tokens", on, x.data_ptr(), W1.data_ptr(), S1.data_ptr(), W2.data_ptr(), S2.data_ptr(),
          ids.data_ptr(), weights.data_ptr(), out.data_ptr(), _ROW_TYPES[out.dtype], T, topk, E, H, I, ws, ws_bytes)
    return out
