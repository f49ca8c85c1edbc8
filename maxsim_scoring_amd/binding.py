"""Python binding of the C ABI in include/maxsim.h (argument marshalling only).

Every function takes torch tensors that live on the GPU, checks that they have
the layout the ABI documents, allocates missing outputs with torch (device
memory is PyTorch's job here) and calls the C entry point of the same name on
the current HIP stream. All arithmetic runs in the HIP kernels; there is no
CPU path. When the library is missing, or a tensor is not on the GPU, the call
raises.
"""

from __future__ import annotations

import ctypes
import math
import os
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmaxsim_amd.so")

MAXSIM_F16 = 0
MAXSIM_BF16 = 1
MAXSIM_F32 = 2
MAXSIM_I8 = 3
D_MODEL = 128

_lib = None


class MaxSimError(RuntimeError):
    """A non-zero status from the library."""

    def __init__(self, fn: str, status: int):
        msg = lib().maxsim_status_string(status).decode()
        super().__init__(f"{fn}: status {status} ({msg})")
        self.status = status


def lib() -> ctypes.CDLL:
    """The loaded C library (loaded once)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"HIP library {LIB_PATH} is not built; run __graft_entry__.build()")
        L = ctypes.CDLL(LIB_PATH)
        vp, i64, i32, f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float
        ci = ctypes.c_int
        L.maxsim_fwd.argtypes = [ci, vp, vp, i64, i64, i64, i64, i64, vp, vp, vp, vp, vp]
        L.maxsim_fwd_varlen.argtypes = [ci, vp, vp, i64, i32, vp, vp, i64, i64, vp, vp, vp]
        L.maxsim_fwd_i8.argtypes = [vp, f32, vp, f32, i64, i64, i64, i64, i64, vp, vp, vp, vp, vp, vp]
        L.maxsim_bwd.argtypes = [ci, vp, vp, i64, i64, i64, i64, i64, vp, vp, vp, vp, vp, vp, vp,
                                 vp, vp]
        L.maxsim_fwd_i8_tok.argtypes = [vp, vp, vp, vp, i64, i64, i64, i64, i64, vp, vp, vp, vp, vp]
        L.maxsim_fwd_pairs.argtypes = [ci, vp, vp, i64, i64, i64, i64, i64, vp, vp, vp, vp, i64, vp,
                                       vp, vp]
        L.maxsim_topk.argtypes = [vp, i64, i64, i64, vp, vp, vp, vp, vp]
        L.maxsim_fwd_pairs_varlen.argtypes = [ci, vp, vp, i64, i32, vp, vp, i64, i64, vp, vp, i64,
                                              vp, vp, vp]
        L.maxsim_bwd_varlen.argtypes = [ci, vp, vp, i64, i64, i32, vp, vp, i64, i64, i64, vp, vp,
                                        vp, vp, vp, vp, vp]
        L.maxsim_chamfer_fwd.argtypes = [vp, vp, i64, i64, i64, vp, vp, vp, vp, vp, vp]
        L.maxsim_chamfer_bwd.argtypes = [vp, vp, i64, i64, i64, vp, vp, vp, vp, vp, vp, vp, vp, vp,
                                         vp, vp]
        u64, f64 = ctypes.c_uint64, ctypes.c_double
        L.maxsim_quantize_tok.argtypes = [ci, vp, i64, i64, vp, ci, vp, vp, vp]
        L.maxsim_linear_i8.argtypes = [ci, vp, vp, vp, vp, vp, i64, i64, i64, vp, vp]
        L.maxsim_embed_i8.argtypes = [ci, vp, vp, vp, vp, vp, vp, i64, i64, i64, vp, vp, vp]
        L.maxsim_normalize_fwd.argtypes = [ci, vp, i64, i64, vp, ci, vp, vp, vp]
        L.maxsim_normalize_bwd.argtypes = [ci, vp, vp, vp, i64, i64, ci, vp, vp]
        L.maxsim_dropout_fwd.argtypes = [ci, vp, i64, f64, u64, u64, vp, vp, vp]
        L.maxsim_dropout_bwd.argtypes = [ci, vp, i64, f64, u64, u64, vp, vp, vp]
        L.maxsim_quantize_mx4.argtypes = [ci, vp, i64, i64, vp, ci, vp, vp, vp]
        L.maxsim_dequantize_mx4.argtypes = [vp, vp, i64, i64, ci, vp, vp]
        L.maxsim_linear_mx4.argtypes = [ci, vp, vp, vp, vp, vp, i64, i64, i64, vp, vp]
        L.maxsim_fwd_mx4.argtypes = [vp, vp, vp, vp, i64, i64, i64, i64, i64, vp, vp, vp, vp, vp]
        L.maxsim_logprob_workspace.argtypes = [i64, i64, i64, i64]
        L.maxsim_logprob_workspace.restype = i64
        L.maxsim_logprob_fwd.argtypes = [ci, vp, i64, i64, f32, vp, vp, i64, i64, vp, vp, vp, vp, vp,
                                         vp, vp, i64, vp]
        L.maxsim_logprob_bwd.argtypes = [ci, vp, i64, i64, f32, vp, vp, i64, vp, vp, vp, vp, ci, vp,
                                         vp]
        L.maxsim_logprob_fwd.restype = L.maxsim_logprob_bwd.restype = ci
        for f in (L.maxsim_quantize_mx4, L.maxsim_dequantize_mx4, L.maxsim_linear_mx4,
                  L.maxsim_fwd_mx4):
            f.restype = ci
        for f in (L.maxsim_quantize_tok, L.maxsim_linear_i8, L.maxsim_embed_i8,
                  L.maxsim_normalize_fwd, L.maxsim_normalize_bwd, L.maxsim_dropout_fwd,
                  L.maxsim_dropout_bwd):
            f.restype = ci
        for f in (L.maxsim_fwd, L.maxsim_fwd_varlen, L.maxsim_fwd_i8, L.maxsim_bwd,
                  L.maxsim_fwd_i8_tok, L.maxsim_fwd_pairs, L.maxsim_topk,
                  L.maxsim_fwd_pairs_varlen, L.maxsim_bwd_varlen, L.maxsim_chamfer_fwd,
                  L.maxsim_chamfer_bwd):
            f.restype = ci
        L.maxsim_status_string.argtypes = [ci]
        L.maxsim_status_string.restype = ctypes.c_char_p
        L.maxsim_abi_version.argtypes = []
        L.maxsim_abi_version.restype = ci
        _lib = L
    return _lib


def _p(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _dev(name: str, t: Optional[torch.Tensor], dtype=None) -> None:
    if t is None:
        return
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")


def _out(name: str, t: Optional[torch.Tensor], dtype, shape) -> None:
    """An output the caller passed in: on the GPU, contiguous, of `dtype` and
    exactly the documented `shape` (the kernels write every element of it)."""
    if t is None:
        return
    _dev(name, t, dtype)
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {list(shape)}, got {list(t.shape)}")


def _out_flat(name: str, t: torch.Tensor, dtype, n: int) -> None:
    """A flat output of n elements; with n == 0 a placeholder of at most one
    element is accepted (the default allocation keeps one)."""
    _dev(name, t, dtype)
    if t.dim() != 1 or (t.numel() != n if n > 0 else t.numel() > 1):
        raise ValueError(f"{name} must have shape [{n}], got {list(t.shape)}")


def _mask(name: str, t: Optional[torch.Tensor], shape) -> None:
    _dev(name, t, torch.uint8)
    if t is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {list(shape)}, got {list(t.shape)}")


def _stream(stream) -> ctypes.c_void_p:
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float16:
        return MAXSIM_F16
    if t.dtype == torch.bfloat16:
        return MAXSIM_BF16
    raise ValueError(f"embeddings must be float16 or bfloat16, got {t.dtype}")


def _check(fn: str, status: int) -> None:
    if status != 0:
        raise MaxSimError(fn, status)


def maxsim_fwd(Q: torch.Tensor, D: torch.Tensor, q_mask: Optional[torch.Tensor] = None,
               d_mask: Optional[torch.Tensor] = None, want_argmax: bool = False,
               scores: Optional[torch.Tensor] = None, argmax: Optional[torch.Tensor] = None,
               stream=None):
    """Cross-product forward. Q [Nq,Lq,d], D [Nd,Ld,d] fp16/bf16; masks uint8.
    Returns (scores float32 [Nq,Nd], argmax int32 [Nq,Nd,Lq] or None)."""
    Nq, Lq, d = Q.shape
    Nd, Ld, d2 = D.shape
    if d2 != d or D.dtype != Q.dtype:
        raise ValueError("Q and D must share d and dtype")
    _dev("Q", Q)
    _dev("D", D)
    _mask("q_mask", q_mask, (Nq, Lq))
    _mask("d_mask", d_mask, (Nd, Ld))
    if scores is None:
        scores = torch.empty((Nq, Nd), dtype=torch.float32, device=Q.device)
    if argmax is None and want_argmax:
        argmax = torch.empty((Nq, Nd, Lq), dtype=torch.int32, device=Q.device)
    _out("scores", scores, torch.float32, (Nq, Nd))
    _out("argmax", argmax, torch.int32, (Nq, Nd, Lq))
    st = lib().maxsim_fwd(_dtype_code(Q), _p(Q), _p(D), Nq, Nd, Lq, Ld, d, _p(q_mask), _p(d_mask),
                          _p(scores), _p(argmax), _stream(stream))
    _check("maxsim_fwd", st)
    return scores, argmax


def maxsim_fwd_varlen(Q: torch.Tensor, cu_q: torch.Tensor, max_lq: int, D: torch.Tensor,
                      cu_d: torch.Tensor, want_argmax: bool = False,
                      scores: Optional[torch.Tensor] = None,
                      argmax: Optional[torch.Tensor] = None, stream=None):
    """Padding-free forward. Q [Tq,d], D [Td,d] packed; cu_* int32 [N+1].
    Returns (scores [Nq,Nd], argmax [Nq,Nd,max_lq] or None)."""
    if Q.dim() != 2 or D.dim() != 2 or Q.shape[1] != D.shape[1] or Q.dtype != D.dtype:
        raise ValueError("Q and D must be packed [tokens, d] of one dtype")
    d = Q.shape[1]
    for n, t in (("Q", Q), ("D", D)):
        _dev(n, t)
    _dev("cu_q", cu_q, torch.int32)
    _dev("cu_d", cu_d, torch.int32)
    if cu_q.dim() != 1 or cu_d.dim() != 1:
        raise ValueError("cu_q and cu_d must be [N+1]")
    Nq, Nd = cu_q.numel() - 1, cu_d.numel() - 1
    if scores is None:
        scores = torch.empty((Nq, Nd), dtype=torch.float32, device=Q.device)
    if argmax is None and want_argmax:
        argmax = torch.empty((Nq, Nd, max_lq), dtype=torch.int32, device=Q.device)
    _out("scores", scores, torch.float32, (Nq, Nd))
    _out("argmax", argmax, torch.int32, (Nq, Nd, max_lq))
    st = lib().maxsim_fwd_varlen(_dtype_code(Q), _p(Q), _p(cu_q), Nq, int(max_lq), _p(D),
                                 _p(cu_d), Nd, d, _p(scores), _p(argmax), _stream(stream))
    _check("maxsim_fwd_varlen", st)
    return scores, argmax


def maxsim_fwd_i8(Q: torch.Tensor, q_scale: float, D: torch.Tensor, d_scale: float,
                  q_mask: Optional[torch.Tensor] = None, d_mask: Optional[torch.Tensor] = None,
                  want_argmax: bool = False, want_int: bool = True, want_float: bool = True,
                  scores_i32: Optional[torch.Tensor] = None, scores: Optional[torch.Tensor] = None,
                  argmax: Optional[torch.Tensor] = None, stream=None):
    """INT8 forward with per-tensor scales. Returns (scores_i32, scores, argmax)."""
    Nq, Lq, d = Q.shape
    Nd, Ld, d2 = D.shape
    if d2 != d:
        raise ValueError("Q and D must share d")
    _dev("Q", Q, torch.int8)
    _dev("D", D, torch.int8)
    _mask("q_mask", q_mask, (Nq, Lq))
    _mask("d_mask", d_mask, (Nd, Ld))
    dev = Q.device
    if scores_i32 is None and want_int:
        scores_i32 = torch.empty((Nq, Nd), dtype=torch.int32, device=dev)
    if scores is None and want_float:
        scores = torch.empty((Nq, Nd), dtype=torch.float32, device=dev)
    if argmax is None and want_argmax:
        argmax = torch.empty((Nq, Nd, Lq), dtype=torch.int32, device=dev)
    _out("scores_i32", scores_i32, torch.int32, (Nq, Nd))
    _out("scores", scores, torch.float32, (Nq, Nd))
    _out("argmax", argmax, torch.int32, (Nq, Nd, Lq))
    st = lib().maxsim_fwd_i8(_p(Q), float(q_scale), _p(D), float(d_scale), Nq, Nd, Lq, Ld, d,
                             _p(q_mask), _p(d_mask), _p(scores_i32), _p(scores), _p(argmax),
                             _stream(stream))
    _check("maxsim_fwd_i8", st)
    return scores_i32, scores, argmax


def maxsim_bwd(Q: torch.Tensor, D: torch.Tensor, argmax: torch.Tensor, grad_scores: torch.Tensor,
               q_mask: Optional[torch.Tensor] = None, d_mask: Optional[torch.Tensor] = None,
               dQ: Optional[torch.Tensor] = None, dD: Optional[torch.Tensor] = None,
               csr_row_ptr: Optional[torch.Tensor] = None,
               csr_col_idx: Optional[torch.Tensor] = None, stream=None):
    """Backward through a saved argmax. Returns (dQ, dD, csr_row_ptr, csr_col_idx)."""
    Nq, Lq, d = Q.shape
    Nd, Ld, d2 = D.shape
    if d2 != d or D.dtype != Q.dtype:
        raise ValueError("Q and D must share d and dtype")
    _dev("Q", Q)
    _dev("D", D)
    _dev("argmax", argmax, torch.int32)
    _dev("grad_scores", grad_scores, torch.float32)
    _mask("q_mask", q_mask, (Nq, Lq))
    _mask("d_mask", d_mask, (Nd, Ld))
    if tuple(argmax.shape) != (Nq, Nd, Lq) or tuple(grad_scores.shape) != (Nq, Nd):
        raise ValueError("argmax must be [Nq,Nd,Lq] and grad_scores [Nq,Nd]")
    dev = Q.device
    if dQ is None:
        dQ = torch.empty((Nq, Lq, d), dtype=torch.float32, device=dev)
    if dD is None:
        dD = torch.empty((Nd, Ld, d), dtype=torch.float32, device=dev)
    if csr_row_ptr is None:
        csr_row_ptr = torch.empty((Nd * Ld + 1,), dtype=torch.int32, device=dev)
    if csr_col_idx is None:
        csr_col_idx = torch.empty((max(1, Nq * Nd * Lq),), dtype=torch.int32, device=dev)
    _out("dQ", dQ, torch.float32, (Nq, Lq, d))
    _out("dD", dD, torch.float32, (Nd, Ld, d))
    _out("csr_row_ptr", csr_row_ptr, torch.int32, (Nd * Ld + 1,))
    _out_flat("csr_col_idx", csr_col_idx, torch.int32, Nq * Nd * Lq)
    st = lib().maxsim_bwd(_dtype_code(Q), _p(Q), _p(D), Nq, Nd, Lq, Ld, d, _p(q_mask), _p(d_mask),
                          _p(argmax), _p(grad_scores), _p(dQ), _p(dD), _p(csr_row_ptr),
                          _p(csr_col_idx), _stream(stream))
    _check("maxsim_bwd", st)
    return dQ, dD, csr_row_ptr, csr_col_idx[:Nq * Nd * Lq]


def maxsim_fwd_pairs_varlen(Q: torch.Tensor, cu_q: torch.Tensor, max_lq: int, D: torch.Tensor,
                            cu_d: torch.Tensor, pair_q: torch.Tensor, pair_d: torch.Tensor,
                            want_argmax: bool = False, scores: Optional[torch.Tensor] = None,
                            argmax: Optional[torch.Tensor] = None, stream=None):
    """Scores of listed (query, doc) pairs of packed batches. Q [Tq,d], D [Td,d]
    packed; pair_q, pair_d int32 [P]. Returns (scores [P], argmax [P,max_lq] or None)."""
    if Q.dim() != 2 or D.dim() != 2 or Q.shape[1] != D.shape[1] or Q.dtype != D.dtype:
        raise ValueError("Q and D must be packed [tokens, d] of one dtype")
    d = Q.shape[1]
    for n, t in (("Q", Q), ("D", D)):
        _dev(n, t)
    for n, t in (("cu_q", cu_q), ("cu_d", cu_d), ("pair_q", pair_q), ("pair_d", pair_d)):
        _dev(n, t, torch.int32)
    if pair_q.shape != pair_d.shape or pair_q.dim() != 1:
        raise ValueError("pair_q and pair_d must be [P]")
    Nq, Nd, P = cu_q.numel() - 1, cu_d.numel() - 1, pair_q.numel()
    if scores is None:
        scores = torch.empty((P,), dtype=torch.float32, device=Q.device)
    if argmax is None and want_argmax:
        argmax = torch.empty((P, max_lq), dtype=torch.int32, device=Q.device)
    _out("scores", scores, torch.float32, (P,))
    _out("argmax", argmax, torch.int32, (P, max_lq))
    st = lib().maxsim_fwd_pairs_varlen(_dtype_code(Q), _p(Q), _p(cu_q), Nq, int(max_lq), _p(D),
                                       _p(cu_d), Nd, d, _p(pair_q), _p(pair_d), P, _p(scores),
                                       _p(argmax), _stream(stream))
    _check("maxsim_fwd_pairs_varlen", st)
    return scores, argmax


def maxsim_bwd_varlen(Q: torch.Tensor, cu_q: torch.Tensor, max_lq: int, D: torch.Tensor,
                      cu_d: torch.Tensor, argmax: torch.Tensor, grad_scores: torch.Tensor,
                      dQ: Optional[torch.Tensor] = None, dD: Optional[torch.Tensor] = None,
                      csr_row_ptr: Optional[torch.Tensor] = None,
                      csr_col_idx: Optional[torch.Tensor] = None, stream=None):
    """Padding-free backward through the saved [Nq,Nd,max_lq] argmax. Q [Tq,d],
    D [Td,d] packed. Returns (dQ [Tq,d], dD [Td,d], csr_row_ptr [Td+1],
    csr_col_idx [Tq*Nd]: the first Tq*(docs with a token) entries are the CSR)."""
    if Q.dim() != 2 or D.dim() != 2 or Q.shape[1] != D.shape[1] or Q.dtype != D.dtype:
        raise ValueError("Q and D must be packed [tokens, d] of one dtype")
    Tq, d = Q.shape
    Td = D.shape[0]
    for n, t in (("Q", Q), ("D", D)):
        _dev(n, t)
    _dev("cu_q", cu_q, torch.int32)
    _dev("cu_d", cu_d, torch.int32)
    _dev("argmax", argmax, torch.int32)
    _dev("grad_scores", grad_scores, torch.float32)
    Nq, Nd = cu_q.numel() - 1, cu_d.numel() - 1
    if tuple(argmax.shape) != (Nq, Nd, max_lq) or tuple(grad_scores.shape) != (Nq, Nd):
        raise ValueError("argmax must be [Nq,Nd,max_lq] and grad_scores [Nq,Nd]")
    dev = Q.device
    if dQ is None:
        dQ = torch.empty((Tq, d), dtype=torch.float32, device=dev)
    if dD is None:
        dD = torch.empty((Td, d), dtype=torch.float32, device=dev)
    if csr_row_ptr is None:
        csr_row_ptr = torch.empty((Td + 1,), dtype=torch.int32, device=dev)
    if csr_col_idx is None:
        csr_col_idx = torch.empty((max(1, Tq * Nd),), dtype=torch.int32, device=dev)
    _out("dQ", dQ, torch.float32, (Tq, d))
    _out("dD", dD, torch.float32, (Td, d))
    _out("csr_row_ptr", csr_row_ptr, torch.int32, (Td + 1,))
    _out_flat("csr_col_idx", csr_col_idx, torch.int32, Tq * Nd)
    st = lib().maxsim_bwd_varlen(_dtype_code(Q), _p(Q), _p(cu_q), Nq, Tq, int(max_lq), _p(D),
                                 _p(cu_d), Nd, Td, d, _p(argmax), _p(grad_scores), _p(dQ), _p(dD),
                                 _p(csr_row_ptr), _p(csr_col_idx), _stream(stream))
    _check("maxsim_bwd_varlen", st)
    return dQ, dD, csr_row_ptr, csr_col_idx


def maxsim_chamfer_fwd(P: torch.Tensor, Q: torch.Tensor, want_loss: bool = True,
                       dist1: Optional[torch.Tensor] = None, idx1: Optional[torch.Tensor] = None,
                       dist2: Optional[torch.Tensor] = None, idx2: Optional[torch.Tensor] = None,
                       loss: Optional[torch.Tensor] = None, stream=None):
    """Chamfer distance of point-set batches P [B,N,3], Q [B,M,3] float32.
    Returns (dist1 [B,N], idx1 [B,N], dist2 [B,M], idx2 [B,M], loss [B] or None)."""
    if P.dim() != 3 or Q.dim() != 3 or P.shape[2] != 3 or Q.shape[2] != 3 or P.shape[0] != Q.shape[0]:
        raise ValueError("P and Q must be [B,N,3] and [B,M,3]")
    _dev("P", P, torch.float32)
    _dev("Q", Q, torch.float32)
    B, N, _ = P.shape
    M = Q.shape[1]
    dev = P.device
    if dist1 is None:
        dist1 = torch.empty((B, N), dtype=torch.float32, device=dev)
    if idx1 is None:
        idx1 = torch.empty((B, N), dtype=torch.int32, device=dev)
    if dist2 is None:
        dist2 = torch.empty((B, M), dtype=torch.float32, device=dev)
    if idx2 is None:
        idx2 = torch.empty((B, M), dtype=torch.int32, device=dev)
    if loss is None and want_loss:
        loss = torch.empty((B,), dtype=torch.float32, device=dev)
    _out("dist1", dist1, torch.float32, (B, N))
    _out("idx1", idx1, torch.int32, (B, N))
    _out("dist2", dist2, torch.float32, (B, M))
    _out("idx2", idx2, torch.int32, (B, M))
    _out("loss", loss, torch.float32, (B,))
    st = lib().maxsim_chamfer_fwd(_p(P), _p(Q), B, N, M, _p(dist1), _p(idx1), _p(dist2), _p(idx2),
                                  _p(loss), _stream(stream))
    _check("maxsim_chamfer_fwd", st)
    return dist1, idx1, dist2, idx2, loss


def maxsim_chamfer_bwd(P: torch.Tensor, Q: torch.Tensor, idx1: torch.Tensor, idx2: torch.Tensor,
                       grad_dist1: torch.Tensor, grad_dist2: torch.Tensor,
                       dP: Optional[torch.Tensor] = None, dQ: Optional[torch.Tensor] = None,
                       csr_row_ptr1: Optional[torch.Tensor] = None,
                       csr_col_idx1: Optional[torch.Tensor] = None,
                       csr_row_ptr2: Optional[torch.Tensor] = None,
                       csr_col_idx2: Optional[torch.Tensor] = None, stream=None):
    """Chamfer backward through the saved indices. Returns (dP [B,N,3],
    dQ [B,M,3], row_ptr1 [B*M+1], col_idx1 [B*N], row_ptr2 [B*N+1], col_idx2 [B*M])."""
    B, N, _ = P.shape
    M = Q.shape[1]
    _dev("P", P, torch.float32)
    _dev("Q", Q, torch.float32)
    for n, t, shp in (("idx1", idx1, (B, N)), ("idx2", idx2, (B, M))):
        _dev(n, t, torch.int32)
        if tuple(t.shape) != shp:
            raise ValueError(f"{n} must be {list(shp)}")
    for n, t, shp in (("grad_dist1", grad_dist1, (B, N)), ("grad_dist2", grad_dist2, (B, M))):
        _dev(n, t, torch.float32)
        if tuple(t.shape) != shp:
            raise ValueError(f"{n} must be {list(shp)}")
    dev = P.device
    if dP is None:
        dP = torch.empty((B, N, 3), dtype=torch.float32, device=dev)
    if dQ is None:
        dQ = torch.empty((B, M, 3), dtype=torch.float32, device=dev)
    if csr_row_ptr1 is None:
        csr_row_ptr1 = torch.empty((B * M + 1,), dtype=torch.int32, device=dev)
    if csr_col_idx1 is None:
        csr_col_idx1 = torch.empty((max(1, B * N),), dtype=torch.int32, device=dev)
    if csr_row_ptr2 is None:
        csr_row_ptr2 = torch.empty((B * N + 1,), dtype=torch.int32, device=dev)
    if csr_col_idx2 is None:
        csr_col_idx2 = torch.empty((max(1, B * M),), dtype=torch.int32, device=dev)
    _out("dP", dP, torch.float32, (B, N, 3))
    _out("dQ", dQ, torch.float32, (B, M, 3))
    _out("csr_row_ptr1", csr_row_ptr1, torch.int32, (B * M + 1,))
    _out_flat("csr_col_idx1", csr_col_idx1, torch.int32, B * N)
    _out("csr_row_ptr2", csr_row_ptr2, torch.int32, (B * N + 1,))
    _out_flat("csr_col_idx2", csr_col_idx2, torch.int32, B * M)
    st = lib().maxsim_chamfer_bwd(_p(P), _p(Q), B, N, M, _p(idx1), _p(idx2), _p(grad_dist1),
                                  _p(grad_dist2), _p(dP), _p(dQ), _p(csr_row_ptr1), _p(csr_col_idx1),
                                  _p(csr_row_ptr2), _p(csr_col_idx2), _stream(stream))
    _check("maxsim_chamfer_bwd", st)
    return dP, dQ, csr_row_ptr1, csr_col_idx1[:B * N], csr_row_ptr2, csr_col_idx2[:B * M]


def maxsim_status_string(status: int) -> str:
    return lib().maxsim_status_string(status).decode()


def maxsim_abi_version() -> int:
    return lib().maxsim_abi_version()


def maxsim_fwd_i8_tok(Q: torch.Tensor, q_scale: torch.Tensor, D: torch.Tensor,
                      d_scale: torch.Tensor, q_mask: Optional[torch.Tensor] = None,
                      d_mask: Optional[torch.Tensor] = None, want_argmax: bool = False,
                      scores: Optional[torch.Tensor] = None,
                      argmax: Optional[torch.Tensor] = None, stream=None):
    """INT8 forward with per-token scales q_scale [Nq,Lq], d_scale [Nd,Ld]
    (float32, positive). Returns (scores float32 [Nq,Nd], argmax or None)."""
    Nq, Lq, d = Q.shape
    Nd, Ld, d2 = D.shape
    if d2 != d or Q.dtype != torch.int8 or D.dtype != torch.int8:
        raise ValueError("Q and D must be int8 with the same d")
    for n, t in (("Q", Q), ("D", D)):
        _dev(n, t)
    _dev("q_scale", q_scale, torch.float32)
    _dev("d_scale", d_scale, torch.float32)
    if tuple(q_scale.shape) != (Nq, Lq) or tuple(d_scale.shape) != (Nd, Ld):
        raise ValueError("scales must be [Nq, Lq] and [Nd, Ld]")
    _mask("q_mask", q_mask, (Nq, Lq))
    _mask("d_mask", d_mask, (Nd, Ld))
    if scores is None:
        scores = torch.empty((Nq, Nd), dtype=torch.float32, device=Q.device)
    if argmax is None and want_argmax:
        argmax = torch.empty((Nq, Nd, Lq), dtype=torch.int32, device=Q.device)
    _out("scores", scores, torch.float32, (Nq, Nd))
    _out("argmax", argmax, torch.int32, (Nq, Nd, Lq))
    st = lib().maxsim_fwd_i8_tok(_p(Q), _p(q_scale), _p(D), _p(d_scale), Nq, Nd, Lq, Ld, d,
                                 _p(q_mask), _p(d_mask), _p(scores), _p(argmax), _stream(stream))
    _check("maxsim_fwd_i8_tok", st)
    return scores, argmax


def maxsim_fwd_pairs(Q: torch.Tensor, D: torch.Tensor, pair_q: torch.Tensor,
                     pair_d: torch.Tensor, q_mask: Optional[torch.Tensor] = None,
                     d_mask: Optional[torch.Tensor] = None, want_argmax: bool = False,
                     scores: Optional[torch.Tensor] = None,
                     argmax: Optional[torch.Tensor] = None, stream=None):
    """Scores of the listed (query, doc) pairs of dense Q, D (fp16/bf16).
    pair_q, pair_d int32 [P]. Returns (scores [P], argmax [P,Lq] or None)."""
    Nq, Lq, d = Q.shape
    Nd, Ld, d2 = D.shape
    if d2 != d or D.dtype != Q.dtype:
        raise ValueError("Q and D must share d and dtype")
    for n, t in (("Q", Q), ("D", D)):
        _dev(n, t)
    _dev("pair_q", pair_q, torch.int32)
    _dev("pair_d", pair_d, torch.int32)
    P = pair_q.numel()
    if pair_d.numel() != P:
        raise ValueError("pair_q and pair_d must have the same length")
    _mask("q_mask", q_mask, (Nq, Lq))
    _mask("d_mask", d_mask, (Nd, Ld))
    if scores is None:
        scores = torch.empty((P,), dtype=torch.float32, device=Q.device)
    if argmax is None and want_argmax:
        argmax = torch.empty((P, Lq), dtype=torch.int32, device=Q.device)
    _out("scores", scores, torch.float32, (P,))
    _out("argmax", argmax, torch.int32, (P, Lq))
    st = lib().maxsim_fwd_pairs(_dtype_code(Q), _p(Q), _p(D), Nq, Nd, Lq, Ld, d, _p(q_mask),
                                _p(d_mask), _p(pair_q), _p(pair_d), P, _p(scores), _p(argmax),
                                _stream(stream))
    _check("maxsim_fwd_pairs", st)
    return scores, argmax


def maxsim_topk(scores: torch.Tensor, k: int, ids: Optional[torch.Tensor] = None,
                want_rows: bool = False, idx: Optional[torch.Tensor] = None,
                val: Optional[torch.Tensor] = None, rows: Optional[torch.Tensor] = None,
                stream=None):
    """Per-row top-k of scores [Nq,Nd] float32: (idx int32 [Nq,k], val float32
    [Nq,k], rows int32 [Nq,k] or None), values decreasing, equal values in
    increasing column order. With ``ids`` [Nq,Nd] int32, idx reports
    ids[row, column] instead of the column; ``rows`` holds each entry's row."""
    if scores.dim() != 2:
        raise ValueError("scores must be [Nq, Nd]")
    _dev("scores", scores, torch.float32)
    Nq, Nd = scores.shape
    _dev("ids", ids, torch.int32)
    if ids is not None and tuple(ids.shape) != (Nq, Nd):
        raise ValueError("ids must have the shape of scores")
    if idx is None:
        idx = torch.empty((Nq, k), dtype=torch.int32, device=scores.device)
    if val is None:
        val = torch.empty((Nq, k), dtype=torch.float32, device=scores.device)
    if rows is None and want_rows:
        rows = torch.empty((Nq, k), dtype=torch.int32, device=scores.device)
    _out("idx", idx, torch.int32, (Nq, k))
    _out("val", val, torch.float32, (Nq, k))
    _out("rows", rows, torch.int32, (Nq, k))
    st = lib().maxsim_topk(_p(scores), Nq, Nd, k, _p(ids), _p(idx), _p(val), _p(rows),
                           _stream(stream))
    _check("maxsim_topk", st)
    return idx, val, rows


def two_stage_topk(Qi8: torch.Tensor, q_scale: torch.Tensor, Di8: torch.Tensor,
                   d_scale: torch.Tensor, Qf: torch.Tensor, Df: torch.Tensor, k: int,
                   candidates: int, q_mask: Optional[torch.Tensor] = None,
                   d_mask: Optional[torch.Tensor] = None, stream=None):
    """The INT8 -> FP16 top-K scan ("Flash-MaxSim" Sec. 4.1.4): per-token INT8
    scores of every doc, the `candidates` best docs per query, exact fp16/bf16
    scores of those (query, doc) pairs, and the top-k of the rescored
    candidates. Four library calls. Returns (doc idx int32 [Nq,k], exact
    scores float32 [Nq,k], int8-stage scores [Nq,Nd])."""
    Nq = Qi8.shape[0]
    s8, _ = maxsim_fwd_i8_tok(Qi8, q_scale, Di8, d_scale, q_mask, d_mask, stream=stream)
    cand, _, cand_q = maxsim_topk(s8, candidates, want_rows=True, stream=stream)
    exact, _ = maxsim_fwd_pairs(Qf, Df, cand_q.view(-1), cand.view(-1), q_mask, d_mask,
                                stream=stream)
    doc, val, _ = maxsim_topk(exact.view(Nq, candidates), k, ids=cand, stream=stream)
    return doc, val, s8


# ---------------------------------------------------------------------------
# The embedding head (include/maxsim_embed.h): hidden states to token
# embeddings. Rows may have any leading dimensions ([T, d], [Nd, Ld, d], ...).
# ---------------------------------------------------------------------------

_ROW_TYPES = {torch.float16: MAXSIM_F16, torch.bfloat16: MAXSIM_BF16, torch.float32: MAXSIM_F32}


def _row_type(name: str, dtype) -> int:
    if dtype not in _ROW_TYPES:
        raise ValueError(f"{name} must be float16, bfloat16 or float32, got {dtype}")
    return _ROW_TYPES[dtype]


def _place(names: str, *tensors) -> int:
    """The device index of one call's tensors (None for those left out): all on
    one GPU, all contiguous."""
    index = tensors[0].get_device()
    if index >= 0:
        for t in tensors:
            if t is not None and (t.get_device() != index or not t.is_contiguous()):
                break
        else:
            return index
    for name, t in zip(names.split(), tensors):
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError(f"{name} must be a GPU tensor")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        if t.get_device() != index:
            raise ValueError(f"{name} must be on GPU {index}, got {t.device}")
    raise AssertionError("unreachable")


def _elsewhere(stream, index: int):
    """None where a call can launch at once: on its tensors' device, which is the
    current one, and that device's current stream. Otherwise the context in
    which it can, so that the outputs it allocates belong to that stream too."""
    if stream is None:
        return None if index == torch._C._cuda_getDevice() else torch.cuda.device(index)
    if stream.device.index != index:
        raise ValueError(f"stream must be one of GPU {index}, got {stream.device}")
    return torch.cuda.stream(stream)


# the current stream's handle: building a Stream object takes longer than the
# call's checks
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _at(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _new(shape, dtype, device):
    """torch.empty; with the strides named it takes two thirds of the host time."""
    if len(shape) == 2:
        return torch.empty_strided(shape, (shape[1], 1), dtype=dtype, device=device)
    if len(shape) == 1:
        return torch.empty_strided(shape, (1,), dtype=dtype, device=device)
    return torch.empty(shape, dtype=dtype, device=device)


def _has(name: str, t: Optional[torch.Tensor], dtype, shape) -> None:
    if t is not None and (t.dtype != dtype or t.shape != shape):
        raise ValueError(f"{name} must be {dtype} of shape {list(shape)}, got {t.dtype} {list(t.shape)}")


def _rows(name: str, t: torch.Tensor):
    """(shape, leading shape, rows, width) of a tensor of rows."""
    shape = t.shape
    if not shape:
        raise ValueError(f"{name} must have rows in its last dimension")
    lead, d = shape[:-1], shape[-1]
    return shape, lead, t.numel() // d if d else math.prod(lead), d


def maxsim_quantize_tok(X: torch.Tensor, mask: Optional[torch.Tensor] = None,
                        normalize: bool = False, codes: Optional[torch.Tensor] = None,
                        scale: Optional[torch.Tensor] = None, stream=None):
    """Rows X [..., d] fp16/bf16/fp32 to int8 codes and one scale per token, the
    inputs of maxsim_fwd_i8_tok and maxsim_linear_i8: codes * scale is X, or with
    ``normalize`` X over its row norms. mask uint8 [...]: masked rows (and rows
    of zeros) get codes 0, scale 1. Returns (codes int8 [..., d], scale float32 [...])."""
    code = _row_type("X", X.dtype)
    shape, lead, T, d = _rows("X", X)
    _has("mask", mask, torch.uint8, lead)
    _has("codes", codes, torch.int8, shape)
    _has("scale", scale, torch.float32, lead)
    index = _place("X mask codes scale", X, mask, codes, scale)
    there = _elsewhere(stream, index)
    if there is not None:
        with there:
            return maxsim_quantize_tok(X, mask, normalize, codes, scale)
    if codes is None:
        codes = torch.empty_like(X, dtype=torch.int8)
    if scale is None:
        scale = torch.empty(lead, dtype=torch.float32, device=X.device)
    _check("maxsim_quantize_tok",
           lib().maxsim_quantize_tok(code, X.data_ptr(), T, d, _at(mask), bool(normalize),
                                     codes.data_ptr(), scale.data_ptr(), _raw_stream(index)))
    return codes, scale


def _linear_args(A, a_scale, W, w_scale, bias):
    _, lead, T, K = _rows("A", A)
    if W.dim() != 2 or W.shape[1] != K:
        raise ValueError(f"W must be [N, {K}], got {list(W.shape)}")
    N = W.shape[0]
    if A.dtype != torch.int8 or W.dtype != torch.int8:
        raise ValueError("A and W must be int8")
    _has("a_scale", a_scale, torch.float32, lead)
    _has("w_scale", w_scale, torch.float32, (N,))
    _has("bias", bias, torch.float32, (N,))
    return T, K, N, lead + (N,)


def maxsim_linear_i8(A: torch.Tensor, a_scale: torch.Tensor, W: torch.Tensor,
                     w_scale: torch.Tensor, bias: Optional[torch.Tensor] = None,
                     out_dtype=torch.bfloat16, Y: Optional[torch.Tensor] = None, stream=None):
    """8-bit product a_scale * w_scale * (A W^T) + bias. A int8 [..., K], a_scale
    float32 [...], W int8 [N, K], w_scale and bias float32 [N]. Returns Y [..., N]
    of ``out_dtype`` (fp16, bf16 or fp32)."""
    T, K, N, shape = _linear_args(A, a_scale, W, w_scale, bias)
    dt = out_dtype if Y is None else Y.dtype
    code = _row_type("out_dtype", dt)
    _has("Y", Y, dt, shape)
    index = _place("A a_scale W w_scale bias Y", A, a_scale, W, w_scale, bias, Y)
    there = _elsewhere(stream, index)
    if there is not None:
        with there:
            return maxsim_linear_i8(A, a_scale, W, w_scale, bias, dt, Y)
    if Y is None:
        Y = torch.empty(shape, dtype=dt, device=A.device)
    _check("maxsim_linear_i8",
           lib().maxsim_linear_i8(code, A.data_ptr(), a_scale.data_ptr(), W.data_ptr(),
                                  w_scale.data_ptr(), _at(bias), T, N, K, Y.data_ptr(),
                                  _raw_stream(index)))
    return Y


def maxsim_embed_i8(A: torch.Tensor, a_scale: torch.Tensor, W: torch.Tensor,
                    w_scale: torch.Tensor, bias: Optional[torch.Tensor] = None,
                    mask: Optional[torch.Tensor] = None, out_dtype=torch.int8,
                    E: Optional[torch.Tensor] = None, e_scale: Optional[torch.Tensor] = None,
                    stream=None):
    """Token embeddings from 8-bit hidden states: maxsim_linear_i8 with W [d, K],
    each row over its norm. ``out_dtype`` int8 gives codes and scales for
    maxsim_fwd_i8_tok, fp16, bf16 or fp32 the embeddings themselves. mask uint8
    [...]: masked rows give zeros (codes 0, scale 1). Returns (E [..., d],
    e_scale float32 [...] or None)."""
    T, K, d, shape = _linear_args(A, a_scale, W, w_scale, bias)
    lead = shape[:-1]
    _has("mask", mask, torch.uint8, lead)
    dt = out_dtype if E is None else E.dtype
    code = MAXSIM_I8 if dt == torch.int8 else _row_type("out_dtype", dt)
    if code != MAXSIM_I8 and e_scale is not None:
        raise ValueError("e_scale is an output of int8 embeddings only")
    _has("E", E, dt, shape)
    _has("e_scale", e_scale, torch.float32, lead)
    index = _place("A a_scale W w_scale bias mask E e_scale", A, a_scale, W, w_scale, bias, mask, E,
                   e_scale)
    there = _elsewhere(stream, index)
    if there is not None:
        with there:
            return maxsim_embed_i8(A, a_scale, W, w_scale, bias, mask, dt, E, e_scale)
    if E is None:
        E = torch.empty(shape, dtype=dt, device=A.device)
    if e_scale is None and code == MAXSIM_I8:
        e_scale = torch.empty(lead, dtype=torch.float32, device=A.device)
    _check("maxsim_embed_i8",
           lib().maxsim_embed_i8(code, A.data_ptr(), a_scale.data_ptr(), W.data_ptr(),
                                 w_scale.data_ptr(), _at(bias), _at(mask), T, d, K, E.data_ptr(),
                                 _at(e_scale), _raw_stream(index)))
    return E, e_scale


def embed_tokens_i8(H: torch.Tensor, W: torch.Tensor, w_scale: torch.Tensor,
                    bias: Optional[torch.Tensor] = None, mask: Optional[torch.Tensor] = None,
                    out_dtype=torch.int8, stream=None):
    """Hidden states H [..., K] fp16/bf16/fp32 to token embeddings through an
    8-bit projection (W int8 [d, K], w_scale [d]): the states are quantised per
    token, multiplied and normalised. Two library calls. Returns
    (E [..., d], e_scale [...] or None), as maxsim_embed_i8."""
    codes, scale = maxsim_quantize_tok(H, mask, stream=stream)
    return maxsim_embed_i8(codes, scale, W, w_scale, bias, mask, out_dtype=out_dtype, stream=stream)


def maxsim_normalize_fwd(X: torch.Tensor, mask: Optional[torch.Tensor] = None, out_dtype=None,
                         Y: Optional[torch.Tensor] = None, rnorm: Optional[torch.Tensor] = None,
                         stream=None):
    """Rows X [..., d] (fp16/bf16/fp32) over their Euclidean norms. mask uint8
    [...]: masked rows (and rows of zeros) give zeros. Returns (Y [..., d] of
    ``out_dtype``, X's by default, rnorm float32 [...] = 1/norm)."""
    xt = _row_type("X", X.dtype)
    dt = Y.dtype if Y is not None else X.dtype if out_dtype is None else out_dtype
    yt = _row_type("out_dtype", dt)
    shape, lead, T, d = _rows("X", X)
    _has("mask", mask, torch.uint8, lead)
    _has("Y", Y, dt, shape)
    _has("rnorm", rnorm, torch.float32, lead)
    index = _place("X mask Y rnorm", X, mask, Y, rnorm)
    there = _elsewhere(stream, index)
    if there is not None:
        with there:
            return maxsim_normalize_fwd(X, mask, dt, Y, rnorm)
    if Y is None:
        Y = torch.empty_like(X, dtype=dt)
    if rnorm is None:
        rnorm = torch.empty(lead, dtype=torch.float32, device=X.device)
    _check("maxsim_normalize_fwd",
           lib().maxsim_normalize_fwd(xt, X.data_ptr(), T, d, _at(mask), yt, Y.data_ptr(),
                                      rnorm.data_ptr(), _raw_stream(index)))
    return Y, rnorm


def maxsim_normalize_bwd(X: torch.Tensor, rnorm: torch.Tensor, dY: torch.Tensor, out_dtype=None,
                         dX: Optional[torch.Tensor] = None, stream=None):
    """Gradient of maxsim_normalize_fwd: X and rnorm as there, dY float32 [..., d]
    (the dQ or dD of maxsim_bwd). Returns dX [..., d] of ``out_dtype``, X's by
    default."""
    xt = _row_type("X", X.dtype)
    dt = dX.dtype if dX is not None else X.dtype if out_dtype is None else out_dtype
    gt = _row_type("out_dtype", dt)
    shape, lead, T, d = _rows("X", X)
    _has("rnorm", rnorm, torch.float32, lead)
    _has("dY", dY, torch.float32, shape)
    _has("dX", dX, dt, shape)
    index = _place("X rnorm dY dX", X, rnorm, dY, dX)
    there = _elsewhere(stream, index)
    if there is not None:
        with there:
            return maxsim_normalize_bwd(X, rnorm, dY, dt, dX)
    if dX is None:
        dX = torch.empty_like(X, dtype=dt)
    _check("maxsim_normalize_bwd",
           lib().maxsim_normalize_bwd(xt, X.data_ptr(), rnorm.data_ptr(), dY.data_ptr(), T, d, gt,
                                      dX.data_ptr(), _raw_stream(index)))
    return dX


def _dropout(fn: str, X, p, seed, step, step_dev, Y, stream, names):
    code = _row_type(names[0], X.dtype)
    for name, v in (("seed", seed), ("step", step)):
        if not 0 <= int(v) < 1 << 64:
            raise ValueError(f"{name} must be in [0, 2^64), got {v}")
    if step_dev is not None and (step_dev.dtype != torch.int64 or step_dev.numel() != 1):
        raise ValueError("step_dev must be one int64")
    _has(names[1], Y, X.dtype, X.shape)
    index = _place(f"{names[0]} step_dev {names[1]}", X, step_dev, Y)
    there = _elsewhere(stream, index)
    if there is not None:
        with there:
            return _dropout(fn, X, p, seed, step, step_dev, Y, None, names)
    if Y is None:
        Y = torch.empty_like(X)
    _check(fn, getattr(lib(), fn)(code, X.data_ptr(), X.numel(), float(p), int(seed), int(step),
                                  _at(step_dev), Y.data_ptr(), _raw_stream(index)))
    return Y


def maxsim_dropout_fwd(X: torch.Tensor, p: float, seed: int, step: int = 0,
                       step_dev: Optional[torch.Tensor] = None, Y: Optional[torch.Tensor] = None,
                       stream=None):
    """Dropout of X (any shape, fp16/bf16/fp32) with probability p, kept elements
    times 1/(1-p). The mask is a function of (seed, step + step_dev, element) and
    is not stored; step_dev is one int64 on the GPU, read when the kernel runs.
    Returns Y."""
    return _dropout("maxsim_dropout_fwd", X, p, seed, step, step_dev, Y, stream, ("X", "Y"))


def maxsim_dropout_bwd(dY: torch.Tensor, p: float, seed: int, step: int = 0,
                       step_dev: Optional[torch.Tensor] = None, dX: Optional[torch.Tensor] = None,
                       stream=None):
    """Gradient of maxsim_dropout_fwd with the same p, seed and step. Returns dX."""
    return _dropout("maxsim_dropout_bwd", dY, p, seed, step, step_dev, dX, stream, ("dY", "dX"))


# ---------------------------------------------------------------------------
# 4-bit embeddings (include/maxsim_mx4.h): a row of d values is uint8 codes
# [..., 16 B], two in a byte, and uint8 scales [..., B], B = ceil(d / 32).
# ---------------------------------------------------------------------------

def _mx4_rows(name: str, codes: torch.Tensor, scale: torch.Tensor, d: Optional[int]):
    """(leading shape, rows, width, blocks) of 4-bit rows. Without d the width is
    that of whole blocks."""
    if codes.dtype is not torch.uint8 or scale.dtype is not torch.uint8:
        raise ValueError(f"{name} and its scale must be uint8")
    shape = tuple(scale.shape)
    if not shape:
        raise ValueError(f"{name} must be [..., 16 B] and its scale [..., B]")
    lead, B = shape[:-1], shape[-1]
    if codes.shape != lead + (16 * B,):
        raise ValueError(f"{name} must have shape {list(lead) + [16 * B]}, got {list(codes.shape)}")
    if B > 4096:
        raise ValueError(f"{name} has {B} blocks of 32 in a row, 4096 are the most")
    if d is None:
        d = min(32 * B, 131071)  # the widest row
    elif (int(d) + 31) // 32 != B:
        raise ValueError(f"{name} has {B} blocks of 32 in a row, not those of d = {d}")
    return lead, math.prod(lead), int(d), B


def maxsim_quantize_mx4(X: torch.Tensor, mask: Optional[torch.Tensor] = None,
                        normalize: bool = False, codes: Optional[torch.Tensor] = None,
                        scale: Optional[torch.Tensor] = None, stream=None):
    """Rows X [..., d] fp16/bf16/fp32 (with ``normalize`` over their norms) to
    4-bit codes and one power of two for each 32 of them. mask uint8 [...]: masked
    rows give codes 0, scales 127 (2^0). Returns (codes uint8 [..., 16 B], scale
    uint8 [..., B])."""
    code = _row_type("X", X.dtype)
    shape, lead, T, d = _rows("X", X)
    B = (d + 31) // 32
    _has("mask", mask, torch.uint8, lead)
    _has("codes", codes, torch.uint8, lead + (16 * B,))
    _has("scale", scale, torch.uint8, lead + (B,))
    index = _place("X mask codes scale", X, mask, codes, scale)
    there = _elsewhere(stream, index)
    if there is not None:
        with there:
            return maxsim_quantize_mx4(X, mask, normalize, codes, scale)
    if codes is None:
        codes = _new(lead + (16 * B,), torch.uint8, X.device)
    if scale is None:
        scale = _new(lead + (B,), torch.uint8, X.device)
    _check("maxsim_quantize_mx4",
           lib().maxsim_quantize_mx4(code, X.data_ptr(), T, d, _at(mask), bool(normalize),
                                     codes.data_ptr(), scale.data_ptr(), _raw_stream(index)))
    return codes, scale


def maxsim_dequantize_mx4(codes: torch.Tensor, scale: torch.Tensor, d: Optional[int] = None,
                          out_dtype=torch.bfloat16, Y: Optional[torch.Tensor] = None, stream=None):
    """The values of 4-bit rows: codes [..., 16 B], scale [..., B] to Y [..., d] of
    ``out_dtype`` (fp16, bf16 or fp32); d is 32 B by default (at most 131071)."""
    lead, T, d, _ = _mx4_rows("codes", codes, scale, d)
    dt = out_dtype if Y is None else Y.dtype
    code = _row_type("out_dtype", dt)
    _has("Y", Y, dt, lead + (d,))
    index = _place("codes scale Y", codes, scale, Y)
    there = _elsewhere(stream, index)
    if there is not None:
        with there:
            return maxsim_dequantize_mx4(codes, scale, d, dt, Y)
    if Y is None:
        Y = _new(lead + (d,), dt, codes.device)
    _check("maxsim_dequantize_mx4",
           lib().maxsim_dequantize_mx4(codes.data_ptr(), scale.data_ptr(), T, d, code,
                                       Y.data_ptr(), _raw_stream(index)))
    return Y


def maxsim_linear_mx4(A: torch.Tensor, a_scale: torch.Tensor, W: torch.Tensor,
                      w_scale: torch.Tensor, bias: Optional[torch.Tensor] = None,
                      out_dtype=torch.bfloat16, Y: Optional[torch.Tensor] = None, stream=None):
    """Product A W^T + bias of 4-bit rows. A [..., 16 B] with a_scale [..., B], W
    [N, 16 B] with w_scale [N, B], bias float32 [N]. Returns Y [..., N] of
    ``out_dtype`` (fp16, bf16 or fp32)."""
    lead, T, K, B = _mx4_rows("A", A, a_scale, None)
    wlead, N, _, wB = _mx4_rows("W", W, w_scale, None)
    if len(wlead) != 1 or wB != B:
        raise ValueError(f"W must be [N, {16 * B}], got {list(W.shape)}")
    _has("bias", bias, torch.float32, (N,))
    dt = out_dtype if Y is None else Y.dtype
    code = _row_type("out_dtype", dt)
    _has("Y", Y, dt, lead + (N,))
    index = _place("A a_scale W w_scale bias Y", A, a_scale, W, w_scale, bias, Y)
    there = _elsewhere(stream, index)
    if there is not None:
        with there:
            return maxsim_linear_mx4(A, a_scale, W, w_scale, bias, dt, Y)
    if Y is None:
        Y = _new(lead + (N,), dt, A.device)
    _check("maxsim_linear_mx4",
           lib().maxsim_linear_mx4(code, A.data_ptr(), a_scale.data_ptr(), W.data_ptr(),
                                   w_scale.data_ptr(), _at(bias), T, N, K, Y.data_ptr(),
                                   _raw_stream(index)))
    return Y


def maxsim_fwd_mx4(Q: torch.Tensor, q_scale: torch.Tensor, D: torch.Tensor, d_scale: torch.Tensor,
                   q_mask: Optional[torch.Tensor] = None, d_mask: Optional[torch.Tensor] = None,
                   want_argmax: bool = False, scores: Optional[torch.Tensor] = None,
                   argmax: Optional[torch.Tensor] = None, stream=None):
    """MaxSim of 4-bit token embeddings: Q [Nq,Lq,16 B], q_scale [Nq,Lq,B],
    D [Nd,Ld,16 B], d_scale [Nd,Ld,B] uint8; masks uint8. Returns (scores float32
    [Nq,Nd], argmax int32 [Nq,Nd,Lq] or None)."""
    qlead, _, d, B = _mx4_rows("Q", Q, q_scale, None)
    dlead, _, _, dB = _mx4_rows("D", D, d_scale, None)
    if len(qlead) != 2 or len(dlead) != 2 or dB != B:
        raise ValueError("Q and D must be [N, L, 16 B] with the same number of blocks")
    (Nq, Lq), (Nd, Ld) = qlead, dlead
    _has("q_mask", q_mask, torch.uint8, qlead)
    _has("d_mask", d_mask, torch.uint8, dlead)
    _has("scores", scores, torch.float32, (Nq, Nd))
    _has("argmax", argmax, torch.int32, (Nq, Nd, Lq))
    index = _place("Q q_scale D d_scale q_mask d_mask scores argmax", Q, q_scale, D, d_scale, q_mask,
                   d_mask, scores, argmax)
    there = _elsewhere(stream, index)
    if there is not None:
        with there:
            return maxsim_fwd_mx4(Q, q_scale, D, d_scale, q_mask, d_mask, want_argmax, scores, argmax)
    if scores is None:
        scores = _new((Nq, Nd), torch.float32, Q.device)
    if argmax is None and want_argmax:
        argmax = _new((Nq, Nd, Lq), torch.int32, Q.device)
    _check("maxsim_fwd_mx4",
           lib().maxsim_fwd_mx4(Q.data_ptr(), q_scale.data_ptr(), D.data_ptr(), d_scale.data_ptr(),
                                Nq, Nd, Lq, Ld, d, _at(q_mask), _at(d_mask), scores.data_ptr(),
                                _at(argmax), _raw_stream(index)))
    return scores, argmax


def embed_tokens_mx4(H: torch.Tensor, W: torch.Tensor, w_scale: torch.Tensor,
                     bias: Optional[torch.Tensor] = None, mask: Optional[torch.Tensor] = None,
                     stream=None):
    """Hidden states H [..., K] fp16/bf16/fp32 to 4-bit token embeddings through a
    4-bit projection (W [d, 16 B], w_scale [d, B]): the states are quantised,
    multiplied, normalised and quantised again. Three library calls. Returns
    (codes, scale) as maxsim_quantize_mx4, masked rows as there."""
    a, a_scale = maxsim_quantize_mx4(H, mask, stream=stream)
    y = maxsim_linear_mx4(a, a_scale, W, w_scale, bias, out_dtype=torch.float32, stream=stream)
    return maxsim_quantize_mx4(y, mask, normalize=True, stream=stream)


def two_stage_topk_mx4(Qm: torch.Tensor, q_scale: torch.Tensor, Dm: torch.Tensor,
                       d_scale: torch.Tensor, Qf: torch.Tensor, Df: torch.Tensor, k: int,
                       candidates: int, q_mask: Optional[torch.Tensor] = None,
                       d_mask: Optional[torch.Tensor] = None, stream=None):
    """two_stage_topk with a 4-bit scan: maxsim_fwd_mx4 scores of every doc, the
    `candidates` best docs per query, exact fp16/bf16 scores of those (query, doc)
    pairs, and the top-k of the rescored candidates. Four library calls. Returns
    (doc idx int32 [Nq,k], exact scores float32 [Nq,k], scan scores [Nq,Nd])."""
    Nq = Qm.shape[0]
    scan, _ = maxsim_fwd_mx4(Qm, q_scale, Dm, d_scale, q_mask, d_mask, stream=stream)
    cand, _, cand_q = maxsim_topk(scan, candidates, want_rows=True, stream=stream)
    exact, _ = maxsim_fwd_pairs(Qf, Df, cand_q.view(-1), cand.view(-1), q_mask, d_mask,
                                stream=stream)
    doc, val, _ = maxsim_topk(exact.view(Nq, candidates), k, ids=cand, stream=stream)
    return doc, val, scan


# ---------------------------------------------------------------------------
# Log probabilities of columns of a score matrix (include/maxsim_loss.h)
# ---------------------------------------------------------------------------

def _logprob_args(X, targets, mask):
    if X.dim() != 2 or targets.dim() != 2 or targets.shape[0] != X.shape[0]:
        raise ValueError("X must be [Nq, Nd] and targets [Nq, P]")
    code = _row_type("X", X.dtype)
    if targets.dtype != torch.int32:
        raise ValueError(f"targets must be int32, got {targets.dtype}")
    _has("mask", mask, torch.uint8, X.shape)
    return code, X.shape[0], X.shape[1], targets.shape[1]


def maxsim_logprob_workspace(Nq: int, Nd: int, P: int, k: int = 0) -> int:
    """Bytes of workspace that maxsim_logprob_fwd needs for these sizes, 0 for rows of up
    to 4096 columns. Calls that may run at the same time need one each."""
    need = lib().maxsim_logprob_workspace(Nq, Nd, P, k)
    if need < 0:
        raise ValueError(f"sizes {Nq}, {Nd}, {P}, {k} are refused")
    return need


def maxsim_logprob_fwd(X: torch.Tensor, targets: torch.Tensor, mask: Optional[torch.Tensor] = None,
                       scale: float = 1.0, k: int = 0, logp: Optional[torch.Tensor] = None,
                       rank: Optional[torch.Tensor] = None, norm: Optional[torch.Tensor] = None,
                       entropy: Optional[torch.Tensor] = None,
                       top_idx: Optional[torch.Tensor] = None,
                       top_logp: Optional[torch.Tensor] = None,
                       workspace: Optional[torch.Tensor] = None, stream=None):
    """Log probabilities of columns ``targets`` [Nq, P] int32 under the softmax of
    ``scale`` X (2^-64 to 2^64), rows of scores X [Nq, Nd] (fp16/bf16/fp32), mask uint8 [Nq, Nd].
    Returns (logp [Nq, P], rank int32 [Nq, P], norm [Nq, 2], entropy [Nq],
    top_idx int32 [Nq, k], top_logp [Nq, k]; the last two None with k = 0).
    ``workspace`` is uint8 of maxsim_logprob_workspace bytes (allocated if left out)."""
    code, Nq, Nd, P = _logprob_args(X, targets, mask)
    k = int(k)
    if not 0 <= k <= 1024:
        raise ValueError(f"k must be in [0, 1024], got {k}")
    _has("logp", logp, torch.float32, (Nq, P))
    _has("rank", rank, torch.int32, (Nq, P))
    _has("norm", norm, torch.float32, (Nq, 2))
    _has("entropy", entropy, torch.float32, (Nq,))
    _has("top_idx", top_idx, torch.int32, (Nq, k))
    _has("top_logp", top_logp, torch.float32, (Nq, k))
    need = lib().maxsim_logprob_workspace(Nq, Nd, P, k) if Nd > 4096 else 0
    if workspace is not None and (workspace.dtype != torch.uint8 or workspace.numel() < need):
        raise ValueError(f"workspace must be uint8 of at least {need} bytes")
    index = _place("X targets mask logp rank norm entropy top_idx top_logp workspace", X, targets, mask,
                   logp, rank, norm, entropy, top_idx, top_logp, workspace)
    there = _elsewhere(stream, index)
    if there is not None:
        with there:
            return maxsim_logprob_fwd(X, targets, mask, scale, k, logp, rank, norm, entropy, top_idx,
                                      top_logp, workspace)
    dev = X.device
    if logp is None:
        logp = _new((Nq, P), torch.float32, dev)
    if rank is None:
        rank = _new((Nq, P), torch.int32, dev)
    if norm is None:
        norm = _new((Nq, 2), torch.float32, dev)
    if entropy is None:
        entropy = _new((Nq,), torch.float32, dev)
    if k and top_idx is None:
        top_idx = _new((Nq, k), torch.int32, dev)
    if k and top_logp is None:
        top_logp = _new((Nq, k), torch.float32, dev)
    if workspace is None and need > 0:
        workspace = _new((need,), torch.uint8, dev)
    _check("maxsim_logprob_fwd",
           lib().maxsim_logprob_fwd(code, X.data_ptr(), Nq, Nd, float(scale), _at(mask),
                                    targets.data_ptr(), P, k, logp.data_ptr(), rank.data_ptr(),
                                    norm.data_ptr(), entropy.data_ptr(), _at(top_idx),
                                    _at(top_logp), _at(workspace),
                                    0 if workspace is None else workspace.numel(),
                                    _raw_stream(index)))
    return logp, rank, norm, entropy, top_idx, top_logp


def maxsim_logprob_bwd(X: torch.Tensor, targets: torch.Tensor, norm: torch.Tensor,
                       grad_logp: torch.Tensor, mask: Optional[torch.Tensor] = None,
                       scale: float = 1.0, entropy: Optional[torch.Tensor] = None,
                       grad_entropy: Optional[torch.Tensor] = None, out_dtype=torch.float32,
                       dX: Optional[torch.Tensor] = None, stream=None):
    """Gradient of maxsim_logprob_fwd with respect to X, from its norm (and, with
    grad_entropy [Nq], its entropy): grad_logp float32 [Nq, P]. Returns dX [Nq, Nd]
    of ``out_dtype``; in float32 it is the grad_scores of maxsim_bwd."""
    code, Nq, Nd, P = _logprob_args(X, targets, mask)
    _has("norm", norm, torch.float32, (Nq, 2))
    _has("grad_logp", grad_logp, torch.float32, (Nq, P))
    if (entropy is None) != (grad_entropy is None):
        raise ValueError("entropy and grad_entropy go together")
    _has("entropy", entropy, torch.float32, (Nq,))
    _has("grad_entropy", grad_entropy, torch.float32, (Nq,))
    dt = out_dtype if dX is None else dX.dtype
    xt = _row_type("out_dtype", dt)
    _has("dX", dX, dt, X.shape)
    index = _place("X targets norm grad_logp mask entropy grad_entropy dX", X, targets, norm, grad_logp,
                   mask, entropy, grad_entropy, dX)
    there = _elsewhere(stream, index)
    if there is not None:
        with there:
            return maxsim_logprob_bwd(X, targets, norm, grad_logp, mask, scale, entropy, grad_entropy,
                                      dt, dX)
    if dX is None:
        dX = torch.empty_like(X, dtype=dt)
    _check("maxsim_logprob_bwd",
           lib().maxsim_logprob_bwd(code, X.data_ptr(), Nq, Nd, float(scale), _at(mask),
                                    targets.data_ptr(), P, norm.data_ptr(), _at(entropy),
                                    grad_logp.data_ptr(), _at(grad_entropy), xt, dX.data_ptr(),
                                    _raw_stream(index)))
    return dX
