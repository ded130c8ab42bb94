"""Thin ctypes binding of ``libmsa.so`` -- argument marshalling only.

Each function has the name of the C entry point it calls (``include/msa.h``)
and takes torch CUDA tensors; it passes raw device pointers, element strides
and the current CUDA stream, raises ``MSAError`` on a non-OK status, and does
no arithmetic of its own.  If the library is missing this module raises on
first use: there is no fallback path.
"""
from __future__ import annotations

import ctypes
import os
import threading

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "lib", "libmsa.so")

BLOCK = 128
TOPK = 16
HEAD_DIM = 128

STATUS = {0: "MSA_OK", 1: "MSA_ERR_INVALID_ARG", 2: "MSA_ERR_UNSUPPORTED",
          3: "MSA_ERR_ALIGNMENT", 4: "MSA_ERR_WORKSPACE_TOO_SMALL", 5: "MSA_ERR_CUDA",
          6: "MSA_ERR_SCRATCH_LIMIT"}
DEVERR = {1: "MSA_DEVERR_TIMEOUT", 2: "MSA_DEVERR_BAD_BLOCK", 3: "MSA_DEVERR_BAD_ENTRY",
          4: "MSA_DEVERR_BAD_POSITION", 5: "MSA_DEVERR_BAD_PAGE", 6: "MSA_DEVERR_BAD_LENGTH"}


class MSAError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn} returned {STATUS.get(status, status)}")
        self.status = status


class Dims(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("n_q", ctypes.c_int64), ("n_kv", ctypes.c_int64),
                ("q_pos0", ctypes.c_int64), ("h_q", ctypes.c_int32), ("h_kv", ctypes.c_int32),
                ("h_kidx", ctypes.c_int32), ("d_idx", ctypes.c_int32), ("scale", ctypes.c_float),
                ("q_window", ctypes.c_int32)]


class Tensor(ctypes.Structure):
    _fields_ = [("ptr", ctypes.c_void_p), ("s_batch", ctypes.c_int64), ("s_tok", ctypes.c_int64),
                ("s_head", ctypes.c_int64)]


class NormRopeDims(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("n_tok", ctypes.c_int64), ("pos0", ctypes.c_int64),
                ("h_q", ctypes.c_int32), ("h_k", ctypes.c_int32), ("d", ctypes.c_int32),
                ("rot", ctypes.c_int32), ("interleaved", ctypes.c_int32),
                ("eps", ctypes.c_float)]


class PagedKV(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("n_pages", ctypes.c_int64),
                ("s_page", ctypes.c_int64), ("s_tok", ctypes.c_int64), ("s_head", ctypes.c_int64),
                ("block_table", ctypes.c_void_p), ("table_stride", ctypes.c_int64),
                ("seq_lens", ctypes.c_void_p), ("page_size", ctypes.c_int32),
                ("h_kv", ctypes.c_int32)]


_lib = None
_lock = threading.Lock()
_P = ctypes.c_void_p
_PD = ctypes.POINTER(Dims)


def load_library(path: str) -> ctypes.CDLL:
    """Load a build of the library from `path` with every signature declared."""
    if not os.path.exists(path):
        raise RuntimeError(
            f"{path} is missing: build it with "
            "`python -m block_sparse_attention_32_b200.build` (no CPU fallback exists)")
    L = ctypes.CDLL(path)
    L.msa_num_blocks.argtypes = [_PD]
    L.msa_num_blocks.restype = ctypes.c_int64
    L.msa_num_entries.argtypes = [_PD]
    L.msa_num_entries.restype = ctypes.c_int64
    L.msa_query_window.argtypes = [_PD]
    L.msa_query_window.restype = ctypes.c_int64
    L.msa_num_segments.argtypes = [_PD]
    L.msa_num_segments.restype = ctypes.c_int64
    L.msa_index_score_maxpool.argtypes = [_PD, Tensor, Tensor, _P, ctypes.c_int64, _P, _P]
    L.msa_topk_blocks.argtypes = [_PD, _P, ctypes.c_int64, _P, _P, _P]
    L.msa_block_query_lists_workspace.argtypes = [_PD]
    L.msa_block_query_lists_workspace.restype = ctypes.c_size_t
    L.msa_build_block_query_lists.argtypes = [_PD, _P, _P, _P, _P, _P, ctypes.c_size_t, _P, _P]
    L.msa_build_block_query_lists_noalloc.argtypes = [_PD, _P, _P, _P, _P, _P, _P]
    L.msa_sparse_attn_fwd.argtypes = [_PD, Tensor, Tensor, Tensor, _P, _P, _P, _P, _P, _P]
    L.msa_merge_partials.argtypes = [_PD, _P, _P, _P, _P, _P, _P, _P]
    L.msa_sparse_attn_fwd_compact.argtypes = [_PD, Tensor, Tensor, Tensor, _P, _P, _P, _P, _P,
                                              _P]
    L.msa_merge_partials_compact.argtypes = [_PD, _P, _P, _P, _P, _P, _P, _P]
    L.msa_quantize_e4m3.argtypes = [_P, ctypes.c_int64, _P, _P, _P]
    L.msa_index_score_maxpool_e4m3.argtypes = [_PD, Tensor, Tensor, _P, _P, _P, ctypes.c_int64,
                                               _P, _P]
    L.msa_selection_recall_workspace.argtypes = [_PD, ctypes.c_int64]
    L.msa_selection_recall_workspace.restype = ctypes.c_size_t
    L.msa_selection_recall.argtypes = [_PD, Tensor, Tensor, Tensor, Tensor, _P, _P, ctypes.c_int64,
                                       _P, ctypes.c_int64, _P, _P, _P, _P, _P, ctypes.c_size_t,
                                       _P, _P]
    L.msa_sparse_attn_bwd.argtypes = [_PD, Tensor, Tensor, Tensor, Tensor, Tensor, _P, _P, _P,
                                      _P, _P, _P, _P, _P, _P, _P]
    L.msa_token_select_workspace.argtypes = [_PD, ctypes.c_int64]
    L.msa_token_select_workspace.restype = ctypes.c_size_t
    L.msa_token_select_attention.argtypes = [_PD, Tensor, Tensor, Tensor, Tensor, Tensor, _P,
                                             ctypes.c_int64, ctypes.c_int64, _P, _P, _P, _P,
                                             ctypes.c_size_t, _P, _P]
    _PN, _PC, _I64 = ctypes.POINTER(NormRopeDims), ctypes.POINTER(PagedKV), ctypes.c_int64
    L.msa_qk_norm_rope.argtypes = [_PN, Tensor, Tensor, _P, _P, _P, _I64, _P, Tensor, Tensor, _P,
                                   _P]
    L.msa_qk_norm_rope_paged.argtypes = [_PN, Tensor, Tensor, Tensor, _P, _P, _P, _I64, _P,
                                         Tensor, _PC, _P, _P]
    L.msa_qk_norm_rope_bwd_workspace.argtypes = [_PN]
    L.msa_qk_norm_rope_bwd_workspace.restype = ctypes.c_size_t
    L.msa_qk_norm_rope_bwd.argtypes = [_PN, Tensor, Tensor, _P, _P, _P, _I64, _P, Tensor, Tensor,
                                       ctypes.c_int32, Tensor, Tensor, _P, _P, _P,
                                       ctypes.c_size_t, _P, _P]
    L.msa_paged_decode_attn_workspace.argtypes = [_PD]
    L.msa_paged_decode_attn_workspace.restype = ctypes.c_size_t
    L.msa_paged_decode_attn.argtypes = [_PD, _I64, _I64, Tensor, _PC, _P, _P, _P,
                                        ctypes.c_size_t, _P, _P]
    L.msa_window_attn_fwd.argtypes = [_PD, _I64, _I64, Tensor, Tensor, Tensor, _P, _P, _P, _P,
                                      _P]
    L.msa_window_attn_bwd_workspace.argtypes = [_PD, _I64, _I64]
    L.msa_window_attn_bwd_workspace.restype = ctypes.c_size_t
    L.msa_window_attn_bwd.argtypes = [_PD, _I64, _I64, Tensor, Tensor, Tensor, Tensor, Tensor,
                                      _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P, _P]
    L.msa_debug_set_attn_wait_limit_ns.argtypes = [ctypes.c_uint64]
    L.msa_debug_set_attn_wait_limit_ns.restype = ctypes.c_uint64
    L.msa_status_string.argtypes = [ctypes.c_int]
    L.msa_status_string.restype = ctypes.c_char_p
    for f in (L.msa_index_score_maxpool, L.msa_topk_blocks, L.msa_build_block_query_lists,
              L.msa_build_block_query_lists_noalloc, L.msa_sparse_attn_fwd, L.msa_merge_partials,
              L.msa_sparse_attn_fwd_compact, L.msa_merge_partials_compact,
              L.msa_selection_recall, L.msa_quantize_e4m3, L.msa_index_score_maxpool_e4m3,
              L.msa_token_select_attention, L.msa_sparse_attn_bwd, L.msa_qk_norm_rope,
              L.msa_qk_norm_rope_paged, L.msa_qk_norm_rope_bwd, L.msa_paged_decode_attn,
              L.msa_window_attn_fwd, L.msa_window_attn_bwd):
        f.restype = ctypes.c_int
    return L


def lib() -> ctypes.CDLL:
    """Load libmsa.so (raises if it has not been built)."""
    global _lib
    with _lock:
        if _lib is None:
            _lib = load_library(LIB_PATH)
    return _lib


def make_dims(batch, n_q, n_kv, q_pos0, h_q, h_kv, d_idx, h_kidx=1, scale=None,
              q_window=0) -> Dims:
    if scale is None:
        scale = HEAD_DIM ** -0.5
    return Dims(batch, n_q, n_kv, q_pos0, h_q, h_kv, h_kidx, d_idx, scale, q_window)


def _ptr(t) -> int:
    return 0 if t is None else t.data_ptr()


def _stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def tensor_btd(t: torch.Tensor) -> Tensor:
    """[B, T, H, D] layout (q, q_idx)."""
    assert t.dim() == 4 and t.stride(3) == 1 and t.dtype == torch.bfloat16 and t.is_cuda
    return Tensor(t.data_ptr(), t.stride(0), t.stride(1), t.stride(2))


def tensor_bhtd(t: torch.Tensor) -> Tensor:
    """[B, H, T, D] layout (k, v, k_idx)."""
    assert t.dim() == 4 and t.stride(3) == 1 and t.dtype == torch.bfloat16 and t.is_cuda
    return Tensor(t.data_ptr(), t.stride(0), t.stride(2), t.stride(1))


def _check(fn, status):
    if status != 0:
        raise MSAError(fn, status)


def msa_num_blocks(d: Dims) -> int:
    return lib().msa_num_blocks(ctypes.byref(d))


def msa_num_entries(d: Dims) -> int:
    return lib().msa_num_entries(ctypes.byref(d))


def msa_query_window(d: Dims) -> int:
    return lib().msa_query_window(ctypes.byref(d))


def msa_num_segments(d: Dims) -> int:
    return lib().msa_num_segments(ctypes.byref(d))


def msa_debug_set_attn_wait_limit_ns(ns: int) -> int:
    """Time limit (ns) of the attention kernel's barrier waits for later calls;
    returns the previous one (0 restores the default 2 s)."""
    return int(lib().msa_debug_set_attn_wait_limit_ns(ns))


def msa_block_query_lists_workspace(d: Dims) -> int:
    return lib().msa_block_query_lists_workspace(ctypes.byref(d))


def msa_index_score_maxpool(d: Dims, q_idx, k_idx, pooled, pooled_row_stride, dev_err=None):
    _check("msa_index_score_maxpool",
           lib().msa_index_score_maxpool(ctypes.byref(d), tensor_btd(q_idx), tensor_bhtd(k_idx),
                                         _ptr(pooled), pooled_row_stride, _ptr(dev_err), _stream()))


def msa_topk_blocks(d: Dims, pooled, pooled_row_stride, sel, dev_err=None):
    _check("msa_topk_blocks",
           lib().msa_topk_blocks(ctypes.byref(d), _ptr(pooled), pooled_row_stride, _ptr(sel),
                                 _ptr(dev_err), _stream()))


def msa_build_block_query_lists(d: Dims, sel, blk_offsets, entries, entry_pos, ws, dev_err=None):
    """entry_pos (int32, the shape of sel) receives the position in entries of
    each (b, g, query, slot), -1 for an empty slot."""
    nbytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check("msa_build_block_query_lists",
           lib().msa_build_block_query_lists(ctypes.byref(d), _ptr(sel), _ptr(blk_offsets),
                                             _ptr(entries), _ptr(entry_pos), _ptr(ws), nbytes,
                                             _ptr(dev_err), _stream()))


def msa_build_block_query_lists_noalloc(d: Dims, sel, blk_offsets, entries, entry_pos,
                                        dev_err=None):
    """Same lists as msa_build_block_query_lists, with the library's built-in
    device scratch instead of a caller workspace (nothing is allocated)."""
    _check("msa_build_block_query_lists_noalloc",
           lib().msa_build_block_query_lists_noalloc(ctypes.byref(d), _ptr(sel), _ptr(blk_offsets),
                                                     _ptr(entries), _ptr(entry_pos),
                                                     _ptr(dev_err), _stream()))


def msa_sparse_attn_fwd(d: Dims, q, k, v, blk_offsets, entries, part_ml, part_acc, dev_err=None):
    _check("msa_sparse_attn_fwd",
           lib().msa_sparse_attn_fwd(ctypes.byref(d), tensor_btd(q), tensor_bhtd(k),
                                     tensor_bhtd(v), _ptr(blk_offsets), _ptr(entries),
                                     _ptr(part_ml), _ptr(part_acc), _ptr(dev_err), _stream()))


def msa_sparse_attn_fwd_compact(d: Dims, q, k, v, blk_offsets, entries, part_ml, part_acc16,
                                dev_err=None):
    """As msa_sparse_attn_fwd with compact pieces: part_acc16 bf16 [entries, R, 128]
    holds acc / l."""
    assert part_acc16.dtype == torch.bfloat16
    _check("msa_sparse_attn_fwd_compact",
           lib().msa_sparse_attn_fwd_compact(ctypes.byref(d), tensor_btd(q), tensor_bhtd(k),
                                             tensor_bhtd(v), _ptr(blk_offsets), _ptr(entries),
                                             _ptr(part_ml), _ptr(part_acc16), _ptr(dev_err),
                                             _stream()))


def msa_merge_partials_compact(d: Dims, entry_pos, part_ml, part_acc16, out, lse, dev_err=None):
    assert part_acc16.dtype == torch.bfloat16
    _check("msa_merge_partials_compact",
           lib().msa_merge_partials_compact(ctypes.byref(d), _ptr(entry_pos), _ptr(part_ml),
                                            _ptr(part_acc16), _ptr(out), _ptr(lse),
                                            _ptr(dev_err), _stream()))


def msa_sparse_attn_bwd(d: Dims, q, k, v, o, d_o, lse, blk_offsets, entries, delta, part_dq, dq,
                        dk, dv, dev_err=None):
    """dq [B,n_q,H,128], dk/dv [B,G,n_kv,128] (fp32) for upstream d_o (bf16)."""
    for t in (delta, part_dq, dq, dk, dv):
        assert t.dtype == torch.float32 and t.is_contiguous()
    _check("msa_sparse_attn_bwd",
           lib().msa_sparse_attn_bwd(ctypes.byref(d), tensor_btd(q), tensor_bhtd(k),
                                     tensor_bhtd(v), tensor_btd(o), tensor_btd(d_o), _ptr(lse),
                                     _ptr(blk_offsets), _ptr(entries), _ptr(delta),
                                     _ptr(part_dq), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dev_err),
                                     _stream()))


def msa_merge_partials(d: Dims, entry_pos, part_ml, part_acc, out, lse, dev_err=None):
    """Pieces in list order: slot s of (b, g, query) is at row entry_pos * R + r."""
    _check("msa_merge_partials",
           lib().msa_merge_partials(ctypes.byref(d), _ptr(entry_pos), _ptr(part_ml), _ptr(part_acc),
                                    _ptr(out), _ptr(lse), _ptr(dev_err), _stream()))


def msa_selection_recall_workspace(d: Dims, n_rows: int) -> int:
    return int(lib().msa_selection_recall_workspace(ctypes.byref(d), n_rows))


def msa_selection_recall(d: Dims, q, k, q_idx, k_idx, sel, rows, block_mass, recall, kl_pq, kl_qp,
                         ws, dev_err=None, lse_full=None):
    """Teacher block mass, recall and KL divergences for the sampled rows
    (rows: int64 device tensor of b * n_q + qi; block_mass [n * G, >= nblk]);
    lse_full [n, H] (optional) receives each head's full causal log-normaliser."""
    nbytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check("msa_selection_recall",
           lib().msa_selection_recall(ctypes.byref(d), tensor_btd(q), tensor_bhtd(k),
                                      tensor_btd(q_idx), tensor_bhtd(k_idx), _ptr(sel), _ptr(rows),
                                      rows.numel(), _ptr(block_mass), block_mass.stride(0),
                                      _ptr(recall), _ptr(kl_pq), _ptr(kl_qp), _ptr(lse_full),
                                      _ptr(ws), nbytes, _ptr(dev_err), _stream()))


def msa_token_select_workspace(d: Dims, n_rows: int) -> int:
    return int(lib().msa_token_select_workspace(ctypes.byref(d), n_rows))


def msa_token_select_attention(d: Dims, q, k, v, q_idx, k_idx, rows, budget, tokens, out, lse, ws,
                               dev_err=None):
    """Top-budget tokens by index score per (sampled row, group) and attention
    over them: tokens int32 [n, G, budget], out fp32 [n, H, 128], lse fp32 [n, H]."""
    nbytes = 0 if ws is None else ws.numel() * ws.element_size()
    assert tokens.dtype == torch.int32 and out.dtype == torch.float32 and lse.dtype == torch.float32
    _check("msa_token_select_attention",
           lib().msa_token_select_attention(ctypes.byref(d), tensor_btd(q), tensor_bhtd(k),
                                            tensor_bhtd(v), tensor_btd(q_idx), tensor_bhtd(k_idx),
                                            _ptr(rows), rows.numel(), budget, _ptr(tokens),
                                            _ptr(out), _ptr(lse), _ptr(ws), nbytes,
                                            _ptr(dev_err), _stream()))


def tensor_u8(t: torch.Tensor, bhtd: bool) -> Tensor:
    """uint8 [B, T, H, D] (q_idx codes) or [B, H, T, D] (k_idx codes), strides in bytes."""
    assert t.dim() == 4 and t.stride(3) == 1 and t.dtype == torch.uint8 and t.is_cuda
    if bhtd:
        return Tensor(t.data_ptr(), t.stride(0), t.stride(2), t.stride(1))
    return Tensor(t.data_ptr(), t.stride(0), t.stride(1), t.stride(2))


def msa_quantize_e4m3(x, codes, scale):
    """x bf16 contiguous -> codes uint8 (same numel); scale: 2 device floats."""
    assert x.is_contiguous() and codes.is_contiguous() and codes.numel() == x.numel()
    assert scale.dtype == torch.float32 and scale.numel() >= 2
    _check("msa_quantize_e4m3",
           lib().msa_quantize_e4m3(_ptr(x), x.numel(), _ptr(codes), _ptr(scale), _stream()))


def msa_index_score_maxpool_e4m3(d: Dims, q_idx8, k_idx8, scale_q, scale_k, pooled, stride,
                                 dev_err=None):
    _check("msa_index_score_maxpool_e4m3",
           lib().msa_index_score_maxpool_e4m3(ctypes.byref(d), tensor_u8(q_idx8, False),
                                              tensor_u8(k_idx8, True), _ptr(scale_q),
                                              _ptr(scale_k), _ptr(pooled), stride,
                                              _ptr(dev_err), _stream()))


# ---------------------------------------------------------------------------
# operators around the sparse path
# ---------------------------------------------------------------------------
def _need(cond, what):
    if not cond:
        raise ValueError(what)


def _on_current(*tensors):
    """The call is enqueued on the current device's current stream: every
    tensor has to live there."""
    dev = torch.cuda.current_device()
    for t in tensors:
        if t is not None:
            _need(t.is_cuda and t.get_device() == dev,
                  f"every tensor must be on the current device cuda:{dev}")


def _rows(name, t, shape, dtype=torch.bfloat16):
    """A [B, T, H, D] tensor as msa_tensor, after checking its shape and type."""
    _need(tuple(t.shape) == tuple(shape), f"{name}: shape {tuple(t.shape)}, expected {shape}")
    _need(t.dtype == dtype, f"{name}: {t.dtype}, expected {dtype}")
    _need(t.stride(3) == 1, f"{name}: the last dimension must be contiguous")
    return Tensor(t.data_ptr(), t.stride(0), t.stride(1), t.stride(2))


def _heads_first(name, t, shape, dtype=torch.bfloat16):
    """A [B, H, T, D] tensor as msa_tensor."""
    _need(tuple(t.shape) == tuple(shape), f"{name}: shape {tuple(t.shape)}, expected {shape}")
    return _rows(name, t.transpose(1, 2), (shape[0], shape[2], shape[1], shape[3]), dtype)


def _flat(name, t, shape, dtype):
    """A contiguous tensor of the given shape (None: passed as a null pointer)."""
    if t is None:
        return 0
    _need(tuple(t.shape) == tuple(shape), f"{name}: shape {tuple(t.shape)}, expected {shape}")
    _need(t.dtype == dtype and t.is_contiguous(), f"{name}: must be contiguous {dtype}")
    return t.data_ptr()


_NO_TENSOR = Tensor(0, 0, 0, 0)


def _norm_rope_dims(q, k, table, positions, pos0, eps, interleaved):
    some = q if q is not None else k
    _need(some is not None and some.dim() == 4, "q or k must be given, [B, T, H, D]")
    B, T, D = some.shape[0], some.shape[1], some.shape[3]
    rot = 0 if table is None else table.shape[1]
    return NormRopeDims(B, T, pos0, 0 if q is None else q.shape[2],
                        0 if k is None else k.shape[2], D, rot, 1 if interleaved else 0, eps)


def _norm_rope_common(d, q, k, w_q, w_k, table, positions):
    B, T, D = d.batch, d.n_tok, d.d
    n_pos = 0 if table is None else table.shape[0]
    if table is None and positions is None:
        n_pos = d.pos0 + T                 # no rotation: every position is in range
    elif table is None:
        n_pos = (1 << 63) - 1
    return (_NO_TENSOR if q is None else _rows("q", q, (B, T, d.h_q, D)),
            _NO_TENSOR if k is None else _rows("k", k, (B, T, d.h_k, D)),
            _flat("w_q", w_q, (D,), torch.float32), _flat("w_k", w_k, (D,), torch.float32),
            _flat("table", table, (n_pos, d.rot), torch.float32), n_pos,
            _flat("positions", positions, (B, T), torch.int64))


def _out_rows(name, t, like, shape):
    if like is None:
        return _NO_TENSOR
    _need(t is not None, f"{name} is missing")
    return _rows(name, t, shape)


def msa_qk_norm_rope(q, k, w_q, w_k, table, q_out, k_out, positions=None, pos0=0, eps=1e-6,
                     interleaved=False, dev_err=None):
    """q [B,T,Hq,D], k [B,T,Hk,D] (either may be None) -> q_out [B,T,Hq,D], k_out
    [B,Hk,T,D] (the attention's layout; any strides).  table fp32 [n_pos, rot]."""
    d = _norm_rope_dims(q, k, table, positions, pos0, eps, interleaved)
    _on_current(q, k, w_q, w_k, table, q_out, k_out, positions, dev_err)
    qt, kt, wq, wk, tab, n_pos, pos = _norm_rope_common(d, q, k, w_q, w_k, table, positions)
    qo = _out_rows("q_out", q_out, q, (d.batch, d.n_tok, d.h_q, d.d))
    _need(k is None or k_out is not None, "k_out is missing")
    ko = _NO_TENSOR if k is None else _heads_first("k_out", k_out,
                                                   (d.batch, d.h_k, d.n_tok, d.d))
    _check("msa_qk_norm_rope",
           lib().msa_qk_norm_rope(ctypes.byref(d), qt, kt, wq, wk, tab, n_pos, pos, qo, ko,
                                  _ptr(dev_err), _stream()))


def paged_kv(k_pages, v_pages, block_table, seq_lens=None) -> PagedKV:
    """Descriptor of a paged cache: k_pages, v_pages bf16 [n_pages, h_kv,
    page_size, 128] of equal strides (a permuted view when tokens are stored
    outermost), block_table int32 [B, pages per sequence], seq_lens int32 [B]."""
    _on_current(k_pages, v_pages, block_table, seq_lens)
    for name, t in (("k_pages", k_pages), ("v_pages", v_pages)):
        _need(t.dim() == 4 and t.shape[3] == HEAD_DIM and t.dtype == torch.bfloat16,
              f"{name}: must be bf16 [n_pages, h_kv, page_size, {HEAD_DIM}]")
        _need(t.stride(3) == 1, f"{name}: the last dimension must be contiguous")
    _need(k_pages.shape == v_pages.shape and k_pages.stride() == v_pages.stride(),
          "k_pages and v_pages must have the same shape and strides")
    _need(block_table.dim() == 2, "block_table: must be [B, pages per sequence]")
    B, per = block_table.shape
    _flat("block_table", block_table, (B, per), torch.int32)
    _flat("seq_lens", seq_lens, (B,), torch.int32)
    return PagedKV(k_pages.data_ptr(), v_pages.data_ptr(), k_pages.shape[0], k_pages.stride(0),
                   k_pages.stride(2), k_pages.stride(1), block_table.data_ptr(), per,
                   _ptr(seq_lens), k_pages.shape[2], k_pages.shape[1])


def msa_qk_norm_rope_paged(q, k, v, w_q, w_k, table, q_out, cache: PagedKV, cache_batch,
                           positions=None, pos0=0, eps=1e-6, interleaved=False, dev_err=None):
    """As msa_qk_norm_rope, keys and the values v [B,T,Hk,128] into the paged cache
    (cache_batch: the sequences its block table has)."""
    _need(k is not None and v is not None, "k and v must be given")
    d = _norm_rope_dims(q, k, table, positions, pos0, eps, interleaved)
    _on_current(q, k, v, w_q, w_k, table, q_out, positions, dev_err)
    _need(cache_batch == d.batch, "the block table must have a row for each sequence")
    qt, kt, wq, wk, tab, n_pos, pos = _norm_rope_common(d, q, k, w_q, w_k, table, positions)
    vt = _rows("v", v, (d.batch, d.n_tok, d.h_k, d.d))
    qo = _out_rows("q_out", q_out, q, (d.batch, d.n_tok, d.h_q, d.d))
    _check("msa_qk_norm_rope_paged",
           lib().msa_qk_norm_rope_paged(ctypes.byref(d), qt, kt, vt, wq, wk, tab, n_pos, pos, qo,
                                        ctypes.byref(cache), _ptr(dev_err), _stream()))


def msa_qk_norm_rope_bwd_workspace(d_head) -> int:
    d = NormRopeDims(1, 1, 0, 1, 1, d_head, 0, 0, 0.0)
    return int(lib().msa_qk_norm_rope_bwd_workspace(ctypes.byref(d)))


def msa_qk_norm_rope_bwd(q, k, w_q, w_k, table, d_q, d_k, dx_q, dx_k, dw_q, dw_k, ws,
                         positions=None, pos0=0, eps=1e-6, interleaved=False, dev_err=None):
    """d_q [B,T,Hq,D], d_k [B,Hk,T,D] (both bf16 or both fp32) -> dx_q [B,T,Hq,D], dx_k
    [B,T,Hk,D] bf16, dw_q, dw_k [D] fp32 (None: not wanted)."""
    d = _norm_rope_dims(q, k, table, positions, pos0, eps, interleaved)
    _on_current(q, k, w_q, w_k, table, d_q, d_k, dx_q, dx_k, dw_q, dw_k, ws, positions, dev_err)
    qt, kt, wq, wk, tab, n_pos, pos = _norm_rope_common(d, q, k, w_q, w_k, table, positions)
    _need((q is None or d_q is not None) and (k is None or d_k is not None),
          "an upstream gradient is missing")
    t = (d_q if q is not None else d_k).dtype
    _need(t in (torch.bfloat16, torch.float32), "gradients must be bf16 or fp32")
    dq = _NO_TENSOR if q is None else _rows("d_q", d_q, (d.batch, d.n_tok, d.h_q, d.d), t)
    dk = _NO_TENSOR if k is None else _heads_first("d_k", d_k,
                                                   (d.batch, d.h_k, d.n_tok, d.d), t)
    xq = _out_rows("dx_q", dx_q, q, (d.batch, d.n_tok, d.h_q, d.d))
    xk = _out_rows("dx_k", dx_k, k, (d.batch, d.n_tok, d.h_k, d.d))
    nbytes = ws.numel() * ws.element_size()
    _check("msa_qk_norm_rope_bwd",
           lib().msa_qk_norm_rope_bwd(ctypes.byref(d), qt, kt, wq, wk, tab, n_pos, pos, dq, dk,
                                      1 if t == torch.float32 else 0, xq, xk,
                                      _flat("dw_q", dw_q, (d.d,), torch.float32),
                                      _flat("dw_k", dw_k, (d.d,), torch.float32), _ptr(ws),
                                      nbytes, _ptr(dev_err), _stream()))


def msa_paged_decode_attn_workspace(d: Dims) -> int:
    return int(lib().msa_paged_decode_attn_workspace(ctypes.byref(d)))


def msa_paged_decode_attn(d: Dims, q, cache: PagedKV, cache_batch, out, lse, ws, window=0,
                          n_sink=0, dev_err=None):
    """One new token per sequence over the paged cache: q, out [B,1,H,128] bf16,
    lse [B,1,H] fp32."""
    _on_current(q, out, lse, ws, dev_err)
    _need(cache_batch == d.batch, "the block table must have a row for each sequence")
    shape = (d.batch, 1, d.h_q, HEAD_DIM)
    qt = _rows("q", q, shape)
    _check("msa_paged_decode_attn",
           lib().msa_paged_decode_attn(ctypes.byref(d), window, n_sink, qt, ctypes.byref(cache),
                                       _flat("out", out, shape, torch.bfloat16),
                                       _flat("lse", lse, shape[:3], torch.float32), _ptr(ws),
                                       ws.numel() * ws.element_size(), _ptr(dev_err), _stream()))


def msa_window_attn_fwd(d: Dims, window, n_sink, q, k, v, out, lse, kv_len=None, dev_err=None):
    """Sliding-window attention with sinks: q, out [B,n_q,H,128], k, v [B,G,n_kv,128]
    bf16, lse [B,n_q,H] fp32, kv_len int32 [B] (padded batch) or None."""
    _on_current(q, k, v, out, lse, kv_len, dev_err)
    qs, ks = (d.batch, d.n_q, d.h_q, HEAD_DIM), (d.batch, d.h_kv, d.n_kv, HEAD_DIM)
    _check("msa_window_attn_fwd",
           lib().msa_window_attn_fwd(ctypes.byref(d), window, n_sink, _rows("q", q, qs),
                                     _heads_first("k", k, ks), _heads_first("v", v, ks),
                                     _flat("kv_len", kv_len, (d.batch,), torch.int32),
                                     _flat("out", out, qs, torch.bfloat16),
                                     _flat("lse", lse, qs[:3], torch.float32), _ptr(dev_err),
                                     _stream()))


def msa_window_attn_bwd_workspace(d: Dims, window, n_sink) -> int:
    return int(lib().msa_window_attn_bwd_workspace(ctypes.byref(d), window, n_sink))


def msa_window_attn_bwd(d: Dims, window, n_sink, q, k, v, o, d_o, lse, dq, dk, dv, ws,
                        kv_len=None, dev_err=None):
    """dq [B,n_q,H,128], dk, dv [B,G,n_kv,128] (bf16) for the upstream d_o (bf16)."""
    _on_current(q, k, v, o, d_o, lse, dq, dk, dv, ws, kv_len, dev_err)
    qs, ks = (d.batch, d.n_q, d.h_q, HEAD_DIM), (d.batch, d.h_kv, d.n_kv, HEAD_DIM)
    _check("msa_window_attn_bwd",
           lib().msa_window_attn_bwd(ctypes.byref(d), window, n_sink, _rows("q", q, qs),
                                     _heads_first("k", k, ks), _heads_first("v", v, ks),
                                     _rows("o", o, qs), _rows("d_o", d_o, qs),
                                     _flat("lse", lse, qs[:3], torch.float32),
                                     _flat("kv_len", kv_len, (d.batch,), torch.int32),
                                     _flat("dq", dq, qs, torch.bfloat16),
                                     _flat("dk", dk, ks, torch.bfloat16),
                                     _flat("dv", dv, ks, torch.bfloat16), _ptr(ws),
                                     ws.numel() * ws.element_size(), _ptr(dev_err), _stream()))
