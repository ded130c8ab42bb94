"""Thin ctypes binding of ``libmsa.so`` -- argument marshalling only.

Each function has the name of the C entry point it calls (``include/msa.h``)
and takes torch CUDA tensors; it passes raw device pointers, element strides
and the current CUDA stream, raises ``MSAError`` on a non-OK status, and does
no arithmetic of its own.  If the library is missing this module raises on
first use: there is no fallback path.
"""
from __future__ import annotations

import ctypes
import importlib.util
import os
import threading

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "lib", "libmsa.so")
CALLS_PATH = os.path.join(_HERE, "lib", "msa_calls.so")

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
                                      _P, _P]
    L.msa_window_attn_bwd_workspace.argtypes = [_PD, _I64, _I64]
    L.msa_window_attn_bwd_workspace.restype = ctypes.c_size_t
    L.msa_window_attn_bwd.argtypes = [_PD, _I64, _I64, Tensor, Tensor, Tensor, Tensor, _P, Tensor,
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
# operators around the sparse path: checks and marshalling in lib/msa_calls.so
# (csrc/calls.cpp).  Tensors that do not fit together raise ValueError, a refusal
# of the C entry point MSAError; every tensor has to be on the current device,
# whose current stream the call is enqueued on.
# ---------------------------------------------------------------------------
_calls = None


def _load_calls():
    if not os.path.exists(CALLS_PATH):
        raise RuntimeError(
            f"{CALLS_PATH} is missing: build it with "
            "`python -m block_sparse_attention_32_b200.build` (no fallback exists)")
    spec = importlib.util.spec_from_file_location("msa_calls", CALLS_PATH)
    rebuild = "build it again with `python -m block_sparse_attention_32_b200.build`"
    try:
        mod = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(mod)
    except ImportError as e:               # libmsa.so missing, or the symbols of another torch
        raise RuntimeError(f"{CALLS_PATH} does not load ({e}): {rebuild}") from e
    built_for = getattr(mod, "torch_version", "of another build")
    if built_for != str(torch.__version__):
        raise RuntimeError(f"{CALLS_PATH} was built for torch {built_for}, this is "
                           f"{torch.__version__}: {rebuild}")
    return mod


def calls():
    """The msa_calls module (raises if it has not been built)."""
    global _calls
    if _calls is None:
        with _lock:
            if _calls is None:
                _calls = _load_calls()
    return _calls


def msa_qk_norm_rope(q, k, w_q, w_k, table, q_out, k_out, positions=None, pos0=0, eps=1e-6,
                     interleaved=False, dev_err=None):
    """q [B,T,Hq,D], k [B,T,Hk,D] (either may be None) -> q_out [B,T,Hq,D], k_out
    [B,Hk,T,D] (the attention's layout; any strides).  table fp32 [n_pos, rot]."""
    st = calls().norm_rope(q, k, w_q, w_k, table, q_out, k_out, positions, pos0, eps, interleaved,
                           dev_err)
    if st:
        raise MSAError("msa_qk_norm_rope", st)


def msa_qk_norm_rope_paged(q, k, v, w_q, w_k, table, q_out, k_pages, v_pages, block_table,
                           positions=None, pos0=0, eps=1e-6, interleaved=False, dev_err=None):
    """As msa_qk_norm_rope, keys and the values v [B,T,Hk,128] into the pages
    [n_pages, h_kv, page_size, 128] (K and V of equal strides; a permuted view when
    tokens are stored outermost) that block_table int32 [B, pages per sequence] names."""
    st = calls().norm_rope_paged(q, k, v, w_q, w_k, table, q_out, k_pages, v_pages, block_table,
                                 positions, pos0, eps, interleaved, dev_err)
    if st:
        raise MSAError("msa_qk_norm_rope_paged", st)


def msa_qk_norm_rope_bwd_workspace(d_head) -> int:
    d = NormRopeDims(1, 1, 0, 1, 1, d_head, 0, 0, 0.0)
    return int(lib().msa_qk_norm_rope_bwd_workspace(ctypes.byref(d)))


def msa_qk_norm_rope_bwd(q, k, w_q, w_k, table, d_q, d_k, dx_q, dx_k, dw_q, dw_k, ws,
                         positions=None, pos0=0, eps=1e-6, interleaved=False, dev_err=None):
    """d_q [B,T,Hq,D], d_k [B,Hk,T,D] (both bf16 or both fp32) -> dx_q [B,T,Hq,D], dx_k
    [B,T,Hk,D] bf16, dw_q, dw_k [D] fp32 (None: not wanted)."""
    st = calls().norm_rope_bwd(q, k, w_q, w_k, table, d_q, d_k, dx_q, dx_k, dw_q, dw_k, ws,
                               positions, pos0, eps, interleaved, dev_err)
    if st:
        raise MSAError("msa_qk_norm_rope_bwd", st)


def msa_paged_decode_attn_workspace(d: Dims) -> int:
    return int(lib().msa_paged_decode_attn_workspace(ctypes.byref(d)))


def msa_paged_decode_attn(d: Dims, q, k_pages, v_pages, block_table, seq_lens, out, lse, ws,
                          window=0, n_sink=0, dev_err=None):
    """One new token per sequence over the paged cache: q, out [B,1,H,128] bf16,
    lse [B,1,H] fp32, seq_lens int32 [B]."""
    st = calls().paged_decode(d, window, n_sink, q, k_pages, v_pages, block_table, seq_lens, out,
                              lse, ws, dev_err)
    if st:
        raise MSAError("msa_paged_decode_attn", st)


def msa_window_attn_fwd(d: Dims, window, n_sink, q, k, v, out, lse, kv_len=None, out_rest=None,
                        dev_err=None):
    """Sliding-window attention with sinks: q, out [B,n_q,H,128], k, v [B,G,n_kv,128]
    bf16, lse [B,n_q,H] fp32, kv_len int32 [B] (padded batch) or None, out_rest int8 like
    out (the bits behind it, for the backward) or None."""
    st = calls().window_fwd(d, window, n_sink, q, k, v, out, out_rest, lse, kv_len, dev_err)
    if st:
        raise MSAError("msa_window_attn_fwd", st)


def msa_window_attn_bwd_workspace(d: Dims, window, n_sink) -> int:
    return int(lib().msa_window_attn_bwd_workspace(ctypes.byref(d), window, n_sink))


def msa_window_attn_bwd(d: Dims, window, n_sink, q, k, v, o, d_o, lse, dq, dk, dv, ws,
                        kv_len=None, o_rest=None, dev_err=None):
    """dq [B,n_q,H,128], dk, dv [B,G,n_kv,128] (bf16) for the upstream d_o (bf16); o,
    o_rest (or None) and lse as the forward left them."""
    st = calls().window_bwd(d, window, n_sink, q, k, v, o, o_rest, d_o, lse, dq, dk, dv, ws, kv_len,
                            dev_err)
    if st:
        raise MSAError("msa_window_attn_bwd", st)
