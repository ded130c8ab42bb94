"""The whole MSA hot path as five C-ABI calls on one stream.

``Buffers`` owns the intermediate device tensors (torch allocates them: the
library itself never allocates); ``forward`` enqueues

  msa_index_score_maxpool -> msa_topk_blocks -> msa_build_block_query_lists
  -> msa_sparse_attn_fwd -> msa_merge_partials

and returns the bf16 output and the fp32 log-sum-exp.  Beside it:
``select_e4m3`` (8-bit index branch), ``selection_recall`` (recall / KL
alignment target, optionally the full causal lse), ``token_select_attention``
(token-level selection at the same key budget), ``backward`` with ``Grads``
(dq, dk, dv for an upstream gradient) and ``HostPipeline`` (host buffers,
copies overlapped).  Around the path: ``NormRope`` with ``norm_rope`` /
``norm_rope_backward`` / ``norm_rope_append`` (per-head norms and rotation of
queries and keys, dense or into a ``PagedCache``), ``paged_decode`` (one new token
over the paged cache) and ``window_forward`` / ``window_backward`` (sliding-window
or full causal attention).  Every step runs in the library's kernels; this
module only marshals arguments.
"""
from __future__ import annotations

import dataclasses

import torch

from . import capi

# kernels each step launches (for launch accounting; with one query per row the
# block lists take 2 launches instead of 6)
LAUNCHES_PER_STEP = {"index": 1, "topk": 1, "block_lists": 6, "attn": 1, "merge": 1}


@dataclasses.dataclass
class Buffers:
    dims: capi.Dims
    pooled: torch.Tensor
    pooled_stride: int
    sel: torch.Tensor
    blk_offsets: torch.Tensor
    entries: torch.Tensor
    entry_pos: torch.Tensor
    ws: torch.Tensor
    part_ml: torch.Tensor
    part_acc: torch.Tensor
    out: torch.Tensor
    lse: torch.Tensor
    dev_err: torch.Tensor
    compact: bool = False

    @staticmethod
    def allocate(d: capi.Dims, device="cuda", compact: bool = False) -> "Buffers":
        """Intermediate buffers of one problem.  compact=True: the pieces' acc
        in bf16 (acc / l), read and written by the compact attention and merge
        calls."""
        B, n_q, G, H = d.batch, d.n_q, d.h_kv, d.h_q
        nblk = capi.msa_num_blocks(d)
        stride = (nblk + 3) // 4 * 4
        n_ent = capi.msa_num_entries(d)
        ws_bytes = capi.msa_block_query_lists_workspace(d)
        dev = torch.device(device)
        return Buffers(
            dims=d,
            pooled=torch.empty((B, G, n_q, stride), dtype=torch.float32, device=dev),
            pooled_stride=stride,
            sel=torch.empty((B, G, n_q, capi.TOPK), dtype=torch.int32, device=dev),
            blk_offsets=torch.empty((capi.msa_num_segments(d) + 1,), dtype=torch.int32,
                                    device=dev),
            entries=torch.empty((max(n_ent, 1),), dtype=torch.int32, device=dev),
            entry_pos=torch.empty((B, G, n_q, capi.TOPK), dtype=torch.int32, device=dev),
            ws=torch.empty(((ws_bytes + 15) // 16 * 4,), dtype=torch.int32, device=dev),
            # pieces in list order, [entries, R, ...]; sized for 16 slots per
            # (query, group), so the fp32 buffer also serves as the backward's
            # dq scratch [B, n_q, G, 16, R, 128]
            part_ml=torch.empty((B * n_q * G * capi.TOPK, H // G, 2), dtype=torch.float32,
                                device=dev),
            part_acc=torch.empty((B * n_q * G * capi.TOPK, H // G, capi.HEAD_DIM),
                                 dtype=torch.bfloat16 if compact else torch.float32, device=dev),
            out=torch.empty((B, n_q, H, capi.HEAD_DIM), dtype=torch.bfloat16, device=dev),
            lse=torch.empty((B, n_q, H), dtype=torch.float32, device=dev),
            dev_err=torch.zeros((4,), dtype=torch.int32, device=dev),
            compact=compact,
        )


def dims_for(w) -> capi.Dims:
    """Dims of a workloads.Workload."""
    return capi.make_dims(w.batch, w.n_q, w.n_kv, w.q_pos0, w.h_q, w.h_kv, w.d_idx,
                          h_kidx=w.h_kidx, scale=w.scale, q_window=w.q_window)


def select(buf: Buffers, q_idx, k_idx):
    """Index scores + max-pool + top-16 selection -> buf.sel."""
    d = buf.dims
    capi.msa_index_score_maxpool(d, q_idx, k_idx, buf.pooled, buf.pooled_stride, buf.dev_err)
    capi.msa_topk_blocks(d, buf.pooled, buf.pooled_stride, buf.sel, buf.dev_err)


def select_e4m3(buf: Buffers, q_idx, k_idx):
    """Selection from 8-bit index scores: per-tensor e4m3 copies of q_idx and
    k_idx, the tcgen05 kind::f8f6f4 score + max-pool kernel, then top-16 ->
    buf.sel.  Returns the codes and the two scales (device)."""
    d = buf.dims
    q8 = torch.empty(q_idx.shape, dtype=torch.uint8, device=q_idx.device)
    k8 = torch.empty(k_idx.shape, dtype=torch.uint8, device=k_idx.device)
    sq = torch.empty((2,), dtype=torch.float32, device=q_idx.device)
    sk = torch.empty((2,), dtype=torch.float32, device=q_idx.device)
    capi.msa_quantize_e4m3(q_idx, q8, sq)
    capi.msa_quantize_e4m3(k_idx, k8, sk)
    capi.msa_index_score_maxpool_e4m3(d, q8, k8, sq, sk, buf.pooled, buf.pooled_stride,
                                      buf.dev_err)
    capi.msa_topk_blocks(d, buf.pooled, buf.pooled_stride, buf.sel, buf.dev_err)
    return q8, k8, sq, sk


def attend(buf: Buffers, q, k, v, sel=None):
    """Block lists + KV-block-outer attention + merge over `sel` (default buf.sel)."""
    d = buf.dims
    s = buf.sel if sel is None else sel
    capi.msa_build_block_query_lists(d, s, buf.blk_offsets, buf.entries, buf.entry_pos, buf.ws,
                                     buf.dev_err)
    if buf.compact:
        capi.msa_sparse_attn_fwd_compact(d, q, k, v, buf.blk_offsets, buf.entries, buf.part_ml,
                                         buf.part_acc, buf.dev_err)
        capi.msa_merge_partials_compact(d, buf.entry_pos, buf.part_ml, buf.part_acc, buf.out,
                                        buf.lse, buf.dev_err)
    else:
        capi.msa_sparse_attn_fwd(d, q, k, v, buf.blk_offsets, buf.entries, buf.part_ml,
                                 buf.part_acc, buf.dev_err)
        capi.msa_merge_partials(d, buf.entry_pos, buf.part_ml, buf.part_acc, buf.out, buf.lse,
                                buf.dev_err)


def forward(buf: Buffers, q, k, v, q_idx, k_idx):
    """The whole hot path; returns (out bf16 [B,n_q,H,128], lse fp32 [B,n_q,H])."""
    select(buf, q_idx, k_idx)
    attend(buf, q, k, v)
    return buf.out, buf.lse


@dataclasses.dataclass
class Grads:
    delta: torch.Tensor
    dq: torch.Tensor
    dk: torch.Tensor
    dv: torch.Tensor

    @staticmethod
    def allocate(d: capi.Dims, device="cuda") -> "Grads":
        B, n_q, n_kv, G, H = d.batch, d.n_q, d.n_kv, d.h_kv, d.h_q
        dev = torch.device(device)
        return Grads(
            delta=torch.empty((B, n_q, H), dtype=torch.float32, device=dev),
            dq=torch.empty((B, n_q, H, capi.HEAD_DIM), dtype=torch.float32, device=dev),
            dk=torch.empty((B, G, n_kv, capi.HEAD_DIM), dtype=torch.float32, device=dev),
            dv=torch.empty((B, G, n_kv, capi.HEAD_DIM), dtype=torch.float32, device=dev),
        )


def backward(buf: Buffers, grads: Grads, q, k, v, d_out):
    """Gradients of the attention for upstream d_out (bf16 [B,n_q,H,128]) after a
    forward on the same buffers (its out, lse and block lists; the selection is
    fixed).  The forward's piece buffer holds the dQ pieces, so it must be the
    fp32 one (Buffers allocated with compact=False).  Returns (dq, dk, dv)."""
    if buf.compact:
        raise ValueError("the backward keeps fp32 dq pieces in the piece buffer: "
                         "allocate the Buffers with compact=False")
    capi.msa_sparse_attn_bwd(buf.dims, q, k, v, buf.out, d_out, buf.lse, buf.blk_offsets,
                             buf.entries, grads.delta, buf.part_acc, grads.dq, grads.dk,
                             grads.dv, buf.dev_err)
    return grads.dq, grads.dk, grads.dv


def selection_recall(buf: Buffers, q, k, q_idx, k_idx, rows, lse_full=None):
    """For sampled rows (int64 device tensor of b * n_q + qi): the main branch's
    block mass [n, G, nblk], the recall of buf.sel and KL(P||Q), KL(Q||P) [n, G].
    A given lse_full [n, H] fp32 receives each head's full causal log-normaliser."""
    d = buf.dims
    n, G = rows.numel(), d.h_kv
    nblk = capi.msa_num_blocks(d)
    dev = rows.device
    mass = torch.empty((n, G, nblk), dtype=torch.float32, device=dev)
    rec = torch.empty((n, G), dtype=torch.float32, device=dev)
    kpq = torch.empty((n, G), dtype=torch.float32, device=dev)
    kqp = torch.empty((n, G), dtype=torch.float32, device=dev)
    ws_bytes = capi.msa_selection_recall_workspace(d, n)
    ws = torch.empty(((ws_bytes + 15) // 16 * 4,), dtype=torch.int32, device=dev)
    capi.msa_selection_recall(d, q, k, q_idx, k_idx, buf.sel, rows, mass.view(n * G, nblk), rec,
                              kpq, kqp, ws, buf.dev_err, lse_full=lse_full)
    return mass, rec, kpq, kqp


def token_select_attention(d, q, k, v, q_idx, k_idx, rows, budget=2048, dev_err=None):
    """Token-level selection at the same key budget for sampled rows: tokens
    int32 [n, G, budget] (ascending, -1 padded), out fp32 [n, H, 128] and lse
    fp32 [n, H] of the attention over them."""
    n, G, H = rows.numel(), d.h_kv, d.h_q
    dev = rows.device
    tokens = torch.empty((n, G, budget), dtype=torch.int32, device=dev)
    out = torch.empty((n, H, 128), dtype=torch.float32, device=dev)
    lse = torch.empty((n, H), dtype=torch.float32, device=dev)
    ws_bytes = capi.msa_token_select_workspace(d, n)
    ws = torch.empty(((ws_bytes + 15) // 16 * 4,), dtype=torch.int32, device=dev)
    capi.msa_token_select_attention(d, q, k, v, q_idx, k_idx, rows, budget, tokens, out, lse, ws,
                                    dev_err)
    return tokens, out, lse


INPUT_NAMES = ("q", "k", "v", "q_idx", "k_idx")


class HostPipeline:
    """The hot path on batches held in pinned host memory, copies overlapped.

    ``run(host_in, host_out)`` takes a list of host input dicts (pinned q, k,
    v, q_idx, k_idx of the problem ``buf`` was allocated for) and a matching
    list of pinned host (out, lse) pairs.  For every batch it enqueues the
    host-to-device copy of the inputs (upload stream), the five library calls
    (the caller's current stream) and the device-to-host copy of out and lse
    (download stream).  Two device sets of inputs and outputs alternate, so
    batch i+1's upload and batch i-1's download run while batch i's kernels
    do; events order the three streams.  On return the caller's stream has
    waited for every download.
    """

    def __init__(self, buf: Buffers, like: dict):
        self.buf = buf
        self.dev_in = [{k: torch.empty_like(like[k]) for k in INPUT_NAMES} for _ in range(2)]
        self.dev_out = [(buf.out, buf.lse), (torch.empty_like(buf.out), torch.empty_like(buf.lse))]
        self.s_up = torch.cuda.Stream()
        self.s_down = torch.cuda.Stream()

    def run(self, host_in, host_out):
        comp = torch.cuda.current_stream()
        n = len(host_in)
        comp_done, down_done = [None] * n, [None] * n
        try:
            for i in range(n):
                slot = i % 2
                dev = self.dev_in[slot]
                out, lse = self.dev_out[slot]
                up = torch.cuda.Event()
                with torch.cuda.stream(self.s_up):
                    if i >= 2:                      # the kernels of batch i-2 read this set
                        self.s_up.wait_event(comp_done[i - 2])
                    for k in INPUT_NAMES:
                        dev[k].copy_(host_in[i][k], non_blocking=True)
                    up.record(self.s_up)
                comp.wait_event(up)
                if i >= 2:                          # batch i-2's output has left this set
                    comp.wait_event(down_done[i - 2])
                self.buf.out, self.buf.lse = out, lse
                forward(self.buf, dev["q"], dev["k"], dev["v"], dev["q_idx"], dev["k_idx"])
                comp_done[i] = torch.cuda.Event()
                comp_done[i].record(comp)
                down_done[i] = torch.cuda.Event()
                with torch.cuda.stream(self.s_down):
                    self.s_down.wait_event(comp_done[i])
                    host_out[i][0].copy_(out, non_blocking=True)
                    host_out[i][1].copy_(lse, non_blocking=True)
                    down_done[i].record(self.s_down)
            if n:
                comp.wait_event(down_done[n - 1])
        finally:
            self.buf.out, self.buf.lse = self.dev_out[0]


def check_device_errors(buf):
    """Raise if any kernel reported a device-side error (synchronises).  buf: Buffers, or
    whatever else holds a dev_err (a paged cache, the buffers of decode and window)."""
    code = int(buf.dev_err[0].item())
    if code:
        raise capi.MSAError("device", 0) from RuntimeError(capi.DEVERR.get(code, code))


# ---------------------------------------------------------------------------
# around the sparse path: norms + rotation, the paged cache, window attention
# ---------------------------------------------------------------------------
def rope_table(n_pos, rot, theta=1.0e6, device="cuda"):
    """The rotation table [n_pos, rot] fp32 of angles p * theta^(-2 i / rot): rot / 2
    cosines, then rot / 2 sines; the angles in 64 bits, so far positions keep
    their precision.  Any other table of this layout (scaled angles) serves too."""
    inv = float(theta) ** (-torch.arange(0, rot, 2, device=device, dtype=torch.float64) / rot)
    ang = torch.arange(n_pos, device=device, dtype=torch.float64)[:, None] * inv
    return torch.cat([ang.cos(), ang.sin()], dim=1).to(torch.float32)


@dataclasses.dataclass
class NormRope:
    """What a layer keeps for its per-head norms and rotation: the table (None: no
    rotation), the norm weights fp32 [d] (None: ones), eps and the pairing.  dev_err takes
    the errors of calls that are given none (positions past the table, which leave their
    rows as they were): ``check_device_errors(plan)``."""
    table: torch.Tensor | None
    w_q: torch.Tensor | None = None
    w_k: torch.Tensor | None = None
    eps: float = 1e-6
    interleaved: bool = False
    dev_err: torch.Tensor | None = None

    def __post_init__(self):
        if self.dev_err is None and self.table is not None:
            self.dev_err = torch.zeros((4,), dtype=torch.int32, device=self.table.device)


def norm_rope(plan: NormRope, q, k, q_out=None, k_out=None, positions=None, pos0=0,
              dev_err=None):
    """Normed and rotated queries [B,T,Hq,D] and keys; q [B,T,Hq,D], k [B,T,Hk,D] bf16
    (either may be None), D 64 or 128.  Returns (q_out, k_out [B,Hk,T,D], the
    attention's layout), allocated when not given."""
    if q is not None and q_out is None:
        q_out = torch.empty_like(q, memory_format=torch.contiguous_format)
    if k is not None and k_out is None:
        k_out = torch.empty((k.shape[0], k.shape[2], k.shape[1], k.shape[3]), dtype=k.dtype,
                            device=k.device)
    capi.msa_qk_norm_rope(q, k, plan.w_q, plan.w_k, plan.table, q_out, k_out, positions, pos0,
                          plan.eps, plan.interleaved,
                          plan.dev_err if dev_err is None else dev_err)
    return q_out, k_out


@dataclasses.dataclass
class NormRopeGrads:
    dx_q: torch.Tensor | None
    dx_k: torch.Tensor | None
    dw_q: torch.Tensor | None
    dw_k: torch.Tensor | None
    ws: torch.Tensor

    @staticmethod
    def allocate(q, k) -> "NormRopeGrads":
        some = q if q is not None else k
        d, dev = some.shape[3], some.device
        n = capi.msa_qk_norm_rope_bwd_workspace(d)

        def like(t):
            return None if t is None else torch.empty(t.shape, dtype=torch.bfloat16, device=dev)

        def row(t):
            return None if t is None else torch.empty((d,), dtype=torch.float32, device=dev)

        return NormRopeGrads(like(q), like(k), row(q), row(k),
                             torch.empty((n // 4,), dtype=torch.float32, device=dev))


def norm_rope_backward(plan: NormRope, q, k, d_q, d_k, grads: NormRopeGrads, positions=None,
                       pos0=0, dev_err=None):
    """Gradients of norm_rope for d_q [B,T,Hq,D] and d_k [B,Hk,T,D] (bf16, or fp32 as
    ``backward`` gives them).  Returns (dx_q, dx_k, dw_q, dw_k)."""
    capi.msa_qk_norm_rope_bwd(q, k, plan.w_q, plan.w_k, plan.table, d_q, d_k, grads.dx_q,
                              grads.dx_k, grads.dw_q, grads.dw_k, grads.ws, positions, pos0,
                              plan.eps, plan.interleaved,
                              plan.dev_err if dev_err is None else dev_err)
    return grads.dx_q, grads.dx_k, grads.dw_q, grads.dw_k


@dataclasses.dataclass
class PagedCache:
    """A paged key-value cache: pages seen as [n_pages, h_kv, page_size, 128] (heads
    or tokens stored outermost), the block table [B, pages per sequence] int32 and
    the sequences' lengths [B] int32.  Who calls keeps the table and the lengths.
    dev_err takes the errors of appends (``check_device_errors(cache)``)."""
    k_pages: torch.Tensor
    v_pages: torch.Tensor
    block_table: torch.Tensor
    seq_lens: torch.Tensor
    dev_err: torch.Tensor | None = None

    def __post_init__(self):
        if self.dev_err is None:
            self.dev_err = torch.zeros((4,), dtype=torch.int32, device=self.k_pages.device)

    @staticmethod
    def allocate(batch, max_tokens, h_kv, page_size=64, n_pages=None, tokens_outermost=False,
                 device="cuda") -> "PagedCache":
        """An empty cache.  Without n_pages every sequence owns pages for
        max_tokens, else the table starts out at -1."""
        dev = torch.device(device)
        per = (max_tokens + page_size - 1) // page_size
        own = n_pages is None
        n = batch * per if own else n_pages

        def pages():
            if tokens_outermost:
                t = torch.zeros((n, page_size, h_kv, capi.HEAD_DIM), dtype=torch.bfloat16,
                                device=dev)
                return t.permute(0, 2, 1, 3)
            return torch.zeros((n, h_kv, page_size, capi.HEAD_DIM), dtype=torch.bfloat16,
                               device=dev)

        table = (torch.arange(n, dtype=torch.int32, device=dev).view(batch, per) if own else
                 torch.full((batch, per), -1, dtype=torch.int32, device=dev))
        return PagedCache(pages(), pages(), table,
                          torch.zeros((batch,), dtype=torch.int32, device=dev))

    @property
    def batch(self):
        return self.block_table.shape[0]

    @property
    def h_kv(self):
        return self.k_pages.shape[1]

    @property
    def capacity(self):
        """Tokens a sequence's table row can hold."""
        return self.block_table.shape[1] * self.k_pages.shape[2]


def norm_rope_append(plan: NormRope, q, k, v, positions, q_out, cache: PagedCache, pos0=0,
                     dev_err=None):
    """norm_rope whose keys, and the values v [B,T,Hk,128], go into the cache's pages
    at positions [B, T] int64 (negative: padding; None: pos0 + i).  The table must
    already map them: a token without a page leaves the cache as it was and an error in
    dev_err (the cache's, when not given).  seq_lens is the caller's to advance.  Returns
    q_out."""
    if q is not None and q_out is None:
        q_out = torch.empty_like(q, memory_format=torch.contiguous_format)
    capi.msa_qk_norm_rope_paged(q, k, v, plan.w_q, plan.w_k, plan.table, q_out, cache.k_pages,
                                cache.v_pages, cache.block_table, positions, pos0, plan.eps,
                                plan.interleaved, cache.dev_err if dev_err is None else dev_err)
    return q_out


@dataclasses.dataclass
class DecodeBuffers:
    dims: capi.Dims
    out: torch.Tensor
    lse: torch.Tensor
    ws: torch.Tensor
    dev_err: torch.Tensor

    @staticmethod
    def allocate(cache: PagedCache, h_q, scale=None) -> "DecodeBuffers":
        dev, B = cache.k_pages.device, cache.batch
        cap = max(cache.capacity, 1)
        d = capi.make_dims(B, 1, cap, cap - 1, h_q, cache.h_kv, capi.HEAD_DIM, scale=scale)
        n = capi.msa_paged_decode_attn_workspace(d)
        return DecodeBuffers(
            dims=d,
            out=torch.empty((B, 1, h_q, capi.HEAD_DIM), dtype=torch.bfloat16, device=dev),
            lse=torch.empty((B, 1, h_q), dtype=torch.float32, device=dev),
            ws=torch.empty(((n + 15) // 16 * 4,), dtype=torch.int32, device=dev),
            dev_err=torch.zeros((4,), dtype=torch.int32, device=dev))


def paged_decode(buf: DecodeBuffers, q, cache: PagedCache, window=0, n_sink=0):
    """Attention of each sequence's newest token (token seq_lens[b] - 1, already in
    the cache) over its pages: all of them, or a window and sinks.  q [B,1,H,128].
    Returns (out bf16 [B,1,H,128], lse fp32 [B,1,H]); an empty sequence gives 0, -inf."""
    capi.msa_paged_decode_attn(buf.dims, q, cache.k_pages, cache.v_pages, cache.block_table,
                               cache.seq_lens, buf.out, buf.lse, buf.ws, window, n_sink,
                               buf.dev_err)
    return buf.out, buf.lse


def window_dims(batch, n_q, n_kv, q_pos0, h_q, h_kv, scale=None) -> capi.Dims:
    """Dims of a window-attention problem (there is no index branch)."""
    return capi.make_dims(batch, n_q, n_kv, q_pos0, h_q, h_kv, capi.HEAD_DIM, scale=scale)


@dataclasses.dataclass
class WindowBuffers:
    dims: capi.Dims
    window: int
    n_sink: int
    out: torch.Tensor
    lse: torch.Tensor
    dev_err: torch.Tensor
    dq: torch.Tensor | None = None
    dk: torch.Tensor | None = None
    dv: torch.Tensor | None = None
    ws: torch.Tensor | None = None
    rest: torch.Tensor | None = None     # the 8 bits behind out, for the backward

    @staticmethod
    def allocate(d: capi.Dims, window=0, n_sink=0, backward=False,
                 device="cuda") -> "WindowBuffers":
        """Outputs (and, with backward=True, gradients and workspace) of one
        problem; window 0 is full causal attention."""
        dev = torch.device(device)
        qs = (d.batch, d.n_q, d.h_q, capi.HEAD_DIM)
        ks = (d.batch, d.h_kv, d.n_kv, capi.HEAD_DIM)
        buf = WindowBuffers(d, window, n_sink,
                            torch.empty(qs, dtype=torch.bfloat16, device=dev),
                            torch.empty(qs[:3], dtype=torch.float32, device=dev),
                            torch.zeros((4,), dtype=torch.int32, device=dev))
        if backward:
            n = capi.msa_window_attn_bwd_workspace(d, window, n_sink)
            buf.dq = torch.empty(qs, dtype=torch.bfloat16, device=dev)
            buf.dk = torch.empty(ks, dtype=torch.bfloat16, device=dev)
            buf.dv = torch.empty(ks, dtype=torch.bfloat16, device=dev)
            buf.ws = torch.empty(((n + 31) // 32 * 8,), dtype=torch.int32, device=dev)
            buf.rest = torch.empty(qs, dtype=torch.int8, device=dev)
        return buf


def window_forward(buf: WindowBuffers, q, k, v, kv_len=None):
    """Sliding-window attention with sinks over q [B,n_q,H,128], k, v [B,G,n_kv,128];
    kv_len int32 [B]: queries at positions >= kv_len[b] are padding (0, -inf).
    Returns (out, lse)."""
    capi.msa_window_attn_fwd(buf.dims, buf.window, buf.n_sink, q, k, v, buf.out, buf.lse, kv_len,
                             buf.rest, buf.dev_err)
    return buf.out, buf.lse


def window_backward(buf: WindowBuffers, q, k, v, d_out, kv_len=None):
    """Gradients for upstream d_out (bf16) after window_forward on the same buffers.
    Returns (dq, dk, dv) in bf16."""
    if buf.ws is None:
        raise ValueError("allocate the WindowBuffers with backward=True")
    capi.msa_window_attn_bwd(buf.dims, buf.window, buf.n_sink, q, k, v, buf.out, d_out, buf.lse,
                             buf.dq, buf.dk, buf.dv, buf.ws, kv_len, buf.rest, buf.dev_err)
    return buf.dq, buf.dk, buf.dv
