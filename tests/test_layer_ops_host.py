"""Refusals of the operators around the sparse path, without a GPU: statuses of the
C ABI for bad arguments (nothing is enqueued), and ValueErrors of the Python calls
for tensors that do not fit together."""
import ctypes

import pytest
import torch

from block_sparse_attention_32_b200 import build as msa_build
from block_sparse_attention_32_b200 import capi, pipeline

P = ctypes.c_void_p
INVALID, UNSUPPORTED, ALIGNMENT, WORKSPACE = 1, 2, 3, 4
GOOD = capi.Tensor(0x100000, 0, 256, 128)


@pytest.fixture(scope="module")
def lib():
    msa_build.build()
    return capi.lib()


def _norm(lib, n_pos=100, positions=None, w=0x1000, table=0x2000, q=GOOD, k=GOOD, qo=GOOD,
          ko=GOOD, **dims):
    d = dict(batch=1, n_tok=10, pos0=0, h_q=2, h_k=1, d=128, rot=64, interleaved=0, eps=1e-6)
    d.update(dims)
    d = capi.NormRopeDims(*[d[n] for n, _ in capi.NormRopeDims._fields_])
    return lib.msa_qk_norm_rope(ctypes.byref(d), q, k, P(w), P(w), P(table), n_pos, P(positions),
                                qo, ko, None, None)


@pytest.mark.parametrize("want,kw", [
    (INVALID, dict(batch=0)), (INVALID, dict(n_tok=0)), (INVALID, dict(pos0=-1)),
    (INVALID, dict(h_q=-1)), (INVALID, dict(h_q=0, h_k=0)), (INVALID, dict(eps=-1.0)),
    (INVALID, dict(eps=float("nan"))), (INVALID, dict(interleaved=2)),
    (UNSUPPORTED, dict(d=96)), (UNSUPPORTED, dict(rot=72)), (UNSUPPORTED, dict(rot=144)),
    (UNSUPPORTED, dict(d=64, rot=128)), (UNSUPPORTED, dict(rot=-16)),
    (UNSUPPORTED, dict(batch=1 << 20, n_tok=1 << 20)),
    (INVALID, dict(table=0)), (INVALID, dict(n_pos=9)), (INVALID, dict(pos0=91)),
    (INVALID, dict(pos0=(1 << 63) - 1)), (INVALID, dict(n_pos=-1, positions=0x3000)),
    (ALIGNMENT, dict(table=0x2008)), (ALIGNMENT, dict(w=0x1004)), (ALIGNMENT, dict(positions=0x3004)),
    (INVALID, dict(q=capi.Tensor(0, 0, 256, 128))), (ALIGNMENT, dict(k=capi.Tensor(0x8, 0, 256, 128))),
    (ALIGNMENT, dict(qo=capi.Tensor(0x100000, 0, 260, 128))),
    (INVALID, dict(ko=capi.Tensor(0x100000, 0, -256, 128))),
], ids=str)
def test_norm_rope_statuses(lib, want, kw):
    assert _norm(lib, **kw) == want


def _cache(**kw):
    c = dict(k=0x10000, v=0x20000, n_pages=8, s_page=64 * 256, s_tok=128, s_head=64 * 128,
             block_table=0x3000, table_stride=4, seq_lens=0x4000, page_size=64, h_kv=2)
    c.update(kw)
    return capi.PagedKV(*[c[n] for n, _ in capi.PagedKV._fields_])


BAD_CACHES = [
    (INVALID, dict(k=0)), (INVALID, dict(v=None)), (INVALID, dict(block_table=0)),
    (INVALID, dict(n_pages=0)), (INVALID, dict(table_stride=0)), (INVALID, dict(h_kv=0)),
    (INVALID, dict(s_page=-128)), (INVALID, dict(s_tok=0)), (INVALID, dict(s_head=0)),
    (INVALID, dict(s_page=0)), (UNSUPPORTED, dict(page_size=8)), (UNSUPPORTED, dict(page_size=48)),
    (ALIGNMENT, dict(k=0x10008)), (ALIGNMENT, dict(s_head=132)), (ALIGNMENT, dict(block_table=0x3002)),
]


@pytest.mark.parametrize("want,kw", BAD_CACHES + [(INVALID, dict(h_kv=3))], ids=str)
def test_paged_append_statuses(lib, want, kw):
    d = capi.NormRopeDims(1, 10, 0, 4, 2, 128, 64, 0, 1e-6)
    c = _cache(**kw)
    assert lib.msa_qk_norm_rope_paged(ctypes.byref(d), GOOD, GOOD, GOOD, None, None, P(0x2000),
                                      100, None, GOOD, ctypes.byref(c), None, None) == want


def test_paged_append_needs_128_wide_heads(lib):
    d = capi.NormRopeDims(1, 10, 0, 4, 2, 64, 64, 0, 1e-6)
    assert lib.msa_qk_norm_rope_paged(ctypes.byref(d), GOOD, GOOD, GOOD, None, None, P(0x2000),
                                      100, None, GOOD, ctypes.byref(_cache()), None,
                                      None) == UNSUPPORTED
    assert lib.msa_qk_norm_rope_paged(ctypes.byref(capi.NormRopeDims(1, 1, 0, 4, 2, 128, 0, 0, 0)),
                                      GOOD, GOOD, GOOD, None, None, None, 100, None, GOOD, None,
                                      None, None) == INVALID


def test_norm_rope_backward_statuses(lib):
    d = capi.NormRopeDims(1, 10, 0, 4, 2, 128, 64, 0, 1e-6)
    need = lib.msa_qk_norm_rope_bwd_workspace(ctypes.byref(d))
    assert need > 0

    def call(d=d, fp32=0, dq=GOOD, dk=GOOD, ws=P(0x5000), n=need):
        return lib.msa_qk_norm_rope_bwd(ctypes.byref(d), GOOD, GOOD, None, None, P(0x2000), 100,
                                        None, dq, dk, fp32, GOOD, GOOD, None, None, ws, n, None,
                                        None)

    assert call(fp32=2) == INVALID
    assert call(ws=None) == INVALID
    assert call(ws=P(0x5008)) == ALIGNMENT
    assert call(n=need - 1) == WORKSPACE
    assert call(dq=capi.Tensor(0x100000, 0, 260, 128)) == ALIGNMENT       # bf16: multiples of 8
    # fp32 strides need multiples of 4 only: this gets as far as the workspace check
    assert call(dq=capi.Tensor(0x100000, 0, 260, 128), fp32=1, n=0) == WORKSPACE
    assert call(dq=capi.Tensor(0x100000, 0, 258, 128), fp32=1) == ALIGNMENT
    bad = capi.NormRopeDims(1, 10, 0, 4, 2, 96, 64, 0, 1e-6)
    assert lib.msa_qk_norm_rope_bwd_workspace(ctypes.byref(bad)) == 0
    assert call(d=bad) == UNSUPPORTED


def _decode(lib, cache=None, window=0, sink=0, q=GOOD, out=0x100000, lse=0x2000, ws=0x5000,
            n=None, n_kv=256, n_q=1, batch=1, h_q=8, h_kv=2):
    d = capi.make_dims(batch, n_q, n_kv, max(0, n_kv - 1), h_q, h_kv, 128)
    c = _cache() if cache is None else cache
    if n is None:
        n = capi.msa_paged_decode_attn_workspace(d)
    return lib.msa_paged_decode_attn(ctypes.byref(d), window, sink, q, ctypes.byref(c), P(out),
                                     P(lse), P(ws), n, None, None)


@pytest.mark.parametrize("want,kw", [
    (INVALID, dict(window=-1)), (INVALID, dict(sink=-1)), (INVALID, dict(n_q=2)),
    (INVALID, dict(n_kv=257)),                       # more than the table's row holds
    (INVALID, dict(out=0)), (INVALID, dict(lse=0)), (INVALID, dict(ws=0)),
    (ALIGNMENT, dict(out=0x100008)), (ALIGNMENT, dict(ws=0x5008)), (ALIGNMENT, dict(lse=0x2002)),
    (WORKSPACE, dict(n=64)), (INVALID, dict(q=capi.Tensor(0, 0, 0, 128))),
    (ALIGNMENT, dict(q=capi.Tensor(0x100000, 0, 0, 129))),
    (UNSUPPORTED, dict(h_q=12, h_kv=2)), (UNSUPPORTED, dict(h_q=64, h_kv=2)),
    (UNSUPPORTED, dict(batch=4097)),
], ids=str)
def test_paged_decode_statuses(lib, want, kw):
    assert _decode(lib, **kw) == want


@pytest.mark.parametrize("want,kw", BAD_CACHES + [(INVALID, dict(seq_lens=0)),
                                                  (ALIGNMENT, dict(seq_lens=0x4002))], ids=str)
def test_paged_decode_refuses_bad_caches(lib, want, kw):
    assert _decode(lib, cache=_cache(**kw)) == want


def test_broadcast_strides(lib):
    """Inputs of the norms may be broadcast, outputs not; tensors read by TMA not."""
    flat = capi.Tensor(0x100000, 1 << 20, 0, 128)
    assert _norm(lib, qo=flat) == INVALID and _norm(lib, ko=capi.Tensor(0x100000, 0, 0, 128)) == INVALID
    assert _norm(lib, batch=2, qo=GOOD) == INVALID
    assert _norm(lib, batch=2, q=flat, qo=flat) == INVALID
    d = capi.make_dims(2, 100, 300, 200, 8, 2, 128)
    good, shared = capi.Tensor(0x100000, 1 << 20, 1024, 128), capi.Tensor(0x100000, 0, 1024, 128)
    for q, k, v in ((shared, good, good), (good, shared, good), (good, good, shared)):
        assert lib.msa_window_attn_fwd(ctypes.byref(d), 0, 0, q, k, v, None, P(0x100000), None,
                                       P(0x2000), None, None) == UNSUPPORTED
    assert lib.msa_window_attn_bwd(ctypes.byref(d), 0, 0, good, good, good, good, None, shared,
                                   P(0x2000), None, P(0x100000), P(0x100000), P(0x100000),
                                   P(0x5000), 1 << 40, None, None) == UNSUPPORTED


def test_window_statuses(lib):
    GOOD = capi.Tensor(0x100000, 1 << 20, 256, 128)
    d = capi.make_dims(2, 100, 300, 200, 8, 2, 128)
    f, b = lib.msa_window_attn_fwd, lib.msa_window_attn_bwd

    def fwd(d=d, w=64, s=4, q=GOOD, lens=None, out=0x100000, rest=0x200000, lse=0x2000):
        return f(ctypes.byref(d), w, s, q, GOOD, GOOD, P(lens), P(out), P(rest), P(lse), None,
                 None)

    assert fwd(w=-1) == INVALID and fwd(s=-1) == INVALID
    assert fwd(out=0) == INVALID and fwd(lse=0) == INVALID
    assert fwd(q=capi.Tensor(0, 0, 256, 128)) == INVALID
    assert fwd(q=capi.Tensor(0x100000, 0, 256, 132)) == ALIGNMENT
    assert fwd(out=0x100010) == ALIGNMENT and fwd(rest=0x200008) == ALIGNMENT
    assert fwd(lse=0x2002) == ALIGNMENT and fwd(lens=0x3002) == ALIGNMENT
    assert fwd(d=capi.make_dims(1, 100, 150, 51, 8, 2, 128)) == INVALID      # past the keys
    assert fwd(d=capi.make_dims(1, 100, 300, 200, 12, 2, 128)) == UNSUPPORTED
    need = capi.msa_window_attn_bwd_workspace(d, 64, 4)
    assert need > 0

    def bwd(w=64, q=GOOD, o=GOOD, do=GOOD, rest=0x200000, lse=0x2000, dq=0x100000, dk=0x100000,
            dv=0x100000, ws=0x5000, n=need):
        return b(ctypes.byref(d), w, 4, q, GOOD, GOOD, o, P(rest), do, P(lse), None, P(dq), P(dk),
                 P(dv), P(ws), n, None, None)

    for name in ("lse", "dq", "dk", "dv", "ws"):
        assert bwd(**{name: 0}) == INVALID, name
    for name in ("dq", "dk", "dv", "ws"):
        assert bwd(**{name: 0x100010}) == ALIGNMENT, name
    assert bwd(rest=0x200008) == ALIGNMENT
    assert bwd(o=capi.Tensor(0, 0, 256, 128)) == INVALID
    assert bwd(do=capi.Tensor(0x100008, 0, 256, 128)) == ALIGNMENT
    assert bwd(n=need - 1) == WORKSPACE and bwd(w=-5) == INVALID
    assert capi.msa_window_attn_bwd_workspace(d, -1, 0) == 0
    # wider windows, more chunks: never more than the cut's bound of partial sums
    for w, s in ((0, 0), (1, 0), (0, 300), (300, 300), (1 << 40, 1 << 40)):
        x = capi.msa_window_attn_bwd_workspace(capi.make_dims(1, 32768, 32768, 0, 64, 8, 128), w, s)
        assert 32768 * 64 * 4 < x < 32768 * 64 * 4 + (1 << 20) + 2 * 2 * 148 * 2 * 128 * 128 * 4


# ---------------------------------------------------------------------------
# Python calls
# ---------------------------------------------------------------------------
BF = torch.bfloat16


def _z(*shape, dtype=BF):
    return torch.zeros(shape, dtype=dtype)


def test_python_calls_refuse_what_does_not_fit(lib):
    q, k = _z(2, 5, 4, 128), _z(2, 5, 2, 128)
    ko = _z(2, 2, 5, 128)
    table = _z(10, 64, dtype=torch.float32)
    for match, fn in [
        ("CUDA device", lambda: pipeline.norm_rope(pipeline.NormRope(table), q, k)),
        ("q or k", lambda: pipeline.norm_rope(pipeline.NormRope(table), None, None)),
        ("q: Float", lambda: pipeline.norm_rope(pipeline.NormRope(table), q.float(), None)),
        ("k: shape", lambda: pipeline.norm_rope(pipeline.NormRope(table), q, k[:1])),
        ("k_out: shape", lambda: pipeline.norm_rope(pipeline.NormRope(table), q, k, q, k)),
        ("w_q: shape", lambda: pipeline.norm_rope(pipeline.NormRope(table, _z(64, dtype=torch.float32)), q, k)),
        ("w_k: BFloat16", lambda: pipeline.norm_rope(pipeline.NormRope(table, None, _z(128)), q, k)),
        ("table", lambda: pipeline.norm_rope(pipeline.NormRope(table.t()), q, k)),
        ("positions: Int", lambda: pipeline.norm_rope(pipeline.NormRope(table), q, k, positions=_z(2, 5, dtype=torch.int32))),
        ("contiguous", lambda: pipeline.norm_rope(pipeline.NormRope(table), q.transpose(2, 3).contiguous().transpose(2, 3), None)),
        ("q or k", lambda: pipeline.norm_rope(pipeline.NormRope(table), q[0], k)),
        ("q_out: shape", lambda: capi.msa_qk_norm_rope(q, k, None, None, table, q[:, :, :3], ko)),
    ]:
        with pytest.raises(ValueError, match=match):
            fn()
    grads = pipeline.NormRopeGrads(q, k, None, None, _z(8, dtype=torch.float32))
    for match, dq, dk in [("d_q is missing", None, ko), ("d_k: Float", q, ko.float()),
                          ("bf16 or fp32", q.half(), ko), ("d_k: shape", q, k)]:
        with pytest.raises(ValueError, match=match):
            pipeline.norm_rope_backward(pipeline.NormRope(table), q, k, dq, dk, grads)


def test_python_calls_refuse_caches_that_do_not_fit(lib):
    kp, vp = _z(6, 2, 16, 128), _z(6, 2, 16, 128)
    table, lens = _z(2, 3, dtype=torch.int32), _z(2, dtype=torch.int32)
    q, k, v = _z(2, 1, 4, 128), _z(2, 1, 2, 128), _z(2, 1, 2, 128)
    d = capi.make_dims(2, 1, 48, 47, 4, 2, 128)
    buf = pipeline.DecodeBuffers(d, _z(2, 1, 4, 128), _z(2, 1, 4, dtype=torch.float32),
                                 _z(64, dtype=torch.int32), _z(4, dtype=torch.int32))

    def cache(**kw):
        c = dict(k_pages=kp, v_pages=vp, block_table=table, seq_lens=lens)
        c.update(kw)
        return pipeline.PagedCache(**c)

    bad = [("same shape", dict(v_pages=vp[:5])),
           ("same shape", dict(v_pages=vp.transpose(1, 2).contiguous().transpose(1, 2))),
           ("v_pages: must be", dict(v_pages=vp[..., :64])), ("k_pages: Half", dict(k_pages=kp.half())),
           ("block_table", dict(block_table=table[:1])), ("block_table: Long", dict(block_table=table.long()))]
    for match, kw in bad + [("seq_lens: Long", dict(seq_lens=lens.long())),
                            ("CUDA device", {})]:
        with pytest.raises(ValueError, match=match):
            pipeline.paged_decode(buf, q, cache(**kw))
    for match, kw in bad:
        with pytest.raises(ValueError, match=match):
            pipeline.norm_rope_append(pipeline.NormRope(None), q, k, v, None, None, cache(**kw))
    with pytest.raises(ValueError, match="v: shape"):
        pipeline.norm_rope_append(pipeline.NormRope(None), q, k, v[:, :, :1], None, None, cache())
    with pytest.raises(ValueError, match="k is missing"):
        pipeline.norm_rope_append(pipeline.NormRope(None), q, None, v, None, None, cache())
    with pytest.raises(ValueError, match="q: shape"):
        pipeline.paged_decode(buf, q[:, :, :2], cache())


def test_python_window_calls_refuse_what_does_not_fit(lib):
    d = pipeline.window_dims(2, 5, 9, 4, 4, 2)
    buf = pipeline.WindowBuffers.allocate(d, 4, 1, backward=True, device="cpu")
    q, k = _z(2, 5, 4, 128), _z(2, 2, 9, 128)
    for match, args in [("k: shape", (q, k[:, :1], k)), ("v: Float", (q, k, k.float())),
                        ("kv_len: shape", (q, k, k, _z(3, dtype=torch.int32))),
                        ("CUDA device", (q, k, k))]:
        with pytest.raises(ValueError, match=match):
            pipeline.window_forward(buf, *args)
    with pytest.raises(ValueError, match="d_o: shape"):
        pipeline.window_backward(buf, q, k, k, q[:, :4])
    with pytest.raises(ValueError, match="backward=True"):
        pipeline.window_backward(pipeline.WindowBuffers.allocate(d, device="cpu"), q, k, k, q)
    with pytest.raises(ValueError, match="Dims"):
        capi.msa_window_attn_fwd(capi.Tensor(0, 0, 0, 0), 0, 0, q, k, k, buf.out, buf.lse)
