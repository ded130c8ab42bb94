"""Per-head norm + rotation on the GPU (dense, into a paged cache, backward)
against the 64-bit definition; bounds are derived in _layer_ref.py."""
import pytest
import torch

import _layer_ref as ref
from block_sparse_attention_32_b200 import pipeline

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def _rn(seed, *shape, dtype=BF, scale=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def _w(seed, d):
    return 1.0 + 0.3 * _rn(seed, d, dtype=torch.float32)


def _positions(B, T, n_pos, pad, seed=5):
    g = torch.Generator().manual_seed(seed)
    p = torch.randint(0, n_pos, (B, T), generator=g)
    if pad:
        p[-1, T // 2:] = -1
    return p.cuda()


# batch, tokens, query heads, key heads, width, rot, adjacent pairs, padded
DENSE = [
    (1, 1, 1, 1, 64, 64, False, False),
    (1, 1, 8, 1, 128, 128, False, False),
    (2, 7, 5, 3, 128, 64, True, True),
    (3, 33, 16, 2, 64, 16, False, True),
    (1, 130, 64, 8, 128, 128, True, False),
    (2, 65, 3, 1, 64, 48, False, False),
    (1, 257, 9, 9, 128, 112, True, True),
    (2, 300, 32, 4, 128, 96, False, True),
    (1, 19, 4, 2, 128, 0, False, False),
    (1, 5000, 8, 1, 64, 32, True, False),
]


@pytest.mark.parametrize("B,T,hq,hk,d,rot,inter,pad", DENSE)
def test_dense_forward_and_backward(B, T, hq, hk, d, rot, inter, pad):
    n_pos = 9000
    table = pipeline.rope_table(n_pos, rot) if rot else None
    pos = _positions(B, T, n_pos, pad)
    q, k = _rn(1, B, T, hq, d, scale=1.7), _rn(2, B, T, hk, d, scale=0.4)
    plan = pipeline.NormRope(table, _w(3, d), _w(4, d), eps=1e-5, interleaved=inter)
    qo = torch.full_like(q, 7.0)
    ko = torch.full((B, hk, T, d), 7.0, dtype=BF, device="cuda")
    err = torch.zeros(4, dtype=torch.int32, device="cuda")
    pipeline.norm_rope(plan, q, k, qo, ko, positions=pos, dev_err=err)
    live = pos >= 0
    tab = table if rot else torch.zeros((n_pos, 0), device="cuda")
    cos, sin = ref.angles(tab, pos)
    for got, x, w in ((qo, q, plan.w_q), (ko.transpose(1, 2), k, plan.w_k)):
        want, bound = ref.norm_rope(x, w, cos, sin, inter, 1e-5)
        ref.close("y", got[live], want[live], bound[live])
        assert (got[~live] == 7.0).all()                     # padding is left alone
    for dt in (BF, torch.float32):
        dq, dk = _rn(6, B, T, hq, d, dtype=dt), _rn(7, B, hk, T, d, dtype=dt)
        gr = pipeline.NormRopeGrads.allocate(q, k)
        gr.dx_q.fill_(7.0)
        gr.dx_k.fill_(7.0)
        pipeline.norm_rope_backward(plan, q, k, dq, dk, gr, positions=pos, dev_err=err)
        for x, w, dy, dx, dw in ((q, plan.w_q, dq, gr.dx_q, gr.dw_q),
                                 (k, plan.w_k, dk.transpose(1, 2), gr.dx_k, gr.dw_k)):
            ex, bx, ew, bw = ref.norm_rope_bwd(x, w, dy, cos, sin, inter, 1e-5, live)
            ref.close("dx", dx[live], ex[live], bx[live])
            ref.close("dw", dw, ew, bw, fro=False)
            assert (dx[~live] == 7.0).all()
    assert int(err[0]) == 0


def test_backward_is_the_derivative():
    """dx, dw against central differences of the 64-bit forward."""
    B, T, h, d, rot = 1, 3, 2, 64, 32
    table = pipeline.rope_table(50, rot)
    q = _rn(1, B, T, h, d)
    plan = pipeline.NormRope(table, _w(2, d), None, eps=1e-3, interleaved=True)
    dy = _rn(3, B, T, h, d)
    gr = pipeline.NormRopeGrads.allocate(q, None)
    pipeline.norm_rope_backward(plan, q, None, dy, None, gr, pos0=11)
    pos = 11 + torch.arange(T, device="cuda")[None]
    cos, sin = ref.angles(table, pos)

    def loss(x, w):
        return float((ref.norm_rope(x, w, cos, sin, True, 1e-3)[0] * dy.double()).sum())

    x, w, e = q.double(), plan.w_q.double(), 1e-5
    for i in range(0, B * T * h * d, 29):
        hi, lo = x.clone().view(-1), x.clone().view(-1)
        hi[i] += e
        lo[i] -= e
        num = (loss(hi.view_as(x), w) - loss(lo.view_as(x), w)) / (2 * e)
        got = float(gr.dx_q.view(-1)[i])
        assert abs(got - num) <= 2.0 ** -8 * abs(num) + 1e-4, i
    for i in range(0, d, 7):
        hi, lo = w.clone(), w.clone()
        hi[i] += e
        lo[i] -= e
        num = (loss(x, hi) - loss(x, lo)) / (2 * e)
        assert abs(float(gr.dw_q[i]) - num) <= 1e-4 * max(1.0, abs(num)), i


def test_views_of_a_fused_projection_in_place_and_missing_parts():
    """q, k as slices of one [B, T, (hq + 2 hk) d] projection, rewritten in place;
    no weights; only keys; a far position offset."""
    B, T, hq, hk, d = 2, 37, 6, 2, 128
    table = pipeline.rope_table(1 << 17, d)
    qkv = _rn(1, B, T, (hq + 2 * hk) * d)
    keep = qkv.clone()
    parts = qkv.view(B, T, hq + 2 * hk, d)
    q, k = parts[:, :, :hq], parts[:, :, hq:hq + hk]
    q0, k0 = q.clone(), k.clone()
    plan = pipeline.NormRope(table, None, None)
    pos0 = (1 << 17) - T
    pipeline.norm_rope(plan, q, k, q, k.transpose(1, 2), pos0=pos0)
    pos = (pos0 + torch.arange(T, device="cuda"))[None].expand(B, -1)
    cos, sin = ref.angles(table, pos)
    for got, x in ((q, q0), (k, k0)):
        want, bound = ref.norm_rope(x, None, cos, sin, False, 1e-6)
        ref.close("in place", got, want, bound)
    assert torch.equal(parts[:, :, hq + hk:], keep.view_as(parts)[:, :, hq + hk:])
    none, k_out = pipeline.norm_rope(plan, None, k0, pos0=pos0)
    assert none is None and torch.equal(k_out.transpose(1, 2), k)


def test_broadcast_inputs():
    """One row for all tokens and heads (strides of 0), also as upstream gradient."""
    row, g = _rn(1, 1, 1, 1, 128), _rn(2, 1, 1, 1, 128)
    x, dy = row.expand(2, 5, 3, 128), g.expand(2, 5, 3, 128)
    table = pipeline.rope_table(5, 32)
    plan = pipeline.NormRope(table, _w(3, 128))
    out, _ = pipeline.norm_rope(plan, x, None)
    gr = pipeline.NormRopeGrads.allocate(x, None)
    dx, _, dw, _ = pipeline.norm_rope_backward(plan, x, None, dy, None, gr)
    pos = torch.arange(5, device="cuda")[None].expand(2, -1)
    cos, sin = ref.angles(table, pos)
    want, bound = ref.norm_rope(x, plan.w_q, cos, sin, False, 1e-6)
    ref.close("y", out, want, bound)
    ex, bx, ew, bw = ref.norm_rope_bwd(x, plan.w_q, dy, cos, sin, False, 1e-6, pos >= 0)
    ref.close("dx", dx, ex, bx)
    ref.close("dw", dw, ew, bw, fro=False)


def test_zero_rows_and_eps_zero():
    """A zero row stays zero; with eps = 0 absent rows add nothing to dw."""
    q = _rn(1, 1, 6, 3, 64)
    q[0, 2] = 0.0
    out, _ = pipeline.norm_rope(pipeline.NormRope(None, None, None, eps=1e-6), q, None)
    assert not out[0, 2].any() and torch.isfinite(out.float()).all()
    x, dy = _rn(2, 1, 6, 3, 64), _rn(3, 1, 6, 3, 64)
    pos = torch.tensor([[0, 1, 2, -1, -1, -1]], device="cuda")
    gr = pipeline.NormRopeGrads.allocate(x, None)
    pipeline.norm_rope_backward(pipeline.NormRope(None, None, None, eps=0.0), x, None, dy, None,
                                gr, positions=pos)
    cos = torch.zeros((1, 6, 1, 0), dtype=torch.float64, device="cuda")
    _, _, ew, bw = ref.norm_rope_bwd(x, None, dy, cos, cos, False, 0.0, pos >= 0)
    ref.close("dw", gr.dw_q, ew, bw, fro=False)


def test_position_past_the_table_is_reported_and_left_alone():
    table = pipeline.rope_table(10, 64)
    q = _rn(1, 1, 4, 2, 64)
    out = torch.full_like(q, 7.0)
    err = torch.zeros(4, dtype=torch.int32, device="cuda")
    pos = torch.tensor([[3, 10, 9, 1 << 40]], device="cuda")
    pipeline.norm_rope(pipeline.NormRope(table), q, None, out, positions=pos, dev_err=err)
    assert int(err[0]) == 4                                   # MSA_DEVERR_BAD_POSITION
    assert (out[0, 1] == 7.0).all() and (out[0, 3] == 7.0).all()
    assert not (out[0, 0] == 7.0).all() and not (out[0, 2] == 7.0).all()


# ---------------------------------------------------------------------------
# into a paged cache
# ---------------------------------------------------------------------------
def _cache(B, per, h, page, nhd, seed=9):
    n = B * per + 2
    shape = (n, page, h, 128) if nhd else (n, h, page, 128)
    kp, vp = _rn(seed, *shape), _rn(seed + 1, *shape)
    if nhd:
        kp, vp = kp.permute(0, 2, 1, 3), vp.permute(0, 2, 1, 3)
    g = torch.Generator().manual_seed(seed)
    table = torch.randperm(n, generator=g)[:B * per].view(B, per).int().cuda()
    return pipeline.PagedCache(kp, vp, table, torch.zeros(B, dtype=torch.int32, device="cuda"))


@pytest.mark.parametrize("B,T,hq,hk,page,nhd,rot,inter", [
    (1, 1, 1, 1, 16, False, 128, False),
    (5, 1, 16, 2, 64, True, 64, True),
    (3, 40, 8, 8, 16, True, 128, False),
    (2, 129, 12, 3, 32, False, 32, True),
    (4, 3, 64, 4, 256, False, 128, False),
])
def test_append_writes_its_places_and_nothing_else(B, T, hq, hk, page, nhd, rot, inter):
    per = 5 if page > 32 else 20
    cache = _cache(B, per, hk, page, nhd)
    table = pipeline.rope_table(per * page, rot)
    plan = pipeline.NormRope(table, _w(3, 128), _w(4, 128), interleaved=inter)
    q, k, v = _rn(1, B, T, hq, 128), _rn(2, B, T, hk, 128), _rn(5, B, T, hk, 128)
    starts = [(37 * b) % (per * page - T + 1) for b in range(B)]
    pos = torch.tensor([[s + i for i in range(T)] for s in starts], device="cuda")
    if T > 1:
        pos[0, T - 1] = -1                                    # one padded token
    qo = torch.full_like(q, 7.0)
    want_k, want_v = cache.k_pages.clone(), cache.v_pages.clone()
    err = torch.zeros(4, dtype=torch.int32, device="cuda")
    out = pipeline.norm_rope_append(plan, q, k, v, pos, qo, cache, dev_err=err)
    assert out is qo and int(err[0]) == 0
    live = pos >= 0
    cos, sin = ref.angles(table, pos)
    wq, bq = ref.norm_rope(q, plan.w_q, cos, sin, inter, 1e-6)
    ref.close("q", qo[live], wq[live], bq[live])
    assert (qo[~live] == 7.0).all()
    wk, bk = ref.norm_rope(k, plan.w_k, cos, sin, inter, 1e-6)
    got_k, got_v = cache.k_pages.clone(), cache.v_pages.clone()
    for b in range(B):
        for i in range(T):
            p = int(pos[b, i])
            if p < 0:
                continue
            pg, r = int(cache.block_table[b, p // page]), p % page
            ref.close("k", got_k[pg, :, r], wk[b, i], bk[b, i])
            assert torch.equal(got_v[pg, :, r], v[b, i])
            got_k[pg, :, r], got_v[pg, :, r] = want_k[pg, :, r], want_v[pg, :, r]
    assert torch.equal(got_k, want_k) and torch.equal(got_v, want_v)


def test_append_reports_bad_pages_and_leaves_the_cache_alone():
    cache = _cache(2, 2, 2, 16, False)
    cache.block_table[0, 1] = -1
    cache.block_table[1, 0] = cache.k_pages.shape[0]
    plan = pipeline.NormRope(pipeline.rope_table(100, 64))
    q, k, v = _rn(1, 2, 3, 4, 128), _rn(2, 2, 3, 2, 128), _rn(3, 2, 3, 2, 128)
    # unmapped page, place past the table's row, mapped; page number out of range twice, mapped
    pos = torch.tensor([[20, 40, 1], [0, 15, 31]], device="cuda")
    k0, v0 = cache.k_pages.clone(), cache.v_pages.clone()
    err = torch.zeros(4, dtype=torch.int32, device="cuda")
    qo = torch.full_like(q, 7.0)
    pipeline.norm_rope_append(plan, q, k, v, pos, qo, cache, dev_err=err)
    assert int(err[0]) == 5                                   # MSA_DEVERR_BAD_PAGE
    assert not (qo == 7.0).flatten(2).all(-1).any()
    for b, i in ((0, 2), (1, 2)):
        p = int(pos[b, i])
        pg, r = int(cache.block_table[b, p // 16]), p % 16
        assert torch.equal(cache.v_pages[pg, :, r], v[b, i])
        cache.k_pages[pg, :, r], cache.v_pages[pg, :, r] = k0[pg, :, r], v0[pg, :, r]
    assert torch.equal(cache.k_pages, k0) and torch.equal(cache.v_pages, v0)
