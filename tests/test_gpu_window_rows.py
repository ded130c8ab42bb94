"""Window attention backward, row by row: how exact a row's gradient is depends on what
the row sees, not on the call that it is part of."""
import math

import pytest
import torch

import _layer_ref as ref
from block_sparse_attention_32_b200 import pipeline

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def _rn(seed, *shape):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").to(BF)


def _inputs(B, n_q, n_kv, H, G):
    return (_rn(1, B, n_q, H, 128), _rn(2, B, G, n_kv, 128), _rn(3, B, G, n_kv, 128),
            _rn(4, B, n_q, H, 128))


def _buffers(B, n_q, n_kv, pos0, H, G, W, S):
    return pipeline.WindowBuffers.allocate(pipeline.window_dims(B, n_q, n_kv, pos0, H, G), W, S,
                                           backward=True)


@pytest.mark.parametrize("n_q,pos0,H,G,W,S", [(300, 0, 8, 2, 0, 0), (300, 0, 8, 2, 40, 10),
                                              (90, 30, 16, 1, 0, 0), (200, 500, 4, 2, 70, 3)])
def test_a_sequence_alone_and_in_a_batch(n_q, pos0, H, G, W, S):
    """The same sequence as one of nine: dq has the same bits (the sum over a row's keys has
    one order), from the same forward results."""
    B, b = 9, 5
    q, k, v, d_o = _inputs(B, n_q, pos0 + n_q, H, G)
    many, one = (_buffers(x, n_q, pos0 + n_q, pos0, H, G, W, S) for x in (B, 1))
    pipeline.window_forward(many, q, k, v)
    dq, dk, dv = pipeline.window_backward(many, q, k, v, d_o)
    for name in ("out", "lse", "rest"):
        getattr(one, name).copy_(getattr(many, name)[b:b + 1])
    sq, sk, sv = pipeline.window_backward(one, q[b:b + 1], k[b:b + 1], v[b:b + 1], d_o[b:b + 1])
    assert torch.equal(sq[0], dq[b])
    # dk, dv: their sums over queries may be cut elsewhere, which is fp32 (2^-14 of the terms),
    # and then a rounding may fall to the other side: one step of bf16, 2^-7
    see = ref.visible(n_q, pos0 + n_q, pos0, W, S, pos0 + n_q, "cuda")
    o, _, _, aux = ref.attention(q[b], k[b], v[b], see, 1 / math.sqrt(128))
    _, (ek, bk), (ev, bv) = ref.attention_grads(o, aux, d_o[b], see, 1 / math.sqrt(128), G)
    for x, y, e, bound in ((sk[0], dk[b], ek, bk), (sv[0], dv[b], ev, bv)):
        assert ((x.double() - y.double()).abs() <= 2.0 ** -7 * e.abs() + 2.0 ** -6 * bound).all()


@pytest.mark.parametrize("B,n,H,G,W,S", [(1, 1024, 16, 2, 0, 0), (2, 1500, 8, 8, 100, 3),
                                         (3, 700, 1, 1, 0, 0), (2, 2000, 16, 1, 1, 0)])
def test_rows_of_one_key_in_large_calls(B, n, H, G, W, S):
    """A row that sees one key has p = 1 and dS = 0, exactly, in calls of any size; its whole
    dO goes into dv."""
    q, k, v, d_o = _inputs(B, n, n, H, G)
    buf = _buffers(B, n, n, 0, H, G, W, S)
    pipeline.window_forward(buf, q, k, v)
    dq, dk, dv = pipeline.window_backward(buf, q, k, v, d_o)
    assert torch.count_nonzero(dq[:, 0]) == 0
    assert torch.count_nonzero(dq[:, 1:]) > 0 or W == 1
    if W == 1:                                        # every row is such a row
        assert torch.count_nonzero(dq) == 0 and torch.count_nonzero(dk) == 0
        want = d_o.double().view(B, n, G, H // G, 128).sum(3).transpose(1, 2)
        # p = 1 to 2^-17, the sum in fp32, one rounding
        mag = d_o.double().abs().view(B, n, G, H // G, 128).sum(3).transpose(1, 2)
        assert ((dv.double() - want).abs() <= ref.U * want.abs() + ref.SMALL * mag).all()


@pytest.mark.parametrize("n", [40, 700])
def test_a_sequence_of_one_token_in_a_padded_batch(n):
    """It sees itself only: no gradient of q and k, dO as that of v, whatever the others are."""
    B, H, G = 3, 8, 2
    q, k, v, d_o = _inputs(B, n, n, H, G)
    buf = _buffers(B, n, n, 0, H, G, 0, 0)
    kv_len = torch.tensor([n, 1, n // 2], dtype=torch.int32, device="cuda")
    out, _ = pipeline.window_forward(buf, q, k, v, kv_len)
    dq, dk, dv = pipeline.window_backward(buf, q, k, v, d_o, kv_len)
    assert torch.count_nonzero(dq[1]) == 0 and torch.count_nonzero(dk[1]) == 0
    assert torch.count_nonzero(dv[1, :, 1:]) == 0 and torch.count_nonzero(out[1, 1:]) == 0
    x = d_o[1, 0].double().view(G, H // G, 128)
    want, mag = x.sum(1), x.abs().sum(1)
    # p is within fp32 of 1 and rounds to it; one rounding of the sum
    assert ((dv[1, :, 0].double() - want).abs() <= ref.U * want.abs() + ref.SMALL * mag).all()
    assert torch.count_nonzero(dk[0]) > 0 and torch.count_nonzero(dk[2]) > 0


@pytest.mark.parametrize("B,n,H,G,W,S", [(1, 2048, 8, 1, 0, 0), (2, 1500, 16, 2, 40, 20),
                                         (1, 3000, 4, 4, 1000, 5), (2, 1500, 16, 2, 2, 1),
                                         (3, 2000, 1, 1, 0, 0)])
def test_rows_of_few_keys_keep_one_rounding(B, n, H, G, W, S):
    """Rows that see at most four keys, in calls of any size: dS keeps 16 bits, so their dq is
    off by two things.  Its own rounding is at most half a step, 2^-8 of a value, spread
    evenly: 2^-8 / sqrt(3) in the Frobenius norm over hundreds of values (5 % for the sample),
    and 2^-14 for P, dS and fp32.  And D = dO.o takes the forward's o, whose weights p_j were
    rounded to bf16: o is off by sum_j p_j e_j v_j, |e_j| <= 2^-8, D by at most
    2^-8 sum_j p_j |dO.v_j|, and dq by that times scale |sum_j p_j k_j|.  Where all rows are
    such rows, dk and dv are as exact as their terms."""
    q, k, v, d_o = _inputs(B, n, n, H, G)
    buf = _buffers(B, n, n, 0, H, G, W, S)
    pipeline.window_forward(buf, q, k, v)
    grads = pipeline.window_backward(buf, q, k, v, d_o)
    few = n if W and W + S <= 4 else 4
    limit = 1.05 * 2 ** -8 / 3 ** 0.5 + 2 ** -14
    scale = 1 / math.sqrt(128)
    see = ref.visible(n, n, 0, W, S, n, "cuda")
    for b in range(B):
        o, _, _, aux = ref.attention(q[b], k[b], v[b], see, scale)
        p, _, _, kk, vv = aux
        dp = torch.einsum("ihd,hjd->hij", d_o[b].double(), vv)
        e_d = (p * dp.abs()).sum(-1).T * ref.U                        # [n, H]
        by_d = scale * e_d[..., None] * torch.einsum("hij,hjd->ihd", p, kk).abs()
        (eq, _), (ek, _), (ev, _) = ref.attention_grads(o, aux, d_o[b], see, scale, G)
        off = float((grads[0][b, :few].double() - eq[:few]).norm())
        assert off <= limit * float(eq[:few].norm()) + float(by_d[:few].norm())
        if few == n:
            for x, e in ((grads[1][b], ek), (grads[2][b], ev)):
                assert float((x.double() - e).norm() / e.norm()) <= limit


@pytest.mark.parametrize("n_q,n_kv,pos0,H,G,W,S,lens", [
    (64, 2000, 1000, 32, 2, 0, 0, None), (1, 500, 0, 8, 1, 0, 0, None),
    (130, 700, 300, 8, 2, 70, 5, None), (16, 9000, 8000, 16, 2, 0, 0, None),
    (300, 1000, 200, 4, 4, 100, 40, [1000, 350]), (40, 300, 100, 16, 2, 3, 1, [140, 139])])
def test_keys_behind_the_last_query_may_hold_anything(n_q, n_kv, pos0, H, G, W, S, lens):
    """A cache longer than what has been written: no query sees the keys from q_pos0 + n_q
    on (nor those from kv_len on), whose K and V may be NaN or infinite."""
    B = 2
    q, k, v, d_o = _inputs(B, n_q, n_kv, H, G)
    kv_len, ends = None, [pos0 + n_q] * B
    if lens is not None:
        kv_len = torch.tensor(lens, dtype=torch.int32, device="cuda")
        ends = [min(n, pos0 + n_q) for n in lens]
    for b, n in enumerate(ends):
        k[b, :, n:], v[b, :, n:] = math.nan, math.nan
        k[b, :, n:n + 1], v[b, :, n:n + 1] = math.inf, -math.inf
    buf = _buffers(B, n_q, n_kv, pos0, H, G, W, S)
    for t in (buf.dq, buf.dk, buf.dv):
        t.fill_(7.0)
    out, lse = pipeline.window_forward(buf, q, k, v, kv_len)
    grads = pipeline.window_backward(buf, q, k, v, d_o, kv_len)
    assert int(buf.dev_err[0]) == 0
    scale = 1 / math.sqrt(128)
    for b, n in enumerate(ends):
        see = ref.visible(n_q, n_kv, pos0, W, S, n, "cuda")
        o, l, bound, aux = ref.attention(q[b], k[b], v[b], see, scale)
        ref.close("o", out[b], o, bound)
        ref.close_lse(lse[b], l)
        for x, (e, be) in zip(grads, ref.attention_grads(o, aux, d_o[b], see, scale, G)):
            ref.close("grad", x[b], e, be, fro=n_q > 1)
        assert not grads[1][b, :, n:].any() and not grads[2][b, :, n:].any()
