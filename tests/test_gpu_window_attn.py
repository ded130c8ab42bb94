"""Sliding-window attention with sinks on the GPU, forward and backward, against
the 64-bit definition; bounds are derived in _layer_ref.py."""
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


# batch, n_q, n_kv, first position, query heads, KV heads, window, sinks, lengths (or None)
CASES = [
    (1, 1, 1, 0, 1, 1, 0, 0, None),
    (1, 1, 300, 299, 8, 1, 0, 0, None),
    (2, 5, 130, 125, 16, 1, 3, 0, None),
    (1, 128, 128, 0, 4, 1, 0, 0, None),
    (1, 129, 129, 0, 2, 2, 1, 0, None),
    (1, 300, 300, 0, 8, 1, 64, 0, None),
    (2, 257, 513, 256, 4, 2, 100, 9, None),
    (1, 700, 700, 0, 16, 1, 130, 200, None),
    (1, 1000, 1000, 0, 4, 1, 0, 0, None),
    (1, 64, 2000, 1000, 32, 2, 0, 0, None),          # keys after the last query
    (1, 640, 1500, 860, 4, 4, 333, 1, None),
    (3, 200, 400, 200, 8, 2, 50, 5, [400, 250, 0]),  # padded; one sequence without queries
    (2, 333, 333, 0, 16, 2, 0, 0, [100, 333]),
    (3, 129, 390, 201, 2, 1, 1, 3, [330, 202, 201]),
    (2, 70, 1111, 900, 32, 2, 2000, 0, [905, 1111]),
    (1, 50, 900, 850, 8, 8, 100, 700, None),         # sinks run into the window
    (1, 2500, 2500, 0, 8, 8, 40, 300, None),
    # sinks and window in one key tile; the sequence ends inside the sinks' 32 keys
    (1, 900, 900, 0, 4, 1, 70, 45, None),
    (2, 300, 700, 400, 8, 1, 150, 97, [700, 433]),
    (1, 5, 40, 10, 4, 1, 1, 3, [13]),
    (2, 260, 600, 300, 16, 1, 33, 129, [560, 301]),
    (2, 600, 600, 0, 16, 2, 1, 0, None),             # every row sees itself only
    (1, 1500, 1700, 200, 16, 1, 3, 1, [1650]),
    (2, 130, 130, 0, 8, 1, 0, 0, [130, 77]),
    # few rows of many keys: the row tiles are shared by two, four, eight CTAs
    (1, 16, 2500, 2400, 16, 2, 0, 0, None),
    (2, 40, 6000, 5900, 16, 2, 0, 0, [5930, 100]),
    (1, 33, 5000, 4900, 8, 1, 4500, 70, None),
    (1, 20, 9000, 8900, 8, 1, 0, 0, [8911]),
    (1, 300, 8700, 8400, 1, 1, 0, 0, None),
]


def _inputs(case, seed=1, nan=True):
    B, n_q, n_kv, pos0, H, G, W, S, lens = case
    q, k, v = _rn(seed, B, n_q, H, 128), _rn(seed + 1, B, G, n_kv, 128), _rn(seed + 2, B, G, n_kv, 128)
    d_o = _rn(seed + 3, B, n_q, H, 128)
    kv_len = None
    if lens is not None:
        kv_len = torch.tensor(lens, dtype=torch.int32, device="cuda")
        for b, n in enumerate(lens):                 # what lies behind a sequence may be anything
            if nan:
                k[b, :, n:], v[b, :, n:] = math.nan, math.nan
                q[b, max(0, n - pos0):], d_o[b, max(0, n - pos0):] = math.nan, math.nan
    return q, k, v, d_o, kv_len


def _expect(case, q, k, v, d_o, scale):
    B, n_q, n_kv, pos0, H, G, W, S, lens = case
    for b in range(B):
        n = n_kv if lens is None else lens[b]
        see = ref.visible(n_q, n_kv, pos0, W, S, n, "cuda")
        o, lse, bound, aux = ref.attention(q[b], k[b], v[b], see, scale)
        yield b, o, lse, bound, ref.attention_grads(o, aux, d_o[b], see, scale, G)


@pytest.mark.parametrize("case", CASES, ids=str)
def test_forward(case):
    B, n_q, n_kv, pos0, H, G, W, S, lens = case
    q, k, v, d_o, kv_len = _inputs(case)
    buf = pipeline.WindowBuffers.allocate(pipeline.window_dims(B, n_q, n_kv, pos0, H, G), W, S)
    out, lse = pipeline.window_forward(buf, q, k, v, kv_len)
    assert int(buf.dev_err[0]) == 0
    for b, o, l, bound, _ in _expect(case, q, k, v, d_o, 1 / math.sqrt(128)):
        ref.close(f"o[{b}]", out[b], o, bound, fro=n_kv > 1)
        ref.close_lse(lse[b], l)
    first = out.clone()
    pipeline.window_forward(buf, q, k, v, kv_len)
    assert torch.equal(first, out)


@pytest.mark.parametrize("case", CASES, ids=str)
def test_backward(case):
    B, n_q, n_kv, pos0, H, G, W, S, lens = case
    q, k, v, d_o, kv_len = _inputs(case)
    d = pipeline.window_dims(B, n_q, n_kv, pos0, H, G)
    buf = pipeline.WindowBuffers.allocate(d, W, S, backward=True)
    for t in (buf.dq, buf.dk, buf.dv):
        t.fill_(7.0)
    buf.ws.fill_(-1)
    pipeline.window_forward(buf, q, k, v, kv_len)
    dq, dk, dv = pipeline.window_backward(buf, q, k, v, d_o, kv_len)
    assert int(buf.dev_err[0]) == 0
    for b, o, l, _, ((eq, bq), (ek, bk), (ev, bv)) in _expect(case, q, k, v, d_o,
                                                             1 / math.sqrt(128)):
        # one visible key: dS = p (dP - D) is rounding noise around an exact 0
        ref.close(f"dv[{b}]", dv[b], ev, bv)
        ref.close(f"dq[{b}]", dq[b], eq, bq, fro=W != 1 and n_kv > 1)
        ref.close(f"dk[{b}]", dk[b], ek, bk, fro=W != 1 and n_kv > 1)
    first = [t.clone() for t in (dq, dk, dv)]
    pipeline.window_backward(buf, q, k, v, d_o, kv_len)
    for x, y in zip(first, (dq, dk, dv)):
        assert torch.equal(x, y)                      # no order of sums is left to chance


@pytest.mark.parametrize("case", [CASES[5], CASES[9][:1] + (40, 45, 5, 16, 2, 0, 0, None),
                                  (2, 900, 900, 0, 16, 2, 2, 0, None)], ids=str)
def test_few_terms_keep_one_rounding(case):
    """Few keys a row, or few tiles: P and dS keep 16 bits, so the gradients are off by their
    own rounding alone.  It is at most half a step, 2^-8 of a value, spread evenly: 2^-8 /
    sqrt(3) in the Frobenius norm over thousands of values (5 % for the sample), and 2^-14
    for P, dS and D.  (With P and dS in 8 bits: 2^-8 sqrt(2 / 3), less the values' spread.)"""
    B, n_q, n_kv, pos0, H, G, W, S, lens = case
    q, k, v, d_o, _ = _inputs(case)
    buf = pipeline.WindowBuffers.allocate(pipeline.window_dims(B, n_q, n_kv, pos0, H, G), W, S,
                                          backward=True)
    pipeline.window_forward(buf, q, k, v)
    grads = pipeline.window_backward(buf, q, k, v, d_o)
    for b, o, l, _, want in _expect(case, q, k, v, d_o, 1 / math.sqrt(128)):
        for x, (e, _) in zip(grads, want):
            off = float((x[b].double() - e).norm() / e.norm())
            assert off <= 1.05 * 2 ** -8 / 3 ** 0.5 + 2 ** -14


def test_a_row_that_sees_one_key_has_no_gradient():
    for case in ((2, 1, 1, 0, 8, 2, 0, 0, None), (1, 700, 900, 100, 16, 4, 1, 0, None)):
        B, n_q, n_kv, pos0, H, G, W, S, lens = case
        q, k, v, d_o, _ = _inputs(case)
        buf = pipeline.WindowBuffers.allocate(pipeline.window_dims(B, n_q, n_kv, pos0, H, G), W, S,
                                              backward=True)
        pipeline.window_forward(buf, q, k, v)
        dq, dk, dv = pipeline.window_backward(buf, q, k, v, d_o)
        assert torch.count_nonzero(dq) == 0 and torch.count_nonzero(dk) == 0
        assert torch.count_nonzero(dv[:, :, pos0:pos0 + n_q]) > 0


def test_backward_without_the_kept_bits():
    """o alone gives D to bf16: wider bounds, the same otherwise."""
    case = CASES[6]
    B, n_q, n_kv, pos0, H, G, W, S, lens = case
    q, k, v, d_o, _ = _inputs(case)
    buf = pipeline.WindowBuffers.allocate(pipeline.window_dims(B, n_q, n_kv, pos0, H, G), W, S,
                                          backward=True)
    buf.rest = None
    pipeline.window_forward(buf, q, k, v)
    dq, dk, dv = pipeline.window_backward(buf, q, k, v, d_o)
    scale = 1 / math.sqrt(128)
    for b in range(B):
        see = ref.visible(n_q, n_kv, pos0, W, S, n_kv, "cuda")
        o, lse, bound, aux = ref.attention(q[b], k[b], v[b], see, scale)
        (eq, bq), (ek, bk), (ev, bv) = ref.attention_grads(o, aux, d_o[b], see, scale, G, ref.U)
        ref.close("dq", dq[b], eq, bq)
        ref.close("dk", dk[b], ek, bk)
        ref.close("dv", dv[b], ev, bv)


@pytest.mark.parametrize("case", [CASES[6], CASES[11]], ids=str)
def test_kept_bits_extend_the_output(case):
    """out and its kept bits together are o up to the rounding of P and fp32."""
    B, n_q, n_kv, pos0, H, G, W, S, lens = case
    q, k, v, d_o, kv_len = _inputs(case)
    buf = pipeline.WindowBuffers.allocate(pipeline.window_dims(B, n_q, n_kv, pos0, H, G), W, S,
                                          backward=True)
    buf.rest.fill_(99)
    out, _ = pipeline.window_forward(buf, q, k, v, kv_len)
    bits = (out.view(torch.int16).int() << 16) + (buf.rest.int() << 8)
    full = bits.view(torch.float32)
    # the 8 bits leave half a unit of 2^-16 relative, and keep out as the nearest bf16
    assert ((full - out.float()).abs() <= 2.0 ** -8 * out.float().abs() + 1e-38).all()
    for b, o, l, bound, _ in _expect(case, q, k, v, d_o, 1 / math.sqrt(128)):
        rounded_p = bound - ref.U * o.abs()          # what is left without the rounding of o
        ref.close("full", full[b], o, rounded_p + 2.0 ** -15 * o.abs())


def test_scale_and_strided_views():
    """q, k, v as views of one token-major projection; d_o with heads outermost; a
    scale of its own."""
    B, n, H, G, W, S = 2, 200, 8, 2, 60, 4
    qkv = _rn(1, B, n, H + 2 * G, 128)
    q, k, v = qkv[:, :, :H], qkv[:, :, H:H + G].transpose(1, 2), qkv[:, :, H + G:].transpose(1, 2)
    d_o = _rn(2, B, H, n, 128).transpose(1, 2)
    d = pipeline.window_dims(B, n, n, 0, H, G, scale=0.2)
    buf = pipeline.WindowBuffers.allocate(d, W, S, backward=True)
    out, lse = pipeline.window_forward(buf, q, k, v)
    dq, dk, dv = pipeline.window_backward(buf, q, k, v, d_o)
    case = (B, n, n, 0, H, G, W, S, None)
    for b, o, l, bound, ((eq, bq), (ek, bk), (ev, bv)) in _expect(case, q, k, v, d_o, 0.2):
        ref.close("o", out[b], o, bound)
        ref.close_lse(lse[b], l)
        ref.close("dq", dq[b], eq, bq)
        ref.close("dk", dk[b], ek, bk)
        ref.close("dv", dv[b], ev, bv)


def test_backward_is_the_derivative():
    """dq, dk, dv against central differences of the 64-bit forward."""
    case = (1, 9, 14, 5, 2, 1, 4, 2, None)
    B, n_q, n_kv, pos0, H, G, W, S, _ = case
    q, k, v, d_o, _ = _inputs(case)
    buf = pipeline.WindowBuffers.allocate(pipeline.window_dims(B, n_q, n_kv, pos0, H, G), W, S,
                                          backward=True)
    pipeline.window_forward(buf, q, k, v)
    grads = pipeline.window_backward(buf, q, k, v, d_o)
    see = ref.visible(n_q, n_kv, pos0, W, S, n_kv, "cuda")

    def loss(xs):
        return float((ref.attention(xs[0][0], xs[1][0], xs[2][0], see, 1 / math.sqrt(128))[0] *
                      d_o[0].double()).sum())

    xs = [t.double() for t in (q, k, v)]
    bounds = [x[1] for x in next(_expect(case, q, k, v, d_o, 1 / math.sqrt(128)))[4]]
    bounds = [bounds[0], bounds[1], bounds[2]]
    e = 1e-4
    for which in range(3):
        flat, b = grads[which][0].reshape(-1), bounds[which].reshape(-1)
        for i in range(3, flat.numel(), 137):
            hi, lo = [x.clone() for x in xs], [x.clone() for x in xs]
            hi[which].view(-1)[i] += e
            lo[which].view(-1)[i] -= e
            num = (loss(hi) - loss(lo)) / (2 * e)
            assert abs(float(flat[i]) - num) <= float(b[i]) + 1e-6, (which, i)


def test_rows_far_above_the_first_maximum():
    """Later keys raise a row's maximum by far more than the rescaling threshold,
    others by less than it."""
    n, H = 1024, 4
    q, k, v = _rn(1, 1, n, H, 128), _rn(2, 1, 1, n, 128), _rn(3, 1, 1, n, 128)
    ramp = torch.linspace(0.2, 6.0, n, device="cuda")[:, None]
    k = (k.float() * ramp).to(BF)
    buf = pipeline.WindowBuffers.allocate(pipeline.window_dims(1, n, n, 0, H, 1))
    out, lse = pipeline.window_forward(buf, q, k, v)
    see = ref.visible(n, n, 0, 0, 0, n, "cuda")
    o, l, bound, _ = ref.attention(q[0], k[0], v[0], see, 1 / math.sqrt(128))
    ref.close("o", out[0], o, bound)
    ref.close_lse(lse[0], l)


def test_more_than_31_bits_of_elements():
    """2^31 elements of q and out: rows at both ends against the definition, forward and
    backward."""
    n, H, W = 262144 + 200, 64, 30
    q = torch.empty((1, n, H, 128), dtype=BF, device="cuda").normal_()
    k, v = _rn(2, 1, 4, n, 128), _rn(3, 1, 4, n, 128)
    buf = pipeline.WindowBuffers.allocate(pipeline.window_dims(1, n, n, 0, H, 4), W, 2,
                                          backward=True)
    out, lse = pipeline.window_forward(buf, q, k, v)
    d_o = q
    dq, dk, dv = pipeline.window_backward(buf, q, k, v, d_o)
    assert int(buf.dev_err[0]) == 0
    for i0 in (0, 131072, n - 40):
        # 40 queries, their window's keys and the two sinks
        lo = max(2, i0 - W + 1)
        keys = torch.cat([torch.arange(2), torch.arange(lo, i0 + 40)]).cuda()
        t = torch.arange(i0, i0 + 40, device="cuda")[:, None]
        see = (keys[None] <= t) & ((t - keys[None] < W) | (keys[None] < 2))
        sq, sk, sv = q[0, i0:i0 + 40], k[0][:, keys], v[0][:, keys]
        o, l, bound, aux = ref.attention(sq, sk, sv, see, 1 / math.sqrt(128))
        ref.close("o", out[0, i0:i0 + 40], o, bound)
        ref.close_lse(lse[0, i0:i0 + 40], l)
        (eq, bq), _, _ = ref.attention_grads(o, aux, d_o[0, i0:i0 + 40], see, 1 / math.sqrt(128), 4)
        ref.close("dq", dq[0, i0:i0 + 40], eq, bq)
    # the last keys are seen by the last queries alone
    i0 = n - 60
    keys = torch.arange(i0 - W + 1, n, device="cuda")
    t = torch.arange(i0, n, device="cuda")[:, None]
    see = (keys[None] <= t) & (t - keys[None] < W)
    sinks = torch.arange(2, device="cuda")
    see = torch.cat([torch.ones((60, 2), dtype=torch.bool, device="cuda"), see], 1)
    keys = torch.cat([sinks, keys])
    o, l, bound, aux = ref.attention(q[0, i0:], k[0][:, keys], v[0][:, keys], see, 1 / math.sqrt(128))
    _, (ek, bk), (ev, bv) = ref.attention_grads(o, aux, d_o[0, i0:], see, 1 / math.sqrt(128), 4)
    ref.close("dk", dk[0, :, -31:], ek[:, -31:], bk[:, -31:])
    ref.close("dv", dv[0, :, -31:], ev[:, -31:], bv[:, -31:])


def test_bad_length_is_reported_and_clamped():
    case = (2, 40, 100, 60, 4, 1, 0, 0, [100, 0])
    q, k, v, d_o, _ = _inputs(case, nan=False)
    buf = pipeline.WindowBuffers.allocate(pipeline.window_dims(2, 40, 100, 60, 4, 1))
    out, lse = pipeline.window_forward(buf, q, k, v,
                                       torch.tensor([101, -1], dtype=torch.int32, device="cuda"))
    assert int(buf.dev_err[0]) == 6                   # MSA_DEVERR_BAD_LENGTH
    for b, o, l, bound, _ in _expect(case, q, k, v, d_o, 1 / math.sqrt(128)):
        ref.close("o", out[b], o, bound)
        ref.close_lse(lse[b], l)


def test_captured_training_step():
    """Forward and backward captured into one graph, replayed on other inputs, beside
    a second capture that shares the workspace."""
    case = (2, 150, 250, 100, 8, 2, 70, 3, [250, 170])
    B, n_q, n_kv, pos0, H, G, W, S, lens = case
    q, k, v, d_o, kv_len = _inputs(case, nan=False)
    buf = pipeline.WindowBuffers.allocate(pipeline.window_dims(B, n_q, n_kv, pos0, H, G), W, S,
                                          backward=True)

    def step():
        pipeline.window_forward(buf, q, k, v, kv_len)
        pipeline.window_backward(buf, q, k, v, d_o, kv_len)

    step()
    torch.cuda.synchronize()
    graphs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]
    for g in graphs:
        with torch.cuda.graph(g):
            step()
    for t, s in ((q, 21), (k, 22), (v, 23), (d_o, 24)):
        t.copy_(_rn(s, *t.shape))
    for g in graphs:
        for t in (buf.out, buf.dq, buf.dk, buf.dv):
            t.fill_(7.0)
        g.replay()
        for b, o, l, bound, ((eq, bq), (ek, bk), (ev, bv)) in _expect(case, q, k, v, d_o,
                                                                     1 / math.sqrt(128)):
            ref.close("o", buf.out[b], o, bound)
            ref.close("dq", buf.dq[b], eq, bq)
            ref.close("dk", buf.dk[b], ek, bk)
            ref.close("dv", buf.dv[b], ev, bv)
    assert int(buf.dev_err[0]) == 0
