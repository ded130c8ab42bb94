"""The operators around the sparse path run together, as a model and a server use
them: norm + rotation into attention and back, and a prefill into a paged cache
followed by decode steps.

Every step rounds its results to bf16 once (u = 2^-8 relative); a chain of at most
eight such roundings, added up like random signs and taken at their worst case,
stays under 8 u = 2^-5 relative in the Frobenius norm."""
import math

import pytest
import torch

import _layer_ref as ref
from block_sparse_attention_32_b200 import pipeline, workloads as wl

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
CHAIN = 2.0 ** -5


def _rn(seed, *shape, dtype=BF):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


def _rel(got, want):
    return float((got.double() - want).norm() / want.norm())


def test_training_layer_against_autograd():
    """x_q, x_k -> norm + rotation -> window attention -> loss, and all gradients,
    against 64-bit autograd of the whole."""
    B, n, H, G, W, S, rot = 2, 190, 8, 2, 60, 3, 64
    xq, xk, v, d_o = _rn(1, B, n, H, 128), _rn(2, B, n, G, 128), _rn(3, B, G, n, 128), _rn(4, B, n, H, 128)
    table = pipeline.rope_table(n, rot)
    wq, wk = 1 + 0.2 * _rn(5, 128, dtype=torch.float32), 1 + 0.2 * _rn(6, 128, dtype=torch.float32)
    plan = pipeline.NormRope(table, wq, wk)
    buf = pipeline.WindowBuffers.allocate(pipeline.window_dims(B, n, n, 0, H, G), W, S, backward=True)
    gr = pipeline.NormRopeGrads.allocate(xq, xk)
    q, k = pipeline.norm_rope(plan, xq, xk)
    out, _ = pipeline.window_forward(buf, q, k, v)
    dq, dk, dv = pipeline.window_backward(buf, q, k, v, d_o)
    dxq, dxk, dwq, dwk = pipeline.norm_rope_backward(plan, xq, xk, dq, dk, gr)

    leaves = [t.double().requires_grad_() for t in (xq, xk, v, wq, wk)]
    fq, fk, fv, fwq, fwk = leaves
    pos = torch.arange(n, device="cuda")[None].expand(B, -1)
    cos, sin = ref.angles(table, pos)

    def rope(x, w):
        y = x / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w
        a, b = y[..., :rot // 2], y[..., rot // 2:rot]
        return torch.cat([a * cos - b * sin, b * cos + a * sin, y[..., rot:]], -1)

    yq, yk = rope(fq, fwq), rope(fk, fwk)
    kk = yk.transpose(1, 2).repeat_interleave(H // G, 1)
    vv = fv.repeat_interleave(H // G, 1)
    s = torch.einsum("bihd,bhjd->bhij", yq, kk) / math.sqrt(128)
    see = ref.visible(n, n, 0, W, S, n, "cuda")
    o = torch.einsum("bhij,bhjd->bihd", torch.softmax(s.masked_fill(~see, -math.inf), -1), vv)
    (o * d_o.double()).sum().backward()
    assert _rel(out, o.detach()) <= CHAIN
    for got, leaf in zip((dxq, dxk, dv, dwq, dwk), leaves):
        assert _rel(got, leaf.grad) <= CHAIN
    assert int(buf.dev_err[0]) == 0


def test_norms_before_and_after_the_sparse_attention():
    """The rotated queries and keys feed the sparse attention; its fp32 gradients go
    back through the norm unchanged in type."""
    w = wl.small("chain_sparse", 1, 700, 700, 0, 8, 2, 64, seed=31)
    d = pipeline.dims_for(w)
    xq, xk = _rn(1, 1, 700, 8, 128), _rn(2, 1, 700, 2, 128)
    v, d_out = _rn(3, 1, 2, 700, 128), _rn(4, 1, 700, 8, 128)
    plan = pipeline.NormRope(pipeline.rope_table(700, 128))
    q, k = pipeline.norm_rope(plan, xq, xk)
    buf, grads = pipeline.Buffers.allocate(d), pipeline.Grads.allocate(d)
    sel = wl.random_selection(w, "cuda")
    pipeline.attend(buf, q, k, v, sel=sel)
    out = buf.out
    dq, dk, dv = pipeline.backward(buf, grads, q, k, v, d_out)
    assert dq.dtype == torch.float32 and dk.dtype == torch.float32
    # 700 tokens are six blocks: all of them selected, so this is full causal attention
    win = pipeline.WindowBuffers.allocate(pipeline.window_dims(1, 700, 700, 0, 8, 2, scale=w.scale),
                                          backward=True)
    o2, _ = pipeline.window_forward(win, q, k, v)
    dq2, dk2, dv2 = pipeline.window_backward(win, q, k, v, d_out)
    assert _rel(out, o2.double()) <= CHAIN
    for a, b in ((dq, dq2), (dk, dk2), (dv, dv2)):
        assert _rel(a, b.double()) <= CHAIN
    gr, gr2 = pipeline.NormRopeGrads.allocate(xq, xk), pipeline.NormRopeGrads.allocate(xq, xk)
    a = pipeline.norm_rope_backward(plan, xq, xk, dq, dk, gr)
    b = pipeline.norm_rope_backward(plan, xq, xk, dq2, dk2, gr2)
    for x, y in zip(a, b):
        if x is not None:
            assert _rel(x, y.double()) <= CHAIN


@pytest.mark.parametrize("window,sink,nhd", [(0, 0, False), (50, 6, True)])
def test_prefill_into_pages_then_decode(window, sink, nhd):
    """Two prompts go into the cache in two padded chunks, then tokens are decoded one by
    one: each step's attention equals dense window attention over the same keys."""
    B, H, G, page = 2, 16, 2, 16
    prompt, steps = [75, 40], 4
    cache = pipeline.PagedCache.allocate(B, 96, G, page_size=page, tokens_outermost=nhd)
    plan = pipeline.NormRope(pipeline.rope_table(96, 128), 1 + 0.1 * _rn(9, 128, dtype=torch.float32))
    n_all = [p + steps for p in prompt]
    xq, xk, xv = _rn(1, B, 96, H, 128), _rn(2, B, 96, G, 128), _rn(3, B, 96, G, 128)
    dense_q, dense_k = pipeline.norm_rope(plan, xq, xk)
    dense_v = xv.transpose(1, 2).contiguous()

    def append(at, n):                                  # n[b] tokens from at[b] on
        T = max(n)
        pos = torch.tensor([[at[b] + i if i < n[b] else -1 for i in range(T)] for b in range(B)],
                           device="cuda")
        take = lambda x: torch.stack([x[b, at[b]:at[b] + T] if at[b] + T <= 96 else
                                      torch.cat([x[b, at[b]:], x[b, :at[b] + T - 96]])
                                      for b in range(B)])
        q = pipeline.norm_rope_append(plan, take(xq), take(xk), take(xv), pos, None, cache)
        cache.seq_lens.copy_(torch.tensor([at[b] + n[b] for b in range(B)], dtype=torch.int32))
        return q

    append([0, 0], [50, 40])
    append([50, 40], [25, 0])
    buf = pipeline.DecodeBuffers.allocate(cache, H)
    for i in range(steps):
        at = [p + i for p in prompt]
        q = append(at, [1, 1])
        out, lse = pipeline.paged_decode(buf, q, cache, window, sink)
        for b in range(B):
            n = at[b] + 1
            assert torch.equal(q[b, 0], dense_q[b, at[b]])
            see = ref.visible(1, n, n - 1, window, sink, n, "cuda")
            o, l, bound, _ = ref.attention(q[b], dense_k[b, :, :n], dense_v[b, :, :n], see,
                                           1 / math.sqrt(128))
            ref.close("decode", out[b], o, bound)
            ref.close_lse(lse[b], l)
    assert int(buf.dev_err[0]) == 0
    # the last step's rows as part of one dense call over the padded batch
    n_kv = max(n_all)
    win = pipeline.WindowBuffers.allocate(pipeline.window_dims(B, n_kv, n_kv, 0, H, G), window, sink)
    kv_len = torch.tensor(n_all, dtype=torch.int32, device="cuda")
    o_dense, _ = pipeline.window_forward(win, dense_q[:, :n_kv], dense_k[:, :, :n_kv],
                                         dense_v[:, :, :n_kv], kv_len)
    for b in range(B):
        assert _rel(out[b, 0], o_dense[b, n_all[b] - 1].double()) <= CHAIN


def _step(seed, n=700, H=16, G=2):
    """A layer's training step with buffers of its own: returns (run, outputs)."""
    plan = pipeline.NormRope(pipeline.rope_table(n, 64), 1 + 0.1 * _rn(seed, 128, dtype=torch.float32))
    xq, xk, do = _rn(seed + 1, 2, n, H, 128), _rn(seed + 2, 2, n, G, 128), _rn(seed + 3, 2, n, H, 128)
    v = _rn(seed + 4, 2, G, n, 128)
    q, k = torch.empty_like(xq), torch.empty_like(v)
    win = pipeline.WindowBuffers.allocate(pipeline.window_dims(2, n, n, 0, H, G), 300, 5, backward=True)
    grads = pipeline.NormRopeGrads.allocate(xq, xk)

    def run():
        pipeline.norm_rope(plan, xq, xk, q, k)
        pipeline.window_forward(win, q, k, v)
        pipeline.window_backward(win, q, k, v, do)
        pipeline.norm_rope_backward(plan, xq, xk, win.dq, win.dk, grads)

    return run, [q, k, win.out, win.lse, win.dv, grads.dx_q, grads.dx_k, grads.dw_q, win.dev_err]


def _decode(seed, B=5, H=32, G=4):
    cache = pipeline.PagedCache.allocate(B, 5000, G, page_size=32)
    cache.k_pages.copy_(_rn(seed, *cache.k_pages.shape))
    cache.v_pages.copy_(_rn(seed + 1, *cache.v_pages.shape))
    cache.seq_lens.copy_(torch.tensor([1, 4999, 0, 317, 2048], dtype=torch.int32))
    buf, q = pipeline.DecodeBuffers.allocate(cache, H), _rn(seed + 2, B, 1, H, 128)
    return (lambda: pipeline.paged_decode(buf, q, cache)), [buf.out, buf.lse, buf.dev_err]


def _chunk(seed, n=24, n_kv=5000, H=16, G=2):
    """A few queries over a long context: CTAs share a row tile."""
    q, k, v = _rn(seed, 1, n, H, 128), _rn(seed + 1, 1, G, n_kv, 128), _rn(seed + 2, 1, G, n_kv, 128)
    win = pipeline.WindowBuffers.allocate(pipeline.window_dims(1, n, n_kv, n_kv - n, H, G))
    return (lambda: pipeline.window_forward(win, q, k, v)), [win.out, win.lse, win.dev_err]


@pytest.mark.parametrize("captured", [False, True])
def test_steps_side_by_side_on_streams(captured):
    """Training steps, decode steps and a chunk, each with buffers of its own, run over each
    other on five streams, eagerly or as replayed graphs: the bits of a lone run."""
    jobs = [_step(10), _decode(20), _step(30), _chunk(50), _decode(40)]
    alone = []
    for run, outs in jobs:
        run()
        torch.cuda.synchronize()
        alone.append([o.clone() for o in outs])
        for o in outs:
            o.fill_(77)
        outs[-1].zero_()                                # dev_err
    runs = [run for run, _ in jobs]
    if captured:
        graphs = []
        for run in runs:
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                run()
            graphs.append(g)
        runs = [g.replay for g in graphs]
    streams = [torch.cuda.Stream() for _ in jobs]
    torch.cuda.synchronize()
    for _ in range(5):
        for run, s in zip(runs, streams):
            with torch.cuda.stream(s):
                run()
    torch.cuda.synchronize()
    for (_, outs), want in zip(jobs, alone):
        assert int(outs[-1][0]) == 0
        for o, w in zip(outs, want):
            assert torch.equal(o, w)
