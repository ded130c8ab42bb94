"""Workloads of the operators around the sparse path: per-head norms of
queries and keys with the position rotation (dense, into a paged cache, and
backward), attention of one new token over a paged key-value cache, and
sliding-window attention with sink tokens (forward, and forward + backward).

``listed()`` gives the fixed cases, ``draw(rng)`` more of the same ranges;
``prepare`` makes a case's inputs on the GPU, ``run`` makes one pass, ``work``
counts what the pass cannot do without and ``exact`` evaluates the definition
in 64 bits.  With ``own`` false ``run`` computes the plain form from elementary
torch operations, with ``own`` true it calls the library.
"""
import math
import random

import torch

own = False

D = 128          # head dimension of the attention
EPS = 1e-6


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # the prefill of 32768 tokens with 32 / 8 heads: queries and keys between
        # the projections and the attention
        dict(name="norm_rope_prefill_32k", op="norm_rope", batch=1, n_tok=32768, h_q=32, h_k=8,
             d=128, rot=128, inter=False, pos0=0),
        # a decode step of 64 sequences, 64 / 8 heads: one new token each goes into
        # its page (latency counts)
        dict(name="append_decode_64", op="append", batch=64, n_tok=1, h_q=64, h_k=8, rot=128,
             inter=False, page=64, nhd=False, cap=4096, lens_seed=1, ragged=False),
        # chunks of unequal length for three sequences in one padded batch, small
        # pages with tokens outermost, partial rotation in adjacent pairs
        dict(name="append_chunk_ragged", op="append", batch=3, n_tok=1021, h_q=16, h_k=2, rot=64,
             inter=True, page=16, nhd=True, cap=6000, lens_seed=2, ragged=True),
        # training at 16384 tokens with 64 / 8 heads, bf16 gradients
        dict(name="norm_rope_bwd_16k", op="norm_rope_bwd", batch=1, n_tok=16384, h_q=64, h_k=8,
             d=128, rot=128, inter=False, pos0=0, dy32=False),
        # the index branch's 64-wide heads, one shared key head, fp32 gradients
        dict(name="norm_rope_bwd_index", op="norm_rope_bwd", batch=2, n_tok=2300, h_q=8, h_k=1,
             d=64, rot=32, inter=True, pos0=1000, dy32=True),
        # one sequence of about 4K tokens: the smallest decode step
        dict(name="decode_1x4k", op="decode", batch=1, h_q=64, h_kv=8, page=64, nhd=False,
             len_min=4093, len_max=4093, lens_seed=3, window=0, sink=0),
        # a serving batch: 64 sequences of very different lengths up to 32768
        dict(name="decode_64_ragged", op="decode", batch=64, h_q=64, h_kv=8, page=64, nhd=False,
             len_min=500, len_max=32768, lens_seed=4, window=0, sink=0),
        # a window layer of the same service: small pages, tokens outermost, 16
        # query heads to a key head, sinks beside the window
        dict(name="decode_window_37", op="decode", batch=37, h_q=32, h_kv=2, page=16, nhd=True,
             len_min=1, len_max=20000, lens_seed=5, window=4096, sink=64),
        # the 4096-token prefill with 4 heads on one key head
        dict(name="window_prefill_4k", op="window", batch=1, n_q=4096, n_kv=4096, h_q=4, h_kv=1,
             window=512, sink=0, ragged=False, lens_seed=6, train=False),
        # a window layer beside the sparse ones in the 32768-token prefill
        dict(name="window_prefill_32k", op="window", batch=1, n_q=32768, n_kv=32768, h_q=32,
             h_kv=8, window=4096, sink=64, ragged=False, lens_seed=7, train=False),
        # a training step (forward and backward) of the window layer at 8192 tokens
        dict(name="window_train_8k", op="window", batch=1, n_q=8192, n_kv=8192, h_q=64, h_kv=8,
             window=1024, sink=4, ragged=False, lens_seed=8, train=True),
        # the same for a padded batch of odd lengths behind a cached prefix
        dict(name="window_train_ragged", op="window", batch=3, n_q=1111, n_kv=2411, h_q=16,
             h_kv=2, window=257, sink=37, ragged=True, lens_seed=9, train=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_rope", "append", "norm_rope_bwd", "decode", "decode", "window", "window"])
    r = rng.choice([1, 2, 4, 8, 16])
    seed = rng.randrange(1 << 30)
    if op in ("norm_rope", "norm_rope_bwd"):
        d = rng.choice([64, 128])
        h_k = rng.choice([1, 2, 3, 4, 8])
        h_q = h_k * rng.choice([1, 2, 4, 8])
        n = min(_log(rng, 1, 65536), (1 << 20) // (h_q + h_k))
        batch = rng.choice([b for b in (1, 2, 3, 5) if b <= n])
        c = dict(op=op, batch=batch, n_tok=max(1, n // batch), h_q=h_q, h_k=h_k, d=d,
                 rot=rng.choice([16, 32, 64, d]), inter=rng.random() < 0.5,
                 pos0=rng.choice([0, rng.randrange(1, 100000)]))
        if op == "norm_rope_bwd":
            c["dy32"] = rng.random() < 0.5
        return c
    h_kv = rng.choice([1, 2, 4, 8])
    page = rng.choice([16, 32, 64, 128])
    if op == "append":
        n_tok = rng.choice([1, 1, _log(rng, 2, 2000)])
        batch = min(_log(rng, 1, 200), max(1, 20000 // n_tok))
        return dict(op=op, batch=batch, n_tok=n_tok, h_q=h_kv * r, h_k=h_kv,
                    rot=rng.choice([16, 64, 128]), inter=rng.random() < 0.5, page=page,
                    nhd=rng.random() < 0.5, cap=n_tok + _log(rng, 1, 2500), lens_seed=seed,
                    ragged=rng.random() < 0.5)
    window = rng.choice([0, _log(rng, 1, 8192)])
    sink = rng.choice([0, _log(rng, 1, 300)]) if window else 0
    if op == "decode":
        batch = _log(rng, 1, 128)
        hi = max(2, min(_log(rng, 2, 100000), (1 << 22) // (batch * h_kv)))
        return dict(op=op, batch=batch, h_q=h_kv * r, h_kv=h_kv, page=page,
                    nhd=rng.random() < 0.5, len_min=rng.choice([0, 1, hi // 2]), len_max=hi,
                    lens_seed=seed, window=window, sink=sink)
    train = rng.random() < 0.5
    h_kv = rng.choice([1, 2, 4])
    batch = rng.choice([1, 1, 2, 3])
    n_q = max(1, _log(rng, 1, 4096 if train else 8192) // batch)
    prefix = rng.choice([0, 0, _log(rng, 1, 4096)])
    return dict(op="window", batch=batch, n_q=n_q, n_kv=n_q + prefix, h_q=h_kv * r, h_kv=h_kv,
                window=window, sink=sink, ragged=rng.random() < 0.5, lens_seed=seed, train=train)


def _lens(c):
    """Tokens of each sequence: from the case alone, spread over the logarithm."""
    rng = random.Random(c["lens_seed"])
    if c["op"] == "decode":
        lo, hi = max(1, c["len_min"]), c["len_max"]
        out = [_log(rng, lo, hi) for _ in range(c["batch"])]
        if c["len_min"] == 0 and len(out) > 1:
            out[0] = 0              # a slot of the batch without a sequence
        return out
    if c["op"] == "append":          # (tokens cached before, tokens of this chunk)
        n = [rng.randint(1, c["n_tok"]) if c["ragged"] else c["n_tok"] for _ in range(c["batch"])]
        n[-1] = c["n_tok"]
        return [(rng.randint(0, c["cap"] - c["n_tok"]), x) for x in n]
    if not c["ragged"]:              # window
        return [c["n_kv"]] * c["batch"]
    return [rng.randint(0, c["n_kv"]) for _ in range(c["batch"] - 1)] + [c["n_kv"]]


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _rn(g, *shape, dtype=torch.bfloat16):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _table(n_pos, rot):
    """[n_pos, rot] fp32: rot / 2 cosines, then rot / 2 sines, from 64-bit angles."""
    inv = 1.0e6 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)
    ang = torch.arange(n_pos, device="cuda", dtype=torch.float64)[:, None] * inv[None, :]
    return torch.cat([ang.cos(), ang.sin()], dim=1).float()


def _page_table(g, batch, per_seq):
    perm = torch.randperm(batch * per_seq + 3, generator=g, device="cuda")[:batch * per_seq]
    return perm.view(batch, per_seq).to(torch.int32)


def _pages(g, n_pages, h, page, nhd):
    """Pages seen as [n_pages, h, page, 128], stored heads or tokens outermost."""
    if nhd:
        return _rn(g, n_pages, page, h, D).permute(0, 2, 1, 3)
    return _rn(g, n_pages, h, page, D)


def _raw(case, seed):
    g = _gen(seed)
    s, c = {}, case
    if c["op"] in ("norm_rope", "norm_rope_bwd"):
        s["q"] = _rn(g, c["batch"], c["n_tok"], c["h_q"], c["d"]) * 1.5
        s["k"] = _rn(g, c["batch"], c["n_tok"], c["h_k"], c["d"]) * 0.7
        s["w_q"] = 1.0 + 0.2 * _rn(g, c["d"], dtype=torch.float32)
        s["w_k"] = 1.0 + 0.2 * _rn(g, c["d"], dtype=torch.float32)
        s["table"] = _table(c["pos0"] + c["n_tok"], c["rot"])
        if c["op"] == "norm_rope_bwd":
            t = torch.float32 if c["dy32"] else torch.bfloat16
            s["d_q"] = _rn(g, c["batch"], c["n_tok"], c["h_q"], c["d"], dtype=t)
            s["d_k"] = _rn(g, c["batch"], c["h_k"], c["n_tok"], c["d"], dtype=t)
    elif c["op"] == "append":
        s["q"] = _rn(g, c["batch"], c["n_tok"], c["h_q"], D) * 1.5
        s["k"] = _rn(g, c["batch"], c["n_tok"], c["h_k"], D) * 0.7
        s["v"] = _rn(g, c["batch"], c["n_tok"], c["h_k"], D)
        s["w_q"] = 1.0 + 0.2 * _rn(g, D, dtype=torch.float32)
        s["w_k"] = 1.0 + 0.2 * _rn(g, D, dtype=torch.float32)
        s["table"] = _table(c["cap"], c["rot"])
        per = (c["cap"] + c["page"] - 1) // c["page"]
        s["block_table"] = _page_table(g, c["batch"], per)
        s["k_pages"] = _pages(g, c["batch"] * per + 3, c["h_k"], c["page"], c["nhd"])
        s["v_pages"] = _pages(g, c["batch"] * per + 3, c["h_k"], c["page"], c["nhd"])
        pos = [[a + i if i < n else -1 for i in range(c["n_tok"])] for a, n in _lens(c)]
        s["positions"] = torch.tensor(pos, dtype=torch.int64, device="cuda")
        s["seq_lens"] = torch.tensor([a + n for a, n in _lens(c)], dtype=torch.int32, device="cuda")
    elif c["op"] == "decode":
        s["lens"] = _lens(c)
        per = (max(s["lens"] + [1]) + c["page"] - 1) // c["page"]
        s["q"] = _rn(g, c["batch"], 1, c["h_q"], D)
        s["block_table"] = _page_table(g, c["batch"], per)
        s["k_pages"] = _pages(g, c["batch"] * per + 3, c["h_kv"], c["page"], c["nhd"])
        s["v_pages"] = _pages(g, c["batch"] * per + 3, c["h_kv"], c["page"], c["nhd"])
        s["seq_lens"] = torch.tensor(s["lens"], dtype=torch.int32, device="cuda")
    else:
        s["lens"] = _lens(c)
        s["q"] = _rn(g, c["batch"], c["n_q"], c["h_q"], D)
        s["k"] = _rn(g, c["batch"], c["h_kv"], c["n_kv"], D)
        s["v"] = _rn(g, c["batch"], c["h_kv"], c["n_kv"], D)
        if c["train"]:
            s["d_out"] = _rn(g, c["batch"], c["n_q"], c["h_q"], D)
        s["kv_len"] = None
        if c["ragged"]:
            s["kv_len"] = torch.tensor(s["lens"], dtype=torch.int32, device="cuda")
    return s


def prepare(case, seed):
    s = _raw(case, seed)
    s["case"] = case
    c = case
    if c["op"] == "append":
        s["q_out"] = torch.zeros_like(s["q"])      # rows of padded tokens stay zero
    if own:
        from block_sparse_attention_32_b200 import pipeline
        if c["op"] in ("norm_rope", "append", "norm_rope_bwd"):
            s["plan"] = pipeline.NormRope(s["table"], s["w_q"], s["w_k"], eps=EPS,
                                          interleaved=c["inter"])
        if c["op"] == "norm_rope":
            s["q_out"] = torch.empty_like(s["q"])
            s["k_out"] = torch.empty((c["batch"], c["h_k"], c["n_tok"], c["d"]),
                                     dtype=torch.bfloat16, device="cuda")
        elif c["op"] == "norm_rope_bwd":
            s["grads"] = pipeline.NormRopeGrads.allocate(s["q"], s["k"])
        elif c["op"] == "append":
            s["cache"] = pipeline.PagedCache(s["k_pages"], s["v_pages"], s["block_table"],
                                             s["seq_lens"])
        elif c["op"] == "decode":
            s["cache"] = pipeline.PagedCache(s["k_pages"], s["v_pages"], s["block_table"],
                                             s["seq_lens"])
            s["buf"] = pipeline.DecodeBuffers.allocate(s["cache"], c["h_q"])
        else:
            d = pipeline.window_dims(c["batch"], c["n_q"], c["n_kv"], c["n_kv"] - c["n_q"],
                                     c["h_q"], c["h_kv"])
            s["buf"] = pipeline.WindowBuffers.allocate(d, c["window"], c["sink"],
                                                       backward=c["train"])
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    c = s["case"]
    if own:
        from block_sparse_attention_32_b200 import pipeline
        if c["op"] == "norm_rope":
            return pipeline.norm_rope(s["plan"], s["q"], s["k"], s["q_out"], s["k_out"],
                                      pos0=c["pos0"])
        if c["op"] == "norm_rope_bwd":
            return pipeline.norm_rope_backward(s["plan"], s["q"], s["k"], s["d_q"], s["d_k"],
                                               s["grads"], pos0=c["pos0"])
        if c["op"] == "append":
            pipeline.norm_rope_append(s["plan"], s["q"], s["k"], s["v"], s["positions"],
                                      s["q_out"], s["cache"])
            return s["q_out"], s["k_pages"], s["v_pages"]
        if c["op"] == "decode":
            return pipeline.paged_decode(s["buf"], s["q"], s["cache"], window=c["window"],
                                         n_sink=c["sink"])
        out, lse = pipeline.window_forward(s["buf"], s["q"], s["k"], s["v"], s["kv_len"])
        if not c["train"]:
            return out, lse
        dq, dk, dv = pipeline.window_backward(s["buf"], s["q"], s["k"], s["v"], s["d_out"],
                                              s["kv_len"])
        return out, lse, dq, dk, dv
    return {"norm_rope": _norm_rope, "norm_rope_bwd": _norm_rope_bwd, "append": _append,
            "decode": _decode, "window": _window}[c["op"]](s, c)


def _cos_sin(s, c):
    """fp32 cosines and sines [B or 1, T, 1, rot / 2] of the case's tokens."""
    if c["op"] == "append":
        t = s["table"][s["positions"].clamp(min=0)]
    else:
        t = s["table"][c["pos0"]:c["pos0"] + c["n_tok"]][None]
    half = c["rot"] // 2
    return t[:, :, None, :half], t[:, :, None, half:]


def _rotate(y, cos, sin, rot, inter):
    out = y.clone()
    if inter:
        a, b = y[..., 0:rot:2], y[..., 1:rot:2]
        out[..., 0:rot:2] = a * cos - b * sin
        out[..., 1:rot:2] = b * cos + a * sin
    else:
        a, b = y[..., :rot // 2], y[..., rot // 2:rot]
        out[..., :rot // 2] = a * cos - b * sin
        out[..., rot // 2:rot] = b * cos + a * sin
    return out


def _norm_rotate(x, w, cos, sin, c):
    x = x.float()
    y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w
    return _rotate(y, cos, sin, c["rot"], c["inter"])


def _norm_rope(s, c):
    cos, sin = _cos_sin(s, c)
    q = _norm_rotate(s["q"], s["w_q"], cos, sin, c).to(torch.bfloat16)
    k = _norm_rotate(s["k"], s["w_k"], cos, sin, c).to(torch.bfloat16)
    return q, k.permute(0, 2, 1, 3).contiguous()


def _append(s, c):
    cos, sin = _cos_sin(s, c)
    live = s["positions"] >= 0
    q = _norm_rotate(s["q"], s["w_q"], cos, sin, c).to(torch.bfloat16)
    k = _norm_rotate(s["k"], s["w_k"], cos, sin, c).to(torch.bfloat16)
    s["q_out"].copy_(torch.where(live[:, :, None, None], q, s["q_out"]))
    b, i = live.nonzero(as_tuple=True)
    pos = s["positions"][b, i]
    page = s["block_table"][b, pos // c["page"]].long()
    s["k_pages"][page, :, pos % c["page"]] = k[b, i]
    s["v_pages"][page, :, pos % c["page"]] = s["v"][b, i]
    return s["q_out"], s["k_pages"], s["v_pages"]


def _norm_rope_bwd(s, c):
    cos, sin = _cos_sin(s, c)

    def one(x, w, dy):
        x, dy = x.float(), dy.float()
        r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
        xh = x * r
        dz = _rotate(dy, cos, -sin, c["rot"], c["inter"])
        dw = (dz * xh).sum((0, 1, 2), dtype=torch.float64).float()
        dxh = dz * w
        dx = r * (dxh - xh * (dxh * xh).mean(-1, keepdim=True))
        return dx.to(torch.bfloat16), dw

    dxq, dwq = one(s["q"], s["w_q"], s["d_q"])
    dxk, dwk = one(s["k"], s["w_k"], s["d_k"].permute(0, 2, 1, 3))
    return dxq, dxk, dwq, dwk


def _decode(s, c):
    G, R, page = c["h_kv"], c["h_q"] // c["h_kv"], c["page"]
    scale = D ** -0.5
    out = torch.zeros_like(s["q"])
    lse = torch.full((c["batch"], 1, c["h_q"]), -math.inf, device="cuda")
    for b, n in enumerate(s["lens"]):
        if n == 0:
            continue
        lo = max(0, n - c["window"]) if c["window"] else 0
        j = torch.arange(n, device="cuda")
        j = j[(j >= lo) | (j < c["sink"])]
        pg = s["block_table"][b].long()[j // page]
        k = s["k_pages"][pg, :, j % page].float()          # [keys, G, D]
        v = s["v_pages"][pg, :, j % page].float()
        q = s["q"][b, 0].float().view(G, R, D)
        z = torch.einsum("grd,kgd->grk", q, k) * scale
        m = z.amax(-1, keepdim=True)
        p = torch.exp(z - m)
        l = p.sum(-1, keepdim=True)
        o = torch.einsum("grk,kgd->grd", p, v) / l
        out[b, 0] = o.reshape(c["h_q"], D).to(torch.bfloat16)
        lse[b, 0] = (m + torch.log(l)).reshape(c["h_q"])
    return out, lse


def _window(s, c):
    """Chunks of queries against the keys that their windows and the sinks reach."""
    B, n_q, n_kv, H, G = c["batch"], c["n_q"], c["n_kv"], c["h_q"], c["h_kv"]
    R, W, S, pos0 = H // G, c["window"] or c["n_kv"], c["sink"], c["n_kv"] - c["n_q"]
    scale = D ** -0.5
    train = c["train"]
    out = torch.zeros_like(s["q"])
    lse = torch.full((B, n_q, H), -math.inf, device="cuda")
    if train:
        dq = torch.zeros_like(s["q"])
        dk = torch.zeros((B, G, n_kv, D), device="cuda")
        dv = torch.zeros((B, G, n_kv, D), device="cuda")
    step = 1024
    for b in range(B):
        for i0 in range(0, n_q, step):
            i1 = min(n_q, i0 + step, s["lens"][b] - pos0)
            if i1 <= i0:
                continue
            t = torch.arange(pos0 + i0, pos0 + i1, device="cuda")
            lo, hi = max(0, pos0 + i0 - W + 1), pos0 + i1
            j = torch.cat([torch.arange(min(S, lo), device="cuda"),
                           torch.arange(lo, hi, device="cuda")])
            see = (j[None] <= t[:, None]) & ((t[:, None] - j[None] < W) | (j[None] < S))
            see = see[None, :, None, :]                     # [1, T, 1, keys]
            T = i1 - i0
            q = s["q"][b, i0:i1].float().view(T, G, R, D).permute(1, 0, 2, 3)
            k, v = s["k"][b][:, j].float(), s["v"][b][:, j].float()
            q2 = q.reshape(G, T * R, D)
            z = (q2 @ k.transpose(1, 2) * scale).view(G, T, R, -1)
            z = torch.where(see, z, torch.full_like(z, -math.inf))
            m = z.amax(-1, keepdim=True)
            p = torch.exp(z - m)
            l = p.sum(-1, keepdim=True)
            p = p / l
            o = (p.view(G, T * R, -1) @ v).view(G, T, R, D)
            out[b, i0:i1] = o.permute(1, 0, 2, 3).reshape(T, H, D).to(torch.bfloat16)
            lse[b, i0:i1] = (m + torch.log(l))[..., 0].permute(1, 0, 2).reshape(T, H)
            if not train:
                continue
            do = s["d_out"][b, i0:i1].float().view(T, G, R, D).permute(1, 0, 2, 3)
            do2 = do.reshape(G, T * R, D)
            dp = (do2 @ v.transpose(1, 2)).view(G, T, R, -1)
            delta = (do * o).sum(-1, keepdim=True)
            ds = p * (dp - delta) * scale
            g = (ds.view(G, T * R, -1) @ k).view(G, T, R, D)
            dq[b, i0:i1] = g.permute(1, 0, 2, 3).reshape(T, H, D).to(torch.bfloat16)
            dk[b].index_add_(1, j, ds.view(G, T * R, -1).transpose(1, 2) @ q2)
            dv[b].index_add_(1, j, p.view(G, T * R, -1).transpose(1, 2) @ do2)
    if not train:
        return out, lse
    return out, lse, dq, dk.to(torch.bfloat16), dv.to(torch.bfloat16)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def _visible(first, last, W, S):
    """Sum over positions t = first .. last of the keys that t sees."""
    total = 0
    for a, b in ((first, min(last, W - 1)), (max(first, W), last)):
        if b < a:
            continue
        if b < W:                                   # every earlier key
            total += (a + 1 + b + 1) * (b - a + 1) // 2
        else:                                       # W recent ones and min(S, t - W + 1) sinks
            total += W * (b - a + 1)
            e = min(b, W + S - 1)                   # t - W + 1 <= S up to here
            if e >= a:
                total += (a - W + 1 + e - W + 1) * (e - a + 1) // 2
            total += S * max(0, b - max(a, e + 1) + 1)
    return total


def work(case):
    c = case
    if c["op"] in ("norm_rope", "norm_rope_bwd"):
        rows = c["batch"] * c["n_tok"] * (c["h_q"] + c["h_k"])
        tab = c["n_tok"] * c["rot"] * 4 + 2 * c["d"] * 4
        if c["op"] == "norm_rope":
            return {"bytes": rows * c["d"] * 4 + tab, "flops": rows * c["d"] * 7}
        per = 2 + (4 if c["dy32"] else 2) + 2
        return {"bytes": rows * c["d"] * per + tab + 2 * c["d"] * 4, "flops": rows * c["d"] * 14}
    if c["op"] == "append":
        tok = sum(n for _, n in _lens(c))
        rows = tok * (c["h_q"] + c["h_k"])
        return {"bytes": (rows + tok * c["h_k"]) * D * 4 + tok * (c["rot"] * 4 + 12) + 2 * D * 4,
                "flops": rows * D * 7}
    if c["op"] == "decode":
        keys = sum(n if not c["window"] or n <= c["window"]
                   else c["window"] + min(c["sink"], n - c["window"]) for n in _lens(c))
        return {"bytes": keys * c["h_kv"] * D * 4 + c["batch"] * c["h_q"] * (4 * D + 4)
                + (keys // c["page"] + c["batch"]) * 4, "flops": keys * c["h_q"] * D * 4}
    pos0, W = c["n_kv"] - c["n_q"], c["window"] or c["n_kv"]
    pairs = kv_rows = q_rows = 0
    for n in _lens(c):
        last = n - 1                                # queries pos0 .. last
        if last < pos0:
            continue
        pairs += _visible(pos0, last, W, c["sink"])
        lo = max(0, pos0 - W + 1)
        kv_rows += n - lo + min(c["sink"], lo)
        q_rows += last - pos0 + 1
    q_bytes, kv_bytes = q_rows * c["h_q"] * D * 2, kv_rows * c["h_kv"] * D * 2
    lse = c["batch"] * c["n_q"] * c["h_q"] * 4
    out_bytes = c["batch"] * c["n_q"] * c["h_q"] * D * 2
    if not c["train"]:
        return {"bytes": q_bytes + 2 * kv_bytes + out_bytes + lse,
                "flops": pairs * c["h_q"] * D * 4}
    kv_out = 2 * c["batch"] * c["h_kv"] * c["n_kv"] * D * 2
    return {"bytes": 2 * q_bytes + 2 * kv_bytes + 2 * out_bytes + lse + kv_out,
            "flops": pairs * c["h_q"] * D * 14}


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    c, s = case, _raw(case, seed)
    if c["op"] in ("norm_rope", "append", "norm_rope_bwd"):
        return _exact_norm_rope(c, s)
    if c["op"] == "decode":
        return _exact_decode(c, s)
    return _exact_window(c, s)


def _exact_norm_rope(c, s):
    """Feature pairs as complex numbers, turned by e^{i angle} (or back)."""
    rot, half = c["rot"], c["rot"] // 2
    idx = torch.arange(rot, device="cuda")
    if c["inter"]:
        first, second = idx[0::2], idx[1::2]
    else:
        first, second = idx[:half], idx[half:]
    if c["op"] == "append":
        pos = s["positions"].clamp(min=0)
    else:
        pos = (c["pos0"] + torch.arange(c["n_tok"], device="cuda"))[None].expand(c["batch"], -1)
    tab = s["table"].double()[pos]                            # [B, T, rot]
    turn = torch.complex(tab[..., :half], tab[..., half:])[:, :, None]

    def spin(y, by):
        y = y.clone()
        z = torch.complex(y[..., first], y[..., second]) * by
        y[..., first], y[..., second] = z.real, z.imag
        return y

    def forward(x, w):
        x = x.double()
        return spin(x / ((x ** 2).sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt() * w.double(),
                    turn)

    if c["op"] == "norm_rope":
        return forward(s["q"], s["w_q"]), forward(s["k"], s["w_k"]).transpose(1, 2).contiguous()
    if c["op"] == "append":
        q, k = forward(s["q"], s["w_q"]), forward(s["k"], s["w_k"])
        q[s["positions"] < 0] = 0.0
        kp, vp = s["k_pages"].double(), s["v_pages"].double()
        for b, (a, n) in enumerate(_lens(c)):
            at = a + torch.arange(n, device="cuda")
            pg = s["block_table"][b].long()[torch.div(at, c["page"], rounding_mode="floor")]
            kp[pg, :, at % c["page"]] = k[b, :n]
            vp[pg, :, at % c["page"]] = s["v"][b, :n].double()
        return q, kp, vp

    def backward(x, w, dy):
        x, w = x.double(), w.double()
        g = spin(dy.double(), turn.conj())
        n = ((x ** 2).sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt()
        dw = (g * x / n).flatten(0, 2).sum(0)
        gw = g * w
        return gw / n - x * (gw * x).sum(-1, keepdim=True) / (x.shape[-1] * n ** 3), dw

    dxq, dwq = backward(s["q"], s["w_q"], s["d_q"])
    dxk, dwk = backward(s["k"], s["w_k"], s["d_k"].transpose(1, 2))
    return dxq, dxk, dwq, dwk


def _exact_decode(c, s):
    G, R = c["h_kv"], c["h_q"] // c["h_kv"]
    out = torch.zeros((c["batch"], 1, c["h_q"], D), dtype=torch.float64, device="cuda")
    lse = torch.full((c["batch"], 1, c["h_q"]), -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(_lens(c)):
        keep = [j for j in range(n) if not c["window"] or n - 1 - j < c["window"] or j < c["sink"]]
        if not keep:
            continue
        j = torch.tensor(keep, device="cuda")
        pg = s["block_table"][b].long()[torch.div(j, c["page"], rounding_mode="floor")]
        for g in range(G):
            k = s["k_pages"][pg, g, j % c["page"]].double()
            v = s["v_pages"][pg, g, j % c["page"]].double()
            z = s["q"][b, 0, g * R:(g + 1) * R].double() @ k.T / math.sqrt(D)
            lse[b, 0, g * R:(g + 1) * R] = torch.logsumexp(z, -1)
            out[b, 0, g * R:(g + 1) * R] = torch.softmax(z, -1) @ v
    return out, lse


def _exact_window(c, s):
    """Whole rows of scores, 2048 queries of one head at a time."""
    n_q, n_kv, H, G = c["n_q"], c["n_kv"], c["h_q"], c["h_kv"]
    pos0, R = n_kv - n_q, H // G
    f = dict(dtype=torch.float64, device="cuda")
    out = torch.zeros((c["batch"], n_q, H, D), **f)
    lse = torch.full((c["batch"], n_q, H), -math.inf, **f)
    dq = torch.zeros((c["batch"], n_q, H, D), **f)
    dk = torch.zeros((c["batch"], G, n_kv, D), **f)
    dv = torch.zeros((c["batch"], G, n_kv, D), **f)
    j = torch.arange(n_kv, device="cuda")
    for b, n in enumerate(_lens(c)):
        for h in range(H):
            g = h // R
            k, v = s["k"][b, g].double(), s["v"][b, g].double()
            for i0 in range(0, n_q, 2048):
                i = torch.arange(i0, min(i0 + 2048, n_q), device="cuda")
                i = i[pos0 + i < n]
                if not len(i):
                    continue
                t = (pos0 + i)[:, None]
                hide = (j > t) | ((t - j >= (c["window"] or n_kv)) & (j >= c["sink"]))
                q = s["q"][b, i, h].double()
                z = (q @ k.T / math.sqrt(D)).masked_fill_(hide, -math.inf)
                le = torch.logsumexp(z, -1)
                p = torch.exp_(z - le[:, None])
                o = p @ v
                lse[b, i, h], out[b, i, h] = le, o
                if c["train"]:
                    do = s["d_out"][b, i, h].double()
                    dv[b, g] += p.T @ do
                    ds = p * (do @ v.T - (do * o).sum(-1, keepdim=True)) / math.sqrt(D)
                    dq[b, i, h] = ds @ k
                    dk[b, g] += ds.T @ q
    return (out, lse, dq, dk, dv) if c["train"] else (out, lse)
