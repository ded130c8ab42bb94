"""Plain 64-bit definitions of the operators around the sparse path, and the
error bounds their tests use.

Bounds count roundings.  u = 2^-8 is half a bf16 step relative to the value.
fp32 steps (2^-24 each) come to at most SMALL = 2^-14 relative for every sum
here: a score is 128 exact bf16 products added in fp32, |score error| <=
128 * 2^-24 * sum |q k| scale < 2^-14 for the tests' |q|, |k| of a few units, and
a softmax weight's relative error is that of its exponent.
  attention   P is rounded to bf16 for P V (u sum p |v|), the result once (u |o|).
  gradients   D = dO.o uses o as the forward left it: to 2^-17 with the kept bits, or
              rounded to bf16, |dD| <= sum |dO| (u_o |o| + u sum p |v|), u_o = 2^-16 or u;
              P and dS are rounded once each for their products.
All of these are worst cases per element; FRO bounds the relative Frobenius
error, where the (at most three) roundings of an element add up like random
signs: 3 u < 2^-6.
"""
import math

import torch

U = 2.0 ** -8
SMALL = 2.0 ** -14
FRO = 2.0 ** -6
LSE_ABS = 1e-4


def visible(n_q, n_kv, pos0, window, sink, kv_len, device):
    """[n_q, n_kv] truth table of one sequence."""
    t = pos0 + torch.arange(n_q, device=device)[:, None]
    j = torch.arange(n_kv, device=device)[None]
    see = (j <= t) & (t < kv_len)
    if window:
        see &= (t - j < window) | (j < sink)
    return see


def attention(q, k, v, see, scale):
    """One sequence: q [n_q,H,D], k, v [G,n_kv,D], see [n_q,n_kv].  Returns o, lse and
    the bound of o's error (rows that see nothing: 0, -inf)."""
    H, G = q.shape[1], k.shape[0]
    R = H // G
    q, k, v = q.double(), k.double(), v.double()
    # masked places may hold anything (NaN too): they are not part of the sums
    dead_k = ~see.any(0)
    k, v = k.clone(), v.clone()
    k[:, dead_k], v[:, dead_k] = 0.0, 0.0
    q = torch.where(see.any(1)[:, None, None], q, torch.zeros_like(q))
    kk, vv = k.repeat_interleave(R, 0), v.repeat_interleave(R, 0)     # [H, n_kv, D]
    s = torch.einsum("ihd,hjd->hij", q, kk) * scale
    s = s.masked_fill(~see[None], -math.inf)
    lse = torch.logsumexp(s, -1)                                      # [H, n_q]
    p = torch.exp(s - lse.masked_fill(lse == -math.inf, 0.0)[..., None])
    o = torch.einsum("hij,hjd->ihd", p, vv)
    av = torch.einsum("hij,hjd->ihd", p, vv.abs())
    bound = U * o.abs() + (U + SMALL) * av
    return o, lse.T, bound, (p, av, q, kk, vv)


def attention_grads(o, aux, d_o, see, scale, G, u_o=2.0 ** -16):
    """dq, dk, dv of one sequence and their bounds."""
    p, av, q, kk, vv = aux
    H = q.shape[1]
    R = H // G
    d_o = torch.where(see.any(1)[:, None, None], d_o.double(), torch.zeros_like(d_o.double()))
    dp = torch.einsum("ihd,hjd->hij", d_o, vv)
    D = (d_o * o).sum(-1).T                                           # [H, n_q]
    eD = (d_o.abs() * (u_o * o.abs() + U * av)).sum(-1).T
    ds = p * (dp - D[..., None])
    adp = torch.einsum("ihd,hjd->hij", d_o.abs(), vv.abs())
    eds = U * ds.abs() + p * (eD[..., None] * (1 + U) + SMALL * (adp + D.abs()[..., None]))

    def groups(x):                                                    # [H, n_kv, D] -> [G, ...]
        return x.view(G, R, *x.shape[1:]).sum(1)

    dq = scale * torch.einsum("hij,hjd->ihd", ds, kk)
    dk = scale * groups(torch.einsum("hij,ihd->hjd", ds, q))
    dv = groups(torch.einsum("hij,ihd->hjd", p, d_o))
    bq = U * dq.abs() + 1.01 * scale * torch.einsum("hij,hjd->ihd", eds, kk.abs())
    bk = U * dk.abs() + 1.01 * scale * groups(torch.einsum("hij,ihd->hjd", eds, q.abs()))
    bv = U * dv.abs() + (U + SMALL) * groups(torch.einsum("hij,ihd->hjd", p, d_o.abs()))
    return (dq, bq), (dk, bk), (dv, bv)


def close(name, got, want, bound, fro=True):
    got = got.double()
    assert torch.isfinite(got).all(), f"{name}: not finite"
    err = (got - want).abs()
    over = err - (bound + 1e-30)
    assert (over <= 0).all(), (name, float(over.max()), float(err.max()),
                               tuple(int(x) for x in (over > 0).nonzero()[0]))
    if fro and want.norm() > 0:
        rel = float((got - want).norm() / want.norm())
        assert rel <= FRO, (name, rel)


def close_lse(got, want):
    empty = want == -math.inf
    assert torch.equal(got == -math.inf, empty)
    d = (got.double() - want)[~empty].abs()
    assert d.numel() == 0 or float(d.max()) <= LSE_ABS, float(d.max())


# ---------------------------------------------------------------------------
# norm + rotation
# ---------------------------------------------------------------------------
def angles(table, pos):
    """64-bit cosines and sines [B, T, 1, rot / 2] from the fp32 table."""
    t = table.double()[pos.clamp(min=0)]
    half = table.shape[1] // 2
    return t[:, :, None, :half], t[:, :, None, half:]


def rotate(y, cos, sin, inter):
    rot = 2 * cos.shape[-1]
    out = y.clone()
    if rot == 0:
        return out
    a, b = (y[..., 0:rot:2], y[..., 1:rot:2]) if inter else (y[..., :rot // 2],
                                                             y[..., rot // 2:rot])
    na, nb = a * cos - b * sin, b * cos + a * sin
    if inter:
        out[..., 0:rot:2], out[..., 1:rot:2] = na, nb
    else:
        out[..., :rot // 2], out[..., rot // 2:rot] = na, nb
    return out


def norm_rope(x, w, cos, sin, inter, eps):
    """y and the bound of its error: one bf16 rounding, and fp32 steps against the
    row's largest feature (a rotated feature can be the difference of two)."""
    x = x.double()
    xh = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    y = rotate(xh if w is None else xh * w.double(), cos, sin, inter)
    return y, U * y.abs() + 2.0 ** -17 * y.abs().amax(-1, keepdim=True)


def norm_rope_bwd(x, w, dy, cos, sin, inter, eps, live):
    """dx, its bound, dw, its bound; live [B, T]: tokens that count."""
    x, dy = x.double(), dy.double()
    r = 1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    xh = x * r
    dz = rotate(dy, cos, -sin, inter)
    dxh = dz if w is None else dz * w.double()
    m = (dxh * xh).mean(-1, keepdim=True)
    dx = r * (dxh - xh * m)
    am = (dxh * xh).abs().mean(-1, keepdim=True)
    bx = U * dx.abs() + 2.0 ** -17 * r * (dxh.abs().amax(-1, keepdim=True) + xh.abs() * am)
    t = (dz * xh) * live[:, :, None, None]
    # a lane's rows, a block's 32 lanes and the blocks one after the other: under 1024 terms
    return dx, bx, t.sum((0, 1, 2)), 2.0 ** -14 * t.abs().sum((0, 1, 2))
