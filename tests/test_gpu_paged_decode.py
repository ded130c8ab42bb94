"""Attention of one new token over a paged cache on the GPU against the 64-bit
definition; bounds are derived in _layer_ref.py."""
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


def _cache(lens, h, page, nhd=False, extra_pages=1, seed=3):
    """Shuffled pages; NaN in every place that no sequence owns, -7 for every table
    entry that no sequence needs."""
    B = len(lens)
    per = (max(lens + [1]) + page - 1) // page + extra_pages
    n = sum((x + page - 1) // page for x in lens) + 2
    shape = (n, page, h, 128) if nhd else (n, h, page, 128)
    kp, vp = _rn(seed, *shape), _rn(seed + 1, *shape)
    if nhd:
        kp, vp = kp.permute(0, 2, 1, 3), vp.permute(0, 2, 1, 3)
    g = torch.Generator().manual_seed(seed)
    perm = torch.randperm(n, generator=g).int()
    table = torch.full((B, per), -7, dtype=torch.int32)
    own = torch.zeros((n, page), dtype=torch.bool)
    at = 0
    for b, x in enumerate(lens):
        m = (x + page - 1) // page
        table[b, :m] = perm[at:at + m]
        for j in range(m):
            own[perm[at + j].long(), :min(page, x - j * page)] = True
        at += m
    dead = ~own.cuda()
    kp.permute(0, 2, 1, 3)[dead] = math.nan
    vp.permute(0, 2, 1, 3)[dead] = math.nan
    return pipeline.PagedCache(kp, vp, table.cuda(),
                               torch.tensor(lens, dtype=torch.int32, device="cuda"))


def _check(cache, lens, q, out, lse, window, sink, scale=None):
    page = cache.k_pages.shape[2]
    scale = 1 / math.sqrt(128) if scale is None else scale
    for b, n in enumerate(lens):
        if n == 0:
            assert not out[b].any() and (lse[b] == -math.inf).all()
            continue
        j = torch.arange(n, device="cuda")
        pg = cache.block_table[b].long()[j // page]
        k = cache.k_pages[pg, :, j % page].transpose(0, 1)
        v = cache.v_pages[pg, :, j % page].transpose(0, 1)
        see = ref.visible(1, n, n - 1, window, sink, n, "cuda")
        o, l, bound, _ = ref.attention(q[b], k, v, see, scale)
        ref.close(f"o[{b}]", out[b], o, bound, fro=n > 1)
        ref.close_lse(lse[b], l)


# lengths, query heads, KV heads, page, tokens outermost, window, sinks
CASES = [
    ([1], 1, 1, 16, False, 0, 0),
    ([0, 1, 2, 0, 31, 32, 33, 0], 4, 2, 16, True, 0, 0),
    ([17, 0, 64, 65, 127], 16, 1, 32, False, 0, 0),
    ([1000, 3, 513], 64, 8, 64, False, 0, 0),
    ([4093], 64, 8, 64, False, 0, 0),
    ([9000, 1, 70], 8, 8, 128, True, 0, 0),
    ([700, 699, 32, 5], 32, 2, 16, True, 64, 0),
    ([700, 699, 32, 5], 32, 2, 16, False, 1, 0),
    ([700, 699, 32, 5, 0], 2, 1, 64, False, 100, 7),
    ([2500, 300, 64], 16, 4, 16, True, 257, 33),
    ([2500, 300, 64], 16, 4, 256, False, 257, 1000),
    ([513] * 40, 8, 1, 32, False, 0, 0),
    ([33000, 5, 2000], 32, 4, 64, True, 0, 0),
]


@pytest.mark.parametrize("lens,hq,hkv,page,nhd,window,sink", CASES)
def test_decode_matches_the_definition(lens, hq, hkv, page, nhd, window, sink):
    cache = _cache(lens, hkv, page, nhd)
    q = _rn(1, len(lens), 1, hq, 128)
    buf = pipeline.DecodeBuffers.allocate(cache, hq)
    buf.ws.fill_(-1)                                   # contents on entry do not matter
    out, lse = pipeline.paged_decode(buf, q, cache, window, sink)
    first = out.clone(), lse.clone()
    _check(cache, lens, q, out, lse, window, sink)
    assert int(buf.dev_err[0]) == 0
    pipeline.paged_decode(buf, q, cache, window, sink)
    assert torch.equal(out, first[0]) and torch.equal(lse, first[1])


def test_pages_outside_the_window_need_not_be_mapped():
    lens, page = [1000, 640], 32
    cache = _cache(lens, 2, page)
    want = pipeline.paged_decode(pipeline.DecodeBuffers.allocate(cache, 8), _rn(1, 2, 1, 8, 128),
                                 cache, 100, 40)
    cache.block_table[0, 2:28] = -1                    # tokens 64 .. 895: neither sink nor window
    cache.block_table[1, 2:16] = 1 << 30
    buf = pipeline.DecodeBuffers.allocate(cache, 8)
    got = pipeline.paged_decode(buf, _rn(1, 2, 1, 8, 128), cache, 100, 40)
    assert int(buf.dev_err[0]) == 0
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_bad_pages_and_lengths_are_reported():
    lens, page = [100, 64], 16
    cache = _cache(lens, 2, page)
    q = _rn(1, 2, 1, 4, 128)
    buf = pipeline.DecodeBuffers.allocate(cache, 4)
    good = [t.clone() for t in pipeline.paged_decode(buf, q, cache)]
    cache.block_table[0, 3] = cache.k_pages.shape[0]   # tokens 48 .. 63 of sequence 0
    out, lse = pipeline.paged_decode(buf, q, cache)
    assert int(buf.dev_err[0]) == 5                    # MSA_DEVERR_BAD_PAGE
    assert torch.equal(out[1], good[0][1]) and torch.isfinite(out.float()).all()
    # the page's tokens count as not visible
    j = torch.cat([torch.arange(48), torch.arange(64, 100)]).cuda()
    pg = cache.block_table[0].long()[j // page]
    k = cache.k_pages[pg, :, j % page].transpose(0, 1)
    v = cache.v_pages[pg, :, j % page].transpose(0, 1)
    see = torch.ones((1, len(j)), dtype=torch.bool, device="cuda")
    o, l, bound, _ = ref.attention(q[0], k, v, see, 1 / math.sqrt(128))
    ref.close("o", out[0], o, bound)
    ref.close_lse(lse[0], l)
    buf.dev_err.zero_()
    cache = _cache(lens, 2, page, extra_pages=0)
    buf = pipeline.DecodeBuffers.allocate(cache, 4)
    cap = cache.capacity
    cache.seq_lens.copy_(torch.tensor([-3, cap + 1], dtype=torch.int32))
    cache.block_table[1, :] = cache.block_table[0, :1]
    cache.k_pages.nan_to_num_(0.0)
    cache.v_pages.nan_to_num_(0.0)
    out, lse = pipeline.paged_decode(buf, q, cache)
    assert int(buf.dev_err[0]) == 6                    # MSA_DEVERR_BAD_LENGTH
    assert not out[0].any() and (lse[0] == -math.inf).all()
    _check(cache, [0, cap], q, out, lse, 0, 0)


def test_masked_by_infinite_scores_and_large_values():
    """Scores far apart: the running maximum jumps by more than the fp32 range of
    the weights, forwards and backwards."""
    lens, page = [300], 64
    cache = _cache(lens, 1, page)
    q = _rn(1, 1, 1, 2, 128)
    j = torch.arange(300, device="cuda")
    pg = cache.block_table[0].long()[j // page]
    k = cache.k_pages[pg, 0, j % page].float()
    k[200] = 40.0 * q[0, 0, 0].float()
    k[50] = -40.0 * q[0, 0, 1].float()
    cache.k_pages[pg, 0, j % page] = k.to(BF)
    buf = pipeline.DecodeBuffers.allocate(cache, 2)
    out, lse = pipeline.paged_decode(buf, q, cache)
    v = cache.v_pages[pg, :, j % page].transpose(0, 1)
    see = torch.ones((1, 300), dtype=torch.bool, device="cuda")
    o, l, bound, _ = ref.attention(q[0], k.to(BF)[None], v, see, 1 / math.sqrt(128))
    ref.close("o", out[0], o, bound + 1e-3 * bound)
    # scores near 450: fp32 keeps them to 2^-24 * 450 * a few roundings
    assert float((lse[0].double() - l).abs().max()) <= 450 * 2.0 ** -20


def test_captured_call_follows_lengths_and_streams():
    """A captured decode step replays with other queries, lengths and tables; a call
    on a side stream gives the same bits."""
    lens = [500, 40, 1200]
    cache = _cache(lens, 4, 64)
    q = _rn(1, 3, 1, 16, 128)
    buf = pipeline.DecodeBuffers.allocate(cache, 16)
    pipeline.paged_decode(buf, q, cache)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pipeline.paged_decode(buf, q, cache)
    new = [37, 0, 1100]
    q.copy_(_rn(8, 3, 1, 16, 128))
    cache.seq_lens.copy_(torch.tensor(new, dtype=torch.int32))
    g.replay()
    _check(cache, new, q, buf.out, buf.lse, 0, 0)
    other = pipeline.DecodeBuffers.allocate(cache, 16)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        pipeline.paged_decode(other, q, cache)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(other.out, buf.out) and torch.equal(other.lse, buf.lse)


def test_cache_beyond_31_bits_of_elements():
    """Pages past 2^31 elements (4.3 GB each of K and V)."""
    page, h = 128, 8
    n = (1 << 31) // (page * h * 128) + 5
    kp = torch.empty((n, h, page, 128), dtype=BF, device="cuda")
    vp = torch.empty((n, h, page, 128), dtype=BF, device="cuda")
    kp[-4:], vp[-4:] = _rn(1, 4, h, page, 128), _rn(2, 4, h, page, 128)
    table = torch.tensor([[n - 1, n - 3, n - 2, n - 4]], dtype=torch.int32, device="cuda")
    cache = pipeline.PagedCache(kp, vp, table, torch.tensor([450], dtype=torch.int32,
                                                            device="cuda"))
    q = _rn(3, 1, 1, 32, 128)
    buf = pipeline.DecodeBuffers.allocate(cache, 32)
    out, lse = pipeline.paged_decode(buf, q, cache)
    _check(cache, [450], q, out, lse, 0, 0)
    plan = pipeline.NormRope(pipeline.rope_table(512, 128))
    k, v = _rn(4, 1, 1, h, 128), _rn(5, 1, 1, h, 128)
    pipeline.norm_rope_append(plan, None, k, v, torch.tensor([[450]], device="cuda"), None, cache)
    assert torch.equal(vp[n - 4, :, 450 - 384], v[0, 0])
