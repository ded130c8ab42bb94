"""Errors that the kernels of the operators around the sparse path report, where callers
hand in no place for them."""
import pytest
import torch

from block_sparse_attention_32_b200 import capi, pipeline

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def _rn(seed, *shape):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").to(BF)


def test_an_append_to_an_unmapped_page_is_found():
    cache = pipeline.PagedCache.allocate(2, 48, 2, page_size=16)
    plan = pipeline.NormRope(pipeline.rope_table(64, 64))
    q, k, v = _rn(1, 2, 3, 4, 128), _rn(2, 2, 3, 2, 128), _rn(3, 2, 3, 2, 128)
    pos = torch.tensor([[15, 16, 17], [0, 1, 2]], device="cuda")
    pipeline.norm_rope_append(plan, q, k, v, pos, None, cache)
    pipeline.check_device_errors(cache)
    cache.block_table[0, 1] = -1
    pipeline.norm_rope_append(plan, q, k, v, pos, None, cache)
    with pytest.raises(capi.MSAError) as e:
        pipeline.check_device_errors(cache)
    assert "MSA_DEVERR_BAD_PAGE" in str(e.value.__cause__)


def test_a_position_past_the_table_is_found():
    plan = pipeline.NormRope(pipeline.rope_table(10, 64))
    q, pos = _rn(1, 1, 3, 2, 64), torch.tensor([[3, -1, 9]], device="cuda")
    pipeline.norm_rope(plan, q, None, positions=pos)
    gr = pipeline.NormRopeGrads.allocate(q, None)
    pipeline.norm_rope_backward(plan, q, None, q, None, gr, positions=pos)
    pipeline.check_device_errors(plan)
    pos[0, 1] = 10
    pipeline.norm_rope(plan, q, None, positions=pos)
    with pytest.raises(capi.MSAError) as e:
        pipeline.check_device_errors(plan)
    assert "MSA_DEVERR_BAD_POSITION" in str(e.value.__cause__)
    plan.dev_err.zero_()
    pipeline.norm_rope_backward(plan, q, None, q, None, gr, positions=pos)
    assert int(plan.dev_err[0]) == 4
