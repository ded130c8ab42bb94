"""The Python calls of the operators around the sparse path, without a GPU: what is refused
before anything is enqueued, how their module is loaded, where errors are reported."""
import pytest
import torch

from block_sparse_attention_32_b200 import build as msa_build
from block_sparse_attention_32_b200 import capi, pipeline

BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def built():
    msa_build.build()


def _z(*shape, dtype=BF):
    return torch.zeros(shape, dtype=dtype)


class _NoTruth:
    def __bool__(self):
        raise KeyError("no truth value")


@pytest.mark.parametrize("what", [torch.tensor([1, 0]), _NoTruth()], ids=["tensor", "raises"])
def test_interleaved_without_a_truth_value_is_refused(what):
    """Refused as the other arguments are, before the tensors are looked at for a device."""
    q, k, v = _z(2, 1, 4, 128), _z(2, 1, 2, 128), _z(2, 1, 2, 128)
    table = _z(10, 64, dtype=torch.float32)
    plan = pipeline.NormRope(table, interleaved=what)
    cache = pipeline.PagedCache(_z(6, 2, 16, 128), _z(6, 2, 16, 128), _z(2, 3, dtype=torch.int32),
                                _z(2, dtype=torch.int32))
    grads = pipeline.NormRopeGrads.allocate(q, k)
    for call in (lambda: pipeline.norm_rope(plan, q, k),
                 lambda: pipeline.norm_rope_append(plan, q, k, v, None, None, cache),
                 lambda: pipeline.norm_rope_backward(plan, q, k, q, _z(2, 2, 1, 128), grads)):
        with pytest.raises(ValueError, match="interleaved"):
            call()


def test_the_module_is_loaded_once(monkeypatch):
    """Two first callers at once: one loads it, the other waits and takes the same."""
    import threading
    import time

    load, loads = capi.importlib.util.spec_from_file_location, []

    def slow(*a, **kw):
        loads.append(a)
        time.sleep(0.2)
        return load(*a, **kw)

    monkeypatch.setattr(capi, "_calls", None)
    monkeypatch.setattr(capi.importlib.util, "spec_from_file_location", slow)
    got = []
    threads = [threading.Thread(target=lambda: got.append(capi.calls())) for _ in range(3)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert len(loads) == 1 and len(got) == 3 and all(m is got[0] for m in got)


def test_a_module_built_for_another_torch_is_refused_and_rebuilt(monkeypatch):
    """msa_calls.so is bound to the torch whose headers it was compiled with."""
    assert capi.calls().torch_version == str(torch.__version__)
    assert not msa_build.calls_stale()
    monkeypatch.setattr(capi, "_calls", None)
    monkeypatch.setattr(torch, "__version__", "1.0.0+other")
    assert msa_build.calls_stale()
    with pytest.raises(RuntimeError, match="built for torch .*1.0.0.*build"):
        capi.calls()
    assert capi._calls is None


def test_a_module_that_does_not_load_says_what_to_do(monkeypatch, tmp_path):
    bad = tmp_path / "msa_calls.so"
    bad.write_bytes(b"not a library")
    monkeypatch.setattr(capi, "_calls", None)
    monkeypatch.setattr(capi, "CALLS_PATH", str(bad))
    with pytest.raises(RuntimeError, match="does not load.*build"):
        capi.calls()


def test_the_cache_takes_the_errors_of_appends(monkeypatch):
    """A page that is not in the table drops keys: without a dev_err of the caller's, the
    cache's own reports it."""
    seen = []
    monkeypatch.setattr(capi, "msa_qk_norm_rope_paged", lambda *a: seen.append(a[-1]))
    cache = pipeline.PagedCache.allocate(2, 48, 2, page_size=16, device="cpu")
    made = pipeline.PagedCache(cache.k_pages, cache.v_pages, cache.block_table, cache.seq_lens)
    plan = pipeline.NormRope(_z(48, 64, dtype=torch.float32))
    q, k, v = _z(2, 1, 4, 128), _z(2, 1, 2, 128), _z(2, 1, 2, 128)
    mine = torch.zeros(4, dtype=torch.int32)
    for c in (cache, made):
        pipeline.norm_rope_append(plan, q, k, v, None, None, c)
        pipeline.norm_rope_append(plan, q, k, v, None, None, c, dev_err=mine)
        assert seen[-2] is c.dev_err and seen[-1] is mine
        assert c.dev_err.dtype == torch.int32 and c.dev_err.device == c.k_pages.device
        pipeline.check_device_errors(c)
        c.dev_err[0] = 5
        with pytest.raises(capi.MSAError) as e:
            pipeline.check_device_errors(c)
        assert "BAD_PAGE" in str(e.value.__cause__)
    assert cache.dev_err is not made.dev_err


def test_the_plan_takes_the_errors_of_positions(monkeypatch):
    """A position past the table leaves a row unwritten: reported by the plan's dev_err when
    the caller gives none."""
    seen = []
    monkeypatch.setattr(capi, "msa_qk_norm_rope", lambda *a: seen.append(a[-1]))
    monkeypatch.setattr(capi, "msa_qk_norm_rope_bwd", lambda *a: seen.append(a[-1]))
    q, k = _z(2, 1, 4, 128), _z(2, 1, 2, 128)
    plan = pipeline.NormRope(_z(48, 64, dtype=torch.float32))
    mine = torch.zeros(4, dtype=torch.int32)
    grads = pipeline.NormRopeGrads.allocate(q, k)
    for own, want in ((None, plan.dev_err), (mine, mine)):
        pipeline.norm_rope(plan, q, k, dev_err=own)
        pipeline.norm_rope_backward(plan, q, k, q, k, grads, dev_err=own)
        assert seen[-2] is want and seen[-1] is want
    pipeline.check_device_errors(plan)
    # without a table no position is out of range, and there may be no device to tell
    assert pipeline.NormRope(None).dev_err is None
