"""The speculative calls look at their status tensor before they pass its address on."""
import numpy as np
import pytest
import torch

WRONG = {
    "host": lambda dev: torch.zeros(1, dtype=torch.int32),
    "wide": lambda dev: torch.zeros(1, dtype=torch.int64, device=dev),
    "float": lambda dev: torch.zeros(1, dtype=torch.float32, device=dev),
    "empty": lambda dev: torch.zeros(0, dtype=torch.int32, device=dev),
}


@pytest.fixture(scope="module")
def pkv():
    from paged_kv_cache_180_gb300 import build
    build.build()
    import paged_kv_cache_180_gb300 as p
    return p


@pytest.mark.parametrize("kind", WRONG)
def test_a_status_that_is_no_word_of_the_device_is_refused(pkv, kind):
    with pytest.raises(ValueError, match="status is an int32 word"):
        pkv.binding._status_ptr("call", WRONG[kind]("cpu"), 0)
    assert pkv.binding._status_ptr("call", None, 0) is None


@pytest.mark.gpu
@pytest.mark.parametrize("kind", WRONG)
def test_the_calls_refuse_it_before_they_launch(pkv, kind):
    from tests import spec_util as S
    from tests.test_gpu_speculative import Run
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    run = Run(pkv, S.TreeCase([40], [5], seed=111))
    good, bad = run.status, WRONG[kind]("cuda")
    run.status = bad
    with pytest.raises(ValueError, match="pkv_paged_tree_attention: status"):
        run.call()
    assert torch.isnan(run.out).all()
    bits = run.pool.buffer.view(torch.int16).clone()
    counts = torch.ones(1, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="pkv_tree_commit: status"):
        pkv.tree_commit(run.pool, run.bt, run.bt.shape[1], 0, 1, run.starts, run.lens, torch.full_like(counts, 2)[None],
                        counts, 64, None, bad)
    with pytest.raises(ValueError, match="pkv_kv_copy_pages: status"):
        pkv.kv_copy_pages(run.pool, run.bt[0, :1].contiguous(), run.bt[0, 1:2].contiguous(), bad)
    torch.cuda.synchronize()
    assert torch.equal(run.pool.buffer.view(torch.int16), bits)
    run.status = good
    got, status = run.call().result()
    assert status == 0 and np.isfinite(got).all()
    word = torch.zeros(2, dtype=torch.int32, device="cuda")
    run.status = word.view(torch.uint32)                    # unsigned, and more behind it
    run.out.fill_(float("nan"))
    run.call()
    torch.cuda.synchronize()
    assert np.array_equal(run.out[:5].double().cpu().numpy(), got) and not word.any()
