"""Scales at the end of fp32's range: accepted as long as scale * log2(e), the exponents' factor, is finite."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def pkv():
    from paged_kv_cache_180_gb300 import build
    build.build()
    import paged_kv_cache_180_gb300 as p
    return p


def test_a_scale_whose_factor_is_infinite_is_refused(pkv):
    b = pkv.binding
    base = 1 << 20
    d, p, need = b.kv_pool_create(base, base + 16384, 0, 8), ctypes.c_void_p(base), b.tree_workspace_bytes(4, 16)
    call = lambda scale, ws: b._lib.pkv_paged_tree_attention(  # noqa: E731
        ctypes.byref(d), p, p, 32, 64, p, p, 1, p, 128, p, 4, 16, 2048, scale, p, ws, None, 0, None)
    for scale in (2.36e38, 3e38, 3.4e38, float("inf"), float("nan")):
        assert call(scale, need) == call(-scale, need) == -5, scale
    for scale in (2.3e38, 2.358e38):
        assert call(scale, need - 1) == call(-scale, need - 1) == -6        # on to the next check


@pytest.mark.gpu
@pytest.mark.parametrize("scale", [2.3e38, -2.3e38])
def test_scores_of_zero_stay_an_average_at_the_largest_scale(pkv, scale):
    from tests import spec_util as S
    from tests.test_gpu_speculative import Run
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    c = S.TreeCase([300, 40], [20, 5], seed=112)
    c.q[:] = 0
    got, status = Run(pkv, c, scale=scale).call().result()
    ref, err, size, _ = c.reference(0.125)                 # any scale: all scores are 0
    assert status == err == 0
    S.assert_within(got, ref, S.bound(ref, size, 0.0, 1.0, 300, False), "an average")
