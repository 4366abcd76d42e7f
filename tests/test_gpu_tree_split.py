"""Tree attention in chosen layouts of its split over the CTAs, against the FP64 oracle."""
import numpy as np
import pytest
import torch

from tests import spec_util as S
from tests import tree_split
from tests.test_gpu_speculative import Run
from tests.test_tree_split import RUN_SUMS, has_run_sums_beside_a_one_block_segment

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


@pytest.fixture(scope="module")
def pkv():
    import paged_kv_cache_180_gb300 as p
    return p


def test_run_sums_are_read_before_the_next_unit_writes_them(pkv):
    # a unit of two runs and one block of the next unit in one share: the runs' sums of the first lie where the second
    # one's state goes.
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    whole, shares = tree_split.split(*RUN_SUMS, sms=sms)
    if sms == 152:
        assert not whole and has_run_sums_beside_a_one_block_segment(shares)
    c = S.TreeCase(*RUN_SUMS, seed=101)
    run = Run(pkv, c)
    first, status = run.call().result()
    ref, err, size, _ = c.reference()
    assert status == err == 0
    # weights in two bf16 terms (2^-18 each), 16 truncating blocks a run (2^-18.8), the scores in fp32 (exponents below 2^4:
    # 2^-19), 2 runs and 2 parts: below 2^-16 of the size of the values
    assert (np.abs(first - ref) <= size * 2.0 ** -16).all()
    for _ in range(50):
        run.out[:c.rows].zero_()
        got, status = run.call().result()
        assert status == 0 and np.array_equal(got, first)
