"""Tree attention held to limits that do not grow with the context, in the layouts that split long contexts."""
import numpy as np
import pytest
import torch

from tests import spec_util as S
from tests import tree_limits, tree_split
from tests.test_gpu_speculative import Run
from tests.test_tree_split import RUN_SUMS

pytestmark = pytest.mark.gpu

_r = np.random.RandomState(13)
LONG_AND_SHORT = ([20000] + [int(_r.randint(8, 200)) for _ in range(90)], [8] + [int(_r.randint(1, 8)) for _ in range(90)])
CLAIMED = ([1600 - 9 * s for s in range(72)], [1 + 7 * s % 64 for s in range(72)])
# name: contexts, nodes, whole units, parts of the first sequence's units at the least
LAYOUTS = {
    "parts merged in groups": ([9000], [3], False, 11),
    "two long ones, one of two tiles": ([30000, 700], [40, 64], False, 6),
    "parts of many blocks": ([20000, 64], [8, 64], False, 11),
    "one long unit among short ones": (*LONG_AND_SHORT, False, 2),
    "run sums beside a block": (*RUN_SUMS, False, 1),
    "whole units, claimed": (*CLAIMED, True, 1),
    "units of 47 blocks, some cut": ([3000, 2990, 2500, 3000] * 10, [2, 8, 1, 3] * 10, False, 1),
    "whole units of 47 blocks": ([3000, 2990] * 19, [2, 8] * 19, True, 1),
}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


@pytest.fixture(scope="module")
def pkv():
    import paged_kv_cache_180_gb300 as p
    return p


@pytest.mark.parametrize("name", LAYOUTS)
def test_errors_do_not_grow_with_the_context(pkv, name):
    contexts, nodes, whole, parts = LAYOUTS[name]
    if torch.cuda.get_device_properties(0).multi_processor_count == 152:
        is_whole, shares = tree_split.split(contexts, nodes)
        assert is_whole == whole
        if not whole:
            assert tree_split.parts_of_units(shares)[0, 0, 0] >= parts
    c = S.TreeCase(contexts, nodes, seed=133)
    ref, err, _, _ = c.reference()
    for bf16 in (False, True):
        got, status = Run(pkv, c, bf16).call().result()
        assert status == err == 0
        tree_limits.assert_precise(got, ref, c.starts, bf16)
