"""The bounded calls' limits on lengths, windows and strides, to the last value (no GPU: refused calls never launch)."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def b():
    from paged_kv_cache_180_gb300 import build
    build.build()
    from paged_kv_cache_180_gb300 import binding
    return binding


BASE = 1 << 20  # a fake, aligned device address: refused calls never dereference it
P = ctypes.c_void_p


def _pool(b):
    return ctypes.byref(b.kv_pool_create(BASE, BASE + 16384, 0, 8))


# (the query's pointer is null: what passes the check of the bound is refused for that)
@pytest.mark.parametrize("max_context,code", [((1 << 31) - 64, -1), ((1 << 31) - 63, -2), ((1 << 31) - 1, -2), (0, -1)])
def test_the_longest_context_of_the_window_calls(b, max_context, code):
    decode = b._lib.pkv_paged_window_decode_attention(_pool(b), P(BASE), P(0), 32, P(BASE), 128, P(BASE), 4, max_context, 0.125, 64,
                                                      4, None, 0, None)
    prefill = b._lib.pkv_paged_window_prefill_attention(_pool(b), P(BASE), P(0), 32, 64, P(BASE), P(BASE), 128, P(BASE), 4, 16,
                                                        max_context, 0.125, 64, 4, None, 0, None)
    assert decode == code and prefill == code
