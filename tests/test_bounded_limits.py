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


def _weights(b, **kw):
    g = lambda k, v: kw.get(k, v)  # noqa: E731
    return b._lib.pkv_paged_decode_attention_weights(
        _pool(b), P(BASE), P(BASE), 32, P(BASE), 128, P(g("lens", BASE)), g("n", 4), g("max", 2048), 0.125, P(g("sums", BASE + 2)),
        g("seq", 8 * 2048), g("head", 2048), 1.0, P(0), 0, None, 0, None)


@pytest.mark.parametrize("n,seq,head,code", [
    # heads inside sequences: 8 heads of 2048 to a sequence (sums at an odd address: what passes is refused for that)
    (4, 8 * 2048, 2048, -4), (4, 8 * 2048 - 1, 2048, -2), (4, 8 * 2048, 2047, -2), (4, 1 << 38, 2048, -4), (4, (1 << 38) + 1, 2048, -2),
    # sequences inside heads: 4 sequences of 2048 to a head
    (4, 2048, 4 * 2048, -4), (4, 2047, 4 * 2048, -2), (4, 2048, 4 * 2048 - 1, -2),
    # one sequence: its stride counts for nothing, the heads' does
    (1, 0, 2048, -4), (1, 5, 4 * 2048, -4), (1, 0, 2047, -2),
    # no sequence: the same, and nothing is done
    (0, 2048, 4 * 2048, 0), (0, 0, 2048, 0), (0, 0, 2047, -2), (0, -1, 2048, -2)])
def test_strides_of_the_weight_sums(b, n, seq, head, code):
    assert _weights(b, n=n, seq=seq, head=head) == code


@pytest.mark.parametrize("n,layers,seq,layer,head,code", [
    # layers inside sequences, sequences inside layers, one layer, one sequence, none of either
    (4, 2, 16 * 2048, 8 * 2048, 2048, -4), (4, 2, 16 * 2048 - 1, 8 * 2048, 2048, -2), (4, 2, 16 * 2048, 8 * 2048 - 1, 2048, -2),
    (4, 2, 8 * 2048, 32 * 2048, 2048, -4), (4, 2, 8 * 2048, 32 * 2048 - 1, 2048, -2), (4, 2, 8 * 2048 - 1, 32 * 2048, 2048, -2),
    (4, 1, 8 * 2048, 0, 2048, -4), (4, 1, 8 * 2048 - 1, 0, 2048, -2), (1, 2, 0, 8 * 2048, 2048, -4),
    (1, 2, 0, 8 * 2048 - 1, 2048, -2), (1, 1, 0, 0, 2048, -4), (1, 1, 0, 0, 2047, -2), (0, 2, 0, 0, 2048, 0), (0, 2, 0, 0, 2047, -2)])
def test_strides_of_the_sums_that_eviction_reads(b, n, layers, seq, layer, head, code):
    far = 1 << 36
    assert b._lib.pkv_kv_evict(_pool(b), P(BASE), 256, 128, layers, P(BASE), P(BASE + 64), n, 2048, 1024, 4, 16, P(far + 2),
                               P(2 * far), seq, layer, head, P(3 * far), 1024, P(4 * far), None, None) == code
