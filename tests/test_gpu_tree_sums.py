"""Sums over long contexts whose keys weigh the same: every addition rounds the same way, so errors add up.

All sequences share two pages: the first one's keys differ and one of them outweighs the rest, the second one, repeated up
to the context's end, holds one K row sixteen times.  The expected outputs are sums over 32 keys with multiplicities."""
import numpy as np
import pytest
import torch

import oracle
from tests import gpu_util as U
from tests import tree_split
from workloads import rng

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


@pytest.fixture(scope="module")
def pkv():
    import paged_kv_cache_180_gb300 as p
    return p


def repeated_pages(pkv, pages, bf16, seed, positive=False, order=(0,), keys=None, seconds=None, seqs=None):
    """(output, expected output, weighted sum of |V|) of one drafted token behind a context of `pages` pages: those of `order`,
    then page 1 again and again; as many sequences as make every CTA take one whole unit, or `seqs`.  keys(K): sets the K of
    the pages [page][head][row][dim] as bits.  `seconds`: a list that receives the time the call took."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    cut, seqs = seqs is not None, seqs or 2 * sms // 8
    ctx, ids = 16 * pages, max(2, max(order) + 1)
    if not cut and pages < 10000:
        assert tree_split.split([ctx] * seqs, [1] * seqs, sms=sms)[0]
    host = oracle.Pool(ids)
    draw = lambda tag, n: rng.normal_bf16(rng.stream_key(seed, tag), 0, n)  # noqa: E731
    kv = draw("kv", ids * 2 * 8 * 16 * 64).reshape(ids, 2, 8, 16, 64)
    kv[1, 0] = kv[1, 0, :, :1]                                  # one K row, sixteen times
    if keys is None:
        kv[0, 0, :, 0, 7] = 0x4180                              # token 0: K_7 = 16
    else:
        keys(kv[:, 0])
    if positive:
        kv[:, 1] = kv[:, 1] & 0x7FFF                            # V > 0
    host.data[:] = kv
    q = draw("q", seqs * 32 * 64).reshape(seqs, 32, 64)
    q[..., 7] = (q[..., 7] & 0x7F) | 0x3F80                     # q_7 in [1, 2)
    pool = pkv.KVPool(ids, device=U.dev())
    pool.buffer.copy_(U.to_dev(host.data).view(-1))
    bt = torch.ones(seqs, pages, dtype=torch.int32, device=U.dev())
    bt[:, :len(order)] = torch.tensor(order, dtype=torch.int32, device=U.dev())
    out = torch.full((seqs, 32, 64), float("nan"), device=U.dev(), dtype=torch.bfloat16 if bf16 else torch.float32)
    status = torch.zeros(1, dtype=torch.int32, device=U.dev())
    args = (pool, out, U.to_dev(q), torch.arange(seqs + 1, dtype=torch.int32, device=U.dev()),
            torch.ones(seqs, 1, dtype=torch.int32, device=U.dev()), bt, pages,
            torch.full((seqs,), ctx, dtype=torch.int32, device=U.dev()), 1, ctx, 0.125, pkv.tree_workspace(seqs, 1), status)
    ends = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
    ends[0].record()
    pkv.paged_tree_attention(*args)
    ends[1].record()
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    if seconds is not None:
        seconds.append(ends[0].elapsed_time(ends[1]) * 1e-3)
    K, V = (rng.bf16_bits_to_f64(kv[:, i]).transpose(1, 0, 2, 3).reshape(8, ids * 16, 64) for i in (0, 1))
    times = np.array([order.count(i) for i in range(ids)], float)
    times[1] += pages - len(order)
    times = np.repeat(times, 16)
    x = np.einsum("sghd,gtd->sght", rng.bf16_bits_to_f64(q).reshape(seqs, 8, 4, 64), K) * 0.125
    w = np.exp(x - x[..., times > 0].max(-1, keepdims=True)) * times
    w /= w.sum(-1, keepdims=True)
    ref, size = (np.einsum("sght,gtd->sghd", w, v).reshape(seqs, 32, 64) for v in (V, np.abs(V)))
    return out.double().cpu().numpy(), ref, size


def test_row_sums_of_equal_weights(pkv):
    got, ref, size = repeated_pages(pkv, 1750, False, 121)
    # relative to the weighted |V|: the one weight's split into two bf16 terms 2^-18, 16 truncating blocks a run 2.8e-6, score
    # and exponential 2^-19 + 2^-22, the row sum 16 + 4 + 14 half steps of 2^-24 (block, run, 28 runs), the same 14 for O
    lim = 2.0 ** -18 + 2.8e-6 + 2.0 ** -19 + 2.0 ** -22 + (34 + 14) * 2.0 ** -24
    assert lim < 2.0 ** -16
    assert (np.abs(got - ref) <= size * lim).all(), float((np.abs(got - ref) / size).max())


def test_bf16_output_of_a_context_of_millions_of_equal_weights(pkv):
    got, ref, size = repeated_pages(pkv, 1 << 20, True, 122, positive=True)
    assert np.allclose(ref, size)
    # the one weight as a single bf16 term 2^-8 and the output 2^-8; 256 truncating blocks of four MMAs a run (256 * 4 * 2^-24),
    # 1024 runs added up in O and in the row sum (512 * 2^-24 each), a run's row sum (16 + 64) 2^-24, score and exponential
    lim = 2 * 2.0 ** -8 + (1024 + 1024 + 80) * 2.0 ** -24 + 2.0 ** -19 + 2.0 ** -22
    assert (np.abs(got - ref) <= size * lim).all(), float((np.abs(got - ref) / size).max())


def _grown(K):
    # the first 64 keys score about 0, a later one about 200 and the repeated ones a little less: out of the fast path's range
    K[1, :, :, 7] = 0x447A                                      # 1000
    K[2, :, 5, 7] = 0x447C                                      # 1008


def test_sums_of_rows_that_are_computed_again(pkv):
    got, ref, size = repeated_pages(pkv, 1750, False, 123, order=(0, 0, 0, 0, 2), keys=_grown)
    # 110 stretches of 256 equal weights: (256 + 110) / 2 * 2^-24 in O and in the row sum; the exponential and the division 2^-22;
    # the scores (exponents of up to 2^9.5: 6 roundings of 2^-24) move weight between the one key, 0.2 % at the most, and the others
    lim = (256 + 110) * 2.0 ** -24 + 2.0 ** -22 + 0.002 * 6 * 2.0 ** (9.5 - 24)
    assert (np.abs(got - ref) <= size * lim).all(), float((np.abs(got - ref) / size).max())


def test_rows_computed_again_for_longer_than_a_wait_may_take(pkv):
    # A wait inside the kernel gives up after 3.8e9 cycles, 1.8 s at the highest clock.  Rows that are computed again over a
    # long segment take longer; the other warps wait for them.
    def call(pages, seconds):
        return repeated_pages(pkv, pages, False, 124, order=(0, 0, 0, 0, 2), keys=_grown, seconds=seconds)
    seconds = []
    for _ in range(2):
        call(4000, seconds)
    pages = int(4000 * 3.2 / seconds[-1])
    assert pages < 400_000, seconds                             # (what a key takes: 0.5 us at the least)
    got, ref, size = call(pages, seconds)
    assert seconds[-1] > 2.4, (seconds, pages)
    lim = (256 + 16 * pages / 256) * 2.0 ** -24 + 2.0 ** -22 + 0.002 * 6 * 2.0 ** (9.5 - 24)
    assert (np.abs(got - ref) <= size * lim).all(), float((np.abs(got - ref) / size).max())


@pytest.mark.parametrize("bf16", [False, True])
def test_runs_in_units_that_are_cut(pkv, bf16):
    # one sequence, each unit in 38 parts of over 256 blocks: runs inside parts, parts merged in groups
    whole, shares = tree_split.split([800_000], [1])
    assert not whole and min(j1 - j0 for x in shares for *_, j0, j1, _ in x) > 256
    got, ref, size = repeated_pages(pkv, 50_000, bf16, 125, seqs=1)
    # as above: 21 runs a part and 38 parts for fp32, two runs a part for bf16 output
    if bf16:
        lim = 2 * 2.0 ** -8 + (1024 + 2 * (16 + 64) + 2 * 38) * 2.0 ** -24 + 2.0 ** -19 + 2.0 ** -22
    else:
        lim = 2.0 ** -18 + 2.8e-6 + 2.0 ** -19 + 2.0 ** -22 + (20 + 2 * (21 + 38) / 2) * 2.0 ** -24
    assert (np.abs(got - ref) <= size * lim).all(), float((np.abs(got - ref) / size).max())
