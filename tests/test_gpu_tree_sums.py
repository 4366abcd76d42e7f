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


def repeated_pages(pkv, pages, bf16, seed, positive=False, poke=None):
    """(output, expected output, weighted sum of |V|) of one drafted token behind a context of `pages` pages; as many
    sequences as make every CTA take one whole unit."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    seqs, ctx = 2 * sms // 8, 16 * pages
    if pages < 10000:
        assert tree_split.split([ctx] * seqs, [1] * seqs, sms=sms)[0]
    host = oracle.Pool(2)
    draw = lambda tag, n: rng.normal_bf16(rng.stream_key(seed, tag), 0, n)  # noqa: E731
    kv = draw("kv", 2 * 2 * 8 * 16 * 64).reshape(2, 2, 8, 16, 64)
    kv[1, 0] = kv[1, 0, :, :1]                                  # one K row, sixteen times
    kv[0, 0, :, 0, 7] = 0x4180                                  # token 0: K_7 = 16
    if positive:
        kv[:, 1] = kv[:, 1] & 0x7FFF                            # V > 0
    host.data[:] = kv
    q = draw("q", seqs * 32 * 64).reshape(seqs, 32, 64)
    q[..., 7] = (q[..., 7] & 0x7F) | 0x3F80                     # q_7 in [1, 2)
    if poke:
        poke(host)
    pool = pkv.KVPool(2, device=U.dev())
    pool.buffer.copy_(U.to_dev(host.data).view(-1))
    bt = torch.ones(seqs, pages, dtype=torch.int32, device=U.dev())
    bt[:, 0] = 0
    out = torch.full((seqs, 32, 64), float("nan"), device=U.dev(), dtype=torch.bfloat16 if bf16 else torch.float32)
    status = torch.zeros(1, dtype=torch.int32, device=U.dev())
    pkv.paged_tree_attention(pool, out, U.to_dev(q), torch.arange(seqs + 1, dtype=torch.int32, device=U.dev()),
                             torch.ones(seqs, 1, dtype=torch.int32, device=U.dev()), bt, pages,
                             torch.full((seqs,), ctx, dtype=torch.int32, device=U.dev()), 1, ctx, 0.125,
                             pkv.tree_workspace(seqs, 1), status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    K, V = (rng.bf16_bits_to_f64(kv[:, i]).transpose(1, 0, 2, 3).reshape(8, 32, 64) for i in (0, 1))
    times = np.repeat([1.0, pages - 1.0], 16)
    x = np.einsum("sghd,gtd->sght", rng.bf16_bits_to_f64(q).reshape(seqs, 8, 4, 64), K) * 0.125
    w = np.exp(x - x.max(-1, keepdims=True)) * times
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
