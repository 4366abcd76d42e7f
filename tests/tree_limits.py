"""Limits of tree attention's error that do not grow with the context.

Relative to the output's norm over a sequence's rows.  The errors of different keys are independent of one another and of V's
signs, as the outputs' terms w V are, so both shrink alike as the number of keys grows:

fp32 output: a weight as two bf16 terms is off by at most 2^-18 of itself, 2^-18 / sqrt(3) = 2.2e-6 in the mean square;
the tensor core truncates its accumulator, 2.3e-6 over a run of 16 blocks (V of both signs; taken as 2.8e-6), and what is
added up behind that rounds, (blocks / 16 + parts) 2^-25 in the mean, below 2e-6 for 500 runs; score and exponential 2^-19 / sqrt(3) = 1.1e-6 at
exponents of up to 2^4.  The root of the squares' sum is 4.2e-6; twice that and a little: 1e-5.

bf16 output: half a step of 2^-8 in the weights and in the output, each 2^-8 / sqrt(3) at the most in the mean square (all
mantissas near 1): 3.2e-3 together, and 2e-5 for truncation over 256 blocks; with a half more: 5e-3."""
from __future__ import annotations

import numpy as np

FP32, BF16 = 1e-5, 5e-3


def norm_errors(got, ref, starts):
    """Per sequence with nodes: norm of the error over the output's."""
    pairs = [(a, b) for a, b in zip(starts[:-1], starts[1:]) if b > a]
    return [float(np.linalg.norm(got[a:b] - ref[a:b]) / np.linalg.norm(ref[a:b])) for a, b in pairs]


def assert_precise(got, ref, starts, bf16):
    errors = norm_errors(np.asarray(got, np.float64), ref, starts)
    limit = BF16 if bf16 else FP32
    assert max(errors) <= limit, f"{max(errors):.3g} of the output's norm (sequence {int(np.argmax(errors))}); limit {limit}"
