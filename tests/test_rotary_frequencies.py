"""Frequencies for contexts longer than the trained ones, against the blend's definition."""
import math
import os
import sys

import numpy as np
import pytest

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import tensor_core_gemm_tl_b200 as tg  # noqa: E402


def turns(rot_dim, base, length):
    """Turns of every pair over `length` positions."""
    return length * base ** (-2.0 * np.arange(rot_dim // 2) / rot_dim) / (2 * math.pi)


def share_divided(rot_dim, base, length, fast, slow):
    """How much of each pair is divided: 0 up to the pair that turns `fast` times, 1 from the one that turns `slow`
    times, linear in the index between those (taken outwards to whole indices from 0 to rot_dim - 1, behind the last
    pair too)."""
    per_pair = 2 * math.log(base) / rot_dim  # a pair's turns are exp(-per_pair) of the one's before
    first = math.log(length / (2 * math.pi))
    lo, hi = (first - math.log(fast)) / per_pair, (first - math.log(slow)) / per_pair
    lo, hi = max(math.floor(lo), 0), min(math.ceil(hi), rot_dim - 1)
    return np.interp(np.arange(rot_dim // 2), [lo, hi], [0.0, 1.0])


CASES = [
    # rot_dim, base, length, fast, slow
    (64, 1e4, 4096, 32.0, 1.0),
    (64, 1e4, 65536, 32.0, 1.0),     # the last pair turns 1.39 times: no pair is divided whole
    (64, 1e4, 131072, 32.0, 1.0),
    (128, 1e4, 131072, 32.0, 1.0),
    (32, 1e4, 65536, 32.0, 1.0),
    (128, 5e5, 8192, 32.0, 1.0),
    (64, 1e4, 64, 32.0, 1.0),        # the first pair turns 10 times: the ramp begins with it
    (64, 1e4, 1 << 22, 32.0, 1.0),   # the last pair turns 89 times: all are kept
    (64, 1e4, 65536, 16.0, 1.3),
    (16, 1e4, 1 << 20, 32.0, 1.0),
]


@pytest.mark.parametrize("rot_dim,base,length,fast,slow", CASES)
def test_yarn_blends_by_the_pairs_turns(rot_dim, base, length, fast, slow):
    factor = 4.0
    freq, scale = tg.rotary_frequencies(rot_dim, base, scaling="yarn", factor=factor, original_length=length,
                                        beta_fast=fast, beta_slow=slow)
    plain = base ** (-2.0 * np.arange(rot_dim // 2) / rot_dim)
    share = share_divided(rot_dim, base, length, fast, slow)
    want = plain * (1 - share) + plain / factor * share
    assert np.allclose(freq.numpy(), want, rtol=2.0 ** -23, atol=0)
    assert math.isclose(scale, 0.1 * math.log(factor) + 1)
    t = turns(rot_dim, base, length)
    assert np.all(freq.numpy()[t > slow] > plain[t > slow] / factor)  # only pairs under it are divided whole


def test_yarn_needs_a_base_above_one():
    with pytest.raises(ValueError):
        tg.rotary_frequencies(64, 1.0, scaling="yarn", factor=4.0, original_length=4096)
