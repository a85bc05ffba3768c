"""The "yarn" table against its formula in 64 bits, over original contexts
from one in which every pair turns less than once to one in which none does."""
import math

import numpy as np
import pytest

from fp8_paged_kv_append_gb300.rope import rope_inv_freq


def yarn(rotary, base, factor, original, fast=32.0, slow=1.0):
    """Frequencies by the blend over pair indices, one pair at a time."""
    def pair(turns):
        return rotary * math.log(original / (turns * 2 * math.pi)) / (2 * math.log(base))
    low = max(math.floor(pair(fast)), 0)
    high = min(math.ceil(pair(slow)), rotary - 1)
    out = []
    for i in range(rotary // 2):
        f = base ** (-2 * i / rotary)
        ramp = min(max((i - low) / (high - low if high > low else 1e-3), 0.0), 1.0)
        out.append(f / factor * ramp + f * (1 - ramp))
    return np.array(out)


@pytest.mark.parametrize("base", [10000.0, 500000.0])
@pytest.mark.parametrize("rotary", [32, 64, 96, 128])
@pytest.mark.parametrize("original", [4, 64, 4096, 32768, 62831, 62833, 131072, 1 << 20])
@pytest.mark.parametrize("factor", [1.0, 4.0, 40.0])
def test_yarn_blend(rotary, base, original, factor):
    f, a = rope_inv_freq(rotary, base, scaling="yarn", factor=factor, original_max_position=original)
    want = yarn(rotary, base, factor, original)
    assert a == 0.1 * math.log(factor) + 1
    # one rounding to fp32, and a few in 64 bits
    assert np.all(np.abs(f.double().numpy() - want) <= (2.0 ** -24 + 2.0 ** -45) * want)


def test_only_pairs_below_beta_slow_turns_are_divided_by_the_factor():
    """128 dims over 131,072 positions: the slowest pair makes 2.41 turns, so none is."""
    f, _ = rope_inv_freq(128, scaling="yarn", factor=4.0, original_max_position=131072)
    plain = 10000.0 ** (-np.arange(64) / 64.0)
    assert 131072 * plain[-1] / (2 * math.pi) > 2.4
    r = f.double().numpy() / plain
    assert np.all(r > 0.45) and abs(r[-1] - 0.46) < 1e-6 and np.all(np.abs(r[:46] - 1) < 1e-6)
