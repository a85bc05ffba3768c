"""Rotary frequencies for k16v8_rope_kv_append: the plain ones and those of
contexts longer than the model was trained on.  Host arithmetic in 64 bits;
the result is the fp32 table the call takes."""
from __future__ import annotations

import math

import torch


def rope_inv_freq(rotary_dim: int, base: float = 10000.0, scaling: str = "none",
                  factor: float = 1.0, original_max_position: int = 0, beta_fast: float = 32.0,
                  beta_slow: float = 1.0):
    """(inv_freq fp32 [rotary_dim/2] on the CPU, attn_factor).

    "none":   inv_freq[i] = base^(-2i/rotary_dim)
    "linear": positions interpolated, every frequency divided by factor
    "ntk":    the base raised to base * factor^(d/(d-2)), d = rotary_dim, so
              the slowest pair is slowed by factor and the fastest is kept
    "yarn":   interpolation by parts: a pair that makes more than beta_fast
              turns over original_max_position positions is kept, one with
              fewer than beta_slow is divided by factor, those between are
              blended linearly over the pair's index (the ends of the blend
              rounded outwards to whole pairs and kept within 0 and
              rotary_dim - 1, as in Peng et al., "YaRN: Efficient Context
              Window Extension of Large Language Models", 2023: the upper
              end may lie beyond the last pair); attn_factor is
              0.1 ln(factor) + 1
    attn_factor is 1 for the others."""
    if rotary_dim < 16 or rotary_dim > 128 or rotary_dim % 16:
        raise ValueError(f"rotary_dim must be a multiple of 16 in [16, 128], got {rotary_dim}")
    if not (base > 1.0 and math.isfinite(base)):
        raise ValueError(f"base must be finite and above 1, got {base}")
    if not (factor >= 1.0 and math.isfinite(factor)):
        raise ValueError(f"factor must be finite and at least 1, got {factor}")
    half = rotary_dim // 2
    i = torch.arange(half, dtype=torch.float64)
    if scaling == "ntk":
        base = base * factor ** (rotary_dim / (rotary_dim - 2))
    elif scaling not in ("none", "linear", "yarn"):
        raise ValueError(f"unknown scaling {scaling!r}")
    freq = base ** (-i / half)
    attn_factor = 1.0
    if scaling == "linear":
        freq = freq / factor
    elif scaling == "yarn":
        if original_max_position <= 0:
            raise ValueError("scaling 'yarn' needs original_max_position")
        if not beta_fast > beta_slow > 0:
            raise ValueError("scaling 'yarn' needs beta_fast > beta_slow > 0")

        def pair_with_turns(turns):  # index of the pair that makes so many turns
            return half * math.log(original_max_position / (turns * 2 * math.pi)) / math.log(base)

        low = max(math.floor(pair_with_turns(beta_fast)), 0)
        high = min(math.ceil(pair_with_turns(beta_slow)), rotary_dim - 1)
        slow = ((i - low) / max(high - low, 1e-3)).clamp(0.0, 1.0)
        freq = freq / factor * slow + freq * (1.0 - slow)
        attn_factor = 0.1 * math.log(factor) + 1.0
    return freq.to(torch.float32), attn_factor
