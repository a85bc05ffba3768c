"""Rotary frequencies for k16v8_rope_kv_append: the plain ones and those of
contexts longer than the model was trained on.  Host arithmetic in 64 bits;
the result is the fp32 table the call takes.  And which axis of a position
turns which pair, for the calls whose positions have several."""
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


def rope_pair_axes(rotary_dim: int, sections, interleaved: bool = False) -> bytes:
    """The axis of each of the rotary_dim/2 pairs, as
    k16v8_rope_axes_kv_append takes it.  sections[a] is the number of pairs
    that axis a turns (they sum to rotary_dim/2).

    In blocks: the first sections[0] pairs are axis 0's, the next axis 1's,
    and so on.  Interleaved: the axes take turns -- of n axes, axis a > 0 has
    pairs a, a + n, a + 2n, ... until it has its number, axis 0 the rest."""
    half = rotary_dim // 2
    n = len(sections)
    if rotary_dim < 16 or rotary_dim > 128 or rotary_dim % 16:
        raise ValueError(f"rotary_dim must be a multiple of 16 in [16, 128], got {rotary_dim}")
    if not 1 <= n <= 4:
        raise ValueError(f"1 to 4 axes, got {n}")
    if any(s < 0 for s in sections) or sum(sections) != half:
        raise ValueError(f"sections must sum to {half} pairs, got {tuple(sections)}")
    if not interleaved:
        return bytes(a for a, s in enumerate(sections) for _ in range(s))
    out = bytearray(half)
    for a in range(1, n):
        if sections[a] and a + n * (sections[a] - 1) >= half:
            raise ValueError(f"{sections[a]} pairs of axis {a} do not fit {half} when {n} axes take "
                             "turns")
        for i in range(sections[a]):
            out[a + n * i] = a
    return bytes(out)
