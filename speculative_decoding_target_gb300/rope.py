"""Rotary frequencies for rope_append, with the usual scalings for contexts
longer than the one a model was trained on.

A frequency is the angle in radians that one position adds.  The table is
float64: at position 500,000 an fp32 frequency is off by 0.01 radians.
"""
from __future__ import annotations

import math
from typing import Optional, Tuple

import torch

SCALINGS = ("none", "linear", "ntk", "yarn", "wavelength")


def rope_frequencies(rotary_dim: int, *, base: float = 10000.0,
                     scaling: str = "none", factor: float = 1.0,
                     original_context: int = 8192,
                     beta_fast: float = 32.0, beta_slow: float = 1.0,
                     low_freq_factor: float = 1.0,
                     high_freq_factor: float = 4.0,
                     attn_factor: Optional[float] = None,
                     device=None) -> Tuple[torch.Tensor, float]:
    """Returns (float64 [rotary_dim / 2] radians per position, the factor on
    the rotated channels).

    scaling:
      none        f_j = base^(-2j / rotary_dim)
      linear      f_j / factor (positions interpolated)
      ntk         base * factor^(rotary_dim / (rotary_dim - 2)): the lowest
                  frequency is stretched by factor, the highest is kept
      yarn        f_j / factor for pairs that turn fewer than beta_slow times
                  over original_context, f_j for those above beta_fast, a
                  linear ramp over the pair index between; the rotated
                  channels are scaled by 0.1 ln(factor) + 1 unless attn_factor
                  is given (Peng et al. 2023, "YaRN")
      wavelength  f_j / factor for wavelengths above original_context /
                  low_freq_factor, f_j below original_context /
                  high_freq_factor, blended linearly in the number of turns
                  over original_context between
    """
    if scaling not in SCALINGS:
        raise ValueError(f"scaling {scaling!r}: one of {SCALINGS}")
    if rotary_dim < 8 or rotary_dim > 256 or rotary_dim % 8:
        raise ValueError(f"rotary_dim {rotary_dim}: a multiple of 8 in "
                         "[8, 256]")
    if not (base > 1.0 and math.isfinite(base)):
        raise ValueError(f"base {base}")
    if not (factor >= 1.0 and math.isfinite(factor)):
        raise ValueError(f"factor {factor} must be >= 1")
    if original_context < 1:
        raise ValueError(f"original_context {original_context}")
    pair = torch.arange(0, rotary_dim, 2, dtype=torch.float64)
    m = 1.0
    if scaling == "ntk":
        base = base * factor ** (rotary_dim / (rotary_dim - 2))
    f = base ** (-pair / rotary_dim)
    if scaling == "linear":
        f = f / factor
    elif scaling == "yarn":
        def pair_of(turns):  # the (real) pair that makes this many turns
            return (rotary_dim
                    * math.log(original_context / (turns * 2 * math.pi))
                    / (2 * math.log(base)))
        lo = max(math.floor(pair_of(beta_fast)), 0)
        hi = min(math.ceil(pair_of(beta_slow)), rotary_dim - 1)
        ramp = ((torch.arange(rotary_dim // 2, dtype=torch.float64) - lo)
                / max(hi - lo, 1e-3)).clamp(0, 1)
        f = f / factor * ramp + f * (1 - ramp)
        m = 0.1 * math.log(factor) + 1.0
    elif scaling == "wavelength":
        if not high_freq_factor > low_freq_factor:
            raise ValueError("high_freq_factor must exceed low_freq_factor")
        turns = original_context * f / (2 * math.pi)
        mix = ((turns - low_freq_factor)
               / (high_freq_factor - low_freq_factor)).clamp(0, 1)
        f = (1 - mix) * f / factor + mix * f
    if attn_factor is not None:
        m = float(attn_factor)
    return f.to(device) if device is not None else f, m
