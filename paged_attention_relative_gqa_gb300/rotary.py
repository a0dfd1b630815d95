"""Frequency tables for ``binding.inkling_attn_qk_norm_rope_write``.

Pair i of the rotated channels turns by ``inv_freq[i]`` per position.  Scalings for contexts
longer than the trained one change the table (and multiply cos and sin by a factor), never the
kernel:

* ``linear``: every frequency divided by ``factor`` (positions interpolated);
* ``yarn`` (Peng et al., "YaRN: Efficient Context Window Extension of Large Language Models"):
  with r the turns a pair makes over ``original_len`` positions, pairs with r > beta_fast keep
  their frequency, pairs with r < beta_slow are interpolated, a linear ramp lies between; cos and
  sin are multiplied by 0.1 ln(factor) + 1.  The ramp is linear in r.  Checkpoints are also run with a
  ramp that is linear in the pair's index between two rounded bounds: for those make the table from
  their own formula (the kernel takes any table).
"""
from __future__ import annotations

import math
from typing import Optional, Tuple

import torch


def inv_freq(rot_dim: int, *, base: float = 10000.0, scaling: Optional[str] = None, factor: float = 1.0,
             original_len: int = 4096, beta_fast: float = 32.0, beta_slow: float = 1.0,
             device="cpu") -> Tuple[torch.Tensor, float]:
    """(fp32 [rot_dim / 2] angles per position, factor of cos and sin)."""
    if rot_dim < 2 or rot_dim % 2:
        raise ValueError(f"rot_dim must be even and positive, got {rot_dim}")
    if factor < 1.0 or base <= 1.0 or original_len < 1 or not beta_fast > beta_slow:
        raise ValueError("needs factor >= 1, base > 1, original_len >= 1 and beta_fast > beta_slow")
    f = torch.pow(torch.tensor(base, dtype=torch.float64), -torch.arange(0, rot_dim, 2, dtype=torch.float64) / rot_dim)
    scale = 1.0
    if scaling == "linear":
        f = f / factor
    elif scaling == "yarn":
        turns = original_len * f / (2 * math.pi)
        keep = ((turns - beta_slow) / (beta_fast - beta_slow)).clamp(0.0, 1.0)
        f = f * keep + f / factor * (1.0 - keep)
        scale = 0.1 * math.log(factor) + 1.0
    elif scaling is not None:
        raise ValueError(f"unknown scaling {scaling!r}")
    return f.float().to(device), scale
