"""Dilution attention for GB300 (sm_103a): a C-ABI CUDA library and a thin binding.

The compute path lives in ``csrc/`` and is reached through ``libdilution_attn.so``
(see ``include/dilution_attn.h``).  ``binding`` loads it on first use and
raises if it is missing; there is no CPU fallback.
"""
import math

__all__ = ["yarn_tau", "rope_inv_freq", "rope_pair_axis"]


def yarn_tau(scale: float) -> float:
    """Logit multiplier sqrt(0.1 ln s + 1) for a context extension factor s
    ("YaRN › Attention Temperature Scaling", temperature formula)."""
    return math.sqrt(0.1 * math.log(scale) + 1.0)


def rope_inv_freq(rot_dim: int, base: float = 10000.0):
    """Rotary frequencies base^(-2j / rot_dim) of the rot_dim / 2 pairs (fp32, radians per position)."""
    import torch
    return (base ** (-torch.arange(0, rot_dim, 2, dtype=torch.float64) / max(rot_dim, 1))).float()


def rope_pair_axis(n_pairs: int, axes, interleaved: bool = False) -> list[int]:
    """The position axis of each of n_pairs pairs: runs of the lengths in
    ``axes`` (or of about equal length for a number of axes), or the axes in
    turn with ``interleaved``."""
    if not isinstance(axes, int):
        runs = list(axes)
        if sum(runs) != n_pairs:
            raise ValueError(f"runs of {runs} pairs do not make {n_pairs}")
        return [a for a, n in enumerate(runs) for _ in range(n)]
    if interleaved:
        return [j % axes for j in range(n_pairs)]
    return [min(axes - 1, j * axes // max(1, n_pairs)) for j in range(n_pairs)]
