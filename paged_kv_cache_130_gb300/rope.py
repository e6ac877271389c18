"""Frequencies of rotary positions, on the host in 64 bits.

``pkv_rope_append`` takes the radians that each pair of head elements turns per
position, so any way of stretching positions for long contexts is a matter of
the frequencies handed to it.  The kinds here:

* plain: ``base ** (-2 i / rot_dim)``;
* linear: positions divided by ``factor``;
* ntk: the base raised so that the slowest pair is divided by ``factor`` and the
  fastest stays (``base * factor ** (r / (r - 2))``);
* yarn: by parts (Peng et al., "YaRN", 2023): pairs that turn more than
  ``beta_fast`` times over the trained length stay, pairs that turn less than
  ``beta_slow`` times are divided by ``factor``, linear in the turns between;
  q and K are multiplied by ``0.1 ln(factor) + 1``.  This is the paper's ramp.
  Implementations that ramp linearly over the pair's index instead give other
  frequencies in between: for a checkpoint trained with those, hand its own
  frequencies to the call.
"""
import math

import torch


def inv_freq(rot_dim, base=10000.0, scaling=None, factor=1.0, trained_len=4096, beta_fast=32.0,
             beta_slow=1.0):
    """(float64 [rot_dim / 2] on the host, mscale) for ``pkv_rope_append``."""
    if rot_dim <= 0 or rot_dim % 2:
        raise ValueError("rot_dim must be positive and even")
    if not base > 0 or not factor > 0:
        raise ValueError("base and factor must be positive")
    r = int(rot_dim)
    power = -torch.arange(0, r, 2, dtype=torch.float64) / r
    if scaling is None:
        return float(base) ** power, 1.0
    if scaling == "linear":
        return float(base) ** power / factor, 1.0
    if scaling == "ntk":
        if r == 2:
            raise ValueError("ntk needs more than one pair")
        return (base * factor ** (r / (r - 2))) ** power, 1.0
    if scaling == "yarn":
        if not beta_fast > beta_slow or trained_len <= 0:
            raise ValueError("yarn needs beta_fast > beta_slow and a trained length")
        f = float(base) ** power
        turns = trained_len * f / (2 * math.pi)
        keep = ((turns - beta_slow) / (beta_fast - beta_slow)).clamp(0, 1)
        return f * keep + f / factor * (1 - keep), 0.1 * math.log(factor) + 1 if factor > 1 else 1.0
    raise ValueError("unknown scaling %r" % (scaling,))
