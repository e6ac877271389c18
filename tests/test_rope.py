"""Frequencies of rotary positions against their definitions."""
import math

import pytest

from paged_kv_cache_130_gb300 import rope


def test_plain_and_linear():
    f, m = rope.inv_freq(128)
    assert m == 1.0 and f.shape == (64,) and float(f[0]) == 1.0
    assert math.isclose(float(f[63]), 10000.0 ** (-126 / 128), rel_tol=1e-14)
    g, _ = rope.inv_freq(128, scaling="linear", factor=4)
    assert (g * 4 - f).abs().max() == 0


def test_ntk_keeps_the_fastest_and_divides_the_slowest():
    f, _ = rope.inv_freq(64)
    g, _ = rope.inv_freq(64, scaling="ntk", factor=8)
    assert float(g[0]) == 1.0
    assert math.isclose(float(g[-1]), float(f[-1]) / 8, rel_tol=1e-12)


def test_yarn_by_parts():
    f, _ = rope.inv_freq(128)
    g, m = rope.inv_freq(128, scaling="yarn", factor=32, trained_len=4096)
    turns = 4096 * f / (2 * math.pi)
    assert (g[turns >= 32] == f[turns >= 32]).all()
    assert ((g - f / 32)[turns <= 1].abs() <= 1e-18).all()
    mid = (turns > 1) & (turns < 32)
    assert mid.any() and (g[mid] < f[mid]).all() and (g[mid] > f[mid] / 32).all()
    assert math.isclose(m, 0.1 * math.log(32) + 1)
    assert rope.inv_freq(128, scaling="yarn", factor=1.0)[1] == 1.0


@pytest.mark.parametrize("kw", [dict(rot_dim=0), dict(rot_dim=7), dict(rot_dim=8, base=0),
                                dict(rot_dim=8, scaling="other"), dict(rot_dim=2, scaling="ntk"),
                                dict(rot_dim=8, scaling="linear", factor=0),
                                dict(rot_dim=8, scaling="yarn", beta_fast=1.0)])
def test_refusals(kw):
    with pytest.raises(ValueError):
        rope.inv_freq(**kw)
