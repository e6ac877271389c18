"""Pins of the scaled-cache oracle: scales against their definition, rotations
against complex multiplication, attention against closed forms and against the
oracle of the cache with one scale."""
import numpy as np
import pytest
import torch

import oracle
from oracle import scaled as OS


def test_power_of_two_scale_is_the_smallest():
    for bound in (1e-30, 0.001, 1.0, 447.9, 448.0, 448.1, 1e5, 3e38):
        bound = float(np.float32(bound))
        s = float(OS.power_of_two_scale(bound))
        assert bound <= 448 * s and np.log2(s) == int(np.log2(s))
        assert s == 2.0 ** -126 or bound > 448 * (s / 2)
    assert OS.power_of_two_scale(0.0) == np.float32(2.0 ** -126)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_is_a_complex_product(interleaved):
    r = np.random.default_rng(0)
    x = r.standard_normal((5, 3, 64))
    f = 10000.0 ** (-np.arange(0, 32, 2) / 32)
    pos = np.array([0, 1, 17, 4095, 1 << 20])
    y = OS.rotate(x, pos, f, interleaved, 1.25)
    z = 1.25 * np.exp(1j * pos[:, None] * f)[:, None]
    a = x[..., 0:32:2] + 1j * x[..., 1:32:2] if interleaved else x[..., :16] + 1j * x[..., 16:32]
    w = a * z
    got = y[..., 0:32:2] + 1j * y[..., 1:32:2] if interleaved else y[..., :16] + 1j * y[..., 16:32]
    # np.exp's argument: 2^20 at 2^-53 relative
    np.testing.assert_allclose(got, w, rtol=0, atol=8 * 2.0 ** -32)
    assert np.array_equal(y[..., 32:], x[..., 32:]) and np.array_equal(y[0, :, 32:], x[0, :, 32:])


def test_attention_matches_the_one_scale_oracle_when_all_scales_agree():
    r = np.random.default_rng(1)
    nb, hkv, bs, d, G = 9, 2, 16, 64, 3
    k = r.integers(0, 0x7f, (nb, hkv, bs, d)).astype(np.uint8)
    v = r.integers(0, 0x7f, (nb, hkv, bs, d)).astype(np.uint8)
    scales = np.full((nb, hkv, 2), 2.0 ** -9, np.float32)
    tables = r.permutation(nb).astype(np.int32).reshape(1, nb)
    ctx = np.array([nb * bs - 5], np.int32)
    q = r.standard_normal((1, hkv * G, d)).astype(np.float16)
    ref = oracle.paged_attention_decode(k, v, oracle.E4M3, q.view(np.uint16), oracle.F16, tables,
                                        ctx, 0.125, 2.0 ** -9, 2.0 ** -9)
    got = OS.attention(k, v, scales, q.astype(np.float64), np.array([0, 1]), tables, ctx, 0.125)
    np.testing.assert_allclose(got, ref, rtol=1e-10, atol=1e-12)


def test_append_token_by_token_keeps_the_values():
    """A block filled one token at a time holds what one call would have written,
    but for the older codes' second rounding."""
    r = np.random.default_rng(2)
    raw = r.standard_normal((16, 1, 64)) * np.exp2(np.arange(16) / 2)[:, None, None]
    raw = raw.astype(np.float16).astype(np.float64)
    one = np.full((1, 1, 16, 64), 0xff, np.uint8)
    step = one.copy()
    s1, s2 = np.full((1, 1, 2), np.nan, np.float32), np.full((1, 1, 2), np.nan, np.float32)
    table = np.zeros((1, 1), np.int32)
    OS.append_scaled(one, s1, 0, raw, raw, 1.0, [0, 16], table, [16])
    for i in range(16):
        OS.append_scaled(step, s2, 0, raw[i:i + 1], raw[i:i + 1], 1.0, [0, 1], table, [i + 1])
    assert s1[0, 0, 0] == s2[0, 0, 0]
    a, b = OS.gather(one, s1, 0, table[0], 16, 0), OS.gather(step, s2, 0, table[0], 16, 0)
    # each rounding is half a step of a subnormal at the scale it was made with
    assert np.abs(a - b).max() <= 2 * 2.0 ** -10 * s1[0, 0, 0]
    assert np.abs(a - raw[:, 0]).max() <= np.abs(raw).max() * 2.0 ** -4
    t = torch.from_numpy(one[0, 0].copy()).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(t * float(s1[0, 0, 0]), a)
