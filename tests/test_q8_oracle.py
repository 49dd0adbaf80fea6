"""Pins of the oracle's 8-bit cache format: closed forms and torch's own e4m3 type."""

import numpy as np
import pytest
import torch

import oracle as O


def test_table_and_encode_agree_with_torch():
    codes = torch.arange(256, dtype=torch.uint8)
    want = codes.view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(O.e4m3_table(), want)
    g = np.random.default_rng(0)
    x = np.concatenate([g.standard_normal(4000) * 2.0 ** g.integers(-12, 8, 4000), want[np.isfinite(want)],
                        # halfway between neighbours: ties to the even code
                        (want[:126] + want[1:127]) / 2, -(want[:126] + want[1:127]) / 2])
    x = x[np.abs(x) <= 448].astype(np.float32)
    got = O.e4m3_encode(x)
    ref = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    np.testing.assert_array_equal(got, ref)
    np.testing.assert_array_equal(O.e4m3_encode([1e9, -1e9, np.inf, np.nan, -0.0]), [0x7E, 0xFE, 0x7F, 0x7F, 0x80])


@pytest.mark.parametrize("amax,e", [(448.0, 0), (448.5, 1), (449.0, 1), (224.0, -1), (1.0, -8), (1.75, -8), (1.76, -7),
                                    (3.5, -7), (3.51, -6), (0.0, -100), (1e-38, -100), (3.3e38, 119)])
def test_need(amax, e):
    assert O.q8_need(amax) == 2.0 ** e


def test_append_in_order_keeps_values_and_scales_grow():
    g = np.random.default_rng(1)
    B, H, R, D = 2, 2, 96, 16
    codes, scales = np.zeros((B, H, R, D), np.uint8), np.full((B, H, O.q8_scale_cols(R)), np.nan)
    x = g.standard_normal((B, H, 70, D)) * 2.0 ** g.integers(-2, 5, (B, H, 70, 1))
    for t in range(70):
        codes, scales, _ = O.q8_append(codes, scales, x[:, :, t:t + 1], [t] * B)
    one, s1, kept = O.q8_append(np.zeros_like(codes), np.full_like(scales, np.nan), x, [0] * B)
    np.testing.assert_array_equal(scales[:, :, :3], s1[:, :, :3])
    assert kept[:, :70].all() and not kept[:, 70:].any()
    got, want = O.q8_values(codes, scales)[:, :, :70], O.q8_values(one, s1)[:, :, :70]
    step = np.repeat(s1, 32, axis=2)[:, :, :70, None]
    # token by token: the same but for values below 2^-6 scales, moved once per growth (each
    # time by at most half of their step of 2^-9)
    small = np.abs(want) < step * 2.0 ** -6
    np.testing.assert_array_equal(got[~small], want[~small])
    assert np.all(np.abs(got - want)[small] <= (step * 2.0 ** -9 + 0 * want)[small])
    # and both within half an e4m3 step of the input
    assert np.all(np.abs(want - x) <= np.maximum(np.abs(x) * 2.0 ** -4, step * 2.0 ** -10))


def test_ring_append_restarts_a_block():
    codes, scales = np.full((1, 1, 64, 16), 0x38, np.uint8), np.full((1, 1, 4), 4.0)   # all values 4
    new = np.full((1, 1, 2, 16), 0.875)
    c, s, kept = O.q8_append(codes, scales, new, [64])
    assert s[0, 0, 0] == 2.0 ** -9 and s[0, 0, 1] == 4.0
    assert np.all(O.q8_values(c, s)[0, 0, :2] == 0.875) and not kept[0, 2:32].any() and kept[0, 32:].all()
    c, s, kept = O.q8_append(codes, scales, new, [65])     # joins a block: its larger scale stays
    assert s[0, 0, 0] == 4.0 and np.all(O.q8_values(c, s)[0, 0, 0] == 4.0)
