"""Pins of the oracle's 4-bit cache: the code table, rounding and ties, block scales, row addresses."""

import numpy as np
import pytest
import torch

from oracle import e4m3, fp4, kvcache
from tests.fp4_cases import Fp4Case


def test_code_table_and_ties():
    assert fp4.decode(np.arange(16)).tolist() == [0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6]
    x = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 0.2500001, 0.7499999, 5.0000005, 7.0, np.inf, -0.1, -5.0], np.float32)
    want = [0, 2, 2, 4, 4, 6, 6, 1, 1, 7, 7, 7, 8, 14]
    assert fp4.encode_f32(x).tolist() == want


def test_encode_is_the_nearest_code():
    x = np.random.default_rng(3).standard_normal(20000).astype(np.float32) * 3
    got = fp4.decode(fp4.encode_f32(x))
    best = np.abs(np.clip(x, -6, 6)[:, None].astype(np.float64) - fp4.decode(np.arange(16))[None]).min(1)
    assert np.array_equal(np.abs(np.clip(x, -6, 6).astype(np.float64) - got), best)


def test_block_scale_and_error():
    """The largest of a block lands within a scale rounding of code 6, and no value is off by more than
    half a code step (1/6 of the block's largest, 2^-4 more for the scale's rounding)."""
    x = torch.randn(64, 128, generator=torch.Generator().manual_seed(1)).numpy()
    g = np.float32(np.abs(x).max() / 2688)
    codes, scales = fp4.quantise(x, g)
    y = fp4.dequantise(codes, scales, g)
    amax = np.abs(x.reshape(64, 8, 16)).max(-1).repeat(16, -1).reshape(64, 128)
    assert np.all(np.abs(y - x) <= amax / 6 * (1 + 2.0 ** -4))
    assert np.abs(y - x).mean() < 0.1 * np.abs(x).mean()


def test_block_scale_by_hand():
    """amax 12 and g 1: scale e4m3(2) = 2, codes of 12, 1, 0.5, -3 = 6, 0.5, 0 (0.25 ties to 0), -1.5."""
    x = np.zeros((1, 128), np.float32)
    x[0, :4] = [12, 1, 0.5, -3]
    codes, scales = fp4.quantise(x, 1.0)
    assert e4m3.decode(scales)[0].tolist() == [2, 0, 0, 0, 0, 0, 0, 0]
    assert codes[0, :2].tolist() == [7 | 1 << 4, 0 | 11 << 4] and not codes[0, 2:].any()


@pytest.mark.parametrize("fill,want", [(np.nan, 0.0), (0.0, 0.0), (np.inf, 2688.0), (-np.inf, -2688.0), (1e-30, 0.0)])
def test_special_values(fill, want):
    x = np.zeros((1, 128), np.float32)
    x[0, 3] = fill
    y = fp4.dequantise(*fp4.quantise(x, 1.0), 1.0)
    assert y[0, 3] == want and np.isfinite(y).all()


def test_rows_land_where_the_layout_says():
    c = Fp4Case([300, 400], [True, False], seed=5).fill()
    t = c.segs[0].page_table
    for g in (0, 1):
        codes, scales = fp4.quantise(kvcache.bf16_to_f32(c.k_bits[0][g, 290]), c.cache.k_scale[g])
        block = c.cache.k_pool[t[1], g]                    # position 290: page 1, row 34 of its first half
        assert np.array_equal(block[34 * 64: 35 * 64], codes)
        assert np.array_equal(block[8192 + 34 * 8: 8192 + 35 * 8], scales)
        codes, scales = fp4.quantise(kvcache.bf16_to_f32(c.v_bits[1][g, 399]), c.cache.v_scale[g])
        block = c.segs[1].v_slab[g, 1]                     # position 399: second block, row 143, second half
        assert np.array_equal(block[9216 + 15 * 64: 9216 + 16 * 64], codes)
        assert np.array_equal(block[9216 + 8192 + 15 * 8: 9216 + 8192 + 16 * 8], scales)
    K, V = kvcache.gather(c.cache, c.segs[0], 1, 300)
    assert np.isfinite(K).all() and K.shape == (300, 128)
    x = kvcache.bf16_to_f32(c.k_bits[0][1]).astype(np.float64)
    assert np.abs(K - x).mean() < 0.12 * np.abs(x).mean()
