"""Pins of the attention side's oracle (hand-worked cases) and of the cache's
documented layout (CPU only)."""

import math

import numpy as np
import pytest
import torch

from mxfp8_moe_decode_gb300 import kv_dequant_x8
from oracle import attention as A


def test_add_rounds_once_to_bf16():
    # 1 + 2^-8 is half a bf16 step above 1: to even, 1; 1 + 3 * 2^-8: to 1 + 2^-6
    x = np.array([[1.0, 1.0 + 2.0 ** -7, 3.0e38, -1.0]])
    r = np.array([[2.0 ** -8, 2.0 ** -8, 2.0 ** -60, 1.0]])
    x = A.bf16_rne(x)
    got = A.add(x, r)
    assert got[0, 0] == 1.0 and got[0, 1] == 1.0 + 2.0 ** -6
    assert got[0, 2] == x[0, 2] and got[0, 3] == 0.0


@pytest.mark.parametrize("d", [64, 128, 256])
def test_images_hold_every_byte_once(d):
    for image in A.image_bytes(d):
        assert sorted(image.reshape(-1).tolist()) == list(range(64 * d))


def test_images_by_hand():
    key, value = A.image_bytes(128)
    assert key[0, 0] == 0 and key[0, 17] == 17
    assert key[1, 0] == 128 + 16 and key[9, 16] == 9 * 128  # token 9 swaps chunks 0 and 1
    key, value = A.image_bytes(64)
    assert key[2, 0] == 2 * 64 + 16  # rows of 64 bytes turn every second token
    # value words hold tokens 2i, 2i + 1, 2i + 8, 2i + 9
    assert [int(value[t, 0]) for t in (0, 1, 8, 9, 2, 3, 10, 11, 16)] == [0, 1, 2, 3, 4, 5, 6, 7, 16]
    assert value[0, 2] == 2 * 64 + 16 and value[0, 7] == 7 * 64 + 48


@pytest.mark.parametrize("d", [64, 128, 256])
def test_binding_reads_the_same_layout(d):
    rng = np.random.default_rng(d)
    b = rng.integers(0, 256, (2, 3, 2, 64 * d), dtype=np.uint8)
    c = rng.integers(100, 150, (2, 3, 2), dtype=np.uint8)
    got = kv_dequant_x8(torch.from_numpy(b), torch.from_numpy(c)).numpy()
    np.testing.assert_array_equal(got, A.cache_values(b, c).astype(np.float32))


def test_append_by_hand():
    d = 64
    blocks = np.full((2, 1, 2, 64 * d), 0x7F, dtype=np.uint8)
    codes = np.zeros((2, 1, 2), dtype=np.uint8)
    table = [[1]]
    k = np.zeros((1, 1, d))
    k[0, 0, :3] = [448.0, -1.0, 2.0 ** -9]  # amax 448: code 127, values as they are
    blocks, codes = A.append(blocks, codes, k, -k, table, [0], [0, 1])
    assert codes[1, 0].tolist() == [127, 127] and codes[0].max() == 0
    val = A.cache_values(blocks, codes)[1, 0]
    assert val[0, 0, :3].tolist() == [448.0, -1.0, 2.0 ** -9] and (val[1, 0] == -val[0, 0]).all()
    assert np.isnan(val[0, 1:]).all()
    # a second token of amax 449 (code 128): the first one's bytes halve; its
    # smallest value, half the smallest subnormal, ties to even: 0
    k2 = np.zeros((1, 1, d))
    k2[0, 0, :2] = [449.0, 16.0]
    blocks, codes = A.append(blocks, codes, k2, k2 / 449.0, table, [1], [0, 1])
    assert codes[1, 0].tolist() == [128, 127]  # the values' scale stays
    val = A.cache_values(blocks, codes)[1, 0]
    assert val[0, 0, :3].tolist() == [448.0, -1.0, 0.0]
    assert val[0, 1, :2].tolist() == [448.0, 16.0]  # 449 to the step of 32: 448
    # the same again changes nothing; non-finite values leave the scale alone
    again = A.append(blocks, codes, k2, k2 / 449.0, table, [1], [0, 1])
    assert np.array_equal(again[0], blocks) and np.array_equal(again[1], codes)
    k3 = np.ones((1, 1, d))
    k3[0, 0, :2] = [math.inf, math.nan]
    blocks, codes = A.append(blocks, codes, k3, k3, table, [2], [0, 1])
    assert codes[1, 0].tolist() == [128, 127]
    val = A.cache_values(blocks, codes)[1, 0]
    assert val[0, 2, 0] == 896.0 and np.isnan(val[0, 2, 1]) and val[0, 2, 2] == 1.0


def test_visible_by_hand():
    assert A.visible(3, 10, 0, 0) == [0, 1, 2, 3]
    assert A.visible(5, 10, 2, 0) == [4, 5]
    assert A.visible(5, 10, 2, 1) == [0, 4, 5]
    assert A.visible(1, 10, 4, 9) == [0, 1]  # sinks never reach past the row
    assert A.visible(-1, 0, 0, 0) == []


def test_attention_by_hand():
    d = 64
    values = np.zeros((1, 1, 2, 64, d))
    values[0, 0, 0, :, 0] = [0.0, math.log(3.0)] + [50.0] * 62
    values[0, 0, 1, :, 0] = [4.0, 8.0] + [math.nan] * 62
    q = np.zeros((2, 1, d))
    q[:, 0, 0] = 1.0
    out, lse, spread, _ = A.attention(q, values, [[0]], [2], [0, 2], 1.0)
    # row 0 sees token 0 alone; row 1 weighs 1 : 3
    assert out[0, 0, 0] == 4.0 and lse[0, 0] == 0.0
    assert abs(out[1, 0, 0] - 7.0) < 1e-12 and abs(lse[1, 0] - math.log(4.0)) < 1e-12
    # a row before the first token sees nothing
    out, lse, _, _ = A.attention(q, values, [[0]], [1], [0, 2], 1.0)
    assert (out[0] == 0).all() and lse[0, 0] == -math.inf and out[1, 0, 0] == 4.0
