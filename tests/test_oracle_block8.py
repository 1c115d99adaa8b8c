"""Pins of the 8-bit block-scaled cache's plain definition (oracle/block8.py)."""

import numpy as np
import pytest

from oracle import block8 as o8


def test_e4m3_values_and_rounding():
    v = o8.e4m3_values()
    assert v[0x7e] == 448 and v[0x08] == 2.0 ** -6 and v[0x01] == 2.0 ** -9 and np.isnan(v[0x7f]) and np.isnan(v[0xff])
    assert np.all(np.diff(v[:127]) > 0)
    codes = np.array([c for c in range(256) if c & 127 != 127], dtype=np.uint8)
    assert np.array_equal(o8.codes_of("e4m3_blk", o8.values_of("e4m3_blk", codes)), codes)
    # ties go to the even mantissa, beyond the largest saturates, NaN is 0
    assert o8.values_of("e4m3_blk", o8.codes_of("e4m3_blk", [1.0625, 1.1875, 500.0, -1e9, np.inf, np.nan])).tolist() == \
        [1.0, 1.25, 448.0, -448.0, 448.0, 0.0]
    # half a step of 2^-3 at most
    x = np.random.default_rng(0).uniform(2.0 ** -6, 448, 4000)
    assert np.max(np.abs(o8.values_of("e4m3_blk", o8.codes_of("e4m3_blk", x)) / x - 1)) <= 2.0 ** -4


def test_int8_rounding():
    y = [0.5, 1.5, -2.5, 126.5, 200.0, -np.inf, np.nan]
    assert o8.values_of("int8_blk", o8.codes_of("int8_blk", y)).tolist() == [0, 2, -2, 126, 127, -127, 0]


@pytest.mark.parametrize("fmt", ["e4m3_blk", "int8_blk"])
@pytest.mark.parametrize("block", [16, 64])
def test_rows_of_a_block_cover_it_once(fmt, block):
    f = o8.Block8(fmt, block, 3)
    seen = np.concatenate([o8._row_index(f, h, r, kv) for h in range(3) for r in range(block) for kv in (0, 1)])
    assert np.array_equal(np.sort(seen), np.arange(f.scale_off)) and f.block_bytes == f.scale_off + 128


@pytest.mark.parametrize("fmt,step", [("e4m3_blk", 2.0 ** -4), ("int8_blk", None)])
def test_store_and_read_back_within_half_a_step(fmt, step):
    rng = np.random.default_rng(1)
    f = o8.Block8(fmt, 16, 2)
    x = rng.standard_normal((2, 37, 2, 128)).astype(np.float32)
    cache = np.zeros(4 * f.block_bytes, dtype=np.uint8)
    table = [[3, 0, 2]]
    o8.store(f, cache, x[0], x[1], [0, 37], table, [37])
    k, v = o8.read(f, cache, table[0], 37)
    for got, want in ((k, x[0]), (v, x[1])):
        err = np.abs(got - want)
        for j in range(3):
            rows = slice(16 * j, 16 * j + 16)
            amax = np.abs(want[rows]).max((0, 2), keepdims=True)
            # int8: half a step of amax / 127; e4m3: half a step of the value, or of the smallest normal
            bound = amax / 254 if step is None else np.maximum(np.abs(want[rows]) * step, amax / 448 * 2.0 ** -10)
            assert np.all(err[rows] <= bound * (1 + 1e-5))


def test_a_growing_block_requantises_and_a_reused_one_starts_anew():
    f = o8.Block8("int8_blk", 16, 1)
    cache = np.zeros(f.block_bytes, dtype=np.uint8)
    one = np.full((1, 1, 128), 1.0, dtype=np.float32)
    o8.store(f, cache, one, one, [0, 1], [[0]], [1])
    assert o8.scale(f, cache, 0, 0, 0) == np.float32(1) / np.float32(127)
    o8.store(f, cache, 4 * one, one, [0, 1], [[0]], [2])
    assert o8.scale(f, cache, 0, 0, 0) == np.float32(4) / np.float32(127)
    assert set(o8.row_codes(f, cache, 0, 0, 0, 0).tolist()) == {32}      # 127 / 4, to nearest
    assert set(o8.row_codes(f, cache, 0, 0, 0, 1).tolist()) == {127}     # the values' scale did not grow
    o8.store(f, cache, one, one, [0, 1], [[0]], [1])                     # another sequence begins in the block
    assert o8.scale(f, cache, 0, 0, 0) == np.float32(1) / np.float32(127)


def test_attention_of_equal_keys_is_the_mean():
    v = np.arange(3 * 128, dtype=np.float64).reshape(3, 1, 128)
    out, size, _ = o8.attend(np.ones((2, 128)), np.ones((3, 1, 128)), v, 0.1)
    assert np.allclose(out, v.mean(0)) and np.allclose(size, out)
    assert not o8.attend(np.ones((2, 128)), np.ones((0, 1, 128)), v[:0], 0.1)[0].any()
