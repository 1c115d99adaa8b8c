"""16-bit KV cache: position rotation, addressing and attention, plainly.

Cache: ``cache[num_blocks]`` of n_kv * block * 256 16-bit numbers: tiles [n_kv]
[block / 16] of 16 key rows then 16 value rows of 128 numbers, coordinate j of
row r at number (r // 8) * 1024 + (j // 64) * 512 + (r % 8) * 64 +
8 * ((j // 8 % 8) ^ (r % 8)) + j % 8. Everything is float64; numbers are rounded
once, where they are stored.
"""

from __future__ import annotations

from dataclasses import dataclass

import numpy as np

D = 128


@dataclass(frozen=True)
class Kv16:
    dtype: str          # "bf16" | "fp16"
    block: int
    n_kv: int

    @property
    def block_bytes(self):
        return self.n_kv * self.block * 4 * D


def bits_to_numbers(dtype, bits):
    bits = np.asarray(bits, dtype=np.uint16)
    if dtype == "fp16":
        return bits.view(np.float16).astype(np.float64)
    with np.errstate(invalid="ignore"):
        return (bits.astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def half_step(dtype, x):
    """Half the distance between neighbours of the type around |x|: what one rounding may cost."""
    bits, least = (8, -126) if dtype == "bf16" else (11, -14)
    e = np.maximum(np.frexp(np.abs(x))[1] - 1, least)
    return np.ldexp(0.5, e - bits + 1)


def row_index(f: Kv16, blk, h, row, kv):
    """Places in the cache, in numbers, of the 128 coordinates of one row (arrays of blk and row: [.., 128])."""
    j = np.arange(D)
    blk, row = np.asarray(blk, dtype=np.int64)[..., None], np.asarray(row)[..., None]
    return ((blk * f.n_kv + h) * f.block * 2 * D + (row // 16) * 4096 + kv * 2048 + (row % 16 // 8) * 1024 + (j // 64) * 512 +
            (row % 8) * 64 + 8 * ((j // 8 % 8) ^ (row % 8)) + j % 8)


def rotate(x, angles, style):
    """x [rows, heads, d], angles [rows, rot] (cosines, then sines): the rotated x, and the sum of the
    magnitudes that each coordinate was made of."""
    x = np.asarray(x, dtype=np.float64)
    y, size = x.copy(), np.abs(x)
    half = angles.shape[1] // 2
    for j in range(half):
        a, b = (j, j + half) if style == "halves" else (2 * j, 2 * j + 1)
        c, s = angles[:, j, None].astype(np.float64), angles[:, half + j, None].astype(np.float64)
        with np.errstate(invalid="ignore"):
            y[..., a] = x[..., a] * c - x[..., b] * s
            y[..., b] = x[..., b] * c + x[..., a] * s
        size[..., a] = np.abs(x[..., a] * c) + np.abs(x[..., b] * s)
        size[..., b] = np.abs(x[..., b] * c) + np.abs(x[..., a] * s)
    return y, size


def read(f: Kv16, cache, table_row, length, blocks=None):
    """K, V [length, n_kv, d] float64 of one sequence; positions of a block id outside [0, blocks) are NaN."""
    bits = cache.view(np.uint16)
    out = np.full((2, length, f.n_kv, D), np.nan)
    p = np.arange(length)
    blk = np.asarray(table_row)[p // f.block].astype(np.int64)
    live = blk >= 0 if blocks is None else (blk >= 0) & (blk < blocks)
    for h in range(f.n_kv):
        for kv in (0, 1):
            out[kv, live, h] = bits_to_numbers(f.dtype, bits[row_index(f, blk[live], h, p[live] % f.block, kv)])
    return out[0], out[1]


def put(f: Kv16, cache, table_row, first, key_bits, value_bits):
    """Writes rows (uint16 [n, n_kv, d]) as positions first .. first + n - 1 of a sequence, in place."""
    bits = cache.view(np.uint16)
    p = first + np.arange(len(key_bits))
    blk = np.asarray(table_row)[p // f.block]
    for h in range(f.n_kv):
        bits[row_index(f, blk, h, p % f.block, 0)] = key_bits[:, h]
        bits[row_index(f, blk, h, p % f.block, 1)] = value_bits[:, h]
