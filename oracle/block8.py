"""8-bit KV cache with one fp32 scale per (block, KV head), keys and values apart.

Plain definition of the store, the read-back and the attention over the cache.
Decisions that fix bytes (scales, codes) are taken in IEEE fp32 as the method
states them; everything else is float64.

Cache: ``cache[num_blocks]`` of ``block_bytes``: tiles [n_kv][block / 16] of
4096 bytes (16 key rows of 128 codes, then 16 value rows; coordinate j of row r
at byte 128 r + 16 ((j // 16) ^ (r & 7)) + j % 16), then [n_kv][2] fp32 scales
(key, value), padded to a multiple of 128 bytes.
"""

from __future__ import annotations

from dataclasses import dataclass

import numpy as np

D = 128
FLOOR = np.float32(2.0 ** -100)


@dataclass(frozen=True)
class Block8:
    fmt: str            # "e4m3_blk" | "int8_blk"
    block: int
    n_kv: int

    @property
    def limit(self):
        return np.float32(127 if self.fmt == "int8_blk" else 448)

    @property
    def scale_off(self):
        return self.n_kv * self.block * 2 * D

    @property
    def block_bytes(self):
        return self.scale_off + -(-8 * self.n_kv // 128) * 128


def e4m3_values():
    """The 256 e4m3 numbers by code (NaN at 0x7f and 0xff)."""
    out = np.empty(256)
    for code in range(256):
        e, m = (code >> 3) & 15, code & 7
        x = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        out[code] = np.nan if code & 127 == 127 else (-x if code & 128 else x)
    return out


_E4M3 = e4m3_values()


def values_of(fmt, codes):
    codes = np.asarray(codes, dtype=np.uint8)
    return codes.view(np.int8).astype(np.float64) if fmt == "int8_blk" else _E4M3[codes]


def codes_of(fmt, y):
    """fp32 values to codes: nearest, ties to even, saturated; NaN to 0."""
    y = np.asarray(y, dtype=np.float64)
    y = np.where(np.isnan(y), 0.0, y)
    if fmt == "int8_blk":
        return np.rint(np.clip(y, -127, 127)).astype(np.int8).view(np.uint8)
    grid = _E4M3[:127]                              # ascending, 0 .. 448; even codes have an even mantissa
    a = np.minimum(np.abs(y), 448.0)
    hi = np.clip(np.searchsorted(grid, a), 1, 126)  # grid[hi - 1] < a <= grid[hi]
    lo = hi - 1
    up, down = grid[hi] - a, a - grid[lo]
    code = np.where(up < down, hi, np.where(down < up, lo, np.where(hi % 2 == 0, hi, lo))).astype(np.uint8)
    return np.where(np.signbit(y), code | 128, code).astype(np.uint8)


def _row_index(f: Block8, h, row, kv):
    """Byte offsets in a block of the 128 codes of (head, row, keys or values)."""
    j = np.arange(D)
    return (h * f.block * 2 * D + (row // 16) * 4096 + kv * 2048 + (row % 16) * D +
            16 * ((j // 16) ^ (row % 8)) + j % 16)


def scale(f: Block8, cache, blk, h, kv):
    at = blk * f.block_bytes + f.scale_off + 8 * h + 4 * kv
    return cache[at:at + 4].view(np.float32)[0]


def _set_scale(f: Block8, cache, blk, h, kv, s):
    at = blk * f.block_bytes + f.scale_off + 8 * h + 4 * kv
    cache[at:at + 4] = np.array([s], dtype=np.float32).view(np.uint8)


def row_codes(f: Block8, cache, blk, h, row, kv):
    return cache[blk * f.block_bytes + _row_index(f, h, row, kv)]


def store(f: Block8, cache, key, value, query_start, table, seq_lens):
    """Writes the chunks into `cache` (bytes, in place); key, value [rows, n_kv, d] float32."""
    for b in range(len(seq_lens)):
        q0, q1 = int(query_start[b]), int(query_start[b + 1])
        start, end = int(seq_lens[b]) - (q1 - q0), int(seq_lens[b])
        for j in range(start // f.block, -(-end // f.block)) if end > start else ():
            blk = int(table[b][j])
            first, last = max(start - j * f.block, 0), min(end - j * f.block, f.block)
            for h in range(f.n_kv):
                for kv, src in ((0, key), (1, value)):
                    x = src[q0 + j * f.block + first - start: q0 + j * f.block + last - start, h].astype(np.float32)
                    finite = np.abs(x[np.isfinite(x)])
                    amax = finite.max() if finite.size else np.float32(0)
                    s = max(np.float32(amax / f.limit), FLOOR)
                    old = None
                    if first:
                        old = scale(f, cache, blk, h, kv)
                        s = max(s, old)
                    inv = np.float32(1) / s
                    if old is not None and s > old:
                        ratio = np.float32(old / s)
                        for r in range(first):
                            at = blk * f.block_bytes + _row_index(f, h, r, kv)
                            cache[at] = codes_of(f.fmt, (values_of(f.fmt, cache[at]).astype(np.float32) * ratio))
                    for r in range(first, last):
                        with np.errstate(invalid="ignore", over="ignore"):
                            y = x[r - first] * inv
                        cache[blk * f.block_bytes + _row_index(f, h, r, kv)] = codes_of(f.fmt, y)
                    _set_scale(f, cache, blk, h, kv, s)


def read(f: Block8, cache, table_row, length, blocks=None):
    """K, V [length, n_kv, d] float64 of one sequence; positions of a block id outside [0, blocks) are NaN."""
    out = np.full((2, length, f.n_kv, D), np.nan)
    for p in range(length):
        blk = int(table_row[p // f.block])
        if blocks is not None and not 0 <= blk < blocks:
            continue
        for h in range(f.n_kv):
            for kv in (0, 1):
                out[kv, p, h] = values_of(f.fmt, row_codes(f, cache, blk, h, p % f.block, kv)) * float(scale(f, cache, blk, h, kv))
    return out[0], out[1]


def attend(q, k, v, softmax_scale):
    """q [n_q, d], k, v [n, n_kv, d] float64 -> (out [n_q, d], mean |v| under the weights [n_q, d],
    largest sum of |q k| [n_q]); positions that are NaN are left out; nothing seen gives zeros."""
    n_q, group = q.shape[0], q.shape[0] // k.shape[1]
    out, size, reach = np.zeros((n_q, D)), np.zeros((n_q, D)), np.zeros(n_q)
    for h in range(n_q):
        kk, vv = k[:, h // group], v[:, h // group]
        live = ~np.isnan(kk).any(1)
        kk, vv = kk[live], vv[live]
        if not len(kk):
            continue
        s = kk @ q[h] * softmax_scale
        p = np.exp(s - s.max())
        p /= p.sum()
        out[h], size[h] = p @ vv, p @ np.abs(vv)
        reach[h] = (np.abs(kk) @ np.abs(q[h]) * softmax_scale).max()
    return out, size, reach
