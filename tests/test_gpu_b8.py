"""GPU parity of the 8-bit block-scaled cache (tq_b8_*) with oracle/block8.py.

Store and read-back are compared bit for bit: scales and codes are defined in
IEEE fp32, a read-back value is one fp32 product rounded once. Attention is
compared within ``tolerance``, a bound derived from the arithmetic.
"""

import numpy as np
import pytest
import torch

from oracle import block8 as o8

pytestmark = pytest.mark.gpu

FMTS = ["e4m3_blk", "int8_blk"]
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "f32": torch.float32}
SCALE = 1.0 / np.sqrt(128.0)


@pytest.fixture(scope="module")
def tq():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need CUDA")
    from turboquant_paged_kv_gb300 import build
    build.build()
    import turboquant_paged_kv_gb300 as tq
    return tq


class Case:
    """A cache of random bytes, a shuffled block table with -1 behind each
    sequence, and room for `room` positions of every sequence."""

    def __init__(self, tq, fmt, block, n_q, n_kv, room, seed=0, spare=2):
        self.rng = np.random.default_rng(seed)
        self.f = o8.Block8(fmt, block, n_kv)
        self.cfg = tq.make_config(fmt, n_q, n_kv, block_size=block)
        self.tq, self.n_q, self.n_kv, self.block = tq, n_q, n_kv, block
        need = [-(-r // block) for r in room]
        self.blocks = sum(need) + spare
        perm = self.rng.permutation(self.blocks)
        self.table = np.full((len(room), max(max(need), 1)), -1, dtype=np.int32)
        at = 0
        for b, k in enumerate(need):
            self.table[b, :k] = perm[at:at + k]
            at += k
        self.cache = self.rng.integers(0, 256, self.blocks * self.f.block_bytes, dtype=np.uint8)
        self.lens = np.zeros(len(room), dtype=np.int32)

    def draw(self, rows, heads, dtype="bf16", gain=1.0, outlier=False):
        x = torch.from_numpy(self.rng.standard_normal((rows, heads, 128)).astype(np.float32) * gain)
        if outlier and rows:
            x[:, :, 5] *= 8.0
        return x.to(DT[dtype])

    def fill(self, lens, gain_v=None):
        """Every sequence written by the oracle, in chunks of its own blocks; gain_v(block) scales the values."""
        for b, n in enumerate(lens):
            k = self.draw(n, self.n_kv, outlier=True).float().numpy()
            v = self.draw(n, self.n_kv).float().numpy()
            if gain_v is not None:
                for j in range(0, n, self.block):
                    v[j:j + self.block] *= np.float32(gain_v(j // self.block))
            o8.store(self.f, self.cache, k, v, [0, n], self.table[b:b + 1], [n])
        self.lens = np.array(lens, dtype=np.int32)
        return self

    def gpu(self):
        return (torch.from_numpy(self.cache).cuda(), torch.from_numpy(self.table).cuda(), torch.from_numpy(self.lens).cuda())

    def floor(self, b, n, chunks=False):
        """What the fp16 weights' smallest step may cost (see tolerance), per query head."""
        v = np.abs(self.kv(b, n)[1])
        if chunks:
            s = np.array([[o8.scale(self.f, self.cache, int(self.table[b, p // self.block]), h, 1) if not np.isnan(v[p, h, 0]) else 0.0
                           for h in range(self.n_kv)] for p in range(n)]).reshape(n, self.n_kv, 1)
            v = np.divide(v * s.max(0, initial=0.0), s, out=np.zeros_like(v), where=s > 0)
        return np.repeat(2.0 ** -24 * np.nansum(v, 0), self.n_q // self.n_kv, 0)

    def kv(self, b, length=None, cache=None):
        return o8.read(self.f, self.cache if cache is None else cache, self.table[b], int(self.lens[b] if length is None else length),
                       self.blocks)


def starts_of(q_lens):
    return np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32)


def run_store(c, key, value, starts, lens, max_q=None, status=None, cache=None):
    cache = torch.from_numpy(c.cache).cuda() if cache is None else cache
    q = np.diff(starts)
    c.tq.tq_b8_store(c.cfg, key.cuda() if not key.is_cuda else key, value.cuda() if not value.is_cuda else value,
                     torch.from_numpy(np.asarray(starts, dtype=np.int32)).cuda(), int(q.max(initial=0)) if max_q is None else max_q, cache,
                     torch.from_numpy(c.table).cuda(), torch.from_numpy(np.asarray(lens, dtype=np.int32)).cuda(), dev_status=status)
    torch.cuda.synchronize()
    return cache


def tolerance(ref, size, reach, length, out_dtype, floor, single_p=False):
    """Bound on |kernel - exact| per element. size: sum p |v|; reach: the largest
    softmax_scale sum |q k| of a position.
      scores: 128 exact products summed in fp32 (an add errs by at most 2^-23 of
        the running sum of magnitudes) and 4 more roundings: reach 132 2^-23 in
        natural-log units, in the numerator and in the denominator; x - max once
        more, of magnitude 2 reach at most
      weights: ex2.approx 2^-22, the two fp16 parts of p s_v 2^-21 (one part,
        `single_p`: half a step, 2^-11)
      sums over the positions: length 2^-23 in either sum, and some for the merge
      floor: fp16 weights have no step below 2^-24, so a weight errs by up to
        2^-25 whatever its size. The kernels hold P = 8 p s_v / sigma, the largest
        p of a row being at least 1: the output errs by up to
        2^-28 sum_p |code_p| sigma. One query at a time, sigma <= 16 s_v of the
        position, so floor = 2^-24 sum_p |v_p|; chunks, sigma <= 16 times the
        largest s_v of all positions, so floor = 2^-24 sum_p |v_p| s_max / s_v(p).
    then half a step of the output's type."""
    delta = reach[..., None] * (132 + 4) * 2.0 ** -23
    p = 2.0 ** -11 * 1.01 if single_p else 2.0 ** -21
    rel = 2 * delta * 1.01 + 2.0 ** -21 + p + 2 * (length + 64) * 2.0 ** -23
    t = DT[out_dtype]
    least = {"f32": 1e-37, "bf16": 1e-37, "fp16": 2.0 ** -25}[out_dtype]
    inner = size * rel + floor
    return inner + (np.abs(ref) + inner) * torch.finfo(t).eps / 2 * 1.0001 + least


def run_decode(c, q, lens=None, out_dtype="f32", status=None, max_len=None, scale=0.0, stream=None):
    cache, table, _ = c.gpu()
    lens = c.lens if lens is None else np.asarray(lens, dtype=np.int32)
    lens_d = torch.from_numpy(lens).cuda()
    msl = max(int(lens.max(initial=0)), 1) if max_len is None else max_len
    out = torch.full(q.shape, float("nan"), dtype=DT[out_dtype], device="cuda")
    ws = torch.full((c.tq.tq_b8_decode_workspace_size(c.cfg, q.shape[0], msl),), 255, dtype=torch.uint8, device="cuda")
    c.tq.tq_b8_decode(c.cfg, q.cuda() if not q.is_cuda else q, cache, table, lens_d, msl, out, ws, scale=scale, dev_status=status)
    torch.cuda.synchronize()
    return out.float().cpu().numpy().astype(np.float64)


def check_decode(c, q, got, out_dtype, lens=None, scale=SCALE):
    lens = c.lens if lens is None else lens
    for b in range(q.shape[0]):
        k, v = c.kv(b, lens[b])
        ref, size, reach = o8.attend(q[b].double().numpy(), k, v, scale)
        err, tol = np.abs(got[b] - ref), tolerance(ref, size, reach, int(lens[b]), out_dtype, c.floor(b, int(lens[b])))
        assert np.all(err <= tol), (b, int(lens[b]), float((err / tol).max()))


# ---------------------------------------------------------------- store


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("block,n_kv,dtype", [(16, 8, "bf16"), (32, 1, "fp16"), (64, 3, "bf16"), (128, 2, "fp16")])
def test_store_bytes(tq, fmt, block, n_kv, dtype):
    """Chunks that begin and end anywhere: single tokens, whole blocks, an empty chunk, a chunk over several blocks."""
    hist = [0, 5, block, block - 1, 2 * block + 7, 3, block + 1, 0]
    q_lens = [1, 1, block, 2, 3 * block + 5, 0, block - 1, 2 * block]
    c = Case(tq, fmt, block, n_kv, n_kv, [a + b for a, b in zip(hist, q_lens)], seed=block)
    c.fill(hist)
    rows = sum(q_lens)
    # some chunks outgrow what the block holds, some do not
    key, value = c.draw(rows, n_kv, dtype, 3.0, outlier=True), c.draw(rows, n_kv, dtype, 0.5)
    starts, lens = starts_of(q_lens), np.array(hist) + np.array(q_lens)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = run_store(c, key, value, starts, lens, status=status).cpu().numpy()
    o8.store(c.f, c.cache, key.float().numpy(), value.float().numpy(), starts, c.table, lens)
    assert int(status) == 0
    assert np.array_equal(got, c.cache)          # rows behind the ends and unused blocks too


@pytest.mark.parametrize("fmt", FMTS)
def test_store_token_by_token_with_growing_values(tq, fmt):
    c = Case(tq, fmt, 32, 2, 2, [70, 70, 70], seed=9)
    cache = torch.from_numpy(c.cache).cuda()
    for step in range(70):
        key, value = c.draw(3, 2, gain=1.05 ** step), c.draw(3, 2, gain=1.05 ** -step)
        lens = [step + 1] * 3
        cache = run_store(c, key, value, [0, 1, 2, 3], lens, cache=cache)
        o8.store(c.f, c.cache, key.float().numpy(), value.float().numpy(), [0, 1, 2, 3], c.table, lens)
    assert np.array_equal(cache.cpu().numpy(), c.cache)


@pytest.mark.parametrize("fmt", FMTS)
def test_store_takes_slices_of_a_fused_projection(tq, fmt):
    c = Case(tq, fmt, 16, 8, 2, [40, 9], seed=4)
    fused = c.draw(49, 8 + 2 + 2).cuda()
    got = run_store(c, fused[:, 8:10], fused[:, 10:], [0, 40, 49], [40, 9]).cpu().numpy()
    x = fused.float().cpu().numpy()
    o8.store(c.f, c.cache, x[:, 8:10], x[:, 10:], [0, 40, 49], c.table, [40, 9])
    assert np.array_equal(got, c.cache)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_store_extreme_values(tq, fmt, dtype):
    """Infinities, NaN, all zeros, the smallest and the largest numbers."""
    c = Case(tq, fmt, 16, 1, 1, [64], seed=5)
    key, value = c.draw(64, 1, dtype), c.draw(64, 1, dtype)
    key[3, 0, 7], key[3, 0, 8], key[5, 0, 0] = float("inf"), float("-inf"), float("nan")
    key[16:32] = 0
    value[0:16] = torch.finfo(DT[dtype]).tiny / 4        # subnormal
    value[16:32] *= torch.finfo(DT[dtype]).max / 8
    value[32:48] = float("nan")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = run_store(c, key, value, [0, 64], [64], status=status).cpu().numpy()
    o8.store(c.f, c.cache, key.float().numpy(), value.float().numpy(), [0, 64], c.table, [64])
    assert int(status) == tq.TQ_DEV_NOT_FINITE
    assert np.array_equal(got, c.cache)


def test_store_device_errors_and_padding(tq):
    """A bad block id, a chunk past max_q_len, a chunk longer than its sequence, a
    sequence longer than its row, and rows behind the last sequence: what can be
    stored is, nothing else is touched, the status tells."""
    c = Case(tq, "int8_blk", 16, 2, 2, [48, 32, 32, 32], seed=6)
    key, value = c.draw(200, 2), c.draw(200, 2)
    want = c.cache.copy()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def go(lens, starts, max_q=None):
        status.zero_()
        return run_store(c, key, value, starts, lens, max_q=max_q, status=status).cpu().numpy(), int(status)

    def oracle(x_rows, b, n, seq):
        w = want.copy()
        o8.store(c.f, w, key.float().numpy()[x_rows], value.float().numpy()[x_rows], [0, n], c.table[b:b + 1], [seq])
        return w

    # rows 20 .. 199 behind the last sequence are not used
    got, st = go([20, 0, 0, 0], [0, 20, 20, 20, 20])
    assert st == 0 and np.array_equal(got, oracle(slice(0, 20), 0, 20, 20))
    # a chunk of 30 cut to max_q_len 20
    got, st = go([30, 0, 0, 0], [0, 30, 30, 30, 30], max_q=20)
    assert st == tq.TQ_DEV_SEQ_TOO_LONG and np.array_equal(got, oracle(slice(0, 20), 0, 20, 20))
    # a chunk of 12 of a sequence of 9: its first 3 rows lie before position 0
    got, st = go([9, 0, 0, 0], [0, 12, 12, 12, 12])
    assert st == tq.TQ_DEV_SEQ_TOO_LONG and np.array_equal(got, oracle(slice(3, 12), 0, 9, 9))
    # the row of the table names 3 blocks; positions 48 .. 59 have none
    got, st = go([60, 0, 0, 0], [0, 60, 60, 60, 60])
    assert st == tq.TQ_DEV_SEQ_TOO_LONG and np.array_equal(got, oracle(slice(0, 48), 0, 48, 48))
    # bad block ids
    good = c.table.copy()
    for bad in (-1, c.blocks, 2 ** 31 - 1):
        c.table[0, 1] = bad
        got, st = go([48, 0, 0, 0], [0, 48, 48, 48, 48])
        c.table[:] = good
        w = oracle(slice(0, 48), 0, 48, 48)
        n = c.f.block_bytes
        w[good[0, 1] * n:(good[0, 1] + 1) * n] = want[good[0, 1] * n:(good[0, 1] + 1) * n]
        assert st == tq.TQ_DEV_BLOCK_OUT_OF_RANGE and np.array_equal(got, w)


# ---------------------------------------------------------------- read back


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("block,n_kv,out", [(16, 8, "bf16"), (32, 2, "fp16"), (64, 1, "f32"), (128, 3, "bf16")])
def test_dequant_bits(tq, fmt, block, n_kv, out):
    lens = [0, 1, 15, 16, 17, 77, 130]
    c = Case(tq, fmt, block, n_kv, n_kv, [max(x, 1) for x in lens], seed=block + 1).fill(lens)
    cache, table, lens_d = c.gpu()
    msl = 131
    k = torch.full((len(lens), msl, n_kv, 128), float("nan"), dtype=DT[out], device="cuda")
    v = torch.full_like(k, float("nan"))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    tq.tq_b8_dequant(c.cfg, cache, table, lens_d, msl, k, v, dev_status=status)
    assert int(status) == 0
    for b, n in enumerate(lens):
        kk, vv = c.kv(b)
        for got, ref in ((k[b].cpu(), kk), (v[b].cpu(), vv)):
            want = torch.zeros((msl, n_kv, 128), dtype=DT[out])
            want[:n] = torch.from_numpy(ref.astype(np.float32)).to(DT[out])     # exact in 64 bits, so rounded once to f32
            assert torch.equal(got, want), (b, n)


def test_dequant_device_errors(tq):
    c = Case(tq, "e4m3_blk", 16, 2, 2, [40, 40], seed=2).fill([40, 40])
    good = c.table.copy()
    c.table[0, 1] = c.blocks + 5
    cache, table, lens = c.gpu()
    k = torch.full((2, 24, 2, 128), 7.0, dtype=torch.float32, device="cuda")
    v = torch.full_like(k, 7.0)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    tq.tq_b8_dequant(c.cfg, cache, table, lens, 24, k, v, dev_status=status)
    assert int(status) == tq.TQ_DEV_BLOCK_OUT_OF_RANGE | tq.TQ_DEV_SEQ_TOO_LONG
    assert not k[0, 16:].any() and not v[0, 16:].any()
    c.table[:] = good
    assert torch.equal(k[1].cpu().double(), torch.from_numpy(c.kv(1, 24)[0].astype(np.float32)).double())


# ---------------------------------------------------------------- decode


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("block,n_kv,group,dtype,out", [
    (16, 8, 4, "bf16", "bf16"), (32, 2, 1, "fp16", "fp16"), (64, 1, 8, "bf16", "f32"), (128, 2, 3, "fp16", "f32"),
    (16, 1, 5, "bf16", "f32"), (64, 3, 2, "fp16", "bf16"), (16, 2, 7, "bf16", "fp16"), (32, 1, 6, "fp16", "f32")])
def test_decode(tq, fmt, block, n_kv, group, dtype, out):
    lens = [0, 1, 15, 16, 17, 63, 64, 65, 200, 333]
    c = Case(tq, fmt, block, n_kv * group, n_kv, [max(x, 1) for x in lens], seed=group).fill(lens)
    q = c.draw(len(lens), n_kv * group, dtype, outlier=True)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = run_decode(c, q, out_dtype=out, status=status)
    assert int(status) == 0
    assert not got[0].any()                      # nothing cached: zeros
    check_decode(c, q, got, out)


@pytest.mark.parametrize("lens", [[1], [0], [0, 0, 0], [2100], [700, 0, 0, 1, 900]])
def test_decode_few_and_empty_sequences(tq, lens):
    c = Case(tq, "e4m3_blk", 16, 4, 1, [max(x, 1) for x in lens], seed=3).fill(lens)
    q = c.draw(len(lens), 4)
    check_decode(c, q, run_decode(c, q), "f32")


def test_decode_many_sequences(tq):
    """More (sequence, head) pairs than warps, most of them one tile long."""
    rng = np.random.default_rng(8)
    lens = [int(x) for x in rng.integers(0, 20, 1500)]
    c = Case(tq, "int8_blk", 16, 4, 2, [max(x, 1) for x in lens], seed=8).fill(lens)
    q = c.draw(len(lens), 4)
    check_decode(c, q, run_decode(c, q), "f32")


def test_decode_scale_argument_and_strided_queries(tq):
    lens = [50, 20]
    c = Case(tq, "int8_blk", 32, 8, 2, lens, seed=12).fill(lens)
    fused = c.draw(2, 12).cuda()
    got = run_decode(c, fused[:, :8], scale=0.31)
    check_decode(c, fused[:, :8].cpu(), got, "f32", scale=float(np.float32(0.31)))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("gain", [
    lambda j: 10.0 ** (j % 7 - 3),                      # up and down by up to 10^6
    lambda j: 2.0 ** (60 if j % 2 else -60),            # far apart: the small blocks do not count, the large do
    lambda j: 1e-28, lambda j: 1e30])
def test_decode_blocks_of_very_different_value_scales(tq, fmt, gain):
    lens = [150, 97]
    c = Case(tq, fmt, 16, 4, 1, lens, seed=21).fill(lens, gain)
    q = c.draw(2, 4)
    got = run_decode(c, q)
    check_decode(c, q, got, "f32")


def test_decode_small_values_under_the_weights_of_large_ones(tq):
    """The first block's values are 2^30 times the others', its keys score far
    below: the output comes from the small ones, to full precision."""
    c = Case(tq, "int8_blk", 16, 1, 1, [64], seed=22)
    k = c.draw(64, 1).float().numpy()
    v = c.draw(64, 1).float().numpy()
    q = torch.ones((1, 1, 128), dtype=torch.bfloat16)
    k[:16] = -40.0                       # scores of about -450: no weight left
    v[:16] *= 2.0 ** 30
    o8.store(c.f, c.cache, k, v, [0, 64], c.table, [64])
    c.lens = np.array([64], dtype=np.int32)
    check_decode(c, q, run_decode(c, q), "f32")


def test_decode_device_errors(tq):
    c = Case(tq, "e4m3_blk", 16, 4, 2, [100, 40], seed=14).fill([100, 40])
    good = c.table.copy()
    c.table[0, 2], c.table[1, :] = -1, 2 ** 31 - 1
    q = c.draw(2, 4)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = run_decode(c, q, status=status, max_len=90)
    assert int(status) == tq.TQ_DEV_BLOCK_OUT_OF_RANGE | tq.TQ_DEV_SEQ_TOO_LONG
    check_decode(c, q, got, "f32", lens=[90, 40])      # positions of bad blocks are left out; nothing left: zeros
    c.table[:] = good


def test_decode_not_a_number_query_stays_in_its_row(tq):
    lens = [40, 40]
    c = Case(tq, "int8_blk", 16, 4, 1, lens, seed=15).fill(lens)
    q = c.draw(2, 4)
    q[0, 1, 3] = float("nan")
    got = run_decode(c, q)
    assert np.isnan(got[0, 1]).all() and np.isfinite(got[0, [0, 2, 3]]).all() and np.isfinite(got[1]).all()


def test_decode_on_streams_and_in_graphs(tq):
    """Two calls on two streams with a workspace each, and a captured call
    replayed after the lengths and the query changed, with the indices known
    early too; the same call twice gives the same bits."""
    lens = [300, 45, 0, 128]
    c = Case(tq, "e4m3_blk", 32, 16, 4, [400] * 4, seed=16).fill([400] * 4)
    cache, table, _ = c.gpu()
    lens_d = torch.tensor(lens, dtype=torch.int32, device="cuda")
    q = [c.draw(4, 16).cuda() for _ in range(2)]
    n = tq.tq_b8_decode_workspace_size(c.cfg, 4, 400)
    ws = [torch.empty(n, dtype=torch.uint8, device="cuda") for _ in range(2)]
    out = [torch.empty((4, 16, 128), dtype=torch.float32, device="cuda") for _ in range(2)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for i in range(2):
        with torch.cuda.stream(streams[i]):
            tq.tq_b8_decode(c.cfg, q[i], cache, table, lens_d, 400, out[i], ws[i])
    torch.cuda.synchronize()
    for i in range(2):
        check_decode(c, q[i].cpu(), out[i].cpu().numpy().astype(np.float64), "f32", lens=lens)
    first = out[0].clone()
    tq.tq_b8_decode(c.cfg, q[0], cache, table, lens_d, 400, out[0], ws[0])
    assert torch.equal(first, out[0])
    for flags in (0, tq.TQ_FLAG_INDICES_READY):
        cfg = tq.make_config("e4m3_blk", 16, 4, block_size=32, flags=flags)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            tq.tq_b8_decode(cfg, q[0], cache, table, lens_d, 400, out[0], ws[0])
        for new in ([400, 1, 33, 0], [17, 399, 64, 250]):
            lens_d.copy_(torch.tensor(new, dtype=torch.int32))
            fresh = c.draw(4, 16)
            q[0].copy_(fresh)
            out[0].fill_(float("nan"))
            graph.replay()
            torch.cuda.synchronize()
            check_decode(c, fresh, out[0].cpu().numpy().astype(np.float64), "f32", lens=new)


def test_refusals_with_tensors_on_the_gpu(tq):
    """What the CPU tests cannot reach because a host tensor is refused first."""
    c = Case(tq, "int8_blk", 16, 4, 1, [20, 20], seed=70).fill([20, 20])
    cache, table, lens = c.gpu()
    q = c.draw(2, 4).cuda()
    out = torch.full_like(q, 5.0)
    n = tq.tq_b8_decode_workspace_size(c.cfg, 2, 20)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    for bad, match in ((dict(workspace=torch.empty(1, dtype=torch.uint8, device="cuda").expand(n)), "workspace"),
                       (dict(workspace=ws.cpu()), "one CUDA device"), (dict(seq_lens=lens.cpu()), "one CUDA device"),
                       (dict(num_blocks=c.blocks + 1), "blocks"), (dict(dev_status=torch.zeros(1, device="cuda")), "dev_status")):
        args = dict(cfg=c.cfg, q=q, cache=cache, block_table=table, seq_lens=lens, max_seq_len=20, out=out, workspace=ws)
        with pytest.raises(ValueError, match=match):
            tq.tq_b8_decode(**{**args, **bad})
    with pytest.raises(tq.TQError, match="workspace"):
        tq.tq_b8_decode(c.cfg, q, cache, table, lens, 20, out, ws[:n - 16])
    with pytest.raises(tq.TQError, match="misaligned"):
        tq.tq_b8_decode(c.cfg, q, cache, table, lens, 20, out, torch.empty(n + 8, dtype=torch.uint8, device="cuda")[8:])
    torch.cuda.synchronize()
    assert torch.all(out == 5.0)


# ---------------------------------------------------------------- chunks


def run_continue(c, q, starts, lens, out_dtype="f32", status=None, max_q=None, max_len=None, scale=0.0):
    cache, table, _ = c.gpu()
    lens_d = torch.from_numpy(np.asarray(lens, dtype=np.int32)).cuda()
    msl = max(int(max(lens)), 1) if max_len is None else max_len
    mq = int(np.diff(starts).max(initial=0)) if max_q is None else max_q
    out = torch.full(q.shape, 123.0, dtype=DT[out_dtype], device="cuda")
    n = c.tq.tq_b8_continue_workspace_size(c.cfg, len(lens), q.shape[0], mq, msl)
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    c.tq.tq_b8_continue(c.cfg, q.cuda() if not q.is_cuda else q, torch.from_numpy(np.asarray(starts, dtype=np.int32)).cuda(), mq, cache, table,
                        lens_d, msl, out, ws, scale=scale, dev_status=status)
    torch.cuda.synchronize()
    return out.float().cpu().numpy().astype(np.float64)


def check_continue(c, q, got, starts, lens, out_dtype, rows=None, scale=SCALE):
    """Every query (or the first, the last and some between of a long chunk) against the oracle."""
    for b in range(len(lens)):
        q0, q1 = int(starts[b]), int(starts[b + 1])
        if q0 == q1:
            continue
        k, v = c.kv(b, max(int(lens[b]), 0))
        floor = c.floor(b, max(int(lens[b]), 0), chunks=True)
        n = q1 - q0
        pick = range(n) if n <= 40 or rows is None else sorted({0, 1, n - 1, n - 2, *range(0, n, max(n // rows, 1))})
        for i in pick:
            seen = max(int(lens[b]) - n + i + 1, 0)
            ref, size, reach = o8.attend(q[q0 + i].double().numpy(), k[:seen], v[:seen], scale)
            err, tol = np.abs(got[q0 + i] - ref), tolerance(ref, size, reach, seen, out_dtype, floor, single_p=True)
            assert np.all(err <= tol), (b, i, seen, float((err / tol).max()))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("block,n_kv,group,dtype,out", [
    (16, 2, 4, "bf16", "bf16"), (32, 1, 8, "fp16", "fp16"), (64, 2, 1, "bf16", "f32"), (128, 1, 3, "fp16", "f32"),
    (16, 1, 5, "bf16", "fp16"), (64, 1, 6, "fp16", "bf16"), (32, 1, 7, "bf16", "f32"), (128, 2, 2, "bf16", "f32")])
def test_continue(tq, fmt, block, n_kv, group, dtype, out):
    q_lens, hist = [1, 7, 0, 33, 130, 2], [0, 19, 50, 100, 5, 255]
    lens = [a + b for a, b in zip(q_lens, hist)]
    c = Case(tq, fmt, block, n_kv * group, n_kv, lens, seed=group + 30).fill(lens)
    starts = starts_of(q_lens)
    q = c.draw(int(starts[-1]), n_kv * group, dtype, outlier=True)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = run_continue(c, q, starts, lens, out, status)
    assert int(status) == 0
    check_continue(c, q, got, starts, lens, out, rows=12)


@pytest.mark.parametrize("q_len,hist,group,n_kv", [(300, 0, 4, 1), (257, 700, 1, 2), (128, 1024, 8, 1), (40, 1500, 4, 1)])
def test_continue_long(tq, q_len, hist, group, n_kv):
    c = Case(tq, "e4m3_blk", 64, n_kv * group, n_kv, [q_len + hist], seed=q_len).fill([q_len + hist])
    q = c.draw(q_len, n_kv * group)
    got = run_continue(c, q, [0, q_len], [q_len + hist])
    check_continue(c, q, got, [0, q_len], [q_len + hist], "f32", rows=16)


@pytest.mark.parametrize("fmt,batch", [("int8_blk", 90), ("e4m3_blk", 77), ("int8_blk", 500)])
def test_continue_many_chunks(tq, fmt, batch):
    """More (chunk, head) units than fit one wave, the last ones split over the
    history (180 = 152 + 28, 154 = 152 + 2; 1000 are not split), lengths from one
    position on, empty chunks between; all sequences share their blocks."""
    c = Case(tq, fmt, 32, 8, 2, [700], seed=batch).fill([700])
    c.table = np.repeat(c.table, batch, 0)
    q_lens = c.rng.integers(1, 4, batch)
    if batch == 500:
        q_lens[c.rng.permutation(batch)[:100]] = 0
    lens = np.maximum(c.rng.integers(1, 701, batch), q_lens)
    c.lens = lens.astype(np.int32)
    starts = starts_of(q_lens)
    q = c.draw(int(starts[-1]), 8)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = run_continue(c, q, starts, lens, status=status)
    assert int(status) == 0
    k, v = c.kv(0, 700)
    floors = np.abs(v)
    s = np.array([[o8.scale(c.f, c.cache, int(c.table[0, p // 32]), h, 1) for h in range(2)] for p in range(700)])[..., None]
    floors = np.cumsum(floors * s.max(0) / s, 0) * 2.0 ** -24     # at most: s_max of all positions
    for b in range(batch):
        for i in range(int(q_lens[b])):
            seen = int(lens[b]) - int(q_lens[b]) + i + 1
            row = int(starts[b]) + i
            ref, size, reach = o8.attend(q[row].double().numpy(), k[:seen], v[:seen], SCALE)
            tol = tolerance(ref, size, reach, seen, "f32", np.repeat(floors[seen - 1], 4, 0), single_p=True)
            assert np.all(np.abs(got[row] - ref) <= tol), (b, i, seen)


@pytest.mark.parametrize("q_len", [5, 150])
def test_continue_rows_without_positions_and_padding(tq, q_len):
    """Queries before position 0, past max_q_len and behind the last sequence."""
    c = Case(tq, "int8_blk", 16, 4, 1, [q_len, 200], seed=40).fill([q_len - 3, 200])
    starts = np.array([0, q_len, q_len + 4], dtype=np.int32)
    q = c.draw(int(starts[-1]) + 9, 4)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    # a chunk longer than its sequence: its first 3 queries see nothing
    got = run_continue(c, q, starts, [q_len - 3, 200], status=status)
    assert int(status) == 0
    assert not got[:3].any() and np.all(got[starts[-1]:] == 123.0)
    check_continue(c, q, got, starts, [q_len - 3, 200], "f32", rows=10)
    got = run_continue(c, q, starts, [q_len - 3, 200], status=status, max_q=q_len - 1)
    assert int(status) == tq.TQ_DEV_SEQ_TOO_LONG
    assert not got[q_len - 1].any() and got[q_len - 2].any() and np.all(got[starts[-1]:] == 123.0)


def test_continue_starts_that_go_backwards(tq):
    """Not allowed, but nothing outside the rows is touched: more chunks than the
    rows could hold in order, all of them the same one."""
    batch, n, rows = 401, 600, 32
    c = Case(tq, "int8_blk", 32, 32, 4, [n], seed=47).fill([n])
    c.table = np.repeat(c.table, batch, 0)
    starts = np.array([0, rows] * ((batch + 1) // 2), dtype=np.int32)
    q = c.draw(rows + 5, 32)
    got = run_continue(c, q, starts, [n] * batch)
    assert np.all(got[rows:] == 123.0)
    c.lens = np.array([n], dtype=np.int32)
    check_continue(c, q, got, [0, rows], [n], "f32")


@pytest.mark.parametrize("q_len,length,cut", [(140, 200, 150), (5, 900, 897), (20, 900, 500)])
def test_continue_cuts_long_sequences(tq, q_len, length, cut):
    """Queries keep their places; none sees a position from max_seq_len on."""
    c = Case(tq, "e4m3_blk", 32, 4, 1, [length], seed=49).fill([length])
    q = c.draw(q_len, 4)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = run_continue(c, q, [0, q_len], [length], status=status, max_len=cut)
    assert int(status) == tq.TQ_DEV_SEQ_TOO_LONG
    k, v = c.kv(0)
    floor = c.floor(0, length, chunks=True)
    for i in range(0, q_len, max(q_len // 20, 1)):
        seen = min(length - q_len + i + 1, cut)
        ref, size, reach = o8.attend(q[i].double().numpy(), k[:seen], v[:seen], SCALE)
        assert np.all(np.abs(got[i] - ref) <= tolerance(ref, size, reach, seen, "f32", floor, single_p=True)), (i, seen)


@pytest.mark.parametrize("gain", [lambda j: 0.0, lambda j: j % 3 == 1, lambda j: j < 2])
def test_blocks_of_zero_values(tq, gain):
    """Values of zero take their share of the weights (their scale is the smallest)."""
    c = Case(tq, "int8_blk", 16, 4, 1, [600], seed=51).fill([600], gain)
    q = c.draw(40, 4)
    check_continue(c, q, run_continue(c, q, [0, 40], [600]), [0, 40], [600], "f32", rows=12)
    check_decode(c, q[:1], run_decode(c, q[:1]), "f32")


@pytest.mark.parametrize("fmt", FMTS)
def test_continue_one_position_is_its_value(tq, fmt):
    """The weight of a sequence's only position is exact in fp16, whatever the scale:
    left are two roundings of a score below 64 in the exponent (2^-19 each), the
    logarithm of a scale between 2^-16 and 1 and its power (2^-20 each) and the
    quotient (2^-22): below 2^-16."""
    batch = 40
    c = Case(tq, fmt, 16, 4, 2, [1] * batch, seed=52)
    for b in range(batch):
        o8.store(c.f, c.cache, c.draw(1, 2).float().numpy(), c.draw(1, 2).float().numpy() * np.float32(1.1 ** (b - 20)), [0, 1], c.table[b:b + 1], [1])
    c.lens = np.ones(batch, dtype=np.int32)
    q = c.draw(batch, 4)
    got = run_continue(c, q, np.arange(batch + 1), c.lens)
    for b in range(batch):
        k, v = c.kv(b)
        assert np.abs(q[b].double().numpy() @ k[0].repeat(2, 0).T).max() * SCALE * 1.4427 < 64
        ref = v[0].repeat(2, 0)
        assert np.all(np.abs(got[b] - ref) <= np.abs(ref) * 2.0 ** -16)


@pytest.mark.parametrize("room,stored", [(40, 0), (40, 16), (900, 64)])
def test_blocks_that_nothing_was_stored_to(tq, room, stored):
    """A zeroed cache's fresh blocks (the padding of a batch points there) are left
    out without an error."""
    c = Case(tq, "e4m3_blk", 16, 4, 2, [room], seed=48)
    c.cache[:] = 0
    c.fill([stored])
    q = c.draw(3, 4)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    chunk = run_continue(c, q, [0, 3], [room], status=status)
    step = run_decode(c, q[:1], [room], status=status)
    assert int(status) == 0
    if stored:
        k, v = c.kv(0, stored)
        for i in range(3):
            ref, size, reach = o8.attend(q[i].double().numpy(), k, v, SCALE)
            assert np.all(np.abs(chunk[i] - ref) <= tolerance(ref, size, reach, stored, "f32", c.floor(0, stored, chunks=True), single_p=True))
        check_decode(c, q[:1], step, "f32", [stored])
    else:
        assert not chunk.any() and not step.any()


@pytest.mark.parametrize("hist,dtype", [(20, "bf16"), (2000, "bf16"), (20, "f32")])
def test_continue_output_on_16_bytes(tq, hist, dtype):
    """out and workspace may lie on any 16 bytes (whole and split histories)."""
    c = Case(tq, "int8_blk", 32, 4, 1, [hist + 40], seed=44).fill([hist + 40])
    cache, table, lens = c.gpu()
    q = c.draw(40, 4)
    n = 40 * 4 * 128
    room = torch.empty(n + 16, dtype=DT[dtype], device="cuda")
    ws = torch.empty(tq.tq_b8_continue_workspace_size(c.cfg, 1, 40, 40, hist + 40) + 16, dtype=torch.uint8, device="cuda")
    off = 16 // room.element_size()
    assert room.data_ptr() % 32 == 0 and ws.data_ptr() % 32 == 0
    out = room[off:off + n].view(40, 4, 128)
    starts = torch.tensor([0, 40], dtype=torch.int32, device="cuda")
    tq.tq_b8_continue(c.cfg, q.cuda(), starts, 40, cache, table, lens, hist + 40, out, ws[16:])
    check_continue(c, q, out.float().cpu().numpy().astype(np.float64), [0, 40], [hist + 40], dtype, rows=6)


@pytest.mark.parametrize("q_len", [4, 140])
def test_continue_device_errors(tq, q_len):
    c = Case(tq, "e4m3_blk", 16, 4, 1, [200], seed=41).fill([200])
    c.table[0, 3], c.table[0, 9] = -1, 2 ** 31 - 1
    q = c.draw(q_len, 4)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = run_continue(c, q, [0, q_len], [200], status=status)
    assert int(status) == tq.TQ_DEV_BLOCK_OUT_OF_RANGE
    check_continue(c, q, got, [0, q_len], [200], "f32", rows=10)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("gain", [lambda j: 10.0 ** (j % 7 - 3), lambda j: 1e-28, lambda j: 1e30,
                                  lambda j: 2.0 ** (60 if j % 2 else -60)])
def test_continue_blocks_of_very_different_value_scales(tq, fmt, gain):
    c = Case(tq, fmt, 64, 4, 1, [400], seed=42).fill([400], gain)
    q = c.draw(150, 4)
    got = run_continue(c, q, [0, 150], [400])
    check_continue(c, q, got, [0, 150], [400], "f32", rows=12)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("q_len,hist", [(37, 30), (150, 0), (6, 900)])
@pytest.mark.parametrize("gain_k,gain_q,scale", [(0.0, 0.0, 0.0), (1e-12, 0.0, 0.0), (0.0, 1e-25, 0.0), (1.0, 1e-30, 0.0), (1e-20, 1e-20, 1e-20)])
def test_scores_that_vanish(tq, fmt, q_len, hist, gain_k, gain_q, scale):
    """Scores of nothing, or of so little that a block's factor is not a number of
    fp32 any more: plain means of the values seen."""
    n = q_len + hist
    c = Case(tq, fmt, 16, 4, 1, [n], seed=46)
    o8.store(c.f, c.cache, (c.draw(n, 1).float() * gain_k).numpy(), c.draw(n, 1).float().numpy(), [0, n], c.table, [n])
    c.lens = np.array([n], dtype=np.int32)
    q = c.draw(q_len, 4, gain=gain_q)
    got = run_continue(c, q, [0, q_len], [n], scale=scale)
    check_continue(c, q, got, [0, q_len], [n], "f32", rows=12, scale=scale or SCALE)
    check_decode(c, q[:1], run_decode(c, q[:1], scale=scale), "f32", scale=scale or SCALE)


def test_continue_on_streams_and_in_graphs(tq):
    """As for the decode: two streams, then a captured call replayed with other
    starts, lengths and queries in padded tensors; the same call gives the same bits."""
    c = Case(tq, "int8_blk", 16, 8, 2, [900] * 3, seed=60).fill([900] * 3)
    cache, table, _ = c.gpu()
    rows, msl = 64, 900
    calls = []
    for starts, lens in (([0, 20, 20, 55], [900, 3, 500]), ([0, 1, 40, 64], [7, 899, 64])):
        q = c.draw(rows, 8)
        calls.append((q, starts, lens, q.cuda(), torch.tensor(starts, dtype=torch.int32, device="cuda"),
                      torch.tensor(lens, dtype=torch.int32, device="cuda"),
                      torch.full((rows, 8, 128), 123.0, dtype=torch.float32, device="cuda"),
                      torch.empty(tq.tq_b8_continue_workspace_size(c.cfg, 3, rows, 48, msl), dtype=torch.uint8, device="cuda"),
                      torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _, _, _, q, starts, lens, out, ws, stream in calls:
        with torch.cuda.stream(stream):
            tq.tq_b8_continue(c.cfg, q, starts, 48, cache, table, lens, msl, out, ws)
    torch.cuda.synchronize()
    for q, starts, lens, _, _, _, out, _, _ in calls:
        got = out.cpu().numpy().astype(np.float64)
        check_continue(c, q, got, starts, lens, "f32", rows=5)
        assert np.all(got[starts[-1]:] == 123.0)
    q, _, _, q_d, starts_d, lens_d, out, ws, _ = calls[0]
    first = out.clone()
    tq.tq_b8_continue(c.cfg, q_d, starts_d, 48, cache, table, lens_d, msl, out, ws)
    assert torch.equal(first, out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tq.tq_b8_continue(c.cfg, q_d, starts_d, 48, cache, table, lens_d, msl, out, ws)
    for starts, lens in (([0, 48, 49, 60], [48, 800, 333]), ([0, 0, 0, 5], [10, 20, 700]), ([0, 0, 0, 0], [1, 2, 3])):
        fresh = c.draw(rows, 8)
        q_d.copy_(fresh)
        starts_d.copy_(torch.tensor(starts, dtype=torch.int32))
        lens_d.copy_(torch.tensor(lens, dtype=torch.int32))
        out.fill_(123.0)
        graph.replay()
        torch.cuda.synchronize()
        got = out.cpu().numpy().astype(np.float64)
        check_continue(c, fresh, got, starts, lens, "f32", rows=5)
        assert np.all(got[starts[-1]:] == 123.0)


def test_offsets_past_32_bits(tq):
    """The same sequences in a small cache and behind the first 4 GB of a large one
    give the same bits, written, read back and attended to; and an output of more
    than 2^31 elements is filled to its end."""
    n_q, n_kv, lens = 16, 8, [300, 77]
    cfg = tq.make_config("e4m3_blk", n_q, n_kv, block_size=128)
    bb = tq.tq_b8_layout_for(cfg).block_bytes
    far = (1 << 32) // bb + 3
    c = Case(tq, "e4m3_blk", 128, n_q, n_kv, lens, seed=80)
    key, value, q = c.draw(377, n_kv).cuda(), c.draw(377, n_kv).cuda(), c.draw(377, n_q).cuda()
    starts = torch.tensor([0, 300, 377], dtype=torch.int32, device="cuda")
    lens_d = torch.tensor(lens, dtype=torch.int32, device="cuda")
    results = []
    for base in (0, far):
        cache = torch.empty((base + 8) * bb, dtype=torch.uint8, device="cuda")
        table = torch.tensor([[4, 1, 6], [2, 0, 0]], dtype=torch.int32, device="cuda") + base
        tq.tq_b8_store(cfg, key, value, starts, 300, cache, table, lens_d)
        k = torch.empty((2, 300, n_kv, 128), dtype=torch.float32, device="cuda")
        v = torch.empty_like(k)
        tq.tq_b8_dequant(cfg, cache, table, lens_d, 300, k, v)
        one = torch.empty((2, n_q, 128), dtype=torch.float32, device="cuda")
        ws = torch.empty(max(tq.tq_b8_decode_workspace_size(cfg, 2, 300), tq.tq_b8_continue_workspace_size(cfg, 2, 377, 300, 300)),
                         dtype=torch.uint8, device="cuda")
        tq.tq_b8_decode(cfg, q[:2].contiguous(), cache, table, lens_d, 300, one, ws)
        many = torch.empty((377, n_q, 128), dtype=torch.float32, device="cuda")
        tq.tq_b8_continue(cfg, q, starts, 300, cache, table, lens_d, 300, many, ws)
        results.append((k, v, one, many))
        if base == 0:
            small, small_table = cache, table
    for x, y in zip(*results):
        assert torch.equal(x, y)
    del cache, results
    long = (1 << 31) // (n_kv * 128) + 1001
    k = torch.full((1, long, n_kv, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    v = torch.full_like(k, 3.0)
    tq.tq_b8_dequant(cfg, small, small_table[1:, :1].contiguous(), lens_d[1:], long, k, v)
    assert k[0, :77].any() and v[0, 76].any()
    for x in (k, v):
        assert not x[0, 77:100].any() and not x[0, -5000:].any() and int(torch.count_nonzero(x[0, 100:].view(torch.int16))) == 0


# ---------------------------------------------------------------- chunks, row by row


def check_rows(c, q, got, starts, lens, out_dtype="f32", rows=None, scale=SCALE):
    """As check_continue, the bound taken from what each query sees and weighs.
      weights: P = 8 p s_v / r, rounded to fp16 once, and once more where the row's
        reference r moves within a step: 2 half steps, 2^-10 together
      r is at most the largest p s_v that the row sees: no step below 2^-24 means
        2^-28 of that per code and rounding
      exponents: log2 s_v is off by up to 2 units of its last place (|log2 s_v| < 128:
        2^-16), its difference to the reference by half a unit of a number below 256
        (2^-17), the reference's moves as much: below 2^-14 relative"""
    for b in range(len(lens)):
        k, v = c.kv(b, int(lens[b]))
        s = np.array([[o8.scale(c.f, c.cache, int(c.table[b, p // c.block]), h, 1) for h in range(c.n_kv)] for p in range(int(lens[b]))],
                     dtype=np.float64)
        q0, n = int(starts[b]), int(starts[b + 1] - starts[b])
        for i in range(n) if rows is None else sorted({0, n - 1, *range(0, n, max(n // rows, 1))}):
            seen = int(lens[b]) - n + i + 1
            x = q[q0 + i].double().numpy()
            ref, size, reach = o8.attend(x, k[:seen], v[:seen], scale)
            floor = np.zeros_like(ref)
            for h in range(c.n_q):
                g = h // (c.n_q // c.n_kv)
                z = k[:seen, g] @ x[h] * scale
                p = np.exp(z - z.max())
                codes = np.abs(v[:seen, g]) / s[:seen, g, None]
                floor[h] = 2.0 ** -27 * (p / p.sum() * s[:seen, g]).max() * codes.sum(0)
            tol = tolerance(ref, size, reach, seen, out_dtype, floor + size * (2.0 ** -11 + 2.0 ** -14), single_p=True)
            err = np.abs(got[q0 + i] - ref)
            assert np.all(err <= tol), (b, i, seen, float((err / tol).max()))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("hist,q_len", [(0, 70), (890, 60)])
@pytest.mark.parametrize("r", [10, 18, 24, 28, 60, 110])
def test_continue_small_values_before_large_ones(tq, fmt, hist, q_len, r):
    """Queries among the small values do not see the large ones behind them."""
    n = hist + q_len
    first = -(-(hist + 16) // 16)     # the first block of large values
    c = Case(tq, fmt, 16, 4, 1, [n], seed=90).fill([n], lambda j: 1.0 if j < first else 2.0 ** r)
    q = c.draw(q_len, 4)
    got = run_continue(c, q, [0, q_len], [n])
    assert got[:first * 16 - hist].any(-1).all()
    check_rows(c, q, got, [0, q_len], [n], rows=None if hist == 0 else 12)


@pytest.mark.parametrize("n,q_len,gain", [(64, 20, 30), (64, 64, 30), (700, 20, 30), (400, 150, 100)])
def test_continue_small_values_under_the_weights_of_large_ones(tq, n, q_len, gain):
    """As for the decode: the first block's values are 2^gain times the others', its keys score far below."""
    c = Case(tq, "int8_blk", 16, 1, 1, [n], seed=91)
    k, v = c.draw(n, 1).float().numpy(), c.draw(n, 1).float().numpy()
    q = torch.ones((q_len, 1, 128), dtype=torch.bfloat16)
    k[:16] = -40.0
    v[:16] *= np.float32(2.0 ** gain)
    o8.store(c.f, c.cache, k, v, [0, n], c.table, [n])
    check_rows(c, q, run_continue(c, q, [0, q_len], [n]), [0, q_len], [n], rows=20)


@pytest.mark.parametrize("gap", [0, 20, 60, 80, 100, 118, 122, 130, 200])
@pytest.mark.parametrize("low,high", [(60, -60), (-60, 60), (100, -90)])
def test_continue_scores_and_value_scales_that_rise_and_fall(tq, gap, low, high):
    """Block by block, scores rise by gap / 2 (log2 units) and values go from 2^low over 1 to 2^high."""
    c = Case(tq, "int8_blk", 16, 2, 1, [48], seed=92)
    k = np.zeros((48, 1, 128), dtype=np.float32)
    v = c.draw(48, 1).float().numpy()
    for j, g in enumerate((low, 0, high)):
        k[16 * j:16 * j + 16] = 0.5 * j * gap / (128 * SCALE * np.log2(np.e))
        v[16 * j:16 * j + 16] *= np.float32(2.0 ** g)
    o8.store(c.f, c.cache, k, v, [0, 48], c.table, [48])
    q = torch.ones((48, 2, 128), dtype=torch.bfloat16)
    check_rows(c, q, run_continue(c, q, [0, 48], [48]), [0, 48], [48])


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("hist", [0, 800])
def test_continue_later_positions_change_nothing(tq, fmt, hist):
    """Bit for bit, whatever the keys and values that a query does not see."""
    q_len = 60
    n, out = hist + q_len, []
    for gain in (1.0, 2.0 ** 20, 2.0 ** -20):
        c = Case(tq, fmt, 16, 4, 1, [n], seed=93)
        k, v, q = c.draw(n, 1).float().numpy(), c.draw(n, 1).float().numpy(), c.draw(q_len, 4)
        k[hist + 32:] *= np.float32(gain)
        v[hist + 32:] *= np.float32(gain)
        o8.store(c.f, c.cache, k, v, [0, n], c.table, [n])
        out.append(run_continue(c, q, [0, q_len], [n])[:32])
    assert np.array_equal(out[0], out[1]) and np.array_equal(out[0], out[2])


@pytest.mark.parametrize("block", [16, 64])
@pytest.mark.parametrize("hist,q_len,max_q", [(10, 20, 5), (0, 140, 70), (900, 30, 7)])
def test_continue_rows_that_were_not_stored(tq, block, hist, q_len, max_q):
    """Store and attention cut a chunk at the same max_q_len: what stands in the cache
    behind the last served query (NaN codes, scales of any size) does not count."""
    n, kept = hist + q_len, hist + max_q
    c = Case(tq, "e4m3_blk", block, 4, 1, [n], seed=94)
    c.cache[:] = 0x7f
    c.fill([kept])
    q = c.draw(q_len, 4)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = run_continue(c, q, [0, q_len], [n], max_q=max_q, status=status)
    assert int(status) == tq.TQ_DEV_SEQ_TOO_LONG
    assert not got[max_q:].any()
    check_rows(c, q, got, [0, max_q], [kept], rows=12)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("group", [1, 4, 7])
@pytest.mark.parametrize("hist", [0, 640])
def test_continue_f32_output_has_weights_to_match(tq, fmt, group, hist):
    """Two fp16 parts a weight, as the decode's: the bound without a rounding to fp16.
    Short rows of small scores, where that is the largest term. The exponents: log2 of
    the value scales (of magnitude 8 to 16, off by 2 units of the last place: 2^-19),
    their differences and the reference's moves below that: 2^-17 together."""
    q_lens = [2, 3, 5, 8, 12] * 4
    lens = [x + (hist if i == 7 else 0) for i, x in enumerate(q_lens)]
    c = Case(tq, fmt, 16, group, 1, lens, seed=95).fill(lens)
    starts = starts_of(q_lens)
    q = c.draw(int(starts[-1]), group, gain=0.05)
    got = run_continue(c, q, starts, lens)
    for b, n in enumerate(lens):
        k, v = c.kv(b)
        floor = c.floor(b, n, chunks=True)
        for i in range(q_lens[b]):
            seen = n - q_lens[b] + i + 1
            ref, size, reach = o8.attend(q[starts[b] + i].double().numpy(), k[:seen], v[:seen], SCALE)
            tol = tolerance(ref, size, reach, seen, "f32", floor + size * 2.0 ** -17)
            err = np.abs(got[starts[b] + i] - ref)
            assert np.all(err <= tol), (b, i, seen, float((err / tol).max()))


_CONTEXT_CHILD = """
import ctypes, importlib.util, sys
import numpy as np
spec = importlib.util.spec_from_file_location("abi", sys.argv[1])
abi = importlib.util.module_from_spec(spec)
spec.loader.exec_module(abi)
lib, rt = abi.load(), ctypes.CDLL("libcudart.so.13")     # the runtime that the library is linked to
batch, n_q, n_kv, n = 2, 8, 2, 300
cfg = abi.tq_config(abi.TQ_PRESET_INT8_BLK, 128, 16, n_q, n_kv, 0, 0)
lay = abi.tq_b8_layout()
assert lib.tq_b8_layout_for(ctypes.byref(cfg), ctypes.byref(lay)) == 0
rng = np.random.default_rng(1)
f16 = lambda *shape: rng.standard_normal(shape).astype(np.float16)
host = dict(k=f16(batch * n, n_kv, 128), v=f16(batch * n, n_kv, 128), q=f16(batch * n, n_q, 128),
            starts=np.array([0, n, 2 * n], dtype=np.int32), lens=np.array([n, n], dtype=np.int32),
            table=np.arange(38, dtype=np.int32).reshape(2, 19))
ws = max(lib.tq_b8_decode_workspace_size(ctypes.byref(cfg), batch, n),
         lib.tq_b8_continue_workspace_size(ctypes.byref(cfg), batch, batch * n, n, n))
sizes = dict(cache=38 * lay.block_bytes, ws=ws, one=batch * n_q * 512, many=batch * n * n_q * 512)

def once():
    d = {}
    for name, size in [*((k, x.nbytes) for k, x in host.items()), *sizes.items()]:
        d[name] = ctypes.c_void_p()
        assert rt.cudaMalloc(ctypes.byref(d[name]), ctypes.c_size_t(size)) == 0
        assert rt.cudaMemset(d[name], 0, ctypes.c_size_t(size)) == 0
    for name, x in host.items():
        assert rt.cudaMemcpy(d[name], ctypes.c_void_p(x.ctypes.data), ctypes.c_size_t(x.nbytes), 1) == 0
    status = [lib.tq_b8_store(ctypes.byref(cfg), d["k"], 0, d["v"], 0, 0, d["starts"], batch, 2 * n, n, d["cache"], 38, d["table"], 19,
                              d["lens"], None, None),
              lib.tq_b8_decode(ctypes.byref(cfg), d["q"], 0, 0, d["cache"], 38, d["table"], 19, d["lens"], batch, n, 0.0, d["one"], 2,
                               d["ws"], ws, None, None),
              lib.tq_b8_continue(ctypes.byref(cfg), d["q"], 0, 0, d["starts"], batch, 2 * n, n, d["cache"], 38, d["table"], 19,
                                 d["lens"], n, 0.0, d["many"], 2, d["ws"], ws, None, None)]
    out = []
    for name in ("one", "many"):
        x = np.empty(sizes[name] // 4, dtype=np.float32)
        assert rt.cudaMemcpy(ctypes.c_void_p(x.ctypes.data), d[name], ctypes.c_size_t(x.nbytes), 2) == 0
        out.append(x)
    return status, out

status, first = once()
assert status == [0, 0, 0] and all(x.any() and np.isfinite(x).all() for x in first), status
if sys.argv[2] == "reset":
    assert rt.cudaDeviceReset() == 0
else:
    cu, ctx = ctypes.CDLL("libcuda.so.1"), ctypes.c_void_p()
    assert cu.cuCtxCreate_v2(ctypes.byref(ctx), 0, 0) == 0       # and made current
status, second = once()
assert status == [0, 0, 0], status
assert all(np.array_equal(x, y) for x, y in zip(first, second))
print("same")
"""


@pytest.mark.parametrize("how", ["reset", "another"])
def test_calls_in_a_context_after_the_first(tq, how):
    """A process of its own whose CUDA context ends and begins anew, or is left for
    another one of the same device: nothing is remembered of the first."""
    import subprocess
    import sys
    from turboquant_paged_kv_gb300 import _abi
    run = subprocess.run([sys.executable, "-c", _CONTEXT_CHILD, _abi.__file__, how], capture_output=True, text=True, timeout=300)
    assert run.returncode == 0 and run.stdout.strip() == "same", run.stdout + run.stderr


@pytest.mark.parametrize("group", [2, 6])
@pytest.mark.parametrize("gain", [40, 70, 100, 120, 200])
@pytest.mark.parametrize("even", [False, True])
def test_decode_value_scales_as_far_apart_as_they_get(tq, group, gain, even):
    """Some blocks' values are 2^gain times the others', their keys give them no weight
    (or one around 2^-gain, so that both kinds count) with even query heads and all of
    it with odd ones: each head has its own values.
    Enough tiles for every warp to meet both kinds; all sequences share their blocks."""
    n, batch = 1600, 64
    c = Case(tq, "int8_blk", 16, group, 1, [n], seed=23)
    k, v = c.draw(n, 1).float().numpy(), c.draw(n, 1).float().numpy()
    big = np.arange(n) // 16 % 5 == 1
    k[big] = -gain / (128 * SCALE * np.log2(np.e)) if even else -40.0
    v[big] *= np.float32(2.0 ** (gain // 2))
    v[~big] *= np.float32(2.0 ** (gain // 2 - gain))
    o8.store(c.f, c.cache, k, v, [0, n], c.table, [n])
    c.table = np.repeat(c.table, batch, 0)
    c.lens = np.full(batch, n, dtype=np.int32)
    q = torch.ones((batch, group, 128), dtype=torch.bfloat16)
    q[:, 1::2] = -1.0
    q *= torch.linspace(0.5, 1.5, batch)[:, None, None].to(torch.bfloat16)
    got = run_decode(c, q)
    kk, vv = c.kv(0)
    for b in range(batch):
        ref, size, reach = o8.attend(q[b].double().numpy(), kk, vv, SCALE)
        z = kk[:, 0] @ q[b].double().numpy().T * SCALE
        # the floor of `tolerance`, and no more than the weight itself, where that is less than a step
        floor = np.minimum(2.0 ** -24, np.exp(z - z.max(0))).T @ np.abs(vv[:, 0])
        assert np.all(np.abs(got[b] - ref) <= tolerance(ref, size, reach, n, "f32", floor)), b
        assert np.all(np.abs(got[b]).max(-1) > 0), b


# ---------------------------------------------------------------- together


@pytest.mark.parametrize("fmt,block", [("int8_blk", 16), ("e4m3_blk", 128)])
def test_prompts_then_steps(tq, fmt, block):
    """A batch served as a program would: prompts stored and attended in chunks,
    then decode steps (store, then decode, one captured graph replayed), all
    slices of one projection's output; against the oracle's cache at the end."""
    n_q, n_kv, steps = 8, 2, 20
    prompts = [37, 150, 1]
    c = Case(tq, fmt, block, n_q, n_kv, [p + steps for p in prompts], seed=50)
    cache, table, _ = c.gpu()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    done = [0, 0, 0]
    while any(d < p for d, p in zip(done, prompts)):                 # chunks of at most 64 tokens
        q_lens = [min(64, p - d) for d, p in zip(done, prompts)]
        done = [d + n for d, n in zip(done, q_lens)]
        starts = starts_of(q_lens)
        fused = c.draw(int(starts[-1]), n_q + 2 * n_kv, outlier=True)
        dev, lens_d, starts_d = fused.cuda(), torch.tensor(done, dtype=torch.int32, device="cuda"), torch.from_numpy(starts).cuda()
        q, k, v = dev[:, :n_q], dev[:, n_q:n_q + n_kv], dev[:, n_q + n_kv:]
        out = torch.empty((fused.shape[0], n_q, 128), dtype=torch.float32, device="cuda")
        ws = torch.empty(tq.tq_b8_continue_workspace_size(c.cfg, 3, fused.shape[0], 64, 200), dtype=torch.uint8, device="cuda")
        tq.tq_b8_store(c.cfg, k, v, starts_d, 64, cache, table, lens_d, dev_status=status)
        tq.tq_b8_continue(c.cfg, q, starts_d, 64, cache, table, lens_d, 200, out, ws, dev_status=status)
        x = fused.float().numpy()
        o8.store(c.f, c.cache, x[:, n_q:n_q + n_kv], x[:, n_q + n_kv:], starts, c.table, done)
        check_continue(c, fused[:, :n_q], out.cpu().numpy().astype(np.float64), starts, done, "f32", rows=6)
    fused_d = torch.empty((3, n_q + 2 * n_kv, 128), dtype=torch.bfloat16, device="cuda")
    lens_d, starts_d = torch.zeros(3, dtype=torch.int32, device="cuda"), torch.arange(4, dtype=torch.int32, device="cuda")
    out = torch.empty((3, n_q, 128), dtype=torch.float32, device="cuda")
    ws = torch.empty(tq.tq_b8_decode_workspace_size(c.cfg, 3, 200), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tq.tq_b8_store(c.cfg, fused_d[:, n_q:n_q + n_kv], fused_d[:, n_q + n_kv:], starts_d, 1, cache, table, lens_d, dev_status=status)
        tq.tq_b8_decode(c.cfg, fused_d[:, :n_q], cache, table, lens_d, 200, out, ws, dev_status=status)
    for step in range(steps):
        done = [d + 1 for d in done]
        fused = c.draw(3, n_q + 2 * n_kv, outlier=True)
        fused_d.copy_(fused)
        lens_d.copy_(torch.tensor(done, dtype=torch.int32))
        graph.replay()
        x = fused.float().numpy()
        o8.store(c.f, c.cache, x[:, n_q:n_q + n_kv], x[:, n_q + n_kv:], [0, 1, 2, 3], c.table, done)
        torch.cuda.synchronize()
        check_decode(c, fused[:, :n_q], out.cpu().numpy().astype(np.float64), "f32", lens=done)
    assert int(status) == 0
    assert np.array_equal(cache.cpu().numpy(), c.cache)
