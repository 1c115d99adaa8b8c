"""GPU parity of the 16-bit cache (tq_kv16_*) with oracle/kv16.py: rotation and
placement element by element, attention within ``tolerance``, a bound derived
from the arithmetic.
"""

import numpy as np
import pytest
import torch

from oracle import block8 as o8     # attention over given keys and values
from oracle import kv16 as o16

pytestmark = pytest.mark.gpu

TYPES = ["bf16", "fp16"]
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


def bits_of(x):
    """A 16-bit tensor's bits as uint16."""
    return x.cpu().contiguous().view(torch.int16).numpy().view(np.uint16)


class Case:
    """A cache of random bytes (infinities and NaN among them), a shuffled block
    table with -1 behind each sequence, and room for `room` positions of every
    sequence."""

    def __init__(self, tq, dtype, block, n_q, n_kv, room, seed=0, spare=2, flags=0):
        self.rng = np.random.default_rng(seed)
        self.f = o16.Kv16(dtype, block, n_kv)
        self.cfg = tq.make_config("kv_" + dtype, n_q, n_kv, block_size=block, flags=flags)
        self.tq, self.n_q, self.n_kv, self.block, self.dtype = tq, n_q, n_kv, block, dtype
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

    def draw(self, rows, heads, gain=1.0, outlier=False):
        x = torch.from_numpy(self.rng.standard_normal((rows, heads, 128)).astype(np.float32) * np.float32(gain))
        if outlier and rows:
            x[:, :, 5] *= 8.0
        return x.to(DT[self.dtype])

    def fill(self, lens, gain_v=1.0):
        for b, n in enumerate(lens):
            o16.put(self.f, self.cache, self.table[b], 0, bits_of(self.draw(n, self.n_kv, outlier=True)), bits_of(self.draw(n, self.n_kv, gain_v)))
        self.lens = np.array(lens, dtype=np.int32)
        return self

    def put(self, b, k, v, first=0):
        o16.put(self.f, self.cache, self.table[b], first, bits_of(k), bits_of(v))

    def gpu(self):
        return (torch.from_numpy(self.cache).cuda(), torch.from_numpy(self.table).cuda(), torch.from_numpy(self.lens).cuda())

    def kv(self, b, length=None, cache=None):
        return o16.read(self.f, self.cache if cache is None else cache, self.table[b], int(self.lens[b] if length is None else length),
                        self.blocks)


def starts_of(q_lens):
    return np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32)


def angle_table(positions, rot, base=10000.0):
    a = np.arange(positions)[:, None] * base ** (-np.arange(rot // 2) / max(rot // 2, 1))
    return np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)


# ---------------------------------------------------------------- append


def run_append(c, key, value, starts, lens, angles=None, style="halves", q=None, q_out=None, status=None, cache=None):
    cache = torch.from_numpy(c.cache).cuda() if cache is None else cache
    up = lambda x: x if x is None or x.is_cuda else x.cuda()      # noqa: E731
    if q is not None and q_out is None:
        q_out = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda")
    c.tq.tq_kv16_append(c.cfg, up(key), up(value), torch.from_numpy(np.asarray(starts, dtype=np.int32)).cuda(), cache,
                        torch.from_numpy(c.table).cuda(), torch.from_numpy(np.asarray(lens, dtype=np.int32)).cuda(),
                        cos_sin=None if angles is None else torch.from_numpy(angles).cuda(), style=style, q=up(q), q_out=q_out,
                        dev_status=status)
    torch.cuda.synchronize()
    return cache, q_out


def close(dtype, got_bits, exact, size):
    """got within the roundings of exact: two products and a sum in fp32 (each by 2^-24 of numbers no larger than
    `size`, the products' magnitudes: 3 2^-24), then one rounding to the type. Coordinates that no rotation
    touched are exact as they are: exact == size there, and the rounding of an exact number is itself."""
    got = o16.bits_to_numbers(dtype, got_bits)
    inner = 3 * 2.0 ** -24 * size
    return np.abs(got - exact) <= inner + o16.half_step(dtype, np.abs(exact) + inner)


def check_append(c, before, after, key, value, starts, lens, angles, style, rows=None):
    """The cache afterwards: rows rotated and placed, everything else as it was. `rows`: those that are stored."""
    want = before.copy().view(np.uint16)
    got = after.cpu().numpy().view(np.uint16)
    for b in range(len(lens)):
        q0, n = int(starts[b]), int(starts[b + 1]) - int(starts[b])
        pos = int(lens[b]) - n + np.arange(n)
        keep = np.array([rows is None or rows(b, int(p)) for p in pos], dtype=bool)
        pos, pick = pos[keep], q0 + np.arange(n)[keep]
        if not len(pos):
            continue
        blk = c.table[b][pos // c.block]
        x = key[pick].double().numpy()
        y, size = o16.rotate(x, angles[pos], style) if angles is not None else (x, np.abs(x))
        rot = 0 if angles is None else angles.shape[1]
        for h in range(c.n_kv):
            at = o16.row_index(c.f, blk, h, pos % c.block, 0)
            assert np.all(close(c.dtype, got[at[:, :rot]], y[:, h, :rot], size[:, h, :rot])), (b, h)
            assert np.array_equal(got[at[:, rot:]], bits_of(key[pick, h])[:, rot:]), (b, h)
            want[at] = got[at]
            at = o16.row_index(c.f, blk, h, pos % c.block, 1)
            want[at] = bits_of(value[pick, h])
    assert np.array_equal(got, want)      # values, rows behind the ends, other blocks


def check_queries(c, q, q_out, starts, lens, angles, style):
    got = bits_of(q_out)
    for b in range(len(lens)):
        q0, q1 = int(starts[b]), int(starts[b + 1])
        pos = int(lens[b]) - (q1 - q0) + np.arange(q1 - q0)
        if angles is None:
            assert np.array_equal(got[q0:q1], bits_of(q)[q0:q1])
            continue
        rot = angles.shape[1]
        y, size = o16.rotate(q[q0:q1].double().numpy(), angles[pos], style)
        assert np.all(close(c.dtype, got[q0:q1, :, :rot], y[..., :rot], size[..., :rot])), b
        assert np.array_equal(got[q0:q1, :, rot:], bits_of(q)[q0:q1, :, rot:])


@pytest.mark.parametrize("dtype,block,n_kv,group,rot,style", [
    ("bf16", 16, 8, 4, 128, "halves"), ("fp16", 32, 1, 1, 128, "pairs"), ("bf16", 64, 3, 7, 64, "pairs"), ("fp16", 128, 2, 8, 96, "halves"),
    ("bf16", 16, 2, 5, 16, "halves"), ("fp16", 16, 5, 2, 48, "pairs"), ("fp16", 64, 1, 3, 0, "halves"), ("bf16", 32, 4, 6, 112, "halves")])
def test_append(tq, dtype, block, n_kv, group, rot, style):
    """Chunks that begin and end anywhere: single tokens, whole blocks, an empty chunk, a chunk over several blocks."""
    hist = [0, 5, block, block - 1, 2 * block + 7, 3, block + 1, 0]
    q_lens = [1, 1, block, 2, 3 * block + 5, 0, block - 1, 2 * block]
    lens = np.array(hist) + np.array(q_lens)
    c = Case(tq, dtype, block, n_kv * group, n_kv, lens, seed=block + rot)
    c.fill(hist)
    rows, starts = sum(q_lens), starts_of(q_lens)
    key, value, q = c.draw(rows, n_kv, 3.0, outlier=True), c.draw(rows, n_kv), c.draw(rows, n_kv * group)
    angles = angle_table(int(max(lens)), rot) if rot else None
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    cache, q_out = run_append(c, key, value, starts, lens, angles, style, q, status=status)
    assert int(status) == 0
    check_append(c, c.cache, cache, key, value, starts, lens, angles, style)
    check_queries(c, q, q_out, starts, lens, angles, style)
    # without queries the cache ends up the same
    again, _ = run_append(c, key, value, starts, lens, angles, style)
    assert torch.equal(again, cache)


@pytest.mark.parametrize("batch", [1, 2, 31, 32, 33, 100, 1000, 1025, 2500])
def test_append_finds_the_sequence_of_each_row(tq, batch):
    """Many sequences, most of them of a token or none; all positions from their own lengths."""
    rng = np.random.default_rng(batch)
    q_lens = rng.integers(0, 3, batch)
    q_lens[rng.integers(0, batch)] += 2
    hist = rng.integers(0, 30, batch)
    lens = hist + q_lens
    c = Case(tq, "bf16", 16, 2, 1, np.maximum(lens, 1), seed=batch)
    rows, starts = int(q_lens.sum()), starts_of(q_lens)
    key, value, q = c.draw(rows, 1), c.draw(rows, 1), c.draw(rows, 2)
    angles = angle_table(40, 128)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    cache, q_out = run_append(c, key, value, starts, lens, angles, "pairs", q, status=status)
    assert int(status) == 0
    check_append(c, c.cache, cache, key, value, starts, lens, angles, "pairs")
    check_queries(c, q, q_out, starts, lens, angles, "pairs")


@pytest.mark.parametrize("dtype", TYPES)
def test_append_slices_of_a_fused_projection_in_place(tq, dtype):
    """Queries rotated where they stand, keys and values beside them left as they are."""
    c = Case(tq, dtype, 16, 8, 2, [40, 9], seed=4)
    fused = c.draw(49 + 6, 8 + 2 + 2)
    dev = fused.cuda()
    angles = angle_table(64, 128)
    cache, _ = run_append(c, dev[:49, 8:10], dev[:49, 10:], [0, 40, 49], [40, 9], angles, "halves", dev[:49, :8], dev[:49, :8])
    check_append(c, c.cache, cache, fused[:49, 8:10], fused[:49, 10:], [0, 40, 49], [40, 9], angles, "halves")
    check_queries(c, fused[:49, :8], dev[:49, :8], [0, 40, 49], [40, 9], angles, "halves")
    assert torch.equal(dev[:, 8:].cpu(), fused[:, 8:]) and torch.equal(dev[49:].cpu(), fused[49:])


def test_append_far_positions(tq):
    """Angles of position 131071, in a table of that many rows."""
    n = 131072
    c = Case(tq, "fp16", 128, 4, 1, [200], seed=11)
    c.table = np.tile(c.table, (1, n // c.table.shape[1] + 1))[:, :n // 128].astype(np.int32)
    angles = angle_table(n, 128, 500000.0)
    key, value, q = c.draw(3, 1), c.draw(3, 1), c.draw(3, 4)
    cache, q_out = run_append(c, key, value, [0, 3], [n], angles, "halves", q)
    check_append(c, c.cache, cache, key, value, [0, 3], [n], angles, "halves")
    check_queries(c, q, q_out, [0, 3], [n], angles, "halves")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rot", [0, 128])
def test_append_extreme_values(tq, dtype, rot):
    """Infinities, NaN, numbers that a rotation takes out of the type's range, subnormals."""
    c = Case(tq, dtype, 16, 1, 1, [64], seed=5)
    top, tiny = torch.finfo(DT[dtype]).max, torch.finfo(DT[dtype]).tiny
    key, value, q = c.draw(64, 1), c.draw(64, 1), c.draw(64, 1)
    key[3, 0, 7], key[3, 0, 8], key[5, 0, 0] = float("inf"), float("-inf"), float("nan")
    key[16] = top
    key[17] = -top
    key[18:20] = tiny / 4
    value[1, 0, 3], value[1, 0, 4], value[2, 0, 9] = float("inf"), float("-inf"), float("nan")
    value[20:22] = tiny / 4
    value[22] = top
    q[9, 0, 1] = float("nan")
    angles = angle_table(64, rot) if rot else None
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    cache, q_out = run_append(c, key, value, [0, 64], [64], angles, "halves", q, status=status)
    assert int(status) == tq.TQ_DEV_NOT_FINITE
    k, v = c.kv(0, 64, cache.cpu().numpy())
    assert np.isfinite(k).all() and np.isfinite(v).all()
    assert (v[1, 0, 3], v[1, 0, 4], v[2, 0, 9]) == (top, -top, 0.0)
    x = key.double().numpy()
    y, size = o16.rotate(x, angles[np.arange(64)], "halves") if rot else (x, np.abs(x))
    if not rot:
        assert (k[3, 0, 7], k[3, 0, 8], k[5, 0, 0]) == (top, -top, 0.0)
    else:
        assert k[3, 0, 7] == top or k[3, 0, 7] == -top
        assert k[5, 0, 0] == 0.0 and k[5, 0, 64] == 0.0
    limit = top + float(o16.half_step(dtype, np.array(top)))
    with np.errstate(invalid="ignore"):
        ok = np.isfinite(y) & (np.abs(y) < limit * (1 - 2.0 ** -20))
        over = np.isfinite(y) & (np.abs(y) > limit * (1 + 2.0 ** -20))
    bits = o16.row_index(c.f, c.table[0][np.arange(64) // 16], 0, np.arange(64) % 16, 0)
    good = close(dtype, cache.cpu().numpy().view(np.uint16)[bits][:, None], np.where(ok, y, 0), np.where(ok, size, 0))
    assert np.all(good[ok])
    assert np.array_equal(k[over], np.sign(y[over]) * top)
    if rot:
        assert over.any()
    got_q = q_out.double().cpu().numpy()
    assert np.isnan(got_q[9, 0, 1]) and np.isfinite(np.delete(got_q, 9, 0)).all()


def test_append_device_errors_and_padding(tq):
    """A bad block id, a chunk longer than its sequence, a sequence longer than its row or than the table of angles,
    and rows behind the last sequence: what can be stored is, nothing else is touched, the status tells."""
    c = Case(tq, "bf16", 16, 4, 2, [48, 32, 32, 32], seed=6)
    key, value, q = c.draw(200, 2), c.draw(200, 2), c.draw(200, 4)
    angles = angle_table(100, 64)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def go(lens, starts, want, rows=None, unwritten=(), angles=angles):
        status.zero_()
        cache, q_out = run_append(c, key, value, starts, lens, angles, "halves", q, status=status)
        assert int(status) == want
        check_append(c, c.cache, cache, key, value, starts, lens, angles, "halves", rows)
        left = torch.ones(200, dtype=torch.bool)
        left[:starts[-1]] = False
        left[list(unwritten)] = True
        assert torch.all(q_out[left.cuda()] == 7.0) and not torch.any(torch.all((q_out == 7.0).flatten(1), 1)[~left.cuda()])

    long, bad = tq.TQ_DEV_SEQ_TOO_LONG, tq.TQ_DEV_BLOCK_OUT_OF_RANGE
    go([20, 0, 0, 0], [0, 20, 20, 20, 20], 0)                                           # rows 20 .. 199 are not used
    go([9, 0, 0, 0], [0, 12, 12, 12, 12], long, lambda b, p: p >= 0, range(3))           # 3 rows before position 0
    go([9, 0, 0, 0], [0, 12, 12, 12, 12], long, lambda b, p: p >= 0, range(3), None)
    go([-5, 4, 0, 0], [0, 2, 6, 6, 6], long, lambda b, p: p >= 0, range(2))
    go([60, 0, 0, 0], [0, 60, 60, 60, 60], long, lambda b, p: p < 48)                    # positions 48 .. 59 have no block; queries do
    go([48, 0, 0, 0], [0, 48, 48, 48, 48], long, lambda b, p: p < 30, range(30, 48), angles[:30])
    good = c.table.copy()
    for blk in (-1, c.blocks, 2 ** 31 - 1):
        c.table[0, 1] = blk
        go([48, 0, 0, 0], [0, 48, 48, 48, 48], bad, lambda b, p: not 16 <= p < 32)
        c.table[:] = good
    # starts that go backwards are not allowed, but nothing outside the rows is touched
    status.zero_()
    cache, q_out = run_append(c, key, value, [0, 30, 10, 20, 25], [30, 20, 32, 32], angles, "halves", q, status=status)
    assert torch.all(q_out[30:] == 7.0)


def test_append_in_a_graph_and_on_a_stream(tq):
    """A captured call replayed with other rows, starts and lengths in padded tensors."""
    c = Case(tq, "bf16", 32, 4, 2, [200] * 3, seed=60)
    rows = 64
    key, value, q = (torch.zeros((rows, h, 128), dtype=torch.bfloat16, device="cuda") for h in (2, 2, 4))
    starts, lens = torch.zeros(4, dtype=torch.int32, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda")
    table, angles = torch.from_numpy(c.table).cuda(), angle_table(200, 128)
    turn, cache, q_out = torch.from_numpy(angles).cuda(), torch.empty(c.cache.size, dtype=torch.uint8, device="cuda"), torch.empty_like(q)
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        tq.tq_kv16_append(c.cfg, key, value, starts, cache, table, lens, cos_sin=turn, q=q, q_out=q_out)
    for s, n in (([0, 20, 20, 64], [200, 3, 50]), ([0, 1, 2, 3], [7, 100, 33]), ([0, 0, 0, 0], [1, 2, 3])):
        x = [c.draw(rows, h) for h in (2, 2, 4)]
        for dst, src in zip((key, value, q), x):
            dst.copy_(src)
        starts.copy_(torch.tensor(s, dtype=torch.int32))
        lens.copy_(torch.tensor(n, dtype=torch.int32))
        cache.copy_(torch.from_numpy(c.cache))
        graph.replay()
        torch.cuda.synchronize()
        check_append(c, c.cache, cache, x[0], x[1], s, n, angles, "halves")
        check_queries(c, x[2], q_out, s, n, angles, "halves")
    s, n = [0, 20, 20, 64], [200, 3, 50]
    with torch.cuda.stream(stream):
        starts.copy_(torch.tensor(s, dtype=torch.int32))
        lens.copy_(torch.tensor(n, dtype=torch.int32))
        cache.copy_(torch.from_numpy(c.cache))
        tq.tq_kv16_append(c.cfg, key, value, starts, cache, table, lens, cos_sin=turn, q=q, q_out=q_out)
    stream.synchronize()
    check_append(c, c.cache, cache, x[0], x[1], s, n, angles, "halves")


# ---------------------------------------------------------------- attention


def tolerance(ref, size, reach, length, dtype, out_dtype, spread, chunk=False):
    """Bound on |kernel - exact| per element. size: sum p |v|; reach: the largest
    softmax_scale sum |q k| of a position; spread: sum |v|.
      scores: 128 exact products summed in fp32 (an add errs by at most 2^-23 of
        the running sum of magnitudes) and 4 more roundings: reach 132 2^-23 in
        natural-log units, in the numerator and in the denominator; x - max once
        more, of magnitude 2 reach at most
      weights: ex2.approx 2^-22, then P in two parts of the cache's type: half a step
        of half a step (bf16 2^-16, fp16 2^-22); in one part (a chunk with 16-bit
        output): half a step (bf16 2^-8, fp16 2^-11). A chunk's are rounded once more
        where the row's reference moves within a step: twice that
      sums over the positions: length 2^-23 in either sum, and some for the merge
      floor, fp16 alone: no step below 2^-24, so a weight errs by up to 2^-25
        whatever its size, and twice where it is rounded twice. P = 8 p and the
        largest p of a row is at least 1: the output errs by up to 2^-27 sum |v|
    then half a step of the output's type."""
    delta = reach[..., None] * (132 + 4) * 2.0 ** -23
    single = chunk and out_dtype != "f32"
    p = {("bf16", False): 2.0 ** -16, ("bf16", True): 2.0 ** -8, ("fp16", False): 2.0 ** -22, ("fp16", True): 2.0 ** -11}[dtype, single]
    p *= 2 * 1.01 if chunk else 1.01
    rel = 2 * delta * 1.01 + 2.0 ** -21 + p + 2 * (length + 64) * 2.0 ** -23
    least = {"f32": 1e-37, "bf16": 1e-37, "fp16": 2.0 ** -25}[out_dtype]
    inner = size * rel + (spread * 2.0 ** -27 if dtype == "fp16" else 0.0)
    return inner + (np.abs(ref) + inner) * torch.finfo(DT[out_dtype]).eps / 2 * 1.0001 + least


def check_row(c, q, k, v, got, out_dtype, scale, chunk, where):
    ref, size, reach = o8.attend(q.double().numpy(), k, v, scale)
    spread = np.repeat(np.nansum(np.abs(v), 0), c.n_q // c.n_kv, 0)
    err, tol = np.abs(got - ref), tolerance(ref, size, reach, len(k), c.dtype, out_dtype, spread, chunk)
    assert np.all(err <= tol), (*where, float((err / tol).max()))


def shifted(shape, dtype, value, shift):
    """A tensor of `value` that begins `shift` bytes behind a 32-byte boundary."""
    n, off = int(np.prod(shape)), shift // torch.empty(0, dtype=dtype).element_size()
    room = torch.full((n + 16,), value, dtype=dtype, device="cuda")
    assert room.data_ptr() % 32 == 0
    return room[off:off + n].view(shape)


# Up to so many (sequence, head) pairs go to CTAs of eight, four and two warps; more queries of chunks, and decodes over more
# than 64 tiles a warp, to other kernels
ONE, TWO, FEW = 152, 2 * 152, 4 * 152
LONG = 2064


def widened(table, block):
    """With room for LONG positions a sequence."""
    return torch.nn.functional.pad(table, (0, max(-(-LONG // block) - table.shape[1], 0)), value=-1)


def run_decode(c, q, lens=None, out_dtype="f32", status=None, max_len=None, scale=0.0, line=False, shift=0):
    """`line`: 4 or 2, with empty sequences behind the others until the short kernel's CTAs of so many warps take the call;
    True, and with room for more positions, so that the split and the merge of the line do."""
    cache, table, _ = c.gpu()
    rows = q.shape[0]
    lens = c.lens if lens is None else np.asarray(lens, dtype=np.int32)
    msl = max(int(lens.max(initial=0)), 1) if max_len is None else max_len
    q = q.cuda()
    if line:
        more = max((ONE if line == 4 else TWO) // c.n_kv + 1 - rows, 0)
        q = torch.cat([q, q[:1].repeat(more, 1, 1)])
        lens, table = np.append(lens, np.zeros(more, dtype=np.int32)), torch.cat([table, table[:1].repeat(more, 1)])
    if line is True:
        table = widened(table, c.block)
        msl = max(msl, LONG) if max_len is None else max_len
    out = shifted(q.shape, DT[out_dtype], float("nan"), shift)
    ws = shifted((c.tq.tq_kv16_decode_workspace_size(c.cfg, q.shape[0], msl),), torch.uint8, 255, shift)
    c.tq.tq_kv16_decode(c.cfg, q, cache, table, torch.from_numpy(lens).cuda(), msl, out, ws, scale=scale, dev_status=status)
    torch.cuda.synchronize()
    assert not out[rows:].any()
    return out[:rows].float().cpu().numpy().astype(np.float64)


def check_decode(c, q, got, out_dtype, lens=None, scale=SCALE):
    lens = c.lens if lens is None else lens
    for b in range(q.shape[0]):
        k, v = c.kv(b, int(lens[b]))
        check_row(c, q[b], k, v, got[b], out_dtype, scale, False, (b, int(lens[b])))


@pytest.mark.parametrize("block,n_kv,group,dtype,out", [
    (16, 8, 4, "bf16", "bf16"), (32, 2, 1, "fp16", "fp16"), (64, 1, 8, "bf16", "f32"), (128, 2, 3, "fp16", "f32"),
    (16, 1, 5, "bf16", "f32"), (64, 3, 2, "fp16", "bf16"), (16, 2, 7, "bf16", "fp16"), (32, 1, 6, "fp16", "f32"), (16, 2, 4, "fp16", "f32")])
@pytest.mark.parametrize("line", [False, 4, 2, True])
def test_decode(tq, block, n_kv, group, dtype, out, line):
    lens = [0, 1, 15, 16, 17, 63, 64, 65, 200, 333]
    c = Case(tq, dtype, block, n_kv * group, n_kv, [max(x, 1) for x in lens], seed=group).fill(lens)
    q = c.draw(len(lens), n_kv * group, outlier=True)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = run_decode(c, q, out_dtype=out, status=status, line=line)
    assert int(status) == 0
    assert not got[0].any()                      # nothing cached: zeros
    check_decode(c, q, got, out)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("lens", [[1], [0], [0, 0, 0], [2100], [700, 0, 0, 1, 900], [1500], [9000, 3]])
@pytest.mark.parametrize("line", [False, 4, 2, True])
def test_decode_few_and_empty_sequences(tq, dtype, lens, line):
    c = Case(tq, dtype, 16, 4, 1, [max(x, 1) for x in lens], seed=3).fill(lens)
    q = c.draw(len(lens), 4)
    check_decode(c, q, run_decode(c, q, line=line), "f32")


@pytest.mark.parametrize("batch,n_kv,group,dtype,out,most", [
    (1500, 2, 2, "bf16", "f32", 20), (777, 1, 5, "fp16", "bf16", 20), (199, 3, 7, "bf16", "fp16", 300), (300, 1, 3, "fp16", "f32", 200)])
@pytest.mark.parametrize("line", [False, True])
def test_decode_many_sequences(tq, batch, n_kv, group, dtype, out, most, line):
    """More (sequence, head) pairs than warps, most of them one tile long; heads merged by a warp each, and (the last) by a CTA each."""
    rng = np.random.default_rng(8)
    lens = [int(x) for x in rng.integers(0, most, batch)]
    c = Case(tq, dtype, 16, n_kv * group, n_kv, [max(x, 1) for x in lens], seed=8).fill(lens)
    q = c.draw(len(lens), n_kv * group)
    check_decode(c, q, run_decode(c, q, out_dtype=out, line=line), out)


@pytest.mark.parametrize("lens", [[50, 20], [50, 20, 0, 33] * 40, [2100, 20, 0, 33] * 40])
def test_decode_scale_argument_and_strided_queries(tq, lens):
    c = Case(tq, "fp16", 32, 8, 2, lens, seed=12).fill(lens)
    fused = c.draw(len(lens), 12).cuda()
    got = run_decode(c, fused[:, :8], scale=0.31)
    check_decode(c, fused[:, :8].cpu(), got, "f32", scale=float(np.float32(0.31)))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("gain", [1e-3, 30.0])
@pytest.mark.parametrize("line", [False, 4, 2, True])
def test_decode_scores_that_rise(tq, dtype, gain, line):
    """Keys that grow along the sequence: the running maximum moves again and again, by little or by much."""
    n = 700
    c = Case(tq, dtype, 16, 5, 1, [n], seed=24)
    k = c.draw(n, 1).float() * 0.05 + torch.linspace(-1, 1, n)[:, None, None] * gain / 10
    c.put(0, k.to(DT[dtype]), c.draw(n, 1))
    c.lens = np.array([n], dtype=np.int32)
    q = (torch.ones((1, 5, 128)) * torch.tensor([1.0, -1.0, 0.3, 2.0, 0.0])[None, :, None]).to(DT[dtype])
    check_decode(c, q, run_decode(c, q, line=line), "f32")
    got = run_continue(c, q.repeat(40, 1, 1), [0, 40], [n])
    check_continue(c, q.repeat(40, 1, 1), got, [0, 40], [n], "f32")


@pytest.mark.parametrize("line", [False, 4, 2, True])
def test_decode_device_errors(tq, line):
    length, cut = (2200, 2100) if line is True else (1700, 1600)
    c = Case(tq, "bf16", 16, 4, 2, [length, 40], seed=14).fill([length, 40])
    c.table[0, 2], c.table[0, 95], c.table[1, :] = -1, c.blocks, 2 ** 31 - 1
    q = c.draw(2, 4)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = run_decode(c, q, status=status, max_len=cut, line=line)
    assert int(status) == tq.TQ_DEV_BLOCK_OUT_OF_RANGE | tq.TQ_DEV_SEQ_TOO_LONG
    check_decode(c, q, got, "f32", lens=[cut, 40])      # positions of bad blocks are left out; nothing left: zeros
    assert not got[1].any()


@pytest.mark.parametrize("dtype", TYPES)
def test_not_a_number_query_stays_in_its_row(tq, mode, dtype):
    lens = [40, 40]
    c = Case(tq, dtype, 16, 4, 1, lens, seed=15).fill(lens)
    q = c.draw(2, 4)
    q[0, 1, 3] = float("nan")
    for line in (False, 4, 2, True):
        got = run_decode(c, q, line=line)
        assert np.isnan(got[0, 1]).all() and np.isfinite(got[0, [0, 2, 3]]).all() and np.isfinite(got[1]).all()
    q = c.draw(20, 4)
    q[3, 2, 3], q[5, 0, 7] = float("nan"), float("inf")
    for lens, starts in (([40, 40], [0, 10, 20]), ([40, 40], [0, 1, 20])):
        got = run_continue(c, q, starts, lens)
        assert np.isnan(got[3, 2]).all()
        fine = np.ones((20, 4), dtype=bool)
        fine[3, 2] = fine[5, 0] = False
        assert np.isfinite(got[fine]).all()


@pytest.mark.parametrize("pad,most", [(0, 400), (40, 400), (80, 400), (80, 2100)])      # one launch, or the split and the merge
def test_decode_on_streams_and_in_graphs(tq, pad, most):
    """Two calls on two streams with a workspace each, and a captured call
    replayed after the lengths and the query changed, with the indices known
    early too; the same call twice gives the same bits."""
    lens, rows = [300, 45, 0, 128], 4 + pad
    c = Case(tq, "bf16", 32, 16, 4, [400] * 4, seed=16).fill([400] * 4)
    cache, table, _ = c.gpu()
    table = torch.cat([table, table[:1].repeat(pad, 1)])
    table = widened(table, 32) if most > LONG else table
    lens_d = torch.tensor(lens + [0] * pad, dtype=torch.int32, device="cuda")
    q = [c.draw(rows, 16).cuda() for _ in range(2)]
    n = tq.tq_kv16_decode_workspace_size(c.cfg, rows, most)
    ws = [torch.empty(n, dtype=torch.uint8, device="cuda") for _ in range(2)]
    out = [torch.empty((rows, 16, 128), dtype=torch.float32, device="cuda") for _ in range(2)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for i in range(2):
        with torch.cuda.stream(streams[i]):
            tq.tq_kv16_decode(c.cfg, q[i], cache, table, lens_d, most, out[i], ws[i])
    torch.cuda.synchronize()
    for i in range(2):
        check_decode(c, q[i][:4].cpu(), out[i].cpu().numpy().astype(np.float64), "f32", lens=lens)
    first = out[0].clone()
    tq.tq_kv16_decode(c.cfg, q[0], cache, table, lens_d, most, out[0], ws[0])
    assert torch.equal(first, out[0])
    graphs = []
    for flags in (0, tq.TQ_FLAG_INDICES_READY):      # (the two graphs share a workspace)
        cfg = tq.make_config("kv_bf16", 16, 4, block_size=32, flags=flags)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            tq.tq_kv16_decode(cfg, q[0], cache, table, lens_d, most, out[0], ws[0])
        graphs.append(graph)
    for new in ([400, 1, 33, 0], [17, 399, 64, 250]):
        lens_d[:4].copy_(torch.tensor(new, dtype=torch.int32))
        fresh = c.draw(rows, 16)
        q[0].copy_(fresh)
        for graph in graphs:
            out[0].fill_(float("nan"))
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            check_decode(c, fresh[:4], out[0].cpu().numpy().astype(np.float64), "f32", lens=new)


def test_refusals_with_tensors_on_the_gpu(tq):
    """What the CPU tests cannot reach because a host tensor is refused first."""
    c = Case(tq, "fp16", 16, 4, 1, [20, 20], seed=70).fill([20, 20])
    cache, table, lens = c.gpu()
    q = c.draw(2, 4).cuda()
    out = torch.full_like(q, 5.0)
    n = tq.tq_kv16_decode_workspace_size(c.cfg, 2, 20)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    for bad, match in ((dict(workspace=torch.empty(1, dtype=torch.uint8, device="cuda").expand(n)), "workspace"),
                       (dict(workspace=ws.cpu()), "one CUDA device"), (dict(seq_lens=lens.cpu()), "one CUDA device"),
                       (dict(num_blocks=c.blocks + 1), "blocks"), (dict(dev_status=torch.zeros(1, device="cuda")), "dev_status")):
        args = dict(cfg=c.cfg, q=q, cache=cache, block_table=table, seq_lens=lens, max_seq_len=20, out=out, workspace=ws)
        with pytest.raises(ValueError, match=match):
            tq.tq_kv16_decode(**{**args, **bad})
    with pytest.raises(tq.TQError, match="workspace|invalid"):     # an empty tensor has no address
        tq.tq_kv16_decode(c.cfg, q, cache, table, lens, 20, out, ws[:n - 16])
    with pytest.raises(tq.TQError, match="misaligned"):
        tq.tq_kv16_decode(c.cfg, q, cache, table, lens, 20, out, torch.empty(n + 8, dtype=torch.uint8, device="cuda")[8:])
    kv = c.draw(2, 1).cuda()
    starts = torch.arange(3, dtype=torch.int32, device="cuda")
    before = cache.clone()
    for bad, match in ((dict(cos_sin=torch.zeros((20, 24), device="cuda")), "unsupported"),
                       (dict(cos_sin=torch.zeros((20, 256), device="cuda")), "unsupported"),
                       (dict(cos_sin=torch.zeros(20 * 32 + 2, device="cuda")[2:].view(20, 32)), "misaligned"),
                       (dict(q=out, q_out=torch.empty(1024 + 4, dtype=torch.float16, device="cuda")[4:].view(2, 4, 128)), "misaligned")):
        with pytest.raises(tq.TQError, match=match):
            tq.tq_kv16_append(c.cfg, kv, kv, starts, cache, table, lens, **bad)
    with pytest.raises(ValueError, match="one CUDA device"):
        tq.tq_kv16_append(c.cfg, kv, kv, starts, cache, table, lens, cos_sin=torch.zeros((20, 32)))
    torch.cuda.synchronize()
    assert torch.all(out == 5.0) and torch.equal(cache, before)


# ---------------------------------------------------------------- chunks


MODE = "rows"


@pytest.fixture(params=["rows", 4, 2, "single", "pair"])
def mode(request):
    """Which of its kernels a chunk runs on goes by the sizes of the call: few queries are rows of their own (of CTAs of
    eight warps, 4 or 2); of more, a
    CTA takes 256 rows, or a pair of CTAs 512 where chunks have more than 256 on average. The same chunks come to the
    latter four with rows behind the last sequence, and sequences without queries."""
    global MODE
    MODE = request.param
    yield MODE
    MODE = "rows"


def run_continue(c, q, starts, lens, out_dtype="f32", status=None, max_q=None, max_len=None, scale=0.0, shift=0):
    cache, table, _ = c.gpu()
    rows, batch, group = q.shape[0], len(lens), c.n_q // c.n_kv
    starts, lens = np.asarray(starts, dtype=np.int32), np.asarray(lens, dtype=np.int32)
    msl = max(int(max(lens)), 1) if max_len is None else max_len
    mq = int(np.diff(starts).max(initial=0)) if max_q is None else max_q
    if MODE in (4, 2):
        more = max((ONE if MODE == 4 else TWO) // c.n_kv + 1 - rows, 0)
        q = torch.cat([q.cpu(), torch.zeros((more, *q.shape[1:]), dtype=q.dtype)])
    elif MODE != "rows":
        more = max(FEW + 1 - rows, 0 if MODE == "single" else 256 * batch // group + 1 - rows, 0)
        empty = max(-(-(rows + more) * group // 256) - batch, 0) if MODE == "single" else 0
        q = torch.cat([q.cpu(), torch.zeros((more, *q.shape[1:]), dtype=q.dtype)])
        starts, lens = np.append(starts, [starts[-1]] * empty), np.append(lens, [0] * empty)
        table = torch.cat([table, table[:1].repeat(empty, 1)])
        assert (q.shape[0] * group > 256 * len(lens)) == (MODE == "pair") and q.shape[0] * c.n_kv > FEW
    dev = lambda x: torch.from_numpy(np.asarray(x, dtype=np.int32)).cuda()      # noqa: E731
    out = shifted(q.shape, DT[out_dtype], 123.0, shift)
    ws = shifted((c.tq.tq_kv16_continue_workspace_size(c.cfg, len(lens), q.shape[0], mq, msl),), torch.uint8, 255, shift)
    c.tq.tq_kv16_continue(c.cfg, q.cuda() if not q.is_cuda else q, dev(starts), mq, cache, table, dev(lens), msl, out, ws, scale=scale,
                          dev_status=status)
    torch.cuda.synchronize()
    assert torch.all(out[rows:] == 123.0)
    return out[:rows].float().cpu().numpy().astype(np.float64)


def check_continue(c, q, got, starts, lens, out_dtype, rows=None, scale=SCALE):
    """Every query (or the first, the last and some between of a long chunk) against the oracle."""
    for b in range(len(lens)):
        q0, q1 = int(starts[b]), int(starts[b + 1])
        if q0 == q1:
            continue
        k, v = c.kv(b, max(int(lens[b]), 0))
        n = q1 - q0
        pick = range(n) if n <= 40 or rows is None else sorted({0, 1, n - 1, n - 2, *range(0, n, max(n // rows, 1))})
        for i in pick:
            seen = max(int(lens[b]) - n + i + 1, 0)
            check_row(c, q[q0 + i], k[:seen], v[:seen], got[q0 + i], out_dtype, scale, True, (b, i, seen))


@pytest.mark.parametrize("block,n_kv,group,dtype,out", [
    (16, 2, 4, "bf16", "bf16"), (32, 1, 8, "fp16", "fp16"), (64, 2, 1, "bf16", "f32"), (128, 1, 3, "fp16", "f32"),
    (16, 1, 5, "bf16", "fp16"), (64, 1, 6, "fp16", "bf16"), (32, 1, 7, "bf16", "f32"), (128, 2, 2, "bf16", "f32")])
def test_continue(tq, mode, block, n_kv, group, dtype, out):
    q_lens, hist = [1, 7, 0, 33, 130, 2], [0, 19, 50, 100, 5, 255]
    lens = [a + b for a, b in zip(q_lens, hist)]
    c = Case(tq, dtype, block, n_kv * group, n_kv, lens, seed=group + 30).fill(lens)
    starts = starts_of(q_lens)
    q = c.draw(int(starts[-1]), n_kv * group, outlier=True)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = run_continue(c, q, starts, lens, out, status)
    assert int(status) == 0
    check_continue(c, q, got, starts, lens, out, rows=12)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("q_len,hist,group,n_kv", [(300, 0, 4, 1), (257, 700, 1, 2), (128, 1024, 8, 1), (40, 1500, 4, 1), (1, 3000, 3, 1)])
def test_continue_long(tq, mode, dtype, q_len, hist, group, n_kv):
    c = Case(tq, dtype, 64, n_kv * group, n_kv, [q_len + hist], seed=q_len).fill([q_len + hist])
    q = c.draw(q_len, n_kv * group)
    got = run_continue(c, q, [0, q_len], [q_len + hist])
    check_continue(c, q, got, [0, q_len], [q_len + hist], "f32", rows=16)


@pytest.mark.parametrize("dtype,batch", [("bf16", 90), ("fp16", 77), ("bf16", 500)])
def test_continue_many_chunks(tq, mode, dtype, batch):
    """More (chunk, head) units than SMs, lengths from one position on, empty chunks
    between; all sequences share their blocks."""
    c = Case(tq, dtype, 32, 8, 2, [700], seed=batch).fill([700])
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
    check_continue(c, q, got, starts, lens, "f32")


@pytest.mark.parametrize("n_kv", [1, 2])
def test_continue_lengths_far_apart(tq, mode, n_kv):
    """One long history among short ones, chunks of one query and of many."""
    hist, q_lens = [9000, 3, 0, 700, 0, 17], [5, 200, 1, 64, 0, 1]
    lens = [a + b for a, b in zip(hist, q_lens)]
    c = Case(tq, "bf16", 64, 4 * n_kv, n_kv, [max(x, 1) for x in lens], seed=45).fill(lens)
    starts = starts_of(q_lens)
    q = c.draw(int(starts[-1]), 4 * n_kv)
    for out in ("f32", "bf16"):
        check_continue(c, q, run_continue(c, q, starts, lens, out), starts, lens, out, rows=8)


@pytest.mark.parametrize("q_len", [5, 150])
def test_continue_rows_without_positions_and_padding(tq, mode, q_len):
    """Queries before position 0, past max_q_len and behind the last sequence."""
    c = Case(tq, "fp16", 16, 4, 1, [q_len, 200], seed=40).fill([q_len - 3, 200])
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


def test_continue_starts_that_go_backwards(tq, mode):
    """Not allowed, but nothing outside the rows is touched."""
    batch, n, rows = 401, 600, 32
    c = Case(tq, "bf16", 32, 32, 4, [n], seed=47).fill([n])
    c.table = np.repeat(c.table, batch, 0)
    starts = np.array([0, rows] * ((batch + 1) // 2), dtype=np.int32)
    q = c.draw(rows + 5, 32)
    got = run_continue(c, q, starts, [n] * batch)
    assert np.all(got[rows:] == 123.0)


@pytest.mark.parametrize("q_len,length,cut", [(140, 200, 150), (5, 900, 897), (20, 900, 500)])
def test_continue_cuts_long_sequences(tq, mode, q_len, length, cut):
    """Queries keep their places; none sees a position from max_seq_len on."""
    c = Case(tq, "bf16", 32, 4, 1, [length], seed=49).fill([length])
    q = c.draw(q_len, 4)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = run_continue(c, q, [0, q_len], [length], status=status, max_len=cut)
    assert int(status) == tq.TQ_DEV_SEQ_TOO_LONG
    k, v = c.kv(0)
    for i in range(0, q_len, max(q_len // 20, 1)):
        seen = min(length - q_len + i + 1, cut)
        check_row(c, q[i], k[:seen], v[:seen], got[i], "f32", SCALE, True, (i, seen))


@pytest.mark.parametrize("dtype", TYPES)
def test_one_position_is_its_value(tq, mode, dtype):
    """The weight of a sequence's only position is 1 within ex2's 2^-22, a rounding of a score
    below 64 in the exponent (2^-18) and a rounding of P = 8 p, a number near 8, to the parts
    of the type (2^-16): within 2^-15."""
    batch = 40
    c = Case(tq, dtype, 16, 4, 2, [1] * batch, seed=52).fill([1] * batch)
    q = c.draw(batch, 4)
    for got in (run_continue(c, q, np.arange(batch + 1), c.lens), run_decode(c, q)):
        for b in range(batch):
            k, v = c.kv(b)
            ref = v[0].repeat(2, 0)
            assert np.all(np.abs(got[b] - ref) <= np.abs(ref) * 2.0 ** -15)


@pytest.mark.parametrize("hist,dtype,out", [(20, "bf16", "bf16"), (2000, "fp16", "fp16"), (20, "bf16", "f32"), (2000, "bf16", "f32")])
def test_output_on_16_bytes(tq, mode, hist, dtype, out):
    """out and workspace may lie on any 16 bytes (whole and split histories)."""
    c = Case(tq, dtype, 32, 4, 1, [hist + 40], seed=44).fill([hist + 40])
    q = c.draw(40, 4)
    check_continue(c, q, run_continue(c, q, [0, 40], [hist + 40], out, shift=16), [0, 40], [hist + 40], out, rows=6)
    check_decode(c, q[:1], run_decode(c, q[:1], out_dtype=out, line=mode == "single", shift=16), out)


@pytest.mark.parametrize("q_len", [4, 140])
def test_continue_device_errors(tq, mode, q_len):
    c = Case(tq, "bf16", 16, 4, 1, [200], seed=41).fill([200])
    c.table[0, 3], c.table[0, 9] = -1, 2 ** 31 - 1
    q = c.draw(q_len, 4)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = run_continue(c, q, [0, q_len], [200], status=status)
    assert int(status) == tq.TQ_DEV_BLOCK_OUT_OF_RANGE
    check_continue(c, q, got, [0, q_len], [200], "f32", rows=10)
    c.table[:] = 2 ** 31 - 1                       # nothing left
    assert not run_continue(c, q, [0, q_len], [200], status=status).any()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("q_len,hist", [(37, 30), (150, 0), (6, 900)])
@pytest.mark.parametrize("gain_k,gain_q,scale", [(0.0, 0.0, 0.0), (1e-7, 0.0, 0.0), (0.0, 1e-7, 0.0), (1e-7, 1e-7, 1e-20)])
def test_scores_that_vanish(tq, mode, dtype, q_len, hist, gain_k, gain_q, scale):
    """Scores of nothing or next to it: plain means of the values seen."""
    n = q_len + hist
    c = Case(tq, dtype, 16, 4, 1, [n], seed=46)
    c.put(0, c.draw(n, 1, gain_k), c.draw(n, 1))
    c.lens = np.array([n], dtype=np.int32)
    q = c.draw(q_len, 4, gain_q)
    got = run_continue(c, q, [0, q_len], [n], scale=scale)
    check_continue(c, q, got, [0, q_len], [n], "f32", rows=12, scale=scale or SCALE)
    check_decode(c, q[:1], run_decode(c, q[:1], scale=scale), "f32", scale=scale or SCALE)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("gap", [3, 12, 20, 60, 120, 200])
@pytest.mark.parametrize("step", [1, 16, 100, 130])
def test_continue_scores_that_rise_and_fall(tq, mode, dtype, gap, step):
    """Every `step` positions scores rise by `gap` (log2 units), and fall with the other heads' queries; values as
    large as fp16 has them in the end."""
    n = 8 * step + 5
    c = Case(tq, dtype, 16, 2, 1, [n], seed=92)
    k = torch.zeros((n, 1, 128))
    k += (torch.arange(n) // step)[:, None, None] * (gap / (128 * SCALE * np.log2(np.e)))
    v = c.draw(n, 1).float() * 1000.0
    c.put(0, k.to(DT[dtype]), v.to(DT[dtype]))
    c.lens = np.array([n], dtype=np.int32)
    q = torch.ones((n, 2, 128), dtype=DT[dtype])
    q[:, 1] = -1.0
    for out in ("f32", "bf16"):
        check_continue(c, q, run_continue(c, q, [0, n], [n], out), [0, n], [n], out, rows=40)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("hist", [0, 800])
def test_continue_later_positions_change_nothing(tq, mode, dtype, hist):
    """Bit for bit, whatever the keys and values that a query does not see."""
    q_len = 60
    n, out = hist + q_len, []
    for gain in (1.0, 100.0, 2.0 ** -20, 60000.0):
        c = Case(tq, dtype, 16, 4, 1, [n], seed=93)
        k, v, q = c.draw(n, 1).float(), c.draw(n, 1).float(), c.draw(q_len, 4)
        k[hist + 32:] *= gain
        v[hist + 32:] *= gain
        top = float(torch.finfo(DT[dtype]).max)
        c.put(0, k.clamp(-top, top).to(DT[dtype]), v.clamp(-top, top).to(DT[dtype]))
        c.lens = np.array([n], dtype=np.int32)
        out.append(run_continue(c, q, [0, q_len], [n])[:32])
    for x in out[1:]:
        assert np.array_equal(out[0], x)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("block", [16, 64])
@pytest.mark.parametrize("hist,q_len,max_q", [(10, 20, 5), (0, 140, 70), (900, 30, 7)])
def test_rows_that_were_not_stored(tq, mode, dtype, block, hist, q_len, max_q):
    """What stands in the cache behind the last served query (infinities and NaN) does not count."""
    n, kept = hist + q_len, hist + max_q
    c = Case(tq, dtype, block, 4, 1, [n], seed=94)
    c.cache[:] = 0xff
    c.fill([kept])
    q = c.draw(q_len, 4)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = run_continue(c, q, [0, q_len], [n], max_q=max_q, status=status)
    assert int(status) == tq.TQ_DEV_SEQ_TOO_LONG
    assert not got[max_q:].any()
    check_continue(c, q[:max_q], got[:max_q], [0, max_q], [kept], "f32", rows=12)
    check_decode(c, q[:1], run_decode(c, q[:1], [kept]), "f32", lens=[kept])


@pytest.mark.parametrize("rows,empty", [(64, 0), (200, 0), (400, 5), (400, 0)])      # rows of their own, units of a CTA, of a pair
def test_continue_on_streams_and_in_graphs(tq, rows, empty):
    """As for the decode: two streams, then a captured call replayed with other
    starts, lengths and queries in padded tensors; the same call gives the same bits."""
    c = Case(tq, "fp16", 16, 8, 2, [900] * 3, seed=60).fill([900] * 3)
    cache, table, _ = c.gpu()
    msl, batch = 900, 3 + empty
    table = torch.cat([table, table[:1].repeat(empty, 1)])
    padded = lambda starts, lens: (starts + starts[-1:] * empty, lens + [0] * empty)      # noqa: E731
    assert (rows * 4 > 256 * batch, rows * 2 > FEW) == {64: (False, False), 200: (True, False), 400: (not empty, True)}[rows]
    calls = []
    for starts, lens in (padded([0, 20, 20, 55], [900, 3, 500]), padded([0, 1, 40, 64], [7, 899, 64])):
        q = c.draw(rows, 8)
        calls.append((q, starts, lens, q.cuda(), torch.tensor(starts, dtype=torch.int32, device="cuda"),
                      torch.tensor(lens, dtype=torch.int32, device="cuda"),
                      torch.full((rows, 8, 128), 123.0, dtype=torch.float32, device="cuda"),
                      torch.empty(tq.tq_kv16_continue_workspace_size(c.cfg, batch, rows, 48, msl), dtype=torch.uint8, device="cuda"),
                      torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _, _, _, q, starts, lens, out, ws, stream in calls:
        with torch.cuda.stream(stream):
            tq.tq_kv16_continue(c.cfg, q, starts, 48, cache, table, lens, msl, out, ws)
    torch.cuda.synchronize()
    for q, starts, lens, _, _, _, out, _, _ in calls:
        got = out.cpu().numpy().astype(np.float64)
        check_continue(c, q, got, starts, lens, "f32", rows=5)
        assert np.all(got[starts[-1]:] == 123.0)
    q, _, _, q_d, starts_d, lens_d, out, ws, _ = calls[0]
    first = out.clone()
    tq.tq_kv16_continue(c.cfg, q_d, starts_d, 48, cache, table, lens_d, msl, out, ws)
    assert torch.equal(first, out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tq.tq_kv16_continue(c.cfg, q_d, starts_d, 48, cache, table, lens_d, msl, out, ws)
    for starts, lens in (padded([0, 48, 49, 60], [48, 800, 333]), padded([0, 0, 0, 5], [10, 20, 700]), padded([0, 0, 0, 0], [1, 2, 3])):
        fresh = c.draw(rows, 8)
        q_d.copy_(fresh)
        starts_d.copy_(torch.tensor(starts, dtype=torch.int32))
        lens_d.copy_(torch.tensor(lens, dtype=torch.int32))
        out.fill_(123.0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = out.cpu().numpy().astype(np.float64)
        check_continue(c, fresh, got, starts, lens, "f32", rows=5)
        assert np.all(got[starts[-1]:] == 123.0)


def test_offsets_past_32_bits(tq):
    """The same sequences in a small cache and behind the first 4 GB of a large one
    give the same bits, written and attended to."""
    n_q, n_kv, lens = 16, 8, [300, 77]
    cfg = tq.make_config("kv_bf16", n_q, n_kv, block_size=128)
    bb = tq.tq_kv16_layout_for(cfg).block_bytes
    far = (1 << 32) // bb + 3
    c = Case(tq, "bf16", 128, n_q, n_kv, lens, seed=80)
    key, value, q = c.draw(377, n_kv).cuda(), c.draw(377, n_kv).cuda(), c.draw(377, n_q).cuda()
    starts = torch.tensor([0, 300, 377], dtype=torch.int32, device="cuda")
    lens_d = torch.tensor(lens, dtype=torch.int32, device="cuda")
    turn = torch.from_numpy(angle_table(300, 128)).cuda()
    results = []
    for base in (0, far):
        cache = torch.zeros((base + 8) * bb, dtype=torch.uint8, device="cuda")
        table = torch.tensor([[4, 1, 6], [2, 0, 0]], dtype=torch.int32, device="cuda") + base
        turned = torch.empty_like(q)
        tq.tq_kv16_append(cfg, key, value, starts, cache, table, lens_d, cos_sin=turn, q=q, q_out=turned)
        one = torch.empty((2, n_q, 128), dtype=torch.float32, device="cuda")
        ws = torch.empty(max(tq.tq_kv16_decode_workspace_size(cfg, 2, 300), tq.tq_kv16_continue_workspace_size(cfg, 2, 377, 300, 300)),
                         dtype=torch.uint8, device="cuda")
        tq.tq_kv16_decode(cfg, turned[:2].contiguous(), cache, table, lens_d, 300, one, ws)
        many = torch.empty((377, n_q, 128), dtype=torch.float32, device="cuda")
        tq.tq_kv16_continue(cfg, turned, starts, 300, cache, table, lens_d, 300, many, ws)
        # the same where a decode is the line's, and where a unit is one CTA's
        more = 40
        wide = torch.nn.functional.pad(torch.cat([table, table[:1].repeat(more, 1)]), (0, 14), value=base)
        lens_w = torch.cat([lens_d, lens_d[:1].repeat(more)])
        starts_w = torch.cat([starts, starts[-1:].repeat(more)])
        ws = torch.empty(max(tq.tq_kv16_decode_workspace_size(cfg, 42, LONG), tq.tq_kv16_continue_workspace_size(cfg, 42, 377, 300, 300)),
                         dtype=torch.uint8, device="cuda")
        line = torch.empty((42, n_q, 128), dtype=torch.float32, device="cuda")
        tq.tq_kv16_decode(cfg, turned[:42].contiguous(), cache, wide, lens_w, LONG, line, ws)
        alone = torch.empty((377, n_q, 128), dtype=torch.float32, device="cuda")
        tq.tq_kv16_continue(cfg, turned, starts_w, 300, cache, wide, lens_w, 300, alone, ws)
        results.append((cache[base * bb:].clone(), turned, one, many, line, alone))
    for x, y in zip(*results):
        assert torch.equal(x, y)


def f32_error(c, q, got, seen):
    """2-norm of the difference over that of the exact result, of rows that see `seen` positions of sequence 0."""
    k, v = c.kv(0, max(seen))
    ref = np.stack([o8.attend(q[i].double().numpy(), k[:n], v[:n], SCALE)[0] for i, n in enumerate(seen)])
    return np.sqrt(np.square(got - ref).sum() / np.square(ref).sum())


@pytest.mark.parametrize("dtype", TYPES)
def test_long_sums_in_f32(tq, dtype):
    """The tensor cores cut off what they add to a sum, by half a step of it (2^-24 to 2^-23 of it) on average: 2^-25 of
    the final sum, as the sums before are smaller, for each of the additions. A chunk's sums are of no more than 20 x 8
    additions in 2 parts (320 2^-25), a decode's of 128 in 2 parts or 3 (384 2^-25); the scores' roundings and the
    joining's come to less than half of that. Over 16384 positions in one sum it would be six times as much."""
    n, rows = 16384 + 40, 400
    c = Case(tq, dtype, 128, 8, 1, [n], seed=90).fill([n])
    cache, table, _ = c.gpu()
    batch = 24            # chunks of one sequence: units enough that most are whole
    q = c.draw(64, 8)
    dev = lambda x: torch.from_numpy(np.asarray(x, dtype=np.int32)).cuda()      # noqa: E731
    for q_len in (64, 32):                                                      # a pair's units, and a CTA's
        lens, starts = dev([n] * 8 * batch), dev(np.arange(8 * batch + 1) * q_len)
        out = torch.empty((8 * batch * q_len, 8, 128), dtype=torch.float32, device="cuda")
        ws = torch.empty(tq.tq_kv16_continue_workspace_size(c.cfg, 8 * batch, out.shape[0], q_len, n), dtype=torch.uint8, device="cuda")
        tq.tq_kv16_continue(c.cfg, q[:q_len].cuda().repeat(8 * batch, 1, 1), starts, q_len, cache, table.repeat(8 * batch, 1), lens, n, out, ws)
        got = out.view(8 * batch, q_len, 8, 128)
        # all chunks are the same one: whole or cut anywhere
        assert ((got - got[0]).flatten(1).norm(dim=1) < 2 * 320 * 2.0 ** -25 * 1.5 * got[0].norm()).all()
        for b in (0, 95, 191):
            pick = [0, q_len - 1]
            assert f32_error(c, q[pick], got[b, pick].cpu().numpy().astype(np.float64), [n - q_len + 1 + i for i in pick]) < 320 * 2.0 ** -25 * 1.5
    lens = dev([n] * rows)
    out = torch.empty((rows, 8, 128), dtype=torch.float32, device="cuda")
    ws = torch.empty(tq.tq_kv16_decode_workspace_size(c.cfg, rows, n), dtype=torch.uint8, device="cuda")
    tq.tq_kv16_decode(c.cfg, q[:1].cuda().repeat(rows, 1, 1), cache, table.repeat(rows, 1), lens, n, out, ws)
    assert ((out - out[0]).flatten(1).norm(dim=1) < 2 * 384 * 2.0 ** -25 * 1.5 * out[0].norm()).all()
    for b in (0, 200, 399):
        assert f32_error(c, q[:1], out[b:b + 1].cpu().numpy().astype(np.float64), [n]) < 384 * 2.0 ** -25 * 1.5


_CONTEXT_CHILD = """
import ctypes, importlib.util, sys
import numpy as np
spec = importlib.util.spec_from_file_location("abi", sys.argv[1])
abi = importlib.util.module_from_spec(spec)
spec.loader.exec_module(abi)
lib, rt = abi.load(), ctypes.CDLL("libcudart.so.13")     # the runtime that the library is linked to
batch, n_q, n_kv, n = 2, 8, 2, 300
cfg = abi.tq_config(abi.TQ_PRESET_KV_F16, 128, 16, n_q, n_kv, 0, 0)
lay = abi.tq_kv16_layout()
assert lib.tq_kv16_layout_for(ctypes.byref(cfg), ctypes.byref(lay)) == 0
rng = np.random.default_rng(1)
f16 = lambda *shape: rng.standard_normal(shape).astype(np.float16)
host = dict(k=f16(batch * n, n_kv, 128), v=f16(batch * n, n_kv, 128), q=f16(batch * n, n_q, 128),
            turn=rng.standard_normal((n, 128)).astype(np.float32),
            starts=np.array([0, n, 2 * n], dtype=np.int32), lens=np.array([n, n], dtype=np.int32),
            table=np.arange(38, dtype=np.int32).reshape(2, 19))
ws = max(lib.tq_kv16_decode_workspace_size(ctypes.byref(cfg), batch, n),
         lib.tq_kv16_continue_workspace_size(ctypes.byref(cfg), batch, batch * n, n, n))
sizes = dict(cache=38 * lay.block_bytes, ws=ws, one=batch * n_q * 512, many=batch * n * n_q * 512)

def once():
    d = {}
    for name, size in [*((k, x.nbytes) for k, x in host.items()), *sizes.items()]:
        d[name] = ctypes.c_void_p()
        assert rt.cudaMalloc(ctypes.byref(d[name]), ctypes.c_size_t(size)) == 0
        assert rt.cudaMemset(d[name], 0, ctypes.c_size_t(size)) == 0
    for name, x in host.items():
        assert rt.cudaMemcpy(d[name], ctypes.c_void_p(x.ctypes.data), ctypes.c_size_t(x.nbytes), 1) == 0
    status = [lib.tq_kv16_append(ctypes.byref(cfg), d["k"], 0, d["v"], 0, d["q"], 0, d["q"], 0, d["turn"], 128, n, 0, d["starts"], batch,
                                 2 * n, d["cache"], 38, d["table"], 19, d["lens"], None, None),
              lib.tq_kv16_decode(ctypes.byref(cfg), d["q"], 0, d["cache"], 38, d["table"], 19, d["lens"], batch, n, 0.0, d["one"], 2,
                                 d["ws"], ws, None, None),
              lib.tq_kv16_continue(ctypes.byref(cfg), d["q"], 0, d["starts"], batch, 2 * n, n, d["cache"], 38, d["table"], 19,
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


# ---------------------------------------------------------------- together


@pytest.mark.parametrize("prompts,chunk", [([37, 150, 1], 64), ([700, 1, 433], 256)])
@pytest.mark.parametrize("dtype,block,style", [("bf16", 16, "halves"), ("fp16", 128, "pairs")])
def test_prompts_then_steps(tq, dtype, block, style, prompts, chunk):
    """A batch served as a program would: prompts appended and attended in chunks,
    then decode steps (append, then decode, one captured graph replayed), queries
    rotated in place in one projection's output; attention against the cache as the
    GPU holds it, which is checked against the rotation and the places."""
    n_q, n_kv, steps = 8, 2, 20
    most = max(prompts) + steps
    c = Case(tq, dtype, block, n_q, n_kv, [p + steps for p in prompts], seed=50)
    angles = angle_table(most, 128)
    turn = torch.from_numpy(angles).cuda()
    cache, table, _ = c.gpu()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def after(fused, starts, lens, rotated):
        check_append(c, c.cache, cache, fused[:, n_q:n_q + n_kv], fused[:, n_q + n_kv:], starts, lens, angles, style)
        check_queries(c, fused[:, :n_q], rotated, starts, lens, angles, style)
        c.cache = cache.cpu().numpy()

    done = [0, 0, 0]
    while any(d < p for d, p in zip(done, prompts)):
        q_lens = [min(chunk, p - d) for d, p in zip(done, prompts)]
        done = [d + n for d, n in zip(done, q_lens)]
        starts = starts_of(q_lens)
        fused = c.draw(int(starts[-1]), n_q + 2 * n_kv, outlier=True)
        dev, lens_d, starts_d = fused.cuda(), torch.tensor(done, dtype=torch.int32, device="cuda"), torch.from_numpy(starts).cuda()
        q, k, v = dev[:, :n_q], dev[:, n_q:n_q + n_kv], dev[:, n_q + n_kv:]
        out = torch.empty((fused.shape[0], n_q, 128), dtype=torch.float32, device="cuda")
        ws = torch.empty(tq.tq_kv16_continue_workspace_size(c.cfg, 3, fused.shape[0], chunk, most), dtype=torch.uint8, device="cuda")
        tq.tq_kv16_append(c.cfg, k, v, starts_d, cache, table, lens_d, cos_sin=turn, style=style, q=q, q_out=q, dev_status=status)
        tq.tq_kv16_continue(c.cfg, q, starts_d, chunk, cache, table, lens_d, most, out, ws, dev_status=status)
        after(fused, starts, done, q)
        check_continue(c, q.cpu(), out.cpu().numpy().astype(np.float64), starts, done, "f32", rows=6)
    fused_d = torch.empty((3, n_q + 2 * n_kv, 128), dtype=DT[dtype], device="cuda")
    lens_d, starts_d = torch.zeros(3, dtype=torch.int32, device="cuda"), torch.arange(4, dtype=torch.int32, device="cuda")
    out = torch.empty((3, n_q, 128), dtype=torch.float32, device="cuda")
    ws = torch.empty(tq.tq_kv16_decode_workspace_size(c.cfg, 3, most), dtype=torch.uint8, device="cuda")
    q, k, v = fused_d[:, :n_q], fused_d[:, n_q:n_q + n_kv], fused_d[:, n_q + n_kv:]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tq.tq_kv16_append(c.cfg, k, v, starts_d, cache, table, lens_d, cos_sin=turn, style=style, q=q, q_out=q, dev_status=status)
        tq.tq_kv16_decode(c.cfg, q, cache, table, lens_d, most, out, ws, dev_status=status)
    for step in range(steps):
        done = [d + 1 for d in done]
        fused = c.draw(3, n_q + 2 * n_kv, outlier=True)
        fused_d.copy_(fused)
        lens_d.copy_(torch.tensor(done, dtype=torch.int32))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        after(fused, [0, 1, 2, 3], done, q)
        check_decode(c, q.cpu(), out.cpu().numpy().astype(np.float64), "f32", lens=done)
    assert int(status) == 0


def test_beside_the_other_caches(tq):
    """Layers of one model: the first in 16 bits, the next in 8, with one block table and one set of lengths; the
    queries and keys that append rotated for the first layer are what the 8-bit layer's calls take."""
    n_q, n_kv, lens = 8, 2, [70, 33]
    c = Case(tq, "bf16", 16, n_q, n_kv, lens, seed=55)
    _, table, _ = c.gpu()
    starts, lens_d = torch.tensor([0, 70, 103], dtype=torch.int32, device="cuda"), torch.tensor(lens, dtype=torch.int32, device="cuda")
    turn = torch.from_numpy(angle_table(70, 128)).cuda()
    cfg8 = tq.make_config("e4m3_blk", n_q, n_kv, block_size=16)
    cache16 = torch.zeros(c.blocks * c.f.block_bytes, dtype=torch.uint8, device="cuda")
    cache8 = torch.zeros(c.blocks * tq.tq_b8_layout_for(cfg8).block_bytes, dtype=torch.uint8, device="cuda")
    fused = c.draw(103, n_q + 2 * n_kv).cuda()
    # keys rotated as queries of their own: a config whose query heads are the keys'
    as_keys = tq.make_config("kv_bf16", n_kv, n_kv, block_size=16)
    key = torch.empty((103, n_kv, 128), dtype=torch.bfloat16, device="cuda")
    q, k, v = fused[:, :n_q], fused[:, n_q:n_q + n_kv], fused[:, n_q + n_kv:]
    tq.tq_kv16_append(as_keys, k, v, starts, cache16, table, lens_d, cos_sin=turn, q=k, q_out=key)
    tq.tq_kv16_append(c.cfg, k, v, starts, cache16, table, lens_d, cos_sin=turn, q=q, q_out=q)
    tq.tq_b8_store(cfg8, key, v, starts, 70, cache8, table, lens_d)
    outs = []
    for cfg, cache, size, run in ((c.cfg, cache16, tq.tq_kv16_continue_workspace_size, tq.tq_kv16_continue),
                                  (cfg8, cache8, tq.tq_b8_continue_workspace_size, tq.tq_b8_continue)):
        out = torch.empty((103, n_q, 128), dtype=torch.float32, device="cuda")
        run(cfg, q, starts, 70, cache, table, lens_d, 70, out, torch.empty(size(cfg, 2, 103, 70, 70), dtype=torch.uint8, device="cuda"))
        outs.append(out.cpu().numpy().astype(np.float64))
    c.cache, c.lens = cache16.cpu().numpy(), np.array(lens, dtype=np.int32)
    check_continue(c, q.cpu(), outs[0], [0, 70, 103], lens, "f32", rows=10)
    # e4m3 keys and values are off by up to 2^-4 each: the two layers agree to about that
    assert np.abs(outs[0] - outs[1]).max() < 0.5 and np.corrcoef(outs[0].ravel(), outs[1].ravel())[0, 1] > 0.99


# ---------------------------------------------------------------- steps of many sequences


@pytest.fixture(params=["single", "pair"])
def units(request):
    """A CTA's units or a pair's, as in `mode`."""
    global MODE
    MODE = request.param
    yield MODE
    MODE = "rows"


def mixed_lengths(rng, batch, chunks, most):
    """One query a sequence, none for every ninth, and `chunks` longer ones anywhere."""
    q_lens = np.ones(batch, dtype=np.int64)
    q_lens[::9] = 0
    for b, n in zip(rng.permutation(batch)[:len(chunks)], chunks):
        q_lens[b] = n
    return q_lens, np.maximum(rng.integers(1, most + 1, batch), q_lens)


@pytest.mark.parametrize("batch,n_kv,group,chunks,most,dtype,out", [
    (33, 2, 8, [200, 150, 70], 900, "bf16", "bf16"), (130, 1, 8, [300, 1, 97, 260, 129, 33, 200], 3000, "fp16", "f32"),
    (257, 1, 7, [350, 220, 180], 2500, "bf16", "f32"), (300, 3, 4, [500, 260, 129], 1500, "fp16", "fp16"),
    (1100, 1, 5, [400, 130, 420], 1300, "bf16", "bf16"), (1100, 1, 3, [600, 171, 90], 400, "fp16", "f32")])
def test_continue_chunks_of_several_tiles_among_many_sequences(tq, units, batch, n_kv, group, chunks, most, dtype, out):
    """More sequences than a warp has lanes (1100: than it has for groups of 32), some of three tiles of queries and more."""
    room = max(most, *chunks)
    c = Case(tq, dtype, 32, n_kv * group, n_kv, [room], seed=batch + group).fill([room])
    c.table = np.repeat(c.table, batch, 0)
    q_lens, lens = mixed_lengths(c.rng, batch, chunks, most)
    c.lens = lens.astype(np.int32)
    starts = starts_of(q_lens)
    q = c.draw(int(starts[-1]), n_kv * group)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = run_continue(c, q, starts, lens, out, status)
    assert int(status) == 0
    check_continue(c, q, got, starts, lens, out, rows=10)


def test_continue_more_sequences_than_are_kept(tq):
    """Beyond 16384 sequences chunks are read anew for every sum: long ones on both sides of that."""
    batch, most = 16500, 700
    c = Case(tq, "bf16", 32, 8, 1, [most], seed=5).fill([most])
    c.table = np.repeat(c.table, batch, 0)
    q_lens = (np.arange(batch) % 9 == 0).astype(np.int64)
    lens = np.maximum(c.rng.integers(1, most + 1, batch), q_lens)
    for b, n in ((3, 100), (9000, 65), (16383, 300), (16384, 129), (16499, 260)):
        q_lens[b], lens[b] = n, max(lens[b], n)
    c.lens = lens.astype(np.int32)
    starts = starts_of(q_lens)
    q = c.draw(int(starts[-1]), 8)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = run_continue(c, q, starts, lens, "bf16", status)
    assert int(status) == 0
    check_continue(c, q, got, starts, lens, "bf16", rows=10)


@pytest.mark.parametrize("batch,q_len,group", [(4096, 131072, 8), (2048, 32768, 8)])      # pairs' units, a CTA's
def test_continue_a_long_prompt_among_thousands(tq, batch, q_len, group):
    """The search for a team's work is over long before the others stop waiting for it."""
    at = batch - 7                                     # whose chunk is the prompt
    c = Case(tq, "bf16", 128, group, 1, [q_len], seed=6).fill([q_len])
    c.table = np.repeat(c.table, batch, 0)
    q_lens, lens = np.ones(batch, dtype=np.int64), c.rng.integers(1, 300, batch)
    q_lens[at], lens[at] = q_len, q_len
    starts = starts_of(q_lens)
    rows = int(starts[-1])
    assert (rows * group > 256 * batch) == (batch == 4096)
    q = torch.randn((rows, group, 128), dtype=torch.bfloat16, device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    cache, table, _ = c.gpu()
    out = torch.full_like(q, 123.0)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.empty(tq.tq_kv16_continue_workspace_size(c.cfg, batch, rows, q_len, q_len), dtype=torch.uint8, device="cuda")
    tq.tq_kv16_continue(c.cfg, q, torch.from_numpy(starts).cuda(), q_len, cache, table, torch.from_numpy(lens.astype(np.int32)).cuda(), q_len,
                        out, ws, dev_status=status)
    torch.cuda.synchronize()
    assert int(status) == 0
    assert not torch.any(torch.all(out.view(rows, -1) == 123.0, dim=1))       # every row is written
    k, v = c.kv(0, q_len)
    first = int(starts[at])
    for row, seen in ([(b, int(lens[b])) for b in (0, 31, 32, 1000, at - 1)] + [(first + i, i + 1) for i in (0, 63, q_len // 2 + 5, q_len - 1)] +
                      [(int(starts[b]), int(lens[b])) for b in (at + 1, batch - 1)]):
        check_row(c, q[row].cpu(), k[:seen], v[:seen], out[row].double().cpu().numpy(), "bf16", SCALE, True, (row, seen))


def test_continue_zeros_for_many_queries_past_max_q_len(tq):
    """However many queries are not served: their zeros hold nobody up."""
    rows, group = 600000, 8
    c = Case(tq, "bf16", 64, group, 1, [3000], seed=7).fill([3000])
    c.table = np.repeat(c.table, 3, 0)
    starts, lens = np.array([0, 90, rows - 100, rows], dtype=np.int32), np.array([3000, 2500, 100], dtype=np.int32)
    q = torch.randn((rows, group, 128), dtype=torch.bfloat16, device="cuda", generator=torch.Generator("cuda").manual_seed(2))
    cache, table, _ = c.gpu()
    out = torch.full_like(q, 123.0)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.empty(tq.tq_kv16_continue_workspace_size(c.cfg, 3, rows, 200, 3000), dtype=torch.uint8, device="cuda")
    tq.tq_kv16_continue(c.cfg, q, torch.from_numpy(starts).cuda(), 200, cache, table, torch.from_numpy(lens).cuda(), 3000, out, ws, dev_status=status)
    torch.cuda.synchronize()
    assert int(status) == tq.TQ_DEV_SEQ_TOO_LONG
    assert not out[90 + 200:rows - 100].any()
    k, v = c.kv(0, 3000)
    # row and positions seen: the middle chunk's queries lie past position 0 from its last 2500 on, so those served see none
    for row, seen in ((0, 2911), (89, 3000), (rows - 100, 1), (rows - 1, 100)):
        check_row(c, q[row].cpu(), k[:seen], v[:seen], out[row].double().cpu().numpy(), "bf16", SCALE, True, (row, seen))
    assert not out[90:290].any()


# ---------------------------------------------------------------- prompts: warps of several rounds


def rounds_of(rows, heads):
    """Rounds of 8 head rows that a warp of the append takes, and warps a token."""
    most = -(-heads // 8)
    rounds = min(max(rows * most // (152 * 48), 1), most)
    return rounds, -(-most // rounds)


PROMPTS = [
    # n_kv, group, q_lens, dtype, block, rot, style: the last warp's last rounds lie past the heads, or just end with them
    (8, 4, [1200, 0, 3697, 3], "bf16", 16, 128, "halves"), (2, 8, [5000], "fp16", 64, 64, "pairs"), (5, 5, [1500, 1, 2999], "bf16", 128, 48, "halves"),
    (1, 7, [7000, 7700], "fp16", 32, 112, "pairs"), (8, 1, [4097, 3500], "bf16", 32, 0, "halves"), (6, 3, [9000], "fp16", 16, 16, "halves")]


@pytest.mark.parametrize("n_kv,group,q_lens,dtype,block,rot,style", PROMPTS)
def test_append_of_whole_prompts(tq, n_kv, group, q_lens, dtype, block, rot, style):
    rows, n_q = sum(q_lens), n_kv * group
    assert rounds_of(rows, n_q + 2 * n_kv)[0] > 1
    hist = [7 * i for i in range(len(q_lens))]
    lens = np.array(hist) + np.array(q_lens)
    c = Case(tq, dtype, block, n_q, n_kv, lens, seed=rows)
    starts = starts_of(q_lens)
    key, value, q = c.draw(rows, n_kv, 3.0, outlier=True), c.draw(rows, n_kv), c.draw(rows, n_q)
    angles = angle_table(int(max(lens)), rot) if rot else None
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    cache, q_out = run_append(c, key, value, starts, lens, angles, style, q, status=status)
    assert int(status) == 0
    check_append(c, c.cache, cache, key, value, starts, lens, angles, style)
    check_queries(c, q, q_out, starts, lens, angles, style)


@pytest.mark.parametrize("n_kv,group,q_lens,dtype,block,rot,style", PROMPTS[:3])
def test_append_of_whole_prompts_in_place(tq, n_kv, group, q_lens, dtype, block, rot, style):
    """In a fused projection, with rows behind the last sequence."""
    rows, n_q, extra = sum(q_lens), n_kv * group, 9
    lens = np.array(q_lens)
    c = Case(tq, dtype, block, n_q, n_kv, lens, seed=rows + 1)
    starts = starts_of(q_lens)
    fused = c.draw(rows + extra, n_q + 2 * n_kv)
    dev = fused.cuda()
    angles = angle_table(int(max(lens)), rot)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    cache, _ = run_append(c, dev[:, n_q:n_q + n_kv], dev[:, n_q + n_kv:], starts, lens, angles, style, dev[:, :n_q], dev[:, :n_q], status=status)
    assert int(status) == 0
    check_append(c, c.cache, cache, fused[:, n_q:n_q + n_kv], fused[:, n_q + n_kv:], starts, lens, angles, style)
    check_queries(c, fused[:, :n_q], dev[:, :n_q], starts, lens, angles, style)
    assert torch.equal(dev[:, n_q:].cpu(), fused[:, n_q:]) and torch.equal(dev[rows:].cpu(), fused[rows:])


# ---------------------------------------------------------------- chunks with output of the cache's type


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("q_len,length", [(4, 200), (140, 200), (140, 1500)])
def test_continue_device_errors_with_16_bits(tq, mode, dtype, q_len, length):
    c = Case(tq, dtype, 16, 4, 1, [length], seed=41).fill([length])
    c.table[0, 3], c.table[0, 9], c.table[0, length // 16] = -1, 2 ** 31 - 1, -2
    q = c.draw(q_len, 4)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = run_continue(c, q, [0, q_len], [length], dtype, status=status)
    assert int(status) == tq.TQ_DEV_BLOCK_OUT_OF_RANGE
    check_continue(c, q, got, [0, q_len], [length], dtype, rows=10)
    c.table[:] = 2 ** 31 - 1                       # nothing left
    assert not run_continue(c, q, [0, q_len], [length], dtype, status=status).any()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("block", [16, 64])
@pytest.mark.parametrize("hist,q_len,max_q", [(10, 20, 5), (0, 140, 70), (900, 30, 7), (2000, 90, 85)])
def test_rows_that_were_not_stored_with_16_bits(tq, mode, dtype, block, hist, q_len, max_q):
    n, kept = hist + q_len, hist + max_q
    c = Case(tq, dtype, block, 4, 1, [n], seed=94)
    c.cache[:] = 0xff
    c.fill([kept])
    q = c.draw(q_len, 4)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = run_continue(c, q, [0, q_len], [n], dtype, max_q=max_q, status=status)
    assert int(status) == tq.TQ_DEV_SEQ_TOO_LONG
    assert not got[max_q:].any()
    check_continue(c, q[:max_q], got[:max_q], [0, max_q], [kept], dtype, rows=12)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("hist", [0, 800, 1900])
def test_continue_later_positions_change_nothing_with_16_bits(tq, mode, dtype, hist):
    q_len = 60
    n, out = hist + q_len, []
    for gain in (1.0, 100.0, 2.0 ** -20, 60000.0):
        c = Case(tq, dtype, 16, 4, 1, [n], seed=93)
        k, v, q = c.draw(n, 1).float(), c.draw(n, 1).float(), c.draw(q_len, 4)
        k[hist + 32:] *= gain
        v[hist + 32:] *= gain
        top = float(torch.finfo(DT[dtype]).max)
        c.put(0, k.clamp(-top, top).to(DT[dtype]), v.clamp(-top, top).to(DT[dtype]))
        c.lens = np.array([n], dtype=np.int32)
        out.append(run_continue(c, q, [0, q_len], [n], dtype)[:32])
    for x in out[1:]:
        assert np.array_equal(out[0], x)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("q_len,length,cut", [(140, 200, 150), (5, 900, 897), (20, 900, 500), (200, 2300, 2200)])
def test_continue_cuts_long_sequences_with_16_bits(tq, mode, dtype, q_len, length, cut):
    c = Case(tq, dtype, 32, 4, 1, [length], seed=49).fill([length])
    q = c.draw(q_len, 4)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = run_continue(c, q, [0, q_len], [length], dtype, status=status, max_len=cut)
    assert int(status) == tq.TQ_DEV_SEQ_TOO_LONG
    k, v = c.kv(0)
    for i in range(0, q_len, max(q_len // 20, 1)):
        seen = min(length - q_len + i + 1, cut)
        check_row(c, q[i], k[:seen], v[:seen], got[i], dtype, SCALE, True, (i, seen))


@pytest.mark.parametrize("dtype,batch", [("bf16", 90), ("fp16", 500)])
def test_continue_many_chunks_with_16_bits(tq, mode, dtype, batch):
    c = Case(tq, dtype, 32, 8, 2, [1300], seed=batch).fill([1300])
    c.table = np.repeat(c.table, batch, 0)
    q_lens = c.rng.integers(0, 4, batch)
    lens = np.maximum(c.rng.integers(1, 1301, batch), q_lens)
    c.lens = lens.astype(np.int32)
    starts = starts_of(q_lens)
    q = c.draw(int(starts[-1]), 8)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = run_continue(c, q, starts, lens, dtype, status=status)
    assert int(status) == 0
    check_continue(c, q, got, starts, lens, dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("q_len", [5, 150])
def test_continue_rows_without_positions_with_16_bits(tq, mode, dtype, q_len):
    c = Case(tq, dtype, 16, 4, 1, [q_len, 200], seed=40).fill([q_len - 3, 200])
    starts = np.array([0, q_len, q_len + 4], dtype=np.int32)
    q = c.draw(int(starts[-1]) + 9, 4)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = run_continue(c, q, starts, [q_len - 3, 200], dtype, status=status)
    assert int(status) == 0
    assert not got[:3].any() and np.all(got[starts[-1]:] == 123.0)
    check_continue(c, q, got, starts, [q_len - 3, 200], dtype, rows=10)
    got = run_continue(c, q, starts, [0, 0], dtype, status=status)                  # nobody sees anything
    assert int(status) == 0 and not got[:starts[-1]].any()


@pytest.mark.parametrize("total,shape", [(700, "single"), (5200, "pair")])
def test_continue_of_many_sequences_in_graphs_and_on_streams(tq, total, shape):
    """One captured call on 70 sequences, replayed for other starts, lengths and queries in padded tensors, while another
    stream makes the same calls by itself with a workspace of its own."""
    batch, most, group, n_kv = 70, 1500, 4, 2
    assert (total * group > 256 * batch) == (shape == "pair") and total * n_kv > FEW
    c = Case(tq, "bf16", 16, n_kv * group, n_kv, [most], seed=total).fill([most])
    c.table = np.repeat(c.table, batch, 0)
    cache, table, _ = c.gpu()
    steps = []
    for k, chunks in enumerate(([300, 150], [], [690 if shape == "single" else 1400], [129] * 3)):
        q_lens, lens = mixed_lengths(c.rng, batch, chunks, most)
        if sum(q_lens) > total:
            q_lens[q_lens == 1] = 0
        assert sum(q_lens) <= total
        steps.append((starts_of(q_lens), lens.astype(np.int32), c.draw(total, n_kv * group)))
    up = lambda x: torch.from_numpy(x).cuda()      # noqa: E731
    need = tq.tq_kv16_continue_workspace_size(c.cfg, batch, total, total, most)
    call = lambda q, s, n, out, ws: tq.tq_kv16_continue(c.cfg, q, s, total, cache, table, n, most, out, ws)      # noqa: E731
    s, n, q = up(steps[0][0]), up(steps[0][1]), steps[0][2].cuda()
    out = torch.full_like(q, 123.0)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    main, side = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(main):
        call(q, s, n, out, ws)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=main):
            call(q, s, n, out, ws)
    mine = [(up(a), up(b), x.cuda()) for a, b, x in steps]
    other = [torch.full_like(q, 123.0) for _ in steps]
    ws2 = torch.empty(need, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    for (a, b, x), o in zip(mine, other):
        with torch.cuda.stream(main):
            s.copy_(a)
            n.copy_(b)
            q.copy_(x)
            out.fill_(123.0)
            graph.replay()
        with torch.cuda.stream(side):
            call(x, a, b, o, ws2)
        torch.cuda.synchronize()
        assert torch.equal(out, o)
        a, b = a.cpu().numpy(), b.cpu().numpy()
        c.lens = b
        assert torch.all(out[int(a[-1]):] == 123.0)
        check_continue(c, x.cpu(), out.double().cpu().numpy(), a, b, "bf16", rows=6)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("line", [False, 4, 2, True])
def test_decode_scores_of_a_hundred_million(tq, dtype, line):
    """Scores of 2^27 + 16 and, in the second half, 2^27 + 32 log2 units, which fp32 holds exactly, 16 apart: the former
    weigh 2^-16 of the latter. A record's log-sum-exp, within 8 of its maximum, is rounded to that maximum. The values are
    -1 and 3, the result 3 within 4 2^-16 and the roundings of weights and sums (2^-12 in all, and half of that again)."""
    n, batch = 2048, 40
    c = Case(tq, dtype, 16, 4, 1, [n], seed=3)
    k, v = torch.zeros((n, 1, 128)), torch.full((n, 1, 128), -1.0)
    k[:, :, 0] = 2.0 ** 13
    k[:n // 2, :, 1], k[n // 2:, :, 1], v[n // 2:] = 1.0, 2.0, 3.0
    c.put(0, k.to(DT[dtype]), v.to(DT[dtype]))
    scale = float(np.float32(np.log(2.0)))
    assert np.float32(scale) * np.float32(1.4426950408889634) == 1.0
    for rows in (1, batch):
        c.table, c.lens = np.repeat(c.table[:1], rows, 0), np.full(rows, n, dtype=np.int32)
        q = torch.zeros((rows, 4, 128))
        q[:, :, 0], q[:, :, 1] = 2.0 ** 14, 16.0
        got = run_decode(c, q.to(DT[dtype]), scale=scale, line=line)
        assert np.all(np.abs(got - 3.0) <= 1.5 * 2.0 ** -12), (rows, float(np.abs(got - 3.0).max()))


@pytest.mark.parametrize("top", [1e29, 6e4])
@pytest.mark.parametrize("q_len", [3, 150])
def test_large_values(tq, mode, top, q_len):
    """bf16 values of up to 1e29 over 1500 positions, weighed with up to 60000 before the division by the weights' sum."""
    n = 1500
    c = Case(tq, "bf16", 16, 4, 1, [n], seed=8)
    v = c.draw(n, 1).float()
    c.put(0, c.draw(n, 1, 2.0, outlier=True), (v / v.abs().max() * top).to(torch.bfloat16))
    c.lens = np.array([n], dtype=np.int32)
    q = c.draw(q_len, 4)
    for out in ("f32", "bf16"):
        check_continue(c, q, run_continue(c, q, [0, q_len], [n], out), [0, q_len], [n], out, rows=10)
        check_decode(c, q[:1], run_decode(c, q[:1], out_dtype=out, line={"rows": False, "single": True, "pair": True}.get(mode, mode)), out)
