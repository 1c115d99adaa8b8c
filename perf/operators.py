"""Cases for the operators of the block-scaled 8-bit KV cache.

The cache holds keys and values in 8 bits (e4m3 or int8) with one float32 scale
for each block of tokens and KV head, keys and values apart. Four operators:

  store     new tokens of each sequence quantised into its blocks (a block that
            already holds tokens and whose scale grows is requantised)
  dequant   the cached keys and values of each sequence read back
  decode    attention of one query token a sequence over its cached positions
  continue  causal attention of a chunk of queries a sequence over its cached
            history and the chunk itself

Cache block: n_kv x (block / 16) tiles of 16 tokens, a tile being 16 key rows
then 16 value rows of 128 codes, the 16-byte group c of row r at group
c ^ (r & 7); then n_kv pairs of float32 scales (key, value); the block is padded
to a multiple of 128 bytes.
"""

import math
import random

import torch

own = False

D = 128
FLOOR = 2.0 ** -100
LIMIT = {"e4m3_blk": 448.0, "int8_blk": 127.0}
DTYPE = {"bf16": torch.bfloat16, "fp16": torch.float16, "f32": torch.float32}


def _case(name, op, fmt, block, n_q, n_kv, batch, lens, dtype, hist=(0, 0), out=None, lens_seed=1):
    """`lens`: range of the tokens cached (decode, dequant) or of the chunk (store, continue); `hist`: of the tokens before the chunk."""
    c = {"op": op, "fmt": fmt, "block": block, "n_q": n_q, "n_kv": n_kv, "batch": batch, "len_lo": lens[0], "len_hi": lens[1],
         "hist_lo": hist[0], "hist_hi": hist[1], "dtype": dtype, "out": out or dtype, "lens_seed": lens_seed}
    return {"name": name, **c} if name else c


def listed():
    return [
        # one new token for each of 32 running sequences, most of them in the middle of a block: the write of every serving step
        _case("store one token x 32", "store", "int8_blk", 16, 32, 8, 32, (1, 1), "bf16", (1, 4096)),
        # a batch of prompts and chunks of all lengths, some of them empty, in larger blocks
        _case("store ragged chunks", "store", "e4m3_blk", 64, 28, 4, 24, (0, 700), "fp16", (0, 900)),
        # whole prompts written at once
        _case("store prompts 4 x 8192", "store", "e4m3_blk", 16, 32, 8, 4, (8192, 8192), "bf16"),
        # a few cached histories read back for work outside of the library, odd lengths
        _case("dequant ragged", "dequant", "int8_blk", 32, 8, 2, 5, (33, 777), "fp16"),
        # a whole running batch read back
        _case("dequant 32 x 4096", "dequant", "e4m3_blk", 16, 32, 8, 32, (4096, 4096), "bf16"),
        # one user, a short conversation: latency
        _case("decode one short", "decode", "e4m3_blk", 16, 8, 2, 1, (301, 301), "bf16"),
        # the framework's headline serving batch
        _case("decode 32 x 4096", "decode", "e4m3_blk", 16, 32, 8, 32, (4096, 4096), "bf16"),
        # a batch of all lengths in 64-token blocks
        _case("decode ragged 64", "decode", "int8_blk", 64, 32, 8, 64, (512, 16384), "fp16", lens_seed=3),
        # few long documents, eight query heads a KV head
        _case("decode long 4 x 131072", "decode", "e4m3_blk", 128, 64, 8, 4, (131072, 131072), "bf16"),
        # a few drafted tokens checked at once
        _case("continue drafts", "continue", "int8_blk", 16, 24, 8, 3, (3, 9), "bf16", (150, 420)),
        # 128-token chunks over a cached history
        _case("continue 32 x 128", "continue", "int8_blk", 16, 32, 8, 32, (128, 128), "fp16", (4096, 4096)),
        # long prompts in chunks over histories of all lengths
        _case("continue 4 x 2048", "continue", "e4m3_blk", 64, 32, 8, 4, (2001, 2048), "bf16", (0, 6144), lens_seed=5),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("store", "dequant", "decode", "continue"))
    fmt, block = rng.choice(("e4m3_blk", "int8_blk")), rng.choice((16, 32, 64, 128))
    n_kv, group, dtype = rng.choice((1, 2, 4, 8)), rng.randint(1, 8), rng.choice(("bf16", "fp16"))
    seed = rng.randint(1, 1 << 30)
    if op == "store":
        hi = 1 if rng.random() < 0.4 else _log(rng, 2, 2048)
        batch = _log(rng, 1, 64 if hi < 256 else 12)
        return _case("", op, fmt, block, n_kv * group, n_kv, batch, (min(hi, rng.choice((0, 1))), hi), dtype, (0, _log(rng, 16, 4096)), lens_seed=seed)
    if op == "dequant":
        hi = _log(rng, 16, 4096)
        return _case("", op, fmt, block, n_kv * group, n_kv, _log(rng, 1, 24), (rng.randint(0, hi), hi), dtype, out=rng.choice(("bf16", "fp16", "f32")), lens_seed=seed)
    if op == "decode":
        hi = _log(rng, 1, 100000)
        batch = _log(rng, 1, max(1, min(128, 3000000 // (hi * n_kv))))
        return _case("", op, fmt, block, n_kv * group, n_kv, batch, (rng.randint(0, hi), hi), dtype, out=rng.choice((dtype, dtype, "f32")), lens_seed=seed)
    hi, hist = _log(rng, 1, 2048), _log(rng, 1, 6144)
    room = 4 * 32 * 2048 * 8192 // 2
    batch = _log(rng, 1, max(1, min(24, room // (n_kv * group * hi * (hi + hist)))))
    return _case("", op, fmt, block, n_kv * group, n_kv, batch, (max(1, hi // 3), hi), dtype, (hist // 4, hist), lens_seed=seed)


def _lengths(case):
    """(new tokens, cached tokens with them) of each sequence; new tokens are 0 where an operator has none."""
    r = random.Random(case["lens_seed"])
    a = [r.randint(case["len_lo"], case["len_hi"]) for _ in range(case["batch"])]
    h = [r.randint(case["hist_lo"], case["hist_hi"]) for _ in range(case["batch"])]
    if not any(a):
        a[-1] = 1
    if case["op"] in ("store", "continue"):
        return a, [x + y for x, y in zip(a, h)]
    return [0] * len(a), a


def _block_bytes(case):
    return case["n_kv"] * case["block"] * 2 * D + -(-8 * case["n_kv"] // 128) * 128


def work(case):
    new, total = _lengths(case)
    n_kv, n_q, bs = case["n_kv"], case["n_q"], case["block"]
    size = {"f32": 4}.get(case["out"], 2)
    if case["op"] == "store":
        blocks = sum((t - 1) // bs - (t - n) // bs + 1 for n, t in zip(new, total) if n)
        rows = sum(new) * n_kv
        return {"bytes": rows * 2 * D * 3 + blocks * (8 * n_kv + 4), "flops": rows * 2 * D * 3}
    blocks = sum(-(-t // bs) for t in total)
    read = sum(total) * n_kv * 2 * D + blocks * (8 * n_kv + 4)
    if case["op"] == "dequant":
        return {"bytes": read + case["batch"] * max(total) * n_kv * 2 * D * size, "flops": sum(total) * n_kv * 2 * D}
    if case["op"] == "decode":
        return {"bytes": read + case["batch"] * n_q * D * (2 + size), "flops": 4 * D * n_q * sum(total)}
    seen = sum(n * (t - n) + n * (n + 1) // 2 for n, t in zip(new, total))
    return {"bytes": read + sum(new) * n_q * D * (2 + size), "flops": 4 * D * n_q * seen}


# ---------------------------------------------------------------- inputs


def _split(cache, case):
    """The cache as codes [blocks, n_kv, tiles, 2, 16, 8, 16] (bytes, groups in their stored order) and scales [blocks, n_kv, 2], both views."""
    n_kv, bs = case["n_kv"], case["block"]
    rows = cache.view(-1, _block_bytes(case))
    n = n_kv * bs * 2 * D
    return rows[:, :n].unflatten(1, (n_kv, bs // 16, 2, 16, 8, 16)), rows[:, n:n + 8 * n_kv].view(torch.float32).unflatten(1, (n_kv, 2))


def _order(device):
    r = torch.arange(16, device=device)[:, None]
    return r, torch.arange(8, device=device)[None, :] ^ (r & 7)


def _limit(case):
    """The largest code, on the GPU: a division by a number of the host's would be a product with its reciprocal."""
    return torch.full((), LIMIT[case["fmt"]], device="cuda")


def _encode(x, case):
    """Scaled values to 8-bit codes as bytes: to nearest, ties to even, saturated."""
    if case["fmt"] == "int8_blk":
        return x.round().clamp(-127, 127).to(torch.int8).view(torch.uint8)
    return x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


def _values(codes, case):
    return codes.view(torch.int8 if case["fmt"] == "int8_blk" else torch.float8_e4m3fn).float()


def _normal(shape, g, outlier):
    """Keys have a channel that stands out in each head, as in the framework's own workloads."""
    x = torch.randn(shape, generator=g, device="cuda")
    if outlier:
        ch = torch.randint(0, D, (shape[-2],), generator=g, device="cuda")
        x[..., torch.arange(shape[-2], device="cuda"), ch] *= 8.0
    return x


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 7919 + 17)
    new, total = _lengths(case)
    n_kv, n_q, bs, batch = case["n_kv"], case["n_q"], case["block"], case["batch"]
    blocks = [-(-t // bs) for t in total]
    used, width = sum(blocks), max(max(blocks), 1)
    num_blocks = used + 3
    # the history, quantised block by block; what lies behind a sequence's end is left over from other use
    cache = torch.randint(0, 256, (num_blocks * _block_bytes(case),), generator=g, device="cuda", dtype=torch.uint8)
    if case["op"] == "store":
        cache &= 0xF7  # finite in either format, since the whole cache is compared
    codes, scales = _split(cache, case)
    scales.fill_(0.01)
    r, c = _order("cuda")
    start = [t - n if case["op"] == "store" else t for n, t in zip(new, total)]
    filled = torch.tensor([min(max(s - j * bs, 0), bs) for s, k in zip(start, blocks) for j in range(k)] + [0] * 3, device="cuda")
    perm = torch.randperm(num_blocks, generator=g, device="cuda")
    filled = filled[torch.argsort(perm)]  # tokens held by each physical block
    live = (torch.arange(bs, device="cuda") < filled[:, None])[:, None, :, None]
    for kv in (0, 1):
        x = _normal((num_blocks, bs, n_kv, D), g, kv == 0).transpose(1, 2) * live
        s = (x.abs().amax((2, 3)) / _limit(case)).clamp(min=FLOOR)
        scales[:, :, kv] = torch.where(filled[:, None] > 0, s, scales[:, :, kv])
        y = _encode(x * (1.0 / s)[:, :, None, None], case)
        del x
        rows = codes[:, :, :, kv]
        rows.copy_(torch.where(live.unflatten(2, (bs // 16, 16))[..., None], y.view(num_blocks, n_kv, bs // 16, 16, 8, 16)[:, :, :, r, c], rows))
        del y
    table = torch.full((batch, width), -1, dtype=torch.int32)
    at, perm = 0, perm.cpu().to(torch.int32)
    for b, k in enumerate(blocks):
        table[b, :k] = perm[at:at + k]
        at += k
    rows = sum(new)
    s = {"case": case, "cache": cache, "table": table.cuda(), "max_len": max(max(total), 1),
         "lens": torch.tensor(total, dtype=torch.int32, device="cuda"),
         "starts": torch.tensor([sum(new[:i]) for i in range(batch + 1)], dtype=torch.int32, device="cuda"),
         "max_new": max(new), "rows": rows}
    if case["op"] == "store":
        # the projections' output holds queries, keys and values side by side
        fused = torch.cat([_normal((rows, n_q, D), g, False), _normal((rows, n_kv, D), g, True), _normal((rows, n_kv, D), g, False)], 1).to(DTYPE[case["dtype"]])
        s["key"], s["value"] = fused[:, n_q:n_q + n_kv], fused[:, n_q + n_kv:]
    elif case["op"] != "dequant":
        s["q"] = _normal((batch if case["op"] == "decode" else rows, n_q, D), g, False).to(DTYPE[case["dtype"]])
    if own:
        import turboquant_paged_kv_gb300 as tq
        cfg = s["cfg"] = tq.make_config(case["fmt"], n_q, n_kv, block_size=bs)
        s["tq"] = tq
        if case["op"] == "dequant":
            s["k"] = torch.empty((batch, s["max_len"], n_kv, D), dtype=DTYPE[case["out"]], device="cuda")
            s["v"] = torch.empty_like(s["k"])
        elif case["op"] != "store":
            s["out"] = torch.empty(s["q"].shape, dtype=DTYPE[case["out"]], device="cuda")
            size = tq.tq_b8_decode_workspace_size(cfg, batch, s["max_len"]) if case["op"] == "decode" else \
                tq.tq_b8_continue_workspace_size(cfg, batch, rows, s["max_new"], s["max_len"])
            s["ws"] = torch.empty(size, dtype=torch.uint8, device="cuda")
    return s


# ---------------------------------------------------------------- one pass


def run(s):
    return {"store": _store, "dequant": _dequant, "decode": _one_query, "continue": _chunks}[s["case"]["op"]](s)


def _stored(s):
    """What the store leaves behind: every code as the number it is, and the scales."""
    codes, scales = _split(s["cache"], s["case"])
    return {"codes": codes.view(torch.int8 if s["case"]["fmt"] == "int8_blk" else torch.float8_e4m3fn), "scales": scales}


def _store(s):
    if own:
        s["tq"].tq_b8_store(s["cfg"], s["key"], s["value"], s["starts"], s["max_new"], s["cache"], s["table"], s["lens"])
        return _stored(s)
    case, bs = s["case"], s["case"]["block"]
    codes, scales = _split(s["cache"], case)
    starts, table = s["starts"].long(), s["table"].long()
    count = starts[1:] - starts[:-1]
    first = s["lens"].long() - count  # position of each sequence's first new token
    i = torch.arange(s["rows"], device="cuda")
    b = torch.searchsorted(starts[1:].contiguous(), i, right=True)
    pos = first[b] + i - starts[b]
    blk, row = table[b, pos // bs], pos % bs
    x = torch.stack([s["key"], s["value"]], 2).float()  # [rows, n_kv, 2, d]
    # scales: of the new tokens of each block, and of what its sequence held there before
    new = torch.zeros_like(scales).scatter_reduce_(0, blk[:, None, None].expand(-1, *scales.shape[1:]), x.abs().amax(3), "amax")
    touched = torch.zeros(scales.shape[0], dtype=torch.bool, device="cuda").index_fill_(0, blk, True)[:, None, None]
    new = (new / _limit(case)).clamp(min=FLOOR)
    home = table.gather(1, (first // bs).clamp(max=table.shape[1] - 1)[:, None])[:, 0]
    held = ((first % bs > 0) & (count > 0))[:, None, None]
    home = home.clamp(min=0)
    old = scales[home]
    was = torch.zeros_like(scales).index_put_((home,), torch.where(held, old, torch.zeros_like(old)), accumulate=True)
    scales.copy_(torch.where(touched, torch.maximum(new, was), scales))
    # tokens before the new ones in the blocks that the new ones begin in
    r, c = _order("cuda")
    before = codes[home]  # [batch, n_kv, tiles, 2, 16, 8, 16]
    ratio = torch.where(held, old / scales[home], torch.ones_like(old))[:, :, None, :, None, None, None]
    at = torch.arange(bs, device="cuda").view(bs // 16, 1, 16, 1, 1)
    keep = held[..., None, None, None, None] & (at < (first % bs).view(-1, 1, 1, 1, 1, 1, 1)) & (ratio < 1)
    after = _encode(_values(before, case) * ratio, case)
    # the difference is added (modulo 256): a sequence that changes nothing adds 0, wherever its place in the table points
    codes.index_put_((home,), torch.where(keep, after - before, torch.zeros_like(before)), accumulate=True)
    y = _encode(x * (1.0 / scales)[blk][..., None], case).unflatten(3, (8, 16))
    order = c[row % 16]  # the stored group of each group of a row
    codes[blk[:, None, None, None], torch.arange(case["n_kv"], device="cuda")[None, :, None, None], (row // 16)[:, None, None, None],
          torch.arange(2, device="cuda")[None, None, :, None], (row % 16)[:, None, None, None], order[:, None, None, :]] = y
    return _stored(s)


def _read(s):
    """Keys and values of every sequence as float32 [batch, n_kv, length, d], 0 behind the end."""
    case, bs = s["case"], s["case"]["block"]
    codes, scales = _split(s["cache"], case)
    table = s["table"].long().clamp(min=0)
    r, c = _order("cuda")
    length = table.shape[1] * bs
    live = (torch.arange(length, device="cuda") < s["lens"][:, None])[:, None, :, None]
    both = []
    for kv in (0, 1):
        x = _values(codes[:, :, :, kv][table][..., r, c, :], case)  # [batch, blocks, n_kv, tiles, 16, 8, 16]
        x *= scales[:, :, kv][table][:, :, :, None, None, None, None]
        x = x.transpose(1, 2).reshape(case["batch"], case["n_kv"], length, D)
        both.append(torch.where(live, x, torch.zeros((), device="cuda"))[:, :, :s["max_len"]])
        del x
    return both


def _dequant(s):
    if own:
        s["tq"].tq_b8_dequant(s["cfg"], s["cache"], s["table"], s["lens"], s["max_len"], s["k"], s["v"])
        return {"key": s["k"], "value": s["v"]}
    k, v = _read(s)
    t = DTYPE[s["case"]["out"]]
    return {"key": k.transpose(1, 2).to(t).contiguous(), "value": v.transpose(1, 2).to(t).contiguous()}


def _attend(q, k, v, seen):
    """q [batch, n_kv, rows, d]; seen [batch, rows, length]: a row that sees nothing gives 0."""
    x = q @ k.transpose(2, 3) * (1.0 / math.sqrt(D))
    x = x.masked_fill_(~seen[:, None], -math.inf)
    x = (x - x.amax(3, keepdim=True).clamp(min=-1e30)).exp_()
    total = x.sum(3, keepdim=True)
    return torch.where(total > 0, x @ v / total, torch.zeros((), device="cuda"))


def _one_query(s):
    if own:
        s["tq"].tq_b8_decode(s["cfg"], s["q"], s["cache"], s["table"], s["lens"], s["max_len"], s["out"], s["ws"])
        return s["out"]
    case = s["case"]
    k, v = _read(s)
    q = s["q"].float().view(case["batch"], case["n_kv"], -1, D)
    seen = (torch.arange(s["max_len"], device="cuda") < s["lens"][:, None])[:, None].expand(-1, q.shape[2], -1)
    return _attend(q, k, v, seen).reshape(s["q"].shape).to(DTYPE[case["out"]])


def _chunks(s):
    if own:
        s["tq"].tq_b8_continue(s["cfg"], s["q"], s["starts"], s["max_new"], s["cache"], s["table"], s["lens"], s["max_len"], s["out"], s["ws"])
        return s["out"]
    case, n, group = s["case"], s["max_new"], s["case"]["n_q"] // s["case"]["n_kv"]
    k, v = _read(s)
    starts = s["starts"].long()
    count = starts[1:] - starts[:-1]
    i = torch.arange(n, device="cuda")
    at = (starts[:-1, None] + i).clamp(max=s["rows"] - 1)  # [batch, n]: the rows of each chunk, then others' that are not used
    q = s["q"].float()[at].view(case["batch"], n, case["n_kv"], group, D).transpose(1, 2).reshape(case["batch"], case["n_kv"], n * group, D)
    pos = (s["lens"].long() - count)[:, None] + i
    seen = torch.arange(s["max_len"], device="cuda") <= pos.repeat_interleave(group, 1)[:, :, None]
    o = _attend(q, k, v, seen).view(case["batch"], case["n_kv"], n, group, D).transpose(1, 2).reshape(case["batch"], n, case["n_q"], D)
    j = torch.arange(s["rows"], device="cuda")
    b = torch.searchsorted(starts[1:].contiguous(), j, right=True)
    return o[b, j - starts[b]].to(DTYPE[case["out"]])



# ---------------------------------------------------------------- in 64 bits


def _real(byte, case):
    """The number that a code stands for, from its bits."""
    u = byte.to(torch.int64)
    if case["fmt"] == "int8_blk":
        return (u - 256 * (u >> 7)).double()
    exponent, mantissa = (u >> 3) & 15, (u & 7).double()
    size = torch.where(exponent > 0, (8 + mantissa) * torch.exp2((exponent - 10).double()), mantissa * 2.0 ** -9)
    return torch.where((u & 127) == 127, math.nan, torch.where(u > 127, -size, size))


def _nearest(x, case):
    """The code's number next to x."""
    if case["fmt"] == "int8_blk":
        return torch.round(x).clamp(-127, 127)
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(x / step) * step).clamp(-448, 448)


def _history(s, b, kv):
    """Sequence b's cached rows [length, n_kv, d]."""
    case, bs, n_kv = s["case"], s["case"]["block"], s["case"]["n_kv"]
    length = int(s["lens"][b])
    rows = s["cache"].view(-1, _block_bytes(case))
    p = torch.arange(length, device="cuda")
    blk, row = s["table"][b].long()[p // bs], p % bs
    d = torch.arange(D, device="cuda")
    inside = ((row // 16) * 2 + kv)[:, None] * 2048 + (row % 16)[:, None] * D + ((d // 16)[None, :] ^ (row % 8)[:, None]) * 16 + d % 16
    out = torch.empty((length, n_kv, D), dtype=torch.float64, device="cuda")
    for h in range(n_kv):
        at = n_kv * bs * 2 * D + (2 * h + kv) * 4
        scale = rows[:, at:at + 4].contiguous().view(torch.float32)[blk, 0].double()
        out[:, h] = _real(rows[blk[:, None], h * bs * 2 * D + inside], case) * scale[:, None]
    return out


def _exact_store(s):
    case, bs = s["case"], s["case"]["block"]
    codes, scales = _split(s["cache"], case)
    values, scales = _real(codes, case), scales.double()
    starts, lens, table = s["starts"].tolist(), s["lens"].tolist(), s["table"].tolist()
    x = torch.stack([s["key"], s["value"]]).double()
    for b in range(case["batch"]):
        n = starts[b + 1] - starts[b]
        p = lens[b] - n
        while p < lens[b]:
            j, first = p // bs, p % bs
            end = min(lens[b], (j + 1) * bs) - j * bs
            blk = table[b][j]
            t = x[:, starts[b] + p - (lens[b] - n):][:, :end - first]
            for kv in (0, 1):
                scale = (t[kv].abs().amax((0, 2)) / LIMIT[case["fmt"]]).clamp(min=FLOOR)
                if first:
                    was = scales[blk, :, kv].clone()
                    scale = torch.maximum(scale, was)
                rows = values[blk, :, :, kv].flatten(1, 2)  # [n_kv, block, 8, 16], a copy
                if first:
                    rows[:, :first] = torch.where((scale > was)[:, None, None, None], _nearest(rows[:, :first] * (was / scale)[:, None, None, None], case), rows[:, :first])
                r = torch.arange(first, end, device="cuda")[:, None]
                rows[:, r, torch.arange(8, device="cuda") ^ (r % 8)] = _nearest(t[kv].transpose(0, 1) / scale[:, None, None], case).unflatten(2, (8, 16))
                values[blk, :, :, kv] = rows.unflatten(1, (bs // 16, 16))
                scales[blk, :, kv] = scale
            p = (j + 1) * bs
    return {"codes": values if case["fmt"] == "e4m3_blk" else None, "scales": scales}


def exact(case, seed):
    s = prepare(case, seed)
    starts, lens = s["starts"].tolist(), s["lens"].tolist()
    if case["op"] == "store":
        return _exact_store(s)
    if case["op"] == "dequant":
        out = [torch.zeros((case["batch"], s["max_len"], case["n_kv"], D), dtype=torch.float64, device="cuda") for _ in (0, 1)]
        for b, n in enumerate(lens):
            for kv in (0, 1):
                out[kv][b, :n] = _history(s, b, kv)
        return {"key": out[0], "value": out[1]}
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    group = case["n_q"] // case["n_kv"]
    for b, n in enumerate(lens):
        first, last = (b, b + 1) if case["op"] == "decode" else (starts[b], starts[b + 1])
        if not n or first == last:
            continue
        k, v = _history(s, b, 0), _history(s, b, 1)
        for h in range(case["n_q"]):
            x = s["q"][first:last, h].double() @ k[:, h // group].T / math.sqrt(D)
            if case["op"] == "continue":
                hidden = torch.ones(x.shape, dtype=torch.bool, device="cuda").triu(n - (last - first) + 1)
                x[hidden] = -math.inf
            out[first:last, h] = torch.softmax(x, 1) @ v[:, h // group]
    return out
