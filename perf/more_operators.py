"""Cases for the operators of the 16-bit paged KV cache.

The cache holds the keys and values of the layers that are not quantised, in
bf16 or fp16. Three operators:

  append    new tokens of each sequence: queries and keys are rotated by their
            position, keys and values are written into the sequences' blocks
  decode    attention of one query token a sequence over its cached positions
  continue  causal attention of a chunk of queries a sequence over its cached
            history and the chunk itself

Cache block: n_kv x (block / 16) tiles of 16 tokens; a tile is 16 key rows then
16 value rows of 128 numbers, 4096 bytes each: [2 groups of 8 rows][2 halves of
64 numbers][8 rows][128 bytes], the 16-byte group c of row r at group
c ^ (r & 7).

Rotation: a table of cosines and sines [positions, rot] float32, rot / 2
cosines and then rot / 2 sines a row; number j of the first rot / 2 goes with
number j + rot / 2 ("halves"), or 2 j with 2 j + 1 ("pairs"); numbers from rot
on are left as they are.
"""

import math
import random

import torch

own = False

D = 128
DTYPE = {"bf16": torch.bfloat16, "fp16": torch.float16, "f32": torch.float32}


def _case(name, op, dtype, block, n_q, n_kv, batch, lens, hist=(0, 0), out=None, rot=128, style="halves", lens_seed=1):
    """`lens`: range of the tokens cached (decode) or of the chunk (append, continue); `hist`: of the tokens before the chunk."""
    c = {"op": op, "dtype": dtype, "block": block, "n_q": n_q, "n_kv": n_kv, "batch": batch, "len_lo": lens[0], "len_hi": lens[1],
         "hist_lo": hist[0], "hist_hi": hist[1], "out": out or dtype, "lens_seed": lens_seed}
    if op == "append":
        c["rot"], c["style"] = rot, style
    return {"name": name, **c} if name else c


def listed():
    return [
        # one new token for each of 32 running sequences: the write of every serving step
        _case("append one token x 32", "append", "bf16", 16, 32, 8, 32, (1, 1), (1, 4096)),
        # a batch of prompts and chunks of all lengths, some of them empty, half of each head rotated, in pairs
        _case("append ragged chunks", "append", "fp16", 64, 28, 4, 24, (0, 700), (0, 900), rot=64, style="pairs"),
        # whole prompts written at once
        _case("append prompts 4 x 8192", "append", "bf16", 16, 32, 8, 4, (8192, 8192)),
        # one user, a short conversation: latency
        _case("decode one short", "decode", "bf16", 16, 8, 2, 1, (301, 301)),
        # the framework's headline serving batch, in its unquantised layers
        _case("decode 32 x 4096", "decode", "bf16", 16, 32, 8, 32, (4096, 4096)),
        # a batch of all lengths in 64-token blocks
        _case("decode ragged 64", "decode", "fp16", 64, 32, 8, 64, (512, 16384), lens_seed=3),
        # few long documents, eight query heads a KV head
        _case("decode long 4 x 131072", "decode", "bf16", 128, 64, 8, 4, (131072, 131072)),
        # a few drafted tokens checked at once
        _case("continue drafts", "continue", "fp16", 16, 24, 8, 3, (3, 9), (150, 420)),
        # 128-token chunks over a cached history
        _case("continue 32 x 128", "continue", "bf16", 16, 32, 8, 32, (128, 128), (4096, 4096)),
        # long prompts in chunks over histories of all lengths
        _case("continue 4 x 2048", "continue", "fp16", 64, 32, 8, 4, (2001, 2048), (0, 6144), lens_seed=5),
        # chunks of all lengths, single tokens among them, over histories of all lengths: a mixed serving step
        _case("continue mixed 12", "continue", "bf16", 32, 64, 8, 12, (1, 500), (0, 16384), lens_seed=7),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("append", "decode", "continue"))
    dtype, block = rng.choice(("bf16", "fp16")), rng.choice((16, 32, 64, 128))
    n_kv, group = rng.choice((1, 2, 3, 4, 6, 8)), rng.randint(1, 8)
    seed = rng.randint(1, 1 << 30)
    if op == "append":
        hi = 1 if rng.random() < 0.4 else _log(rng, 2, 4096)
        room = 4 * 8192 * 48 // (n_kv * (group + 2) * hi)
        batch = _log(rng, 1, max(1, min(96, room)))
        return _case("", op, dtype, block, n_kv * group, n_kv, batch, (min(hi, rng.choice((0, 1))), hi), (0, _log(rng, 16, 4096)),
                     rot=rng.choice((0, 32, 64, 96, 128, 128)), style=rng.choice(("halves", "pairs")), lens_seed=seed)
    if op == "decode":
        hi = _log(rng, 1, 100000)
        batch = _log(rng, 1, max(1, min(128, 3000000 // (hi * n_kv))))
        return _case("", op, dtype, block, n_kv * group, n_kv, batch, (rng.randint(0, hi), hi), out=rng.choice((dtype, dtype, "f32")), lens_seed=seed)
    hi, hist = _log(rng, 1, 2048), _log(rng, 1, 16384)
    room = 4 * 32 * 2048 * 8192 // 2
    hist = min(hist, max(1, room // (n_kv * group * hi) - hi))
    batch = _log(rng, 1, max(1, min(32, room // (n_kv * group * hi * (hi + hist)))))
    return _case("", op, dtype, block, n_kv * group, n_kv, batch, (max(1, hi // 3), hi), (hist // 4, hist),
                 out=rng.choice((dtype, dtype, dtype, "f32")), lens_seed=seed)


def _lengths(case):
    """(new tokens, cached tokens with them) of each sequence; new tokens are 0 for the decode."""
    r = random.Random(case["lens_seed"])
    a = [r.randint(case["len_lo"], case["len_hi"]) for _ in range(case["batch"])]
    h = [r.randint(case["hist_lo"], case["hist_hi"]) for _ in range(case["batch"])]
    if not any(a):
        a[-1] = 1
    if case["op"] == "decode":
        return [0] * len(a), a
    return a, [x + y for x, y in zip(a, h)]


def work(case):
    new, total = _lengths(case)
    n_kv, n_q, bs = case["n_kv"], case["n_q"], case["block"]
    size = {"f32": 4}.get(case["out"], 2)
    if case["op"] == "append":
        rows = sum(new)
        seen = set()
        for n, t in zip(new, total):
            seen.update(range(t - n, t))
        blocks = sum((t - 1) // bs - (t - n) // bs + 1 for n, t in zip(new, total) if n)
        return {"bytes": 2 * rows * (n_q + 2 * n_kv) * D * 2 + len(seen) * case["rot"] * 4 + 4 * blocks,
                "flops": 3 * rows * (n_q + n_kv) * case["rot"]}
    read = sum(total) * n_kv * 2 * D * 2 + 4 * sum(-(-t // bs) for t in total)
    if case["op"] == "decode":
        return {"bytes": read + case["batch"] * n_q * D * (2 + size), "flops": 4 * D * n_q * sum(total)}
    pairs = sum(n * (t - n) + n * (n + 1) // 2 for n, t in zip(new, total))
    return {"bytes": read + sum(new) * n_q * D * (2 + size), "flops": 4 * D * n_q * pairs}


# ---------------------------------------------------------------- inputs


def _block_bytes(case):
    return case["n_kv"] * case["block"] * 4 * D


def _numbers(cache, case):
    """The cache as numbers in their stored order: [blocks, n_kv, tiles, keys or values, groups of 8 rows, halves, 8 rows, 8 groups, 8]."""
    return cache.view(DTYPE[case["dtype"]]).view(-1, case["n_kv"], case["block"] // 16, 2, 2, 2, 8, 8, 8)


def _order():
    """Row and stored group of each (row, group) of 8 x 8."""
    r = torch.arange(8, device="cuda")[:, None]
    return r, torch.arange(8, device="cuda")[None, :] ^ r


def _normal(shape, g, outlier, dtype):
    """Keys have a channel that stands out in each head, as in the framework's own workloads."""
    x = torch.randn(shape, generator=g, device="cuda")
    if outlier:
        ch = torch.randint(0, D, (shape[-2],), generator=g, device="cuda")
        x[..., torch.arange(shape[-2], device="cuda"), ch] *= 8.0
    return x.to(DTYPE[dtype])


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 7919 + 29)
    new, total = _lengths(case)
    n_kv, n_q, bs, batch, dtype = case["n_kv"], case["n_q"], case["block"], case["batch"], case["dtype"]
    blocks = [-(-t // bs) for t in total]
    width = max(max(blocks), 1)
    num_blocks = sum(blocks) + 3
    # every place holds numbers: the history, and behind the sequences' ends what is left over from other use
    cache = torch.empty(num_blocks * _block_bytes(case), dtype=torch.uint8, device="cuda")
    numbers = _numbers(cache, case)
    channel = torch.randint(0, D, (n_kv,), generator=g, device="cuda")
    r, c = _order()
    for i in range(0, num_blocks, max(1, (1 << 28) // _block_bytes(case))):
        part = numbers[i:i + max(1, (1 << 28) // _block_bytes(case))]
        x = torch.randn(part.shape, generator=g, device="cuda")
        keys = torch.ones((n_kv, D), device="cuda")
        keys[torch.arange(n_kv, device="cuda"), channel] = 8.0
        # [n_kv, halves, groups, 8] at every row's stored order
        gain = keys.view(n_kv, 2, 8, 8)[:, :, c, :]
        x[:, :, :, 0] *= gain[None, :, None, None]
        part.copy_(x)
        del x
    perm = torch.randperm(num_blocks, generator=g, device="cuda").to(torch.int32)
    table = torch.full((batch, width), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, k in enumerate(blocks):
        table[b, :k] = perm[at:at + k]
        at += k
    rows = sum(new)
    s = {"case": case, "cache": cache, "numbers": numbers, "table": table, "max_len": max(max(total), 1), "new": new, "total": total,
         "lens": torch.tensor(total, dtype=torch.int32, device="cuda"),
         "starts": torch.tensor([sum(new[:i]) for i in range(batch + 1)], dtype=torch.int32, device="cuda"),
         "max_new": max(new), "rows": rows}
    if case["op"] == "append":
        # the projections' output holds queries, keys and values side by side
        fused = torch.cat([_normal((rows, n_q, D), g, False, dtype), _normal((rows, n_kv, D), g, True, dtype),
                           _normal((rows, n_kv, D), g, False, dtype)], 1)
        s["q"], s["key"], s["value"] = fused[:, :n_q], fused[:, n_q:n_q + n_kv], fused[:, n_q + n_kv:]
        s["q_out"] = torch.empty((rows, n_q, D), dtype=DTYPE[dtype], device="cuda")
        # angles of far positions in 64 bits
        half = case["rot"] // 2
        turn = 10000.0 ** (-torch.arange(half, dtype=torch.float64, device="cuda") / max(half, 1))
        angle = torch.arange(s["max_len"] + 5, dtype=torch.float64, device="cuda")[:, None] * turn
        s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float() if half else None
    else:
        s["q"] = _normal((batch if case["op"] == "decode" else rows, n_q, D), g, False, dtype)
    if own:
        import turboquant_paged_kv_gb300 as tq
        cfg = s["cfg"] = tq.make_config("kv_" + dtype, n_q, n_kv, block_size=bs)
        s["tq"] = tq
        if case["op"] != "append":
            s["out"] = torch.empty(s["q"].shape, dtype=DTYPE[case["out"]], device="cuda")
            size = tq.tq_kv16_decode_workspace_size(cfg, batch, s["max_len"]) if case["op"] == "decode" else \
                tq.tq_kv16_continue_workspace_size(cfg, batch, rows, s["max_new"], s["max_len"])
            s["ws"] = torch.empty(size, dtype=torch.uint8, device="cuda")
    return s


# ---------------------------------------------------------------- one pass


def run(s):
    return {"append": _append, "decode": _one_query, "continue": _chunks}[s["case"]["op"]](s)


def _rotated(x, cos, sin, style):
    """x [rows, heads, d] float32; cos, sin [rows, rot / 2]."""
    half = cos.shape[1]
    cos, sin = cos[:, None], sin[:, None]
    y = x.clone()
    a, b = (slice(0, half), slice(half, 2 * half)) if style == "halves" else (slice(0, 2 * half, 2), slice(1, 2 * half, 2))
    y[..., a] = x[..., a] * cos - x[..., b] * sin
    y[..., b] = x[..., b] * cos + x[..., a] * sin
    return y


def _append(s):
    """The cache afterwards, as numbers in their stored order, and the rotated queries."""
    case, bs = s["case"], s["case"]["block"]
    if own:
        s["tq"].tq_kv16_append(s["cfg"], s["key"], s["value"], s["starts"], s["cache"], s["table"], s["lens"], cos_sin=s["cos_sin"],
                               style=case["style"], q=s["q"], q_out=s["q_out"])
        return {"cache": s["numbers"], "q": s["q_out"]}
    t = DTYPE[case["dtype"]]
    starts = s["starts"].long()
    i = torch.arange(s["rows"], device="cuda")
    b = torch.searchsorted(starts[1:].contiguous(), i, right=True)
    pos = s["lens"].long()[b] - starts[b + 1] + i
    q, k, v = s["q"].float(), s["key"].float(), s["value"].float()
    if s["cos_sin"] is not None:
        cos, sin = s["cos_sin"][pos].chunk(2, 1)
        q, k = _rotated(q, cos, sin, case["style"]), _rotated(k, cos, sin, case["style"])
    s["q_out"].copy_(q.to(t))
    blk, row = s["table"].long()[b, pos // bs], pos % bs
    _, c = _order()
    x = torch.stack([k, v], 2).to(t).unflatten(3, (2, 8, 8))  # [rows, n_kv, keys or values, halves, groups, 8]
    at = (slice(None), None, None, None, None)
    s["numbers"][blk[at], torch.arange(case["n_kv"], device="cuda")[None, :, None, None, None], (row // 16)[at],
                 torch.arange(2, device="cuda")[None, None, :, None, None], (row // 8 % 2)[at],
                 torch.arange(2, device="cuda")[None, None, None, :, None], (row % 8)[at], c[row % 8][:, None, None, None, :]] = x
    return {"cache": s["numbers"], "q": s["q_out"]}


def _read(s, table):
    """Keys and values of the blocks in a table [sequences, blocks] as float32 [sequences, n_kv, positions, d]."""
    r, c = _order()
    both = []
    for kv in (0, 1):
        x = s["numbers"][:, :, :, kv][table]  # [sequences, blocks, n_kv, tiles, groups of rows, halves, 8 rows, 8 groups, 8]
        x = x[:, :, :, :, :, :, r, c, :].permute(0, 2, 1, 3, 4, 6, 5, 7, 8)
        both.append(x.reshape(x.shape[0], x.shape[1], -1, D).float())
        del x
    return both


def _attend(q, k, v, seen):
    """q [.., rows, d], k, v [.., length, d]; seen [.., rows, length]: a row that sees nothing gives 0."""
    x = q @ k.transpose(-1, -2) * (1.0 / math.sqrt(D))
    x = x.masked_fill_(~seen, -math.inf)
    x = (x - x.amax(-1, keepdim=True).clamp(min=-1e30)).exp_()
    total = x.sum(-1, keepdim=True)
    return torch.where(total > 0, x @ v / total, torch.zeros((), device="cuda"))


def _one_query(s):
    if own:
        s["tq"].tq_kv16_decode(s["cfg"], s["q"], s["cache"], s["table"], s["lens"], s["max_len"], s["out"], s["ws"])
        return s["out"]
    case = s["case"]
    k, v = _read(s, s["table"].long().clamp(min=0))
    seen = torch.arange(k.shape[2], device="cuda") < s["lens"][:, None]
    q = s["q"].float().view(case["batch"], case["n_kv"], -1, D)
    return _attend(q, k, v, seen[:, None, None]).reshape(s["q"].shape).to(DTYPE[case["out"]])


def _chunks(s):
    if own:
        s["tq"].tq_kv16_continue(s["cfg"], s["q"], s["starts"], s["max_new"], s["cache"], s["table"], s["lens"], s["max_len"], s["out"], s["ws"])
        return s["out"]
    case, group = s["case"], s["case"]["n_q"] // s["case"]["n_kv"]
    out = torch.empty(s["q"].shape, dtype=DTYPE[case["out"]], device="cuda")
    at = 0
    for b, (n, total) in enumerate(zip(s["new"], s["total"])):  # sequence by sequence: scores of all at once would not fit
        k, v = (x[0, :, :total] for x in _read(s, s["table"][b:b + 1, :-(-total // case["block"])].long()))
        q = s["q"][at:at + n].float().view(n, case["n_kv"], group, D).permute(1, 2, 0, 3).reshape(case["n_kv"], group * n, D)
        pos = torch.arange(total - n, total, device="cuda").repeat(group)
        o = _attend(q, k, v, torch.arange(total, device="cuda") <= pos[:, None])
        out[at:at + n] = o.view(case["n_kv"], group, n, D).permute(2, 0, 1, 3).reshape(n, case["n_q"], D).to(out.dtype)
        at += n
    return out


# ---------------------------------------------------------------- in 64 bits


def _place(case, row, kv, d):
    """Where in a head's part of a block number d of row `row` is, in numbers."""
    r = row % 16
    return (row // 16) * 4096 + kv * 2048 + (r // 8) * 1024 + (d // 64) * 512 + (r % 8) * 64 + (((d // 8) % 8) ^ (r % 8)) * 8 + d % 8


def _exact_append(s):
    case, bs, n_kv = s["case"], s["case"]["block"], s["case"]["n_kv"]
    flat = s["cache"].view(DTYPE[case["dtype"]]).double()
    per_head, per_block = bs * 2 * D, n_kv * bs * 2 * D
    q_out = s["q"].double().clone()
    d = torch.arange(D, device="cuda")
    half = case["rot"] // 2
    at = 0
    for b, (n, total) in enumerate(zip(s["new"], s["total"])):
        pos = torch.arange(total - n, total, device="cuda")
        k, v = s["key"][at:at + n].double(), s["value"][at:at + n].double()
        if half:
            turn = torch.complex(s["cos_sin"][pos, :half].double(), s["cos_sin"][pos, half:].double())[:, None]
            first = torch.arange(half, device="cuda") * (1 if case["style"] == "halves" else 2)
            second = first + (half if case["style"] == "halves" else 1)
            for x in (k, q_out[at:at + n]):
                z = torch.complex(x[..., first], x[..., second]) * turn
                x[..., first], x[..., second] = z.real, z.imag
        blk = s["table"][b].long()[pos // bs]
        for kv, x in ((0, k), (1, v)):
            for h in range(n_kv):
                flat[(blk * per_block + h * per_head)[:, None] + _place(case, (pos % bs)[:, None], kv, d)] = x[:, h]
        at += n
    return {"cache": flat.view(s["numbers"].shape), "q": q_out}


def _history(s, b, kv, h):
    """Sequence b's cached rows of head h: [length, d]."""
    case, bs, n_kv = s["case"], s["case"]["block"], s["case"]["n_kv"]
    pos = torch.arange(s["total"][b], device="cuda")
    at = (s["table"][b].long()[pos // bs] * n_kv + h) * bs * 2 * D
    return s["cache"].view(DTYPE[case["dtype"]])[at[:, None] + _place(case, (pos % bs)[:, None], kv, torch.arange(D, device="cuda"))].double()


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "append":
        return _exact_append(s)
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    group, at = case["n_q"] // case["n_kv"], 0
    for b, (n, total) in enumerate(zip(s["new"], s["total"])):
        rows = slice(b, b + 1) if case["op"] == "decode" else slice(at, at + n)
        at += n
        if not total:
            continue
        for h in range(case["n_kv"]):
            k, v = _history(s, b, 0, h), _history(s, b, 1, h)
            for j in range(h * group, (h + 1) * group):
                x = s["q"][rows, j].double() @ k.T / math.sqrt(D)
                if case["op"] == "continue":
                    x[torch.ones(x.shape, dtype=torch.bool, device="cuda").triu(total - n + 1)] = -math.inf
                out[rows, j] = torch.softmax(x, 1) @ v
    return out
