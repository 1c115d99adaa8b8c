"""16-bit cache on the host: layout, workspace sizes, argument checks, and the oracle's own checks.

No test here launches a kernel: every call runs host code only or returns an
error before reaching the GPU.
"""

import ctypes

import numpy as np
import pytest
import torch

from oracle import kv16 as o16


@pytest.fixture(scope="module")
def tq():
    from turboquant_paged_kv_gb300 import build
    build.build()
    import turboquant_paged_kv_gb300 as tq
    return tq


OK = ctypes.c_void_p(0x10000)
ODD = ctypes.c_void_p(0x10008)
ODD4 = ctypes.c_void_p(0x10002)
OTHER = ctypes.c_void_p(0x20000)


def test_oracle_rotation_is_a_complex_product():
    """Pairs are complex numbers times exp(i angle): lengths stay, rotations add up, both pairings are one
    another's permutation, coordinates behind rot_dim stay."""
    rng = np.random.default_rng(0)
    x = rng.standard_normal((5, 3, 128))
    for rot in (16, 64, 96, 128):
        a = rng.uniform(-9, 9, (5, rot // 2))
        angles = np.concatenate([np.cos(a), np.sin(a)], 1)
        for style in ("halves", "pairs"):
            y, _ = o16.rotate(x, angles, style)
            assert np.allclose((y ** 2).sum(-1), (x ** 2).sum(-1)) and np.array_equal(y[..., rot:], x[..., rot:])
            back, _ = o16.rotate(y, np.concatenate([np.cos(a), -np.sin(a)], 1), style)
            assert np.allclose(back, x)
        z = (x[..., 0:rot:2] + 1j * x[..., 1:rot:2]) * np.exp(1j * a)[:, None]
        y, _ = o16.rotate(x, angles, "pairs")
        assert np.allclose(y[..., 0:rot:2], z.real) and np.allclose(y[..., 1:rot:2], z.imag)
        order = np.concatenate([np.arange(0, rot, 2), np.arange(1, rot, 2), np.arange(rot, 128)])
        w, _ = o16.rotate(x[..., order], angles, "halves")
        assert np.allclose(w, y[..., order])


@pytest.mark.parametrize("block,n_kv", [(16, 1), (64, 3), (128, 8)])
def test_oracle_places_fill_a_block(block, n_kv):
    f = o16.Kv16("bf16", block, n_kv)
    at = np.concatenate([o16.row_index(f, 2, h, np.arange(block), kv).ravel() for h in range(n_kv) for kv in (0, 1)])
    assert np.array_equal(np.sort(at), np.arange(2 * f.block_bytes // 2, 3 * f.block_bytes // 2))
    # 8 consecutive coordinates stay together, on 16 bytes
    assert np.all(at.reshape(-1, 8) == at[::8, None] + np.arange(8)) and np.all(at[::8] % 8 == 0)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_oracle_numbers(dtype):
    t = torch.bfloat16 if dtype == "bf16" else torch.float16
    bits = np.arange(1 << 16, dtype=np.uint16)
    want = torch.from_numpy(bits.view(np.int16).copy()).view(t).double().numpy()
    assert np.array_equal(o16.bits_to_numbers(dtype, bits), want, equal_nan=True)
    x = want[np.isfinite(want) & (want > 0)]
    x.sort()
    assert np.array_equal(o16.half_step(dtype, x[:-1]), np.diff(x) / 2)


@pytest.mark.parametrize("fmt", ["kv_bf16", "kv_fp16"])
@pytest.mark.parametrize("bs", [16, 32, 64, 128])
@pytest.mark.parametrize("n_kv", [1, 8, 20])
def test_layout(tq, fmt, bs, n_kv):
    lay = tq.tq_kv16_layout_for(tq.make_config(fmt, n_kv, n_kv, block_size=bs))
    f = o16.Kv16(fmt[3:], bs, n_kv)
    assert (lay.is_bf16, lay.tile_tokens, lay.tile_bytes, lay.k_off, lay.v_off) == (int(fmt == "kv_bf16"), 16, 8192, 0, 4096)
    assert lay.block_bytes == f.block_bytes


def test_layout_refusals(tq):
    from turboquant_paged_kv_gb300 import _abi
    lib, lay = _abi.load(), _abi.tq_kv16_layout()
    for cfg, want in [(tq.make_config("4bit_nc", 8, 8), _abi.TQ_ERR_INVALID_ARG),
                      (tq.make_config("e4m3_blk", 8, 8), _abi.TQ_ERR_INVALID_ARG),
                      (tq.make_config("kv_bf16", 8, 8, head_dim=64), _abi.TQ_ERR_UNSUPPORTED),
                      (tq.make_config("kv_bf16", 8, 8, block_size=24), _abi.TQ_ERR_UNSUPPORTED),
                      (tq.make_config("kv_bf16", 8, 0), _abi.TQ_ERR_INVALID_ARG),
                      (tq.make_config("kv_fp16", 8, 5000), _abi.TQ_ERR_UNSUPPORTED),
                      (tq.make_config("kv_fp16", 8, 8, flags=2), _abi.TQ_ERR_INVALID_ARG),
                      (tq.make_config("kv_fp16", 8, 8, partition_tokens=64), _abi.TQ_ERR_INVALID_ARG)]:
        assert lib.tq_kv16_layout_for(ctypes.byref(cfg), ctypes.byref(lay)) == want
    # the other formats' entry points refuse the 16-bit presets
    cfg = tq.make_config("kv_bf16", 8, 8)
    other, prod, b8 = _abi.tq_layout(), _abi.tq_prod_layout(), _abi.tq_b8_layout()
    assert lib.tq_layout_for(ctypes.byref(cfg), ctypes.byref(other)) == _abi.TQ_ERR_UNSUPPORTED
    assert lib.tq_prod_layout_for(ctypes.byref(cfg), ctypes.byref(prod)) == _abi.TQ_ERR_INVALID_ARG
    assert lib.tq_b8_layout_for(ctypes.byref(cfg), ctypes.byref(b8)) == _abi.TQ_ERR_INVALID_ARG
    assert tq.tq_decode_workspace_size(cfg, 4, 64) == 0 and tq.tq_b8_decode_workspace_size(cfg, 4, 64) == 0


def test_append_refusals(tq):
    from turboquant_paged_kv_gb300 import _abi
    lib = _abi.load()
    base = tq.make_config("kv_bf16", 32, 8)

    def ap(cfg=base, key=OK, ks=0, value=OK, vs=0, q=OK, qst=0, qo=OTHER, qos=0, cs=OK, rot=128, npos=64, style=0, qs=OK,
           batch=2, total=10, cache=OK, nb=4, table=OK, stride=4, lens=OK, status=None):
        return lib.tq_kv16_append(ctypes.byref(cfg), key, ks, value, vs, q, qst, qo, qos, cs, rot, npos, style, qs, batch, total,
                                  cache, nb, table, stride, lens, status, None)

    null = dict(key=None, value=None, qs=None, cache=None, table=None, lens=None)
    for empty in (dict(batch=0), dict(total=0)):
        assert ap(**null, q=None, qo=None, **empty) == _abi.TQ_OK
    for name in null:
        assert ap(**{name: None}) == _abi.TQ_ERR_INVALID_ARG, name
    for bad in (dict(q=None), dict(qo=None), dict(cs=None), dict(rot=0), dict(rot=-16), dict(style=2), dict(npos=-1), dict(batch=-1),
                dict(total=-1), dict(nb=-1), dict(stride=0), dict(ks=1016), dict(vs=1028), dict(ks=-1024), dict(qst=8), dict(qos=4100),
                dict(qo=OK, qst=8192), dict(cfg=tq.make_config("4bit_nc", 32, 8)), dict(cfg=tq.make_config("kv_bf16", 30, 8))):
        assert ap(**bad) == _abi.TQ_ERR_INVALID_ARG, bad
    for bad in (dict(rot=24), dict(rot=144), dict(cfg=tq.make_config("kv_bf16", 32, 2)), dict(cfg=tq.make_config("kv_bf16", 32, 8, head_dim=64))):
        assert ap(**bad) == _abi.TQ_ERR_UNSUPPORTED, bad
    for bad in (dict(key=ODD), dict(value=ODD), dict(q=ODD), dict(qo=ODD), dict(cs=ODD), dict(cache=ODD), dict(qs=ODD4),
                dict(table=ODD4), dict(lens=ODD4), dict(status=ODD4)):
        assert ap(**bad) == _abi.TQ_ERR_MISALIGNED, bad


def test_decode_refusals(tq):
    from turboquant_paged_kv_gb300 import _abi
    lib = _abi.load()
    base = tq.make_config("kv_bf16", 32, 8)
    need = tq.tq_kv16_decode_workspace_size(base, 2, 64)
    assert need > 0 and need % 16 == 0
    assert tq.tq_kv16_decode_workspace_size(base, -1, 64) == 0
    assert tq.tq_kv16_decode_workspace_size(tq.make_config("kv_bf16", 30, 8), 2, 64) == 0
    assert tq.tq_kv16_decode_workspace_size(tq.make_config("kv_bf16", 32, 2), 2, 64) == 0

    def dec(cfg=base, q=OK, qst=0, cache=OK, nb=4, table=OK, stride=4, lens=OK, batch=2, max_len=64, out=OK, od=1,
            ws=OK, size=need, status=None):
        return lib.tq_kv16_decode(ctypes.byref(cfg), q, qst, cache, nb, table, stride, lens, batch, max_len, 0.0, out,
                                  od, ws, size, status, None)

    null = dict(q=None, cache=None, table=None, lens=None, out=None, ws=None)
    assert dec(**null, batch=0) == _abi.TQ_OK
    for name in null:
        assert dec(**{name: None}) == _abi.TQ_ERR_INVALID_ARG, name
    for bad in (dict(od=5), dict(batch=-1), dict(max_len=-1), dict(stride=0), dict(qst=8),
                dict(qst=4100), dict(cfg=tq.make_config("kv_bf16", 30, 8))):
        assert dec(**bad) == _abi.TQ_ERR_INVALID_ARG, bad
    assert dec(cfg=tq.make_config("kv_bf16", 32, 2)) == _abi.TQ_ERR_UNSUPPORTED      # 16 query heads per KV head
    for bad in (dict(q=ODD), dict(out=ODD), dict(ws=ODD), dict(cache=ODD), dict(lens=ODD4)):
        assert dec(**bad) == _abi.TQ_ERR_MISALIGNED, bad
    assert dec(size=need - 1) == _abi.TQ_ERR_WORKSPACE_TOO_SMALL


def test_continue_refusals(tq):
    from turboquant_paged_kv_gb300 import _abi
    lib = _abi.load()
    base = tq.make_config("kv_fp16", 24, 8)
    need = tq.tq_kv16_continue_workspace_size(base, 2, 10, 8, 64)
    assert need > 0 and need % 16 == 0

    def cont(cfg=base, q=OK, qst=0, qs=OK, batch=2, total=10, mql=8, cache=OK, nb=4, table=OK, stride=4, lens=OK,
             max_len=64, out=OK, od=1, ws=OK, size=need, status=None):
        return lib.tq_kv16_continue(ctypes.byref(cfg), q, qst, qs, batch, total, mql, cache, nb, table, stride, lens,
                                    max_len, 0.0, out, od, ws, size, status, None)

    null = dict(q=None, qs=None, cache=None, table=None, lens=None, out=None, ws=None)
    for empty in (dict(batch=0), dict(total=0), dict(mql=0)):
        assert cont(**null, **empty) == _abi.TQ_OK
    for name in null:
        assert cont(**{name: None}) == _abi.TQ_ERR_INVALID_ARG, name
    for bad in (dict(od=5), dict(batch=-1), dict(total=-1), dict(mql=-1), dict(max_len=-1), dict(stride=0),
                dict(qst=8), dict(cfg=tq.make_config("kv_fp16", 30, 8))):
        assert cont(**bad) == _abi.TQ_ERR_INVALID_ARG, bad
    assert cont(cfg=tq.make_config("kv_fp16", 32, 2)) == _abi.TQ_ERR_UNSUPPORTED
    for bad in (dict(q=ODD), dict(out=ODD), dict(ws=ODD), dict(cache=ODD), dict(qs=ODD4), dict(lens=ODD4)):
        assert cont(**bad) == _abi.TQ_ERR_MISALIGNED, bad
    assert cont(size=0) == _abi.TQ_ERR_WORKSPACE_TOO_SMALL
    assert tq.tq_kv16_continue_workspace_size(base, -1, 10, 8, 64) == 0


def test_binding_refusals(tq):
    """Wrong shapes, types, strides and devices raise before anything is launched."""
    cfg = tq.make_config("kv_bf16", 16, 4)
    bb = tq.tq_kv16_layout_for(cfg).block_bytes
    cache = torch.zeros(8 * bb, dtype=torch.uint8)
    table = torch.zeros((2, 4), dtype=torch.int32)
    lens = torch.ones(2, dtype=torch.int32)
    starts = torch.tensor([0, 1, 2], dtype=torch.int32)
    kv = torch.zeros((2, 4, 128), dtype=torch.bfloat16)
    q = torch.zeros((2, 16, 128), dtype=torch.bfloat16)
    turn = torch.zeros((9, 64))
    out = torch.zeros_like(q)
    ws = torch.zeros(16, dtype=torch.uint8)

    def ap(key=kv, value=kv, qs=starts, c=cache, t=table, ln=lens, **more):
        tq.tq_kv16_append(cfg, key, value, qs, c, t, ln, **more)

    with pytest.raises(ValueError, match="CUDA"):        # a host pointer must never reach a kernel
        ap()
    with pytest.raises(ValueError, match="CUDA"):
        ap(cos_sin=turn, q=q, q_out=q)
    with pytest.raises(ValueError, match="CUDA"):
        tq.tq_kv16_decode(cfg, q, cache, table, lens, 64, out, ws)
    for more, match in ((dict(key=kv.half()), "cache's type"), (dict(value=kv.half()), "cache's type"), (dict(key=q), "key must be"),
                        (dict(key=torch.zeros((2, 4, 256), dtype=torch.bfloat16)[..., ::2]), "contiguous"),
                        (dict(key=kv[:1].expand(2, 4, 128)), "overlap"), (dict(value=kv[:1]), "one number of rows"),
                        (dict(qs=starts[:2]), "query_start"), (dict(t=table.long()), "block_table"), (dict(t=table[:1]), "block_table"),
                        (dict(ln=lens.long()), "seq_lens"), (dict(c=cache.float()), "cache"), (dict(q=q), "together"),
                        (dict(q_out=q), "together"), (dict(q=q.half(), q_out=q), "cache's type"), (dict(q=q, q_out=q[:1]), "one number"),
                        (dict(q=q, q_out=out[:1].expand(2, 16, 128)), "overlap"), (dict(cos_sin=turn.double()), "cos_sin"),
                        (dict(cos_sin=turn[:, ::2]), "cos_sin"), (dict(cos_sin=turn[:, :0]), "cos_sin"),
                        (dict(cos_sin=turn, style="both"), "style")):
        with pytest.raises(ValueError, match=match):
            ap(**more)
    with pytest.raises(ValueError, match="out must be"):
        tq.tq_kv16_decode(cfg, q, cache, table, lens, 64, out[:1], ws)
    with pytest.raises(ValueError, match="cache's type"):
        tq.tq_kv16_decode(cfg, q.half(), cache, table, lens, 64, out, ws)
    with pytest.raises(ValueError, match="one row per sequence"):
        tq.tq_kv16_decode(cfg, q[:1], cache, table, lens, 64, out[:1], ws)
    with pytest.raises(ValueError, match="query_start"):
        tq.tq_kv16_continue(cfg, q, starts.long(), 1, cache, table, lens, 64, out, ws)


@pytest.mark.parametrize("group", [1, 3, 4, 5, 8])
def test_continue_workspace_of_the_largest_step_serves_smaller_ones(tq, group):
    """A server keeps one workspace, of its largest step, whatever shape a smaller step's units then have."""
    cfg = tq.make_config("kv_bf16", 2 * group, 2)
    size = lambda *x: tq.tq_kv16_continue_workspace_size(cfg, *x)      # noqa: E731
    steps = [(b, t, m, s) for b in (1, 7, 32, 300) for t in (1, 30, 64, 100, 300, 1000, 9000) for m in (1, 31, 60, 64, 90, 100, 130, 2000)
             for s in (0, 1, 1024, 1025, 50000)]
    for big in [(32, 9000, m, 50000) for m in (31, 64, 90, 100, 130, 2000)] + [(300, 1000, 60, 1025), (7, 100, 100, 1024)]:
        for small in steps:
            if all(x <= y for x, y in zip(small, big)):
                assert size(*small) <= size(*big), (small, big)
