"""8-bit block-scaled cache on the host: layout, workspace sizes, argument checks.

No test here launches a kernel: every call runs host code only or returns an
error before reaching the GPU.
"""

import ctypes

import pytest
import torch

from oracle import block8 as o8


@pytest.fixture(scope="module")
def tq():
    from turboquant_paged_kv_gb300 import build
    build.build()
    import turboquant_paged_kv_gb300 as tq
    return tq


OK = ctypes.c_void_p(0x10000)
ODD = ctypes.c_void_p(0x10008)
ODD4 = ctypes.c_void_p(0x10002)


@pytest.mark.parametrize("fmt", ["e4m3_blk", "int8_blk"])
@pytest.mark.parametrize("bs", [16, 32, 64, 128])
@pytest.mark.parametrize("n_kv", [1, 8, 20])
def test_layout(tq, fmt, bs, n_kv):
    lay = tq.tq_b8_layout_for(tq.make_config(fmt, n_kv, n_kv, block_size=bs))
    f = o8.Block8(fmt, bs, n_kv)
    assert (lay.code_limit, lay.is_int8) == (int(f.limit), int(fmt == "int8_blk"))
    assert (lay.tile_tokens, lay.tile_bytes, lay.k_off, lay.v_off) == (16, 4096, 0, 2048)
    assert (lay.scale_off, lay.block_bytes) == (f.scale_off, f.block_bytes)


def test_layout_refusals(tq):
    from turboquant_paged_kv_gb300 import _abi
    lib, lay = _abi.load(), _abi.tq_b8_layout()
    for cfg, want in [(tq.make_config("4bit_nc", 8, 8), _abi.TQ_ERR_INVALID_ARG),
                      (tq.make_config("e4m3_blk", 8, 8, head_dim=64), _abi.TQ_ERR_UNSUPPORTED),
                      (tq.make_config("e4m3_blk", 8, 8, block_size=24), _abi.TQ_ERR_UNSUPPORTED),
                      (tq.make_config("e4m3_blk", 8, 0), _abi.TQ_ERR_INVALID_ARG),
                      (tq.make_config("e4m3_blk", 8, 5000), _abi.TQ_ERR_UNSUPPORTED),
                      (tq.make_config("e4m3_blk", 8, 8, flags=2), _abi.TQ_ERR_INVALID_ARG),
                      (tq.make_config("e4m3_blk", 8, 8, partition_tokens=64), _abi.TQ_ERR_INVALID_ARG)]:
        assert lib.tq_b8_layout_for(ctypes.byref(cfg), ctypes.byref(lay)) == want
    # the other formats' entry points refuse the 8-bit presets
    cfg = tq.make_config("int8_blk", 8, 8)
    other, prod = _abi.tq_layout(), _abi.tq_prod_layout()
    assert lib.tq_layout_for(ctypes.byref(cfg), ctypes.byref(other)) == _abi.TQ_ERR_UNSUPPORTED
    assert lib.tq_prod_layout_for(ctypes.byref(cfg), ctypes.byref(prod)) == _abi.TQ_ERR_INVALID_ARG
    assert tq.tq_decode_workspace_size(cfg, 4, 64) == 0


def test_store_refusals(tq):
    from turboquant_paged_kv_gb300 import _abi
    lib = _abi.load()
    base = tq.make_config("int8_blk", 32, 8)

    def st(cfg=base, key=OK, ks=0, value=OK, vs=0, dtype=1, qs=OK, batch=2, total=10, mql=8, cache=OK, nb=4, table=OK,
           stride=4, lens=OK, status=None):
        return lib.tq_b8_store(ctypes.byref(cfg), key, ks, value, vs, dtype, qs, batch, total, mql, cache, nb, table,
                               stride, lens, status, None)

    null = dict(key=None, value=None, qs=None, cache=None, table=None, lens=None)
    for empty in (dict(batch=0), dict(total=0), dict(mql=0)):
        assert st(**null, **empty) == _abi.TQ_OK
    for name in null:
        assert st(**{name: None}) == _abi.TQ_ERR_INVALID_ARG, name
    for bad in (dict(dtype=2), dict(batch=-1), dict(total=-1), dict(mql=-1), dict(nb=-1), dict(stride=0), dict(ks=1016),
                dict(vs=1028), dict(ks=-1024), dict(cfg=tq.make_config("4bit_nc", 32, 8))):
        assert st(**bad) == _abi.TQ_ERR_INVALID_ARG, bad
    for bad in (dict(key=ODD), dict(value=ODD), dict(cache=ODD), dict(qs=ODD4), dict(table=ODD4), dict(lens=ODD4),
                dict(status=ODD4)):
        assert st(**bad) == _abi.TQ_ERR_MISALIGNED, bad


def test_dequant_refusals(tq):
    from turboquant_paged_kv_gb300 import _abi
    lib = _abi.load()
    base = tq.make_config("e4m3_blk", 32, 8)

    def dq(cfg=base, cache=OK, nb=4, table=OK, stride=4, lens=OK, batch=2, max_len=64, k=OK, v=OK, dtype=1, status=None):
        return lib.tq_b8_dequant(ctypes.byref(cfg), cache, nb, table, stride, lens, batch, max_len, k, v, dtype, status, None)

    null = dict(cache=None, table=None, lens=None, k=None, v=None)
    assert dq(**null, batch=0) == _abi.TQ_OK and dq(**null, max_len=0) == _abi.TQ_OK
    for name in null:
        assert dq(**{name: None}) == _abi.TQ_ERR_INVALID_ARG, name
    for bad in (dict(dtype=3), dict(batch=-1), dict(max_len=-1), dict(stride=0), dict(nb=-1)):
        assert dq(**bad) == _abi.TQ_ERR_INVALID_ARG, bad
    for bad in (dict(k=ODD), dict(v=ODD), dict(cache=ODD), dict(table=ODD4), dict(lens=ODD4), dict(status=ODD4)):
        assert dq(**bad) == _abi.TQ_ERR_MISALIGNED, bad


def test_decode_refusals(tq):
    from turboquant_paged_kv_gb300 import _abi
    lib = _abi.load()
    base = tq.make_config("e4m3_blk", 32, 8)
    need = tq.tq_b8_decode_workspace_size(base, 2, 64)
    assert need == (2 * 8 + 4096) * 4 * 129 * 4
    assert tq.tq_b8_decode_workspace_size(base, -1, 64) == 0
    assert tq.tq_b8_decode_workspace_size(tq.make_config("e4m3_blk", 30, 8), 2, 64) == 0
    assert tq.tq_b8_decode_workspace_size(tq.make_config("e4m3_blk", 32, 2), 2, 64) == 0

    def dec(cfg=base, q=OK, qst=0, qd=1, cache=OK, nb=4, table=OK, stride=4, lens=OK, batch=2, max_len=64, out=OK, od=1,
            ws=OK, size=need, status=None):
        return lib.tq_b8_decode(ctypes.byref(cfg), q, qst, qd, cache, nb, table, stride, lens, batch, max_len, 0.0, out,
                                od, ws, size, status, None)

    null = dict(q=None, cache=None, table=None, lens=None, out=None, ws=None)
    assert dec(**null, batch=0) == _abi.TQ_OK
    for name in null:
        assert dec(**{name: None}) == _abi.TQ_ERR_INVALID_ARG, name
    for bad in (dict(qd=2), dict(od=5), dict(batch=-1), dict(max_len=-1), dict(stride=0), dict(qst=8),
                dict(qst=4100), dict(cfg=tq.make_config("e4m3_blk", 30, 8))):
        assert dec(**bad) == _abi.TQ_ERR_INVALID_ARG, bad
    assert dec(cfg=tq.make_config("e4m3_blk", 32, 2)) == _abi.TQ_ERR_UNSUPPORTED      # 16 query heads per KV head
    for bad in (dict(q=ODD), dict(out=ODD), dict(ws=ODD), dict(cache=ODD), dict(lens=ODD4)):
        assert dec(**bad) == _abi.TQ_ERR_MISALIGNED, bad
    assert dec(size=need - 1) == _abi.TQ_ERR_WORKSPACE_TOO_SMALL


def test_continue_refusals(tq):
    from turboquant_paged_kv_gb300 import _abi
    lib = _abi.load()
    base = tq.make_config("int8_blk", 24, 8)

    def cont(cfg=base, q=OK, qst=0, qd=1, qs=OK, batch=2, total=10, mql=8, cache=OK, nb=4, table=OK, stride=4, lens=OK,
             max_len=64, out=OK, od=1, ws=OK, size=None, status=None):
        need = tq.tq_b8_continue_workspace_size(base, 2, 10, 8, 64)
        assert need > 0
        return lib.tq_b8_continue(ctypes.byref(cfg), q, qst, qd, qs, batch, total, mql, cache, nb, table, stride, lens,
                                  max_len, 0.0, out, od, ws, need if size is None else size, status, None)

    null = dict(q=None, qs=None, cache=None, table=None, lens=None, out=None, ws=None)
    for empty in (dict(batch=0), dict(total=0), dict(mql=0)):
        assert cont(**null, **empty) == _abi.TQ_OK
    for name in null:
        assert cont(**{name: None}) == _abi.TQ_ERR_INVALID_ARG, name
    for bad in (dict(qd=2), dict(od=5), dict(batch=-1), dict(total=-1), dict(mql=-1), dict(max_len=-1), dict(stride=0),
                dict(qst=8), dict(cfg=tq.make_config("int8_blk", 30, 8))):
        assert cont(**bad) == _abi.TQ_ERR_INVALID_ARG, bad
    assert cont(cfg=tq.make_config("int8_blk", 32, 2)) == _abi.TQ_ERR_UNSUPPORTED
    for bad in (dict(q=ODD), dict(out=ODD), dict(ws=ODD), dict(cache=ODD), dict(qs=ODD4), dict(lens=ODD4)):
        assert cont(**bad) == _abi.TQ_ERR_MISALIGNED, bad
    assert cont(size=0) == _abi.TQ_ERR_WORKSPACE_TOO_SMALL
    # one chunk over a long history is split over CTAs: records of d + 1 floats a query head and part
    split = tq.tq_b8_continue_workspace_size(base, 1, 10, 10, 4096)
    assert split % 16 == 0 and split // (10 * 24 * 129 * 4) >= 2
    assert cont(batch=1, mql=10, max_len=4096, size=split - 16) == _abi.TQ_ERR_WORKSPACE_TOO_SMALL
    assert tq.tq_b8_continue_workspace_size(base, -1, 10, 8, 64) == 0


def test_binding_refusals(tq):
    """Wrong shapes, types, strides and devices raise before anything is launched."""
    cfg = tq.make_config("int8_blk", 16, 4)
    bb = tq.tq_b8_layout_for(cfg).block_bytes
    cache = torch.zeros(8 * bb, dtype=torch.uint8)
    table = torch.zeros((2, 4), dtype=torch.int32)
    lens = torch.ones(2, dtype=torch.int32)
    starts = torch.tensor([0, 1, 2], dtype=torch.int32)
    kv = torch.zeros((2, 4, 128), dtype=torch.bfloat16)
    q = torch.zeros((2, 16, 128), dtype=torch.bfloat16)
    out = torch.zeros_like(q)
    ws = torch.zeros(16, dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA"):        # a host pointer must never reach a kernel
        tq.tq_b8_store(cfg, kv, kv, starts, 1, cache, table, lens)
    with pytest.raises(ValueError, match="CUDA"):
        tq.tq_b8_decode(cfg, q, cache, table, lens, 64, out, ws)
    with pytest.raises(ValueError, match="key must be"):
        tq.tq_b8_store(cfg, kv.float(), kv, starts, 1, cache, table, lens)
    with pytest.raises(ValueError, match="key must be"):
        tq.tq_b8_store(cfg, q, kv, starts, 1, cache, table, lens)
    with pytest.raises(ValueError, match="contiguous"):
        tq.tq_b8_store(cfg, torch.zeros((2, 4, 256), dtype=torch.bfloat16)[..., ::2], kv, starts, 1, cache, table, lens)
    with pytest.raises(ValueError, match="overlap"):     # one row for all of them
        tq.tq_b8_store(cfg, kv[:1].expand(2, 4, 128), kv, starts, 1, cache, table, lens)
    with pytest.raises(ValueError, match="overlap"):
        tq.tq_b8_decode(cfg, q[:1].expand(2, 16, 128), cache, table, lens, 64, out, ws)
    with pytest.raises(ValueError, match="one dtype"):
        tq.tq_b8_store(cfg, kv.half(), kv, starts, 1, cache, table, lens)
    with pytest.raises(ValueError, match="query_start"):
        tq.tq_b8_store(cfg, kv, kv, starts[:2], 1, cache, table, lens)
    with pytest.raises(ValueError, match="block_table"):
        tq.tq_b8_store(cfg, kv, kv, starts, 1, cache, table.long(), lens)
    with pytest.raises(ValueError, match="block_table"):
        tq.tq_b8_store(cfg, kv, kv, starts, 1, cache, table[:1], lens)
    with pytest.raises(ValueError, match="seq_lens"):
        tq.tq_b8_store(cfg, kv, kv, starts, 1, cache, table, lens.long())
    with pytest.raises(ValueError, match="cache"):
        tq.tq_b8_store(cfg, kv, kv, starts, 1, cache.float(), table, lens)
    with pytest.raises(ValueError, match="out must be"):
        tq.tq_b8_decode(cfg, q, cache, table, lens, 64, out[:1], ws)
    with pytest.raises(ValueError, match="one row per sequence"):
        tq.tq_b8_decode(cfg, q[:1], cache, table, lens, 64, out[:1], ws)
    with pytest.raises(ValueError, match="same dtype"):
        tq.tq_b8_dequant(cfg, cache, table, lens, 8, torch.zeros((2, 8, 4, 128)), torch.zeros((2, 8, 4, 128)).half())
    with pytest.raises(ValueError, match="key_out"):
        tq.tq_b8_dequant(cfg, cache, table, lens, 8, torch.zeros((2, 9, 4, 128)), torch.zeros((2, 8, 4, 128)))
    with pytest.raises(ValueError, match="query_start"):
        tq.tq_b8_continue(cfg, q, starts.long(), 1, cache, table, lens, 64, out, ws)
