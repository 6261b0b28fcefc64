"""The attention step's entry points on the host: refusals, page checks and the rotation's table
(nothing here touches a GPU: every refused call returns before any HIP call)."""
import ctypes
import decimal
import math

import numpy as np
import pytest

PTR = 0x10000    # a 16-byte aligned address that no refused call reads


@pytest.fixture(scope="module")
def m():
    from lora_serving_amd import mlora
    return mlora


def cache(m, k=PTR, v=PTR, ks=None, vs=None, pages=8, heads=2, page=16, d=64, dtype=0):
    return m.mlora_cache(k, v, ks, vs, pages, heads, page, d, dtype)


def rope(m, rot=64, turns=PTR, inter=0):
    return m.mlora_rope(turns, rot, inter, 1.0)


def call_rope(m, c=None, slot=None, T=4, stride=512, hq=4, hkv=2, d=64, r=None, qkv=PTR, pos=PTR, q=PTR,
              q_stride=256, k=None, k_stride=0, qw=None, kw=None, eps=1e-6):
    r = rope(m) if r is None else r
    return m._lib.mlora_qk_rope(qkv, T, stride, hq, hkv, d, pos, ctypes.byref(r), qw, kw, eps, q, q_stride, k,
                                k_stride, None if c is None else ctypes.byref(c), slot, None)


def test_qk_rope_refusals(m):
    assert call_rope(m, T=0) == m.MLORA_OK
    assert call_rope(m, T=-1) == m.MLORA_ERR_ARG
    assert call_rope(m, qkv=None) == m.MLORA_ERR_ARG
    assert call_rope(m, q=PTR + 8) == m.MLORA_ERR_ARG
    assert call_rope(m, pos=None) == m.MLORA_ERR_ARG
    assert call_rope(m, qw=PTR + 2) == m.MLORA_ERR_ARG
    assert call_rope(m, hq=0) == m.MLORA_ERR_ARG
    assert call_rope(m, hq=3, hkv=2) == m.MLORA_ERR_SHAPE
    assert call_rope(m, d=96) == m.MLORA_ERR_UNSUPPORTED
    assert call_rope(m, hq=2048, hkv=2) == m.MLORA_ERR_UNSUPPORTED
    assert call_rope(m, stride=504) == m.MLORA_ERR_SHAPE
    assert call_rope(m, stride=516) == m.MLORA_ERR_SHAPE
    assert call_rope(m, q_stride=128) == m.MLORA_ERR_SHAPE
    assert call_rope(m, k=PTR, k_stride=64) == m.MLORA_ERR_SHAPE
    assert call_rope(m, r=rope(m, rot=80)) == m.MLORA_ERR_SHAPE
    assert call_rope(m, r=rope(m, rot=24)) == m.MLORA_ERR_SHAPE
    assert call_rope(m, r=rope(m, turns=None)) == m.MLORA_ERR_ARG
    assert call_rope(m, eps=-1.0) == m.MLORA_ERR_ARG
    assert call_rope(m, eps=math.nan) == m.MLORA_ERR_ARG
    assert call_rope(m, c=cache(m)) == m.MLORA_ERR_ARG                       # a cache without slots
    assert call_rope(m, slot=PTR) == m.MLORA_ERR_ARG                         # slots without a cache
    assert call_rope(m, c=cache(m, heads=4), slot=PTR) == m.MLORA_ERR_SHAPE
    assert call_rope(m, c=cache(m, d=128), slot=PTR) == m.MLORA_ERR_SHAPE
    assert call_rope(m, c=cache(m, page=24), slot=PTR) == m.MLORA_ERR_UNSUPPORTED
    assert call_rope(m, c=cache(m, page=8), slot=PTR) == m.MLORA_ERR_UNSUPPORTED
    assert call_rope(m, c=cache(m, page=512), slot=PTR) == m.MLORA_ERR_UNSUPPORTED
    assert call_rope(m, c=cache(m, dtype=2), slot=PTR) == m.MLORA_ERR_UNSUPPORTED
    assert call_rope(m, c=cache(m, dtype=1), slot=PTR) == m.MLORA_ERR_ARG    # no scales
    assert call_rope(m, c=cache(m, pages=0), slot=PTR) == m.MLORA_ERR_ARG
    assert call_rope(m, c=cache(m, v=None), slot=PTR) == m.MLORA_ERR_ARG


def test_cache_read_refusals(m):
    read = lambda c, slot=PTR, T=4, k=PTR, v=PTR: m._lib.mlora_cache_read(  # noqa: E731
        None if c is None else ctypes.byref(c), slot, T, k, v, None)
    assert read(cache(m), T=0) == m.MLORA_OK
    assert read(cache(m), k=None, v=None) == m.MLORA_OK
    assert read(None) == m.MLORA_ERR_ARG
    assert read(cache(m), T=-1) == m.MLORA_ERR_ARG
    assert read(cache(m), slot=None) == m.MLORA_ERR_ARG
    assert read(cache(m), k=PTR + 2) == m.MLORA_ERR_ARG
    assert read(cache(m, page=48)) == m.MLORA_ERR_UNSUPPORTED
    assert read(cache(m, pages=1 << 27)) == m.MLORA_ERR_UNSUPPORTED


def call_attention(m, q=PTR, k=PTR, v=PTR, out=PTR, Tq=8, Tk=8, n=1, cu=PTR, cu_k=None, hq=4, hkv=2, d=64, max_q=8,
                   window=0, scale=0.0, qs=256, ks=128, vs=128, os=256):
    return m._lib.mlora_attention(q, qs, k, ks, v, vs, Tq, Tk, n, cu, cu_k, hq, hkv, d, max_q, 1, window, scale, out,
                                  os, None, None)


def test_attention_refusals(m):
    assert call_attention(m, Tq=0, Tk=0) == m.MLORA_OK
    assert call_attention(m, n=0) == m.MLORA_OK
    assert call_attention(m, Tq=-1) == m.MLORA_ERR_ARG
    assert call_attention(m, window=-1) == m.MLORA_ERR_ARG
    assert call_attention(m, scale=math.nan) == m.MLORA_ERR_ARG
    assert call_attention(m, q=None) == m.MLORA_ERR_ARG
    assert call_attention(m, v=None) == m.MLORA_ERR_ARG
    assert call_attention(m, out=PTR + 2) == m.MLORA_ERR_ARG
    assert call_attention(m, cu=None) == m.MLORA_ERR_ARG
    assert call_attention(m, Tk=9) == m.MLORA_ERR_SHAPE                  # one table for two lengths
    assert call_attention(m, qs=248) == m.MLORA_ERR_SHAPE
    assert call_attention(m, ks=132) == m.MLORA_ERR_SHAPE
    assert call_attention(m, hq=5) == m.MLORA_ERR_SHAPE
    assert call_attention(m, d=80) == m.MLORA_ERR_UNSUPPORTED
    assert call_attention(m, Tq=1 << 30, Tk=1 << 30) == m.MLORA_ERR_UNSUPPORTED
    assert call_attention(m, Tk=1 << 30, cu_k=PTR) == m.MLORA_ERR_UNSUPPORTED        # positions within 32 bits
    assert call_attention(m, ks=1 << 24) == m.MLORA_ERR_UNSUPPORTED                  # offsets within a tile too
    assert call_attention(m, vs=1 << 24) == m.MLORA_ERR_UNSUPPORTED
    for scale in (-0.5, math.inf, -math.inf):                                        # the largest score leads
        assert call_attention(m, scale=scale) == m.MLORA_ERR_ARG


def call_paged(m, c=None, q=PTR, T=4, hq=4, table=PTR, stride=4, n=4, cu=PTR, lens=PTR, max_q=1, max_kv=64, window=0,
               scale=0.0, out=PTR, qs=256, os=256, ws=None, ws_bytes=0):
    c = cache(m) if c is None else c
    return m._lib.mlora_paged_attention(q, qs, T, hq, ctypes.byref(c), table, stride, n, cu, lens, max_q, max_kv, 1,
                                        window, scale, out, os, None, ws, ws_bytes, None)


def test_paged_refusals(m):
    assert call_paged(m, T=0) == m.MLORA_OK
    assert call_paged(m, n=0) == m.MLORA_OK
    assert call_paged(m, T=-1) == m.MLORA_ERR_ARG
    assert call_paged(m, max_kv=-1) == m.MLORA_ERR_ARG
    assert call_paged(m, window=-2) == m.MLORA_ERR_ARG
    assert call_paged(m, q=None) == m.MLORA_ERR_ARG
    assert call_paged(m, table=None) == m.MLORA_ERR_ARG
    assert call_paged(m, lens=None) == m.MLORA_ERR_ARG
    assert call_paged(m, out=PTR + 4) == m.MLORA_ERR_ARG
    assert call_paged(m, hq=3) == m.MLORA_ERR_SHAPE
    assert call_paged(m, qs=8) == m.MLORA_ERR_SHAPE
    assert call_paged(m, max_kv=1 << 40) == m.MLORA_ERR_UNSUPPORTED
    assert call_paged(m, c=cache(m, dtype=1, ks=PTR)) == m.MLORA_ERR_ARG
    for scale in (-0.5, math.inf, math.nan):
        assert call_paged(m, scale=scale) == m.MLORA_ERR_ARG
    assert call_paged(m, n=1 << 20, max_kv=(1 << 30) - 1) == m.MLORA_ERR_UNSUPPORTED   # units of all heads: 32 bits
    # a long batch is split over keys and needs room for the parts
    need = m._lib.mlora_paged_workspace_size(4, 4, 4, 2, 64, 1, 8192)
    assert need > 4 * 4 * 64 * 4
    assert call_paged(m, stride=512, max_kv=8192) == m.MLORA_ERR_WORKSPACE
    assert call_paged(m, stride=512, max_kv=8192, ws=PTR, ws_bytes=1024) == m.MLORA_ERR_WORKSPACE
    assert m._lib.mlora_paged_workspace_size(4, 4, 3, 2, 64, 1, 64) == 0
    assert m._lib.mlora_paged_workspace_size(-4, 4, 4, 2, 64, 1, 64) == 0


def check_pages(m, table, cu, lens, T, max_q=8, max_kv=64, pages=8):
    c = cache(m, pages=pages)
    bad = ctypes.c_int64(0)
    t = np.ascontiguousarray(table, np.int32)
    u, n = np.ascontiguousarray(cu, np.int32), np.ascontiguousarray(lens, np.int32)
    p = lambda a: a.ctypes.data_as(ctypes.c_void_p)  # noqa: E731
    code = m._lib.mlora_validate_pages(ctypes.byref(c), p(t), t.shape[1], n.size, p(u), p(n), T, max_q, max_kv,
                                       ctypes.byref(bad))
    return code, bad.value


def test_validate_pages(m):
    good = [[0, 7, -1, -1], [3, -5, 99, 0]]
    assert check_pages(m, good, [0, 2, 3], [32, 16], 3) == (m.MLORA_OK, 0)          # unreached entries are free
    assert check_pages(m, good, [0, 2, 3], [33, 16], 3) == (m.MLORA_ERR_INDEX, -1)
    assert check_pages(m, good, [0, 2, 3], [32, 17], 3) == (m.MLORA_ERR_INDEX, -5)
    assert check_pages(m, [[0, 8]], [0, 1], [17], 1) == (m.MLORA_ERR_INDEX, 8)
    assert check_pages(m, good, [0, 2, 3], [65, 16], 3) == (m.MLORA_ERR_SHAPE, 65)
    assert check_pages(m, good, [0, 2, 3], [32, -1], 3) == (m.MLORA_ERR_SHAPE, -1)
    assert check_pages(m, good, [0, 2, 1], [32, 16], 3) == (m.MLORA_ERR_SHAPE, -1)
    assert check_pages(m, good, [0, 9, 10], [32, 16], 10) == (m.MLORA_ERR_SHAPE, 9)
    assert check_pages(m, good, [0, 2, 3], [32, 16], 4) == (m.MLORA_ERR_SHAPE, 3)
    assert check_pages(m, good, [1, 2, 3], [32, 16], 3) == (m.MLORA_ERR_SHAPE, 1)


def test_cache_bytes(m):
    assert m.mlora_cache_bytes(10, 8, 16, 128) == 2 * 10 * 8 * 16 * 128 * 2
    assert m.mlora_cache_bytes(10, 8, 16, 128, m.MLORA_CACHE_E4M3) == 2 * 10 * 8 * 16 * (128 + 4)
    assert m.mlora_cache_bytes(10, 8, 24, 128) == -1
    assert m.mlora_cache_bytes(10, 8, 16, 100) == -1


@pytest.mark.parametrize("rot,base", [(16, 10000.0), (64, 500000.0), (128, 1e6)])
def test_rope_turns(m, rot, base):
    plain = m.mlora_rope_turns(rot, base).numpy().view(np.uint64)
    decimal.getcontext().prec = 50
    pi = decimal.Decimal("3.1415926535897932384626433832795028841971693993751")
    for i in range(rot // 2):
        f = decimal.Decimal(base) ** (decimal.Decimal(-2 * i) / rot) / (2 * pi) * 2 ** 64
        # half a unit of the fixed point, and a 64-bit significand's power and quotient (a few 2^-64, relative)
        assert abs(int(plain[i]) - f) <= decimal.Decimal(0.5) + f * decimal.Decimal(2.0 ** -61)
    slow = m.mlora_rope_turns(rot, base, m.MLORA_ROPE_LINEAR, factor=8.0).numpy().view(np.uint64)
    assert all(abs(int(s) * 8 - int(p)) <= 8 for s, p in zip(slow, plain))
    parts = m.mlora_rope_turns(rot, base, m.MLORA_ROPE_PARTS, factor=8.0, orig_len=4096, fast=32.0,
                               slow=1.0).numpy().view(np.uint64)
    for p, q in zip(plain, parts):
        turns = int(p) / 2.0 ** 64 * 4096
        if turns >= 32:
            assert q == p
        elif turns <= 1:
            assert abs(int(q) * 8 - int(p)) <= 8
        else:
            assert int(p) // 8 <= int(q) <= int(p)


def test_rope_turns_refusals(m):
    for bad in (dict(rot_dim=0), dict(rot_dim=7), dict(rot_dim=16, base=1.0), dict(rot_dim=16, base=math.inf),
                dict(rot_dim=16, scaling=3), dict(rot_dim=16, scaling=1, factor=0.5),
                dict(rot_dim=16, scaling=2, factor=2.0, orig_len=0),
                dict(rot_dim=16, scaling=2, factor=2.0, orig_len=64, fast=1.0, slow=1.0)):
        with pytest.raises(m.MloraError) as e:
            m.mlora_rope_turns(**bad)
        assert e.value.code == m.MLORA_ERR_ARG


def test_binding_refuses_host_tensors(m):
    import torch
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        m.Cache(torch.zeros(2, 2, 16, 64, dtype=torch.bfloat16), torch.zeros(2, 2, 16, 64, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        m.Rope(torch.zeros(32, dtype=torch.int64), 64)
    with pytest.raises(ValueError):
        m.mlora_attention(x, x, x, i, x)
