"""Attention over shared prefixes on the host: refusals, sizes and the check of the groups (nothing here touches a GPU)."""
import ctypes
import math

import numpy as np
import pytest

from tests.test_attention_host import PTR, cache


@pytest.fixture(scope="module")
def m():
    from lora_serving_amd import mlora
    return mlora


def call(m, c=None, q=PTR, T=4, hq=4, table=PTR, stride=1024, n=4, cu=PTR, lens=PTR, groups=1, start=PTR, prefix=PTR, max_q=1,
         max_kv=64, max_prefix=32, scale=0.0, out=PTR, qs=256, ws=None, ws_bytes=0):
    c = cache(m) if c is None else c
    return m._lib.mlora_prefix_attention(q, qs, T, hq, ctypes.byref(c), table, stride, n, cu, lens, groups, start, prefix, max_q,
                                         max_kv, max_prefix, 1, scale, out, 256, None, ws, ws_bytes, None)


def test_refusals(m):
    assert call(m, T=0) == m.MLORA_OK
    assert call(m, n=0) == m.MLORA_OK
    assert call(m, T=-1) == m.MLORA_ERR_ARG
    assert call(m, groups=-1) == m.MLORA_ERR_ARG
    assert call(m, max_prefix=-1) == m.MLORA_ERR_ARG
    assert call(m, q=None) == m.MLORA_ERR_ARG
    assert call(m, start=None) == m.MLORA_ERR_ARG
    assert call(m, prefix=None) == m.MLORA_ERR_ARG
    assert call(m, start=None, max_prefix=0) == m.MLORA_ERR_ARG
    assert call(m, table=None) == m.MLORA_ERR_ARG
    assert call(m, out=PTR + 4) == m.MLORA_ERR_ARG
    assert call(m, hq=3) == m.MLORA_ERR_SHAPE
    assert call(m, qs=8) == m.MLORA_ERR_SHAPE
    assert call(m, max_prefix=1 << 30) == m.MLORA_ERR_UNSUPPORTED
    assert call(m, max_kv=1 << 40) == m.MLORA_ERR_UNSUPPORTED
    for scale in (-0.5, math.inf, math.nan):
        assert call(m, scale=scale) == m.MLORA_ERR_ARG
    assert call(m) == m.MLORA_ERR_WORKSPACE
    assert call(m, ws=PTR, ws_bytes=1024) == m.MLORA_ERR_WORKSPACE


def size(m, *a):
    return m._lib.mlora_prefix_workspace_size(*a)


def test_no_size_for_refused_sizes(m):
    good = [100, 20, 3, 32, 8, 128, 5, 4000, 2000]          # T, n_seqs, n_groups, heads, head_dim, max_q, max_kv, max_prefix
    assert size(m, *good) > size(m, *good[:2], 0, *good[3:]) > 0
    for i, v in ((0, -1), (0, 1 << 61), (1, -1), (1, 1 << 28), (2, -1), (3, 33), (5, 80), (6, -1), (7, 1 << 30), (7, 2 ** 63 - 1),
                 (8, -1), (8, 1 << 30), (8, 2 ** 63 - 1)):
        assert size(m, *[v if j == i else x for j, x in enumerate(good)]) == 0


@pytest.mark.parametrize("hq,hkv,d", [(32, 8, 128), (8, 8, 64), (64, 2, 64), (40, 1, 128), (1024, 1, 64), (6, 3, 128)])
def test_the_workspace_of_the_largest_batch_serves_smaller_ones(m, hq, hkv, d):
    """The size does not fall as any of the sizes rises, and holds two parts of every row at least."""
    r = np.random.default_rng(hq * 7 + hkv + d)
    log = lambda hi: int(np.exp(r.uniform(0, np.log(hi + 1))))  # noqa: E731
    for _ in range(200):
        T, n, g, mk, mp = log(20000), log(2000), log(300), log(200000), log(200000)
        mq = log(T)
        top = size(m, T, n, g, hq, hkv, d, mq, mk, mp)
        assert top >= T * hq * 2 * (d * 4 + 8)
        for _ in range(30):
            T1, n1, g1, mq1, mk1, mp1 = [min(v, log(v)) if r.random() < 0.7 else v for v in (T, n, g, mq, mk, mp)]
            assert size(m, T1, n1, g1, hq, hkv, d, mq1, mk1, mp1) <= top


def groups(m, start, prefix, lens, max_prefix=100, stride=8):
    c = cache(m)
    bad = ctypes.c_int64(0)
    s, p, n = (np.ascontiguousarray(x, np.int32) for x in (start, prefix, lens))
    ptr = lambda a: a.ctypes.data_as(ctypes.c_void_p)  # noqa: E731
    code = m._lib.mlora_validate_prefixes(ctypes.byref(c), stride, n.size, ptr(n), p.size, ptr(s), ptr(p), max_prefix,
                                          ctypes.byref(bad))
    return code, bad.value


def test_validate_prefixes(m):
    ok, shape = (m.MLORA_OK, 0), m.MLORA_ERR_SHAPE
    assert groups(m, [0, 2, 2, 3], [40, 99, 0], [50, 3, 7]) == ok           # an empty group, one of one sequence
    assert groups(m, [0, 2], [50], [50, 3, 7]) == ok                        # the last sequence in none
    assert groups(m, [0], [], [50]) == ok
    assert groups(m, [1, 2], [40], [50, 50]) == (shape, 1)
    assert groups(m, [0, 2, 1], [4, 4], [50, 50]) == (shape, 1)
    assert groups(m, [0, 3], [4], [50, 50]) == (shape, 3)
    assert groups(m, [0, 2], [-1], [50, 50]) == (shape, -1)
    assert groups(m, [0, 2], [51], [50, 90]) == (shape, 51)                 # the first sequence is shorter
    assert groups(m, [0, 2], [101], [128, 128]) == (shape, 101)             # past max_prefix
    assert groups(m, [0, 2], [99], [128, 128], stride=6) == (shape, 99)     # past the table
    assert m._lib.mlora_validate_prefixes(ctypes.byref(cache(m)), 8, 2, None, 1, PTR, PTR, 4, None) == m.MLORA_ERR_ARG
    assert m._lib.mlora_validate_prefixes(ctypes.byref(cache(m)), 1 << 31, 2, PTR, 1, PTR, PTR, 4, None) == m.MLORA_ERR_UNSUPPORTED


def test_binding_checks_shapes(m):
    c = type("C", (), {"ref": ctypes.byref(cache(m))})()
    t = np.zeros((2, 8), np.int32)
    assert m.mlora_validate_prefixes(c, t, [50, 50], [0, 2], [40], 40) == (m.MLORA_OK, 0)
    assert m.mlora_validate_prefixes(c, t, [50, 50], [0, 2], [41], 40) == (m.MLORA_ERR_SHAPE, 41)
    for bad in ((t[0], [50, 50], [0, 2], [40]), (t, [50], [0, 2], [40]), (t, [50, 50], [0, 2], [40, 3])):
        with pytest.raises(ValueError):
            m.mlora_validate_prefixes(c, *bad, 40)
