"""Attention with window and first keys on the host: refusals and page checks (nothing here touches a GPU)."""
import ctypes
import math

import numpy as np
import pytest

from tests.test_attention_host import PTR, cache


@pytest.fixture(scope="module")
def m():
    from lora_serving_amd import mlora
    return mlora


def prompts(m, q=PTR, Tq=8, Tk=8, n=1, hq=4, hkv=2, d=64, window=4, sinks=2, scale=0.0, out=PTR):
    return m._lib.mlora_attention_sinks(q, hq * d, PTR, hkv * d, PTR, hkv * d, Tq, Tk, n, PTR, None, hq, hkv, d, 8, 1,
                                        window, sinks, scale, out, hq * d, None, None)


def paged(m, T=4, n=4, max_q=1, max_kv=64, window=4, sinks=2, scale=0.0, ws=None, ws_bytes=0, stride=1024, lens=PTR):
    c = cache(m)
    return m._lib.mlora_paged_attention_sinks(PTR, 256, T, 4, ctypes.byref(c), PTR, stride, n, PTR, lens, max_q, max_kv, 1,
                                              window, sinks, scale, PTR, 256, None, ws, ws_bytes, None)


def test_refusals(m):
    for call in (prompts, paged):
        assert call(m, n=0) == m.MLORA_OK
        assert call(m, sinks=-1) == m.MLORA_ERR_ARG
        assert call(m, window=-1) == m.MLORA_ERR_ARG
        assert call(m, scale=math.nan) == m.MLORA_ERR_ARG
    assert prompts(m, q=None) == m.MLORA_ERR_ARG
    assert prompts(m, hq=5) == m.MLORA_ERR_SHAPE
    assert prompts(m, Tk=9) == m.MLORA_ERR_SHAPE
    assert paged(m, lens=None) == m.MLORA_ERR_ARG
    assert paged(m, max_kv=1 << 40) == m.MLORA_ERR_UNSUPPORTED


def test_a_window_needs_less_room(m):
    """The keys behind the window are not cut: no parts where the window and the first keys are short."""
    assert paged(m, max_kv=8192, window=0) == m.MLORA_ERR_WORKSPACE
    assert paged(m, max_kv=8192, window=2000) == m.MLORA_ERR_WORKSPACE
    assert paged(m, max_kv=8192, window=100, sinks=4000) == m.MLORA_ERR_WORKSPACE


def check(m, table, cu, lens, window, sinks, pages=8):
    c = cache(m, pages=pages)
    bad = ctypes.c_int64(0)
    t, u, n = (np.ascontiguousarray(x, np.int32) for x in (table, cu, lens))
    p = lambda a: a.ctypes.data_as(ctypes.c_void_p)  # noqa: E731
    code = m._lib.mlora_validate_pages_sinks(ctypes.byref(c), p(t), t.shape[1], n.size, p(u), p(n), int(u[-1]), 64, 64,
                                             window, sinks, ctypes.byref(bad))
    return code, bad.value


def test_validate_pages(m):
    ok = (m.MLORA_OK, 0)
    # 64 keys in 4 pages, one query at 63
    assert check(m, [[0, -1, -1, 7]], [0, 1], [64], 16, 1) == ok                # keys 48 .. 63 and key 0
    assert check(m, [[0, -1, -1, 7]], [0, 1], [64], 17, 1) == (m.MLORA_ERR_INDEX, -1)   # .. and 47
    assert check(m, [[0, -1, 2, 7]], [0, 1], [64], 17, 16) == ok
    assert check(m, [[0, -1, 2, 7]], [0, 1], [64], 17, 17) == (m.MLORA_ERR_INDEX, -1)
    assert check(m, [[-1, -1, -1, 7]], [0, 1], [64], 16, 0) == ok
    assert check(m, [[-1, -1, -1, 7]], [0, 1], [64], 16, 1) == (m.MLORA_ERR_INDEX, -1)
    assert check(m, [[0, -1, -1, 7]], [0, 2], [64], 16, 1) == (m.MLORA_ERR_INDEX, -1)   # the first of two queries sees 47
    assert check(m, [[0, -1, 2, 7]], [0, 1], [64], 0, 16) == (m.MLORA_ERR_INDEX, -1)    # no window: all pages
    assert check(m, [[0, 1, 2, 9]], [0, 1], [64], 16, 1) == (m.MLORA_ERR_INDEX, 9)
    assert check(m, [[0, 1, 2, 3]], [0, 1], [64], -1, 1)[0] == m.MLORA_ERR_ARG
    assert check(m, [[0, 1, 2, 3]], [0, 1], [64], 1, -1)[0] == m.MLORA_ERR_ARG
    assert check(m, [[0, 1, 2, 3]], [0, 1], [65], 1, 1) == (m.MLORA_ERR_SHAPE, 65)


def test_validate_pages_of_a_sequence_without_queries(m):
    assert check(m, [[-1, -1], [1, 2]], [0, 0, 1], [20, 32], 4, 1) == (m.MLORA_OK, 0)
    assert check(m, [[-1, -1], [1, 2]], [0, 0, 1], [20, 32], 0, 1) == (m.MLORA_ERR_INDEX, -1)
