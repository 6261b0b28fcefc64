"""Sizes of the attention step's host helpers (nothing here touches a GPU)."""
import ctypes

import numpy as np
import pytest


@pytest.fixture(scope="module")
def m():
    from lora_serving_amd import mlora
    return mlora


def paged_call(m, T, n_seqs, hq, hkv, d, max_q, max_kv):
    """The paged call for these sizes with a workspace of no bytes: refused before any launch."""
    c = m.mlora_cache(0x10000, 0x10000, None, None, 8, hkv, 16, d, 0)
    return m._lib.mlora_paged_attention(0x10000, hq * d, T, hq, ctypes.byref(c), 0x10000, 1 << 26, n_seqs, 0x10000,
                                        0x10000, max_q, max_kv, 1, 0, 0.0, 0x10000, hq * d, None, None, 0, None)


# T, n_seqs, max_q, max_kv at 32 heads on 8 that the call does not take, some past 64-bit products
REFUSED = [(1 << 30, 4, 1, 64), (1 << 26, 4, 1, 64), (1 << 61, 4, 1, 64), (1 << 58, 1, 1, 64), (4, 4, 1, 1 << 30),
           (4, 4, 1, 1 << 40), (4, 4, 1, 2 ** 63 - 1), (2 ** 63 - 1, 4, 2 ** 63 - 1, 2 ** 63 - 1),
           (4, 1 << 28, 1, 64), (4, 2 ** 31 - 1, 1, 64), (4, 1 << 20, 1, (1 << 30) - 1)]


@pytest.mark.parametrize("T,n,mq,mk", REFUSED)
def test_no_workspace_size_for_refused_sizes(m, T, n, mq, mk):
    assert paged_call(m, T, n, 32, 8, 128, mq, mk) == m.MLORA_ERR_UNSUPPORTED
    assert m._lib.mlora_paged_workspace_size(T, n, 32, 8, 128, mq, mk) == 0


def test_workspace_size_at_the_limits(m):
    for T, n, mq, mk in ((4, 4, 1, (1 << 30) - 1), ((1 << 26) - 1, 1, 1, 64), (4, (1 << 27) - 1, 1, 1)):
        assert m._lib.mlora_paged_workspace_size(T, n, 32, 8, 128, mq, mk) >= 256


def test_cache_bytes_of_too_many_pages(m):
    assert m.mlora_cache_bytes((1 << 27) - 1, 8, 16, 128) == 2 * ((1 << 27) - 1) * 8 * 16 * 128 * 2
    for pages in (1 << 27, 1 << 59, 1 << 60, (1 << 60) + 1, 2 ** 63 - 1):
        assert m.mlora_cache_bytes(pages, 8, 16, 128) == -1
        assert m.mlora_cache_bytes(pages, 8, 256, 64, m.MLORA_CACHE_E4M3) == -1


def test_validate_pages_of_too_wide_tables(m):
    """A table stride that the call refuses is refused, not multiplied past 64 bits."""
    c = m.mlora_cache(0x10000, 0x10000, None, None, 8, 2, 256, 64, 0)
    table, cu, lens = np.zeros(4, np.int32), np.array([0, 1], np.int32), np.array([5], np.int32)
    p = lambda a: a.ctypes.data_as(ctypes.c_void_p)  # noqa: E731
    for stride in (1 << 31, 1 << 55, 1 << 56, 1 << 60):
        assert m._lib.mlora_validate_pages(ctypes.byref(c), p(table), stride, 1, p(cu), p(lens), 1, 1, 64,
                                           None) == m.MLORA_ERR_UNSUPPORTED
    assert m._lib.mlora_validate_pages(ctypes.byref(c), p(table), (1 << 31) - 1, 1, p(cu), p(lens), 1, 1, 64,
                                       None) == m.MLORA_OK


HEADS = [(32, 8, 128), (32, 8, 64), (8, 8, 128), (64, 2, 64), (40, 1, 128), (1024, 1, 64), (6, 3, 128), (16, 1, 64)]


@pytest.mark.parametrize("hq,hkv,d", HEADS)
def test_workspace_of_the_largest_batch_serves_smaller_ones(m, hq, hkv, d):
    """The size does not fall as any of T, n_seqs, max_q or max_kv rises."""
    size = lambda *a: m._lib.mlora_paged_workspace_size(a[0], a[1], hq, hkv, d, a[2], a[3])  # noqa: E731
    r = np.random.default_rng(hq * 7 + hkv + d)
    log = lambda hi: int(np.exp(r.uniform(0, np.log(hi + 1))))  # noqa: E731
    for _ in range(300):
        T, n, mk = log(20000), log(2000), log(200000)
        mq = log(T)
        top = size(T, n, mq, mk)
        assert top > 0
        for _ in range(40):
            low = [min(v, log(v)) if r.random() < 0.7 else v for v in (T, n, mq, mk)]
            assert size(*low) <= top, (T, n, mq, mk, low)


def test_workspace_sizes_stay_small(m):
    """A bound over all smaller batches, not a product of the largest sizes."""
    for hq, hkv, d in HEADS:
        assert m._lib.mlora_paged_workspace_size(100000, 4096, hq, hkv, d, 100000, 200000) < 192 << 20
