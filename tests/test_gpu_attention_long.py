"""Long keys on the GPU: page numbers past the 64 tiles that a wave holds at a time, keys whole and in pieces, and
prompts of more row blocks than CUs, a sample of rows against plain sums in 64 bits."""
import math

import pytest

from tests.test_gpu_attention import check, check_lse, gen, m, randn  # noqa: F401  (m: a fixture)

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


def ref_row(q, k, v, p, causal, window, scale):
    """One query [hq, d] at position p over k, v [L, hkv, d], 64 bits: out, lse, sum p |v|, largest sum |scale q k|."""
    L, hkv, d = k.shape
    hq = q.shape[0]
    lo, hi = max(0, p - window + 1) if window else 0, min(L, p + 1) if causal else L
    if hi <= lo:
        return torch.zeros_like(q), torch.full((hq,), -math.inf, dtype=q.dtype), torch.zeros_like(q), torch.zeros(hq, dtype=q.dtype)
    kk, vv = k[lo:hi].transpose(0, 1).double(), v[lo:hi].transpose(0, 1).double()       # [hkv, keys, d]
    qq = q.view(hkv, hq // hkv, d)
    s = torch.matmul(qq, kk.transpose(1, 2)) * scale                                    # [hkv, group, keys]
    big = torch.matmul(qq.abs(), kk.abs().transpose(1, 2)).amax(-1) * scale
    w = torch.softmax(s, -1)
    return (torch.matmul(w, vv).reshape(hq, d), torch.logsumexp(s, -1).reshape(hq),
            torch.matmul(w, vv.abs()).reshape(hq, d), big.reshape(hq))


def sample(n):
    return sorted({0, n // 3, n - 2, n - 1} & set(range(n)))


def check_rows(out, lse, rows):
    """rows: (row, ref_row's results)."""
    at = torch.tensor([r for r, _ in rows])
    ref, rl, mag, big = [torch.stack([x[i] for _, x in rows]) for i in range(4)]
    check(out.cpu()[at], ref, mag, big)
    check_lse(lse.cpu()[at], rl, big)


TILES = [4096, 4097, 4160, 4161, 8191, 8192, 8193, 9000]
# windows whose first tile is 63, 64 or 65 (128: at or after the second refill), for 40 queries ending at 9000
STARTS = [9000 - 40 + 1 - lo for lo in (64 * 64 - 1, 64 * 64, 65 * 64 - 1, 65 * 64, 128 * 64 - 1, 128 * 64)]

LONG_KEYS = [
    # (queries, keys) of the sequences, hq, hkv, d, page, fp8, window; which keys a workgroup takes
    ([(40, TILES[i % 8]) for i in range(24)], 8, 8, 64, 16, False, 0),              # all (192 row blocks and heads)
    ([(40, TILES[i % 8]) for i in range(24)], 8, 8, 128, 16, True, 0),
    ([(20, TILES[i % 8]) for i in range(24)] + [(1, 9000), (1, 4161)], 16, 8, 128, 64, False, 0),
    ([(40, TILES[i % 8]) for i in range(10)], 64, 2, 64, 32, True, 0),              # groups of 32: no decode rows
    ([(40, TILES[i % 8]) for i in range(22)], 8, 8, 128, 16, False, 0),             # three pieces
    ([(40, TILES[i % 8]) for i in range(22)], 8, 8, 64, 32, True, 0),
    ([(40, 9000)], 8, 2, 128, 16, False, 0),                                        # many pieces
    ([(40, 8193)], 4, 4, 64, 16, True, 0),
    ([(40, 4097)], 36, 2, 128, 32, False, 0),
] + [([(40, 9000)] * 24, 8, 8, 64 << (i & 1), 16, i % 4 > 1, w) for i, w in enumerate(STARTS)] + [
    ([(40, 9000)] * 22, 8, 8, 128, 16, False, STARTS[0]),
    ([(40, 9000)], 8, 2, 64, 16, True, STARTS[3]),
    ([(40, 9000)], 8, 2, 128, 16, False, 130),
    # more row blocks than workgroups launched for them, beside single tokens
    ([(20, TILES[i % 8]) for i in range(30)] + [(1, 9000 - 100 * i) for i in range(60)], 16, 8, 64, 16, False, 0),
    ([(20, TILES[i % 8]) for i in range(30)] + [(1, 9000 - 100 * i) for i in range(60)], 16, 8, 128, 32, True, 0),
]


@pytest.mark.parametrize("case", LONG_KEYS, ids=lambda c: f"{len(c[0])}x{c[0][0]}-" + "-".join(str(v) for v in c[1:]).replace(" ", ""))
def test_long_keys_in_pages(m, case):  # noqa: F811
    seqs, hq, hkv, d, page, fp8, window = case
    g = gen(7 * len(seqs) + seqs[0][1] + 3 * window + hq + d)
    dev = "cuda"
    pages = (9000 + page - 1) // page + 3
    shape = (pages, hkv, page, d)
    raw = [torch.randn(shape, generator=g) for _ in range(2)]
    if fp8:
        store, sc = [x.to(torch.float8_e4m3fn) for x in raw], [0.5 + torch.rand(shape[:3], generator=g) for _ in range(2)]
        value = [x.double() * s[..., None].double() for x, s in zip(store, sc)]
    else:
        store, sc = [x.to(torch.bfloat16) for x in raw], [None, None]
        value = store
    up = lambda t: None if t is None else t.to(dev)  # noqa: E731
    c = m.Cache(*[up(t) for t in store + sc])
    # the sequences share the pages, each from a start of its own
    order = torch.randperm(pages, generator=g)
    width = (max(L for _, L in seqs) + page - 1) // page
    table = torch.stack([order[(torch.arange(width) + 37 * b) % pages] for b in range(len(seqs))]).to(torch.int32)
    T = sum(n for n, _ in seqs)
    q = randn(g, T, hq, d)
    cu = torch.tensor([sum(n for n, _ in seqs[:i]) for i in range(len(seqs) + 1)], dtype=torch.int32)
    lens = torch.tensor([L for _, L in seqs], dtype=torch.int32)
    mq, mk = max(n for n, _ in seqs), max(L for _, L in seqs)
    out = torch.full((T, hq, d), 7.0, device=dev, dtype=torch.bfloat16)
    lse = torch.full((T, hq), 7.0, device=dev)
    ws = m.paged_workspace(T, len(seqs), hq, hkv, d, mq, mk)
    ws.fill_(255)
    m.mlora_paged_attention(q.to(dev), c, table.to(dev), cu.to(dev), lens.to(dev), out, mq, mk, window=window, lse=lse,
                            ws=ws)
    torch.cuda.synchronize()
    assert out.isfinite().all() and lse.isfinite().all()
    rows = []
    for b, (n, L) in enumerate(seqs):
        if b >= 8 and b % 5:
            continue
        j = torch.arange(L)
        k, v = [x[table[b, j // page].long(), :, j % page] for x in value]
        at = int(cu[b])
        for i in sample(n):
            rows.append((at + i, ref_row(q[at + i].double(), k, v, L - n + i, True, window, d ** -0.5)))
    check_rows(out, lse, rows)


MANY_BLOCKS = [
    # lens of queries, lens of keys (None: the same), hq, hkv, d, causal, window: more than 256 row blocks and heads
    ([1100], None, 32, 16, 128, True, 0),
    ([1100], None, 32, 16, 128, True, 500),
    ([1031], [1500], 32, 16, 128, False, 0),
    ([600, 1500], None, 16, 16, 128, True, 0),
    ([1100], None, 64, 16, 64, True, 0),
    ([5, 1200, 300], None, 24, 24, 64, True, 333),
]


@pytest.mark.parametrize("case", MANY_BLOCKS, ids=lambda c: "-".join(str(v) for v in c).replace(" ", ""))
def test_prompts_of_many_row_blocks(m, case):  # noqa: F811
    lq, lk, hq, hkv, d, causal, window = case
    lk = lq if lk is None else lk
    assert sum((n * (hq // hkv) + 127) // 128 for n in lq) * hkv > 256
    g = gen(sum(lq) + 5 * hq + d + window)
    dev = "cuda"
    q, k, v = randn(g, sum(lq), hq, d), randn(g, sum(lk), hkv, d), randn(g, sum(lk), hkv, d)
    cu = lambda n: torch.tensor([sum(n[:i]) for i in range(len(n) + 1)], dtype=torch.int32)  # noqa: E731
    out = torch.full((sum(lq), hq, d), 7.0, device=dev, dtype=torch.bfloat16)
    lse = torch.full((sum(lq), hq), 7.0, device=dev)
    m.mlora_attention(q.to(dev), k.to(dev), v.to(dev), cu(lq).to(dev), out, cu_k=None if lk is lq else cu(lk).to(dev),
                      max_q=max(lq), causal=causal, window=window, lse=lse)
    torch.cuda.synchronize()
    rows, a, c = [], 0, 0
    for n, L in zip(lq, lk):
        for i in sorted(set(sample(n)) | set(range(0, n, 61))):
            rows.append((a + i, ref_row(q[a + i].double(), k[c:c + L], v[c:c + L], L - n + i, causal, window, d ** -0.5)))
        a, c = a + n, c + L
    check_rows(out, lse, rows)
