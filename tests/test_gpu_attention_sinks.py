"""Attention with a sliding window and a few first keys that stay visible (sinks), over packed prompts and over
pages, against a plain implementation in 64 bits on the CPU.  Tolerances as in test_gpu_attention: a probability and
a result are each rounded to bf16 (2^-8 of the value at most), the rest is fp32.
"""
import math
import random

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

from tests.test_gpu_attention import BF, check, check_lse, gen, paged_batch, randn  # noqa: E402


@pytest.fixture(scope="module")
def m():
    from lora_serving_amd import mlora
    return mlora


def seen_keys(p, L, causal, window, sinks):
    """The keys that a query at position p sees."""
    hi = min(L, p + 1) if causal else L
    lo = max(0, p - window + 1) if window else 0
    first = list(range(min(sinks, lo, max(hi, 0)))) if window else []
    return first + list(range(lo, hi))


def reference(q, k, v, causal, window, sinks, scale):
    """q [n, hq, d], k, v [L, hkv, d] fp64 -> out, lse, sum p |v|, largest sum of |scale q k|."""
    n, hq, _ = q.shape
    L, hkv = k.shape[:2]
    out, mag = torch.zeros_like(q), torch.zeros_like(q)
    lse = torch.full((n, hq), -math.inf, dtype=torch.float64)
    big = torch.zeros(n, hq, dtype=torch.float64)
    for i in range(n):
        keys = seen_keys(L - n + i, L, causal, window, sinks)
        if not keys:
            continue
        kk = k[keys].repeat_interleave(hq // hkv, 1)
        vv = v[keys].repeat_interleave(hq // hkv, 1)
        s = (kk * q[i]).sum(-1) * scale
        big[i] = ((kk * q[i]).abs().sum(-1) * scale).amax(0)
        lse[i] = torch.logsumexp(s, 0)
        w = torch.exp(s - lse[i])
        out[i] = (w[..., None] * vv).sum(0)
        mag[i] = (w[..., None] * vv.abs()).sum(0)
    return out, lse, mag, big


PROMPTS = [
    # lens of queries, lens of keys (None: the same), hq, hkv, d, causal, window, sinks
    ([1], None, 1, 1, 64, True, 1, 1),
    ([1, 0, 2, 63, 64, 65, 200], None, 4, 2, 64, True, 7, 4),
    ([127, 129, 5], None, 4, 1, 128, True, 32, 1),
    ([400], None, 6, 2, 128, True, 64, 64),                  # tiles at the border
    ([400], None, 6, 2, 128, True, 65, 65),
    ([390, 31], None, 14, 2, 64, True, 17, 200),             # more first keys than a tile
    ([350], None, 8, 8, 128, True, 100, 1),
    ([190, 40], [400, 300], 2, 1, 64, False, 33, 5),         # not causal: the window's lower end alone
    ([5, 100, 70], [0, 160, 30], 4, 2, 128, True, 12, 3),    # no keys, more keys, fewer keys than queries
    ([70, 9], [600, 64], 4, 4, 128, True, 1, 2),
    ([257], None, 16, 1, 128, True, 100, 2 ** 31 - 1),       # every key is a first one
    ([300], None, 2, 1, 128, True, 2 ** 31 - 1, 4),          # nothing is hidden
    ([300], None, 2, 1, 128, True, 0, 4),
    ([900], None, 2, 1, 128, True, 300, 20),                 # tiles seen in full between two edges
    ([700], None, 1, 1, 64, True, 513, 70),                  # the tiles in two halves of a workgroup, not alike
    ([130], [900], 3, 1, 128, False, 700, 130),
    ([4] * 70 + [250], None, 2, 1, 64, True, 3, 2),          # more than 64 sequences
]


def run_prompts(m, lq, lk, hq, hkv, d, causal, window, sinks, poison=False):
    lk = lq if lk is None else lk
    g = gen(sum(lq) + 7 * hq + d + sinks % 1000)
    Tq, Tk = sum(lq), sum(lk)
    q, kv = randn(g, Tq, hq, d), randn(g, Tk, 2 * hkv, d)
    cu = lambda n: torch.tensor([sum(n[:i]) for i in range(len(n) + 1)], dtype=torch.int32, device="cuda")  # noqa: E731
    dkv = kv.cuda()
    out = torch.full((Tq, hq, d), 7.0, device="cuda", dtype=torch.bfloat16)
    lse = torch.full((Tq, hq), 7.0, device="cuda")
    m.mlora_attention(q.cuda(), dkv[:, :hkv], dkv[:, hkv:], cu(lq), out, cu_k=cu(lk), max_q=max(lq), causal=causal,
                      window=window, sinks=sinks, scale=0.17, lse=lse)
    torch.cuda.synchronize()
    a = c = 0
    for n, L in zip(lq, lk):
        if n:
            ref, rl, mag, big = reference(q[a:a + n].double(), kv[c:c + L, :hkv].double(), kv[c:c + L, hkv:].double(),
                                          causal, window, sinks, 0.17)
            check(out[a:a + n], ref, mag, big)
            check_lse(lse[a:a + n], rl, big)
        a, c = a + n, c + L


@pytest.mark.parametrize("case", PROMPTS, ids=lambda c: "-".join(str(v) for v in c).replace(" ", "")[-60:])
def test_prompts(m, case):
    run_prompts(m, *case)


@pytest.mark.parametrize("seed", range(24))
def test_random_prompts(m, seed):
    r = random.Random(seed)
    hkv = r.choice([1, 2, 3])
    lens = [r.choice([0, 1, 64, 65, r.randint(1, 500)]) for _ in range(r.randint(1, 3))] + [r.randint(1, 300)]
    keys = None if r.random() < 0.5 else [max(0, n + r.randint(-40, 700)) for n in lens]
    run_prompts(m, lens, keys, hkv * r.choice([1, 2, 5]), hkv, r.choice([64, 128]), r.random() < 0.8,
                r.choice([1, 2, 31, 32, 64, 100, r.randint(1, 400)]), r.choice([1, 4, 32, 63, 64, 65, 128, r.randint(1, 300)]))


PAGED = [
    # (queries, keys) of the sequences, hq, hkv, d, page, fp8, causal, window, sinks
    ([(1, 1)], 1, 1, 64, 16, False, True, 1, 1),
    ([(1, 1), (1, 0), (1, 17), (1, 333), (0, 5), (1, 32)], 4, 2, 128, 16, False, True, 20, 4),
    ([(1, 1000), (1, 31), (1, 512)], 8, 1, 64, 32, True, True, 100, 4),
    ([(1, 700), (1, 129), (1, 64)], 4, 4, 128, 64, True, True, 50, 33),
    ([(1, 600), (1, 4)], 6, 2, 64, 16, False, True, 100, 130),                  # more than a unit of 128
    ([(1, 700)], 2, 2, 64, 16, False, True, 250, 400),                          # first keys and unit of the window overlap
    ([(1, 384 + 96)], 2, 1, 128, 16, False, True, 384, 4),                      # the window starts inside the first unit
    ([(1, 1029)], 2, 1, 128, 16, False, True, 1000, 4),                         # .. and in its first block
    ([(1, 513)], 2, 1, 128, 16, True, True, 384, 128),                          # touching: 128 keys, then the window
    ([(1, 560)], 2, 1, 128, 16, True, True, 400, 140),                          # past the window's unit, a gap after it
    ([(4, 300), (3, 3), (4, 2), (1, 77)], 8, 2, 128, 16, False, True, 10, 3),   # 16 rows; fewer keys than queries
    ([(5, 200), (2, 900)], 12, 2, 128, 32, True, True, 60, 20),                 # 30 rows
    ([(8, 140), (8, 8)], 4, 1, 64, 256, False, True, 9, 1),
    ([(5, 500)], 4, 1, 64, 16, False, False, 40, 7),
    ([(1, 500), (40, 300), (1, 20), (130, 930)], 4, 2, 128, 16, False, True, 70, 4),      # decode rows and chunks
    ([(33, 900), (1, 100), (70, 70)], 8, 2, 128, 32, True, True, 128, 64),
    ([(100, 613), (1, 64)], 3, 1, 64, 16, False, True, 75, 90),
    ([(64, 1257), (5, 0)], 40, 2, 64, 64, True, True, 300, 5),
    ([(1, 9000)], 8, 2, 128, 16, False, True, 2000, 4),                         # split over keys
    ([(1, 9000), (1, 40), (1, 7000)], 8, 2, 128, 16, True, True, 1500, 900),    # the first keys split too
    ([(20, 6000)], 8, 4, 128, 16, False, True, 2500, 16),                       # a chunk's tiles in pieces
    ([(50, 5500)], 4, 1, 64, 32, True, True, 3000, 300),
    ([(140, 4000), (1, 2500), (1, 3)], 6, 2, 128, 32, True, True, 900, 64),
    ([(129, 3000)], 2, 2, 64, 64, True, False, 500, 8),
    ([(1, 61 + 61 * i % 1500) for i in range(70)], 2, 1, 64, 16, False, True, 200, 6),   # more than 64 sequences
    ([(1, 1 + i % 50) for i in range(300)] + [(5, 5 + i % 60) for i in range(100)], 64, 16, 64, 16, False, True, 9, 2),
    ([(1, 2000)] * 3, 48, 1, 64, 16, False, True, 300, 4),                      # a group of 48
    ([(1, 300), (2, 90)], 4, 2, 128, 16, False, True, 2 ** 31 - 1, 4),          # nothing is hidden
    ([(1, 700), (40, 90)], 4, 2, 128, 16, True, True, 30, 2 ** 31 - 1),         # every key is a first one
    ([(1, 800), (1, 90)], 24, 1, 128, 16, False, True, 130, 4),                 # single tokens of 24 rows
    ([(1, 700), (4, 333), (60, 900), (1, 9)], 4, 2, 128, 16, False, True, 50, 0),         # a window alone, its past given up
    ([(1, 3000), (1, 2100)], 4, 2, 64, 16, True, True, 1500, 0),
    ([(70, 1900)], 8, 2, 128, 16, True, False, 300, 0),
]


def run_paged(m, seqs, hq, hkv, d, page, fp8, causal, window, sinks, given_up):
    g = gen(sum(L for _, L in seqs) + 13 * hq + d + sinks % 1000)
    c, table, vals = paged_batch(m, g, seqs, hkv, d, page, fp8, given_up)
    if given_up:        # what no query sees holds NaN, and pages of such tokens alone are named no more
        for b, (n, L) in enumerate(seqs):
            seen = set()
            for i in (range(n) if n < 40 else (0, n - 1)):
                seen.update(seen_keys(L - n + i, L, causal, window, sinks))
            if n >= 40:
                lo = max(0, L - n - window + 1) if window else 0
                seen.update(range(lo, L))
            gone = [j for j in range(L) if j not in seen]
            if gone:
                j = torch.tensor(gone)
                pg = table[b, j // page].long().cuda()
                off = (j % page).cuda()
                for t in (c.k, c.v):
                    if fp8:
                        t.view(torch.uint8)[pg, :, off] = 0x7f
                    else:
                        t[pg, :, off] = math.nan
                if fp8:
                    c.k_scale[pg, :, off] = math.nan
                    c.v_scale[pg, :, off] = math.inf
            for p in range((L + page - 1) // page):
                if not seen & set(range(p * page, min(L, p * page + page))):
                    table[b, p] = random.Random(p).choice([-1, 2 ** 31 - 1, -2 ** 31, c.n_pages])
    T = sum(n for n, _ in seqs)
    q = randn(g, T, hq, d)
    cu = torch.tensor([sum(n for n, _ in seqs[:i]) for i in range(len(seqs) + 1)], dtype=torch.int32)
    lens = torch.tensor([L for _, L in seqs], dtype=torch.int32)
    mq, mk = max(n for n, _ in seqs), max(L for _, L in seqs)
    assert m.mlora_validate_pages(c, table, cu, lens, T, mq, mk, window, sinks) == (m.MLORA_OK, 0)
    out = torch.full((T, hq, d), 7.0, device="cuda", dtype=torch.bfloat16)
    lse = torch.full((T, hq), 7.0, device="cuda")
    ws = m.paged_workspace(T, len(seqs), hq, hkv, d, mq, mk)
    ws.fill_(255)                                      # NaN in every word
    m.mlora_paged_attention(q.cuda(), c, table.cuda(), cu.cuda(), lens.cuda(), out, mq, mk, causal=causal,
                            window=window, sinks=sinks, lse=lse, ws=ws)
    torch.cuda.synchronize()
    at = 0
    for (n, L), (k, v) in zip(seqs, vals):
        if n:
            ref, rl, mag, big = reference(q[at:at + n].double(), k, v, causal, window, sinks, d ** -0.5)
            check(out[at:at + n], ref, mag, big)
            check_lse(lse[at:at + n], rl, big)
        at += n


@pytest.mark.parametrize("given_up", [False, True], ids=["", "given_up"])
@pytest.mark.parametrize("case", PAGED, ids=lambda c: "-".join(str(v) for v in c).replace(" ", "")[-60:])
def test_paged(m, case, given_up):
    run_paged(m, *case, given_up)


@pytest.mark.parametrize("seed", range(40))
def test_random_paged(m, seed):
    r = random.Random(1000 + seed)
    hkv = r.choice([1, 2, 3])
    group = r.choice([1, 2, 4, 7])
    seqs = []
    for _ in range(r.randint(1, 6)):
        n = r.choice([0, 1, 1, 1, 1, 2, 5, r.randint(1, 60)])
        seqs.append((n, max(0, n + r.choice([-2, 0, 30, 31, 97, r.randint(0, 900), r.randint(0, 2500)]))))
    seqs.append((1, r.randint(1, 2500)))
    run_paged(m, seqs, hkv * group, hkv, r.choice([64, 128]), r.choice([16, 64, 256]), r.random() < 0.5, r.random() < 0.85,
              r.choice([1, 31, 32, 33, 96, 128, 300, r.randint(1, 1500)]),
              r.choice([1, 4, 31, 32, 33, 96, 127, 128, 129, r.randint(1, 700)]), r.random() < 0.5)


FEW = [
    # (queries, keys) of the sequences, hq, hkv, d, page, fp8, window, sinks
    ([(1, 2), (1, 1), (1, 37), (1, 300), (1, 64)], 4, 2, 128, 16, False, 20, 3),
    ([(1, 5), (1, 41), (1, 150), (1, 2000)], 8, 1, 64, 32, True, 70, 40),
    ([(3, 60), (4, 130), (1, 20)], 8, 2, 64, 16, False, 9, 1),
    ([(1, 140), (1, 8), (1, 900)], 16, 1, 128, 16, True, 100, 4),
    ([(1, 70), (1, 300), (40, 900), (2, 33)], 4, 2, 128, 16, False, 50, 2),        # beside a chunk
]


@pytest.mark.parametrize("case", FEW, ids=lambda c: "-".join(str(v) for v in c).replace(" ", "")[-50:])
def test_few_rows_round_only_the_result(m, case):
    """Sequences of up to 16 rows (queries x heads of a group) keep a probability in two bf16 parts: the second part is at
    most 2^-7 of it and rounded to bf16."""
    seqs, hq, hkv, d, page, fp8, window, sinks = case
    g = gen(5 * hq + d)
    c, table, vals = paged_batch(m, g, seqs, hkv, d, page, fp8)
    T = sum(n for n, _ in seqs)
    q = randn(g, T, hq, d)
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    mq, mk = max(n for n, _ in seqs), max(L for _, L in seqs)
    out = torch.full((T, hq, d), 7.0, device="cuda", dtype=torch.bfloat16)
    m.mlora_paged_attention(q.cuda(), c, table.cuda(), ints([sum(n for n, _ in seqs[:i]) for i in range(len(seqs) + 1)]),
                            ints([L for _, L in seqs]), out, mq, mk, window=window, sinks=sinks,
                            ws=m.paged_workspace(T, len(seqs), hq, hkv, d, mq, mk))
    torch.cuda.synchronize()
    at = 0
    for (n, L), (k, v) in zip(seqs, vals):
        if n * (hq // hkv) <= 16:
            ref, _, mag, big = reference(q[at:at + n].double(), k, v, True, window, sinks, d ** -0.5)
            err = (2 * 2.0 ** -23 * (big[..., None] + 16) * 4 + 2.0 ** -7 * BF) * mag
            bad = ~((out[at:at + n].cpu().double() - ref).abs() <= BF * ref.abs() + (1 + BF) * err + 1e-30)
            assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} at {(n, L)}"
        at += n


@pytest.mark.parametrize("window,sinks", [(1, 1), (5, 2), (30, 1), (64, 4), (64, 70)])
@pytest.mark.parametrize("d", [64, 128])
def test_short_windows_round_only_the_result(m, d, window, sinks):
    """Windows of up to 64 keys: a probability is two bf16 parts in prompts and chunks, too (as above)."""
    g = gen(window + sinks + d)
    n, hq, hkv, page = 300, 4, 2, 16
    q, k, v = randn(g, n, hq, d), randn(g, n, hkv, d), randn(g, n, hkv, d)
    ints = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    out = torch.empty(n, hq, d, device="cuda", dtype=torch.bfloat16)
    m.mlora_attention(q.cuda(), k.cuda(), v.cuda(), ints(0, n), out, window=window, sinks=sinks)
    pages = (n + page - 1) // page
    kc, vc = [torch.zeros(pages * page, hkv, d, dtype=torch.bfloat16) for _ in range(2)]
    kc[:n], vc[:n] = k, v
    c = m.Cache(*[x.view(pages, page, hkv, d).permute(0, 2, 1, 3).contiguous().cuda() for x in (kc, vc)])
    table = torch.arange(pages, dtype=torch.int32, device="cuda")[None]
    w = 90
    chunk = torch.empty(w, hq, d, device="cuda", dtype=torch.bfloat16)
    m.mlora_paged_attention(q[n - w:].cuda(), c, table, ints(0, w), ints(n), chunk, w, n, window=window, sinks=sinks,
                            ws=m.paged_workspace(w, 1, hq, hkv, d, w, n))
    torch.cuda.synchronize()
    ref, _, mag, big = reference(q.double(), k.double(), v.double(), True, window, sinks, d ** -0.5)
    err = (2 * 2.0 ** -23 * (big[..., None] + 16) * 4 + 2.0 ** -7 * BF) * mag
    tol = BF * ref.abs() + (1 + BF) * err + 1e-30
    assert ((out.cpu().double() - ref).abs() <= tol).all()
    assert ((chunk.cpu().double() - ref[n - w:]).abs() <= tol[n - w:]).all()


def test_no_sinks_gives_the_same_bits(m):
    """sinks = 0, and sinks behind a window that reaches them, are the calls without them."""
    g = gen(5)
    seqs, hq, hkv, d = [(1, 900), (3, 500), (40, 700)], 4, 2, 128
    c, table, _ = paged_batch(m, g, seqs, hkv, d, 16, False)
    q = randn(g, 44, hq, d).cuda()
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    cu, lens = ints([0, 1, 4, 44]), ints([L for _, L in seqs])
    ws = m.paged_workspace(44, 3, hq, hkv, d, 40, 900)
    outs = []
    for kw in (dict(window=90), dict(window=90, sinks=0), dict(window=0), dict(window=0, sinks=5), dict(window=900, sinks=5)):
        o = torch.empty(44, hq, d, device="cuda", dtype=torch.bfloat16)
        m.mlora_paged_attention(q, c, table.cuda(), cu, lens, o, 40, 900, ws=ws, **kw)
        p = torch.empty_like(o)
        kv = q[:, :hkv].contiguous()
        m.mlora_attention(q, kv, kv, cu, p, max_q=40, **kw)
        torch.cuda.synchronize()
        outs.append((o.cpu(), p.cpu()))
    for i, j in ((0, 1), (2, 3), (2, 4)):
        assert torch.equal(outs[i][0], outs[j][0]) and torch.equal(outs[i][1], outs[j][1])


@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("d", [64, 128])
def test_values_reach_only_who_sees_them(m, d, bad):
    """An infinity or NaN in K and V of one key, in a prompt and in pages: rows that do not see it keep their bits."""
    g = gen(d + 1)
    n, hq, hkv, window, sinks, page = 500, 4, 2, 90, 70, 16
    q, k, v = randn(g, n, hq, d), randn(g, n, hkv, d), randn(g, n, hkv, d)
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    pages = (n + page - 1) // page
    table = torch.arange(pages, dtype=torch.int32, device="cuda")[None]
    ints = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    spans = [(0, 4), (158, 4), (200, 50), (400, 3), (440, 60)]

    def all_of(kk, vv):
        out = torch.empty(n, hq, d, device="cuda", dtype=torch.bfloat16)
        m.mlora_attention(q.cuda(), kk.cuda(), vv.cuda(), cu, out, window=window, sinks=sinks)
        kc, vc = [torch.zeros(pages * page, hkv, d, dtype=torch.bfloat16) for _ in range(2)]
        kc[:n], vc[:n] = kk, vv
        c = m.Cache(*[x.view(pages, page, hkv, d).permute(0, 2, 1, 3).contiguous().cuda() for x in (kc, vc)])
        parts = [out.cpu()]
        for at, w in spans:
            o = torch.empty(w, hq, d, device="cuda", dtype=torch.bfloat16)
            m.mlora_paged_attention(q[at:at + w].cuda(), c, table, ints(0, w), ints(at + w), o, w, at + w, window=window,
                                    sinks=sinks, ws=m.paged_workspace(w, 1, hq, hkv, d, w, at + w))
            parts.append(o.cpu())
        torch.cuda.synchronize()
        return torch.cat(parts)

    pos = torch.cat([torch.arange(n)] + [torch.arange(at, at + w) for at, w in spans])
    good = all_of(k, v)
    for key in (0, 3, 63, 64, 69, 70, 71, 127, 161, 250, 399, 402, 450, 499):
        kk, vv = k.clone(), v.clone()
        vv[key, :, 3] = bad
        kk[key, :, 5] = bad
        got = all_of(kk, vv)
        seen = (pos >= key) & ((pos - window < key) | (key < sinks))
        assert torch.equal(good[~seen], got[~seen])
        assert got[seen].isnan().any(-1).all()


def test_captured(m):
    """Captured in a graph, on a stream of its own, and replayed with eager work between: the eager bits."""
    g = gen(33)
    seqs, hq, hkv, d = [(1, 3900), (1, 40), (1, 2000), (20, 600)], 8, 2, 128
    c, table, _ = paged_batch(m, g, seqs, hkv, d, 16, True)
    q = randn(g, 23, hq, d).cuda()
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    cu, lens, table = ints([0, 1, 2, 3, 23]), ints([L for _, L in seqs]), table.cuda()
    ws = m.paged_workspace(23, 4, hq, hkv, d, 20, 3900)
    out, outp = [torch.empty(23, hq, d, device="cuda", dtype=torch.bfloat16) for _ in range(2)]
    kv = q[:, :hkv].contiguous()

    def step():
        m.mlora_paged_attention(q, c, table, cu, lens, out, 20, 3900, window=1500, sinks=4, ws=ws)
        m.mlora_attention(q, kv, kv, cu, outp, max_q=20, window=5, sinks=3)
        return [t.clone() for t in (out, outp)]

    eager = step()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        other = step()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(eager, other))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for _ in range(4):
        out.fill_(3.0)
        outp.fill_(3.0)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(eager, held))
        ws.fill_(255)
        torch.cuda.synchronize()


def test_binding_refusals(m):
    x = torch.zeros(5, 4, 64, device="cuda", dtype=torch.bfloat16)
    k = torch.zeros(5, 2, 64, device="cuda", dtype=torch.bfloat16)
    cu = torch.tensor([0, 5], dtype=torch.int32, device="cuda")
    for sinks, error in ((-1, m.MloraError), (2 ** 31, ValueError), ("4", TypeError)):
        with pytest.raises(error):
            m.mlora_attention(x, k, k, cu, torch.empty_like(x), window=2, sinks=sinks)
