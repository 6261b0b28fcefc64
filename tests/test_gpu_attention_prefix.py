"""Attention of sequences that share prefixes against a plain implementation in 64 bits on the CPU, sequence by
sequence over all of its keys.  Tolerances as in test_gpu_attention: a probability and a result are each rounded to bf16
(2^-8 of the value at most), the rest is fp32.
"""
import math
import random

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

from tests.test_gpu_attention import BF, check, check_lse, gen, randn, ref_attention  # noqa: E402


@pytest.fixture(scope="module")
def m():
    from lora_serving_amd import mlora
    return mlora


def ints(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Batch:
    """Sequences (queries, keys) in groups (shared keys, [sequences]).  A sequence that holds the whole prefix shares its
    whole pages and has a copy of the part filled one; a shorter one has pages of its own with other tokens.  Slots
    that no token fills hold NaN, table entries that no token reaches are out of range."""

    def __init__(self, m, g, groups, hq, hkv, d, page, fp8, tail=()):
        self.m, self.hq, self.hkv, self.d, self.page, self.fp8 = m, hq, hkv, d, page, fp8
        self.groups = groups
        self.seqs = [s for _, members in groups for s in members] + list(tail)
        self.start = [sum(len(x) for _, x in groups[:i]) for i in range(len(groups) + 1)]
        self.prefix = [p for p, _ in groups]
        plan, b = [], 0                                     # pages of every sequence; None: copied from
        pages, copies = 0, []
        rows = []
        for p, members in list(groups) + [(0, list(tail))]:
            whole = p // page
            common = list(range(pages, pages + whole)) if any(L >= p for _, L in members) else []
            pages += len(common)
            first = None
            for n, L in members:
                need = (L + page - 1) // page
                mine = L >= p
                own = need - whole if mine else need
                rows.append((common if mine else []) + list(range(pages, pages + own)))
                if mine and p % page:
                    if first is None:
                        first = pages
                    else:
                        copies.append((first, pages, p % page))
                pages += own
        pages += 1
        perm = torch.randperm(pages, generator=g)
        self.table = torch.full((len(self.seqs), max([len(r) for r in rows] + [0]) + 2), 10 ** 6, dtype=torch.int32)
        live = torch.zeros(pages, page, dtype=torch.bool)
        for b, (r, (_, L)) in enumerate(zip(rows, self.seqs)):
            if r:
                self.table[b, :len(r)] = perm[torch.tensor(r)].to(torch.int32)
            j = torch.arange(L)
            live[self.table[b, j // page].long(), j % page] = True
        shape = (pages, hkv, page, d)
        raw = [torch.randn(shape, generator=g) * (0.3 + torch.rand(shape[:3] + (1,), generator=g)) for _ in range(2)]
        store = [x.to(torch.float8_e4m3fn if fp8 else torch.bfloat16) for x in raw]
        scale = [0.1 + torch.rand(shape[:3], generator=g) for _ in range(2)] if fp8 else [None, None]
        for i in range(2):
            s = store[i].view(torch.uint8) if fp8 else store[i]
            for a, b, n in copies:
                a, b = int(perm[a]), int(perm[b])
                s[b, :, :n] = s[a, :, :n]
                if fp8:
                    scale[i][b, :, :n] = scale[i][a, :, :n]
        value = [x.double() * (s[..., None].double() if fp8 else 1.0) for x, s in zip(store, scale)]
        self.vals = []
        for b, (_, L) in enumerate(self.seqs):
            j = torch.arange(L)
            pg = self.table[b, j // page].long()
            self.vals.append([x[pg, :, j % page] for x in value])
        bad = (~live)[:, None, :, None].expand(shape)
        for i in range(2):
            if fp8:
                store[i].view(torch.uint8)[bad] = 0x7f
                scale[i][(~live)[:, None].expand(shape[:3])] = math.nan
            else:
                store[i][bad] = math.nan
        up = lambda t: None if t is None else t.cuda()  # noqa: E731
        self.cache = m.Cache(up(store[0]), up(store[1]), up(scale[0]), up(scale[1]))
        self.T = sum(n for n, _ in self.seqs)
        self.q = randn(g, self.T, hq, d)
        self.cu = [sum(n for n, _ in self.seqs[:i]) for i in range(len(self.seqs) + 1)]
        self.mq, self.mk = max(n for n, _ in self.seqs), max(L for _, L in self.seqs)
        self.mp = max(self.prefix + [0])

    def workspace(self):
        ws = self.m.prefix_workspace(self.T, len(self.seqs), len(self.groups), self.hq, self.hkv, self.d, self.mq, self.mk,
                                     self.mp)
        return ws.fill_(255)                                # NaN in every word

    def args(self):
        return dict(q=self.q.cuda(), cache=self.cache, page_table=self.table.cuda(), cu_q=ints(*self.cu),
                    kv_len=ints(*[L for _, L in self.seqs]), group_start=ints(*self.start), prefix_len=ints(*self.prefix),
                    max_q=self.mq, max_kv=self.mk, max_prefix=self.mp)

    def run(self, causal=True, lse=None, **kw):
        out = torch.full((self.T, self.hq, self.d), 7.0, device="cuda", dtype=torch.bfloat16)
        self.m.mlora_prefix_attention(**{**self.args(), **kw}, out=out, causal=causal, lse=lse, ws=self.workspace())
        torch.cuda.synchronize()
        return out

    def check(self, out, causal=True, lse=None):
        at = 0
        for (n, L), (k, v) in zip(self.seqs, self.vals):
            if n:
                ref, rl, mag, big = ref_attention(self.q[at:at + n].double(), k, v, causal, 0, self.d ** -0.5)
                check(out[at:at + n], ref, mag, big)
                if lse is not None:
                    check_lse(lse[at:at + n], rl, big)
            at += n


def after(p, *seqs):
    """A group: p shared keys, sequences of (queries, own keys with them)."""
    return p, [(n, p + own) for n, own in seqs]


CASES = [
    # groups, sequences of no group, hq, hkv, d, page, fp8, causal
    ([after(64, (1, 1), (1, 5))], [], 1, 1, 64, 16, False, True),
    ([after(100, (1, 1), (1, 17), (1, 130))], [], 4, 2, 128, 16, False, True),
    ([after(1, (1, 1), (1, 9))], [], 4, 2, 128, 16, False, True),                     # one shared key
    ([after(0, (1, 1), (1, 9))], [], 4, 2, 64, 16, False, True),                      # none
    ([after(777, *[(1, 1 + 37 * i % 300) for i in range(40)])], [], 8, 2, 128, 16, False, True),     # 160 rows: two row blocks
    ([after(777, *[(1, 1 + 37 * i % 300) for i in range(40)])], [], 8, 2, 128, 32, True, True),
    ([after(300, (1, 3), (1, 4)), after(65, (1, 1), (1, 2), (1, 3)), after(500, (1, 30))], [(1, 40), (1, 700)],
     6, 2, 64, 16, False, True),                                                      # a group of one, and none
    ([after(300, (1, 3), (1, 4)), (128, []), after(129, (1, 1), (1, 2), (1, 3))], [(0, 9), (1, 0)], 7, 7, 64, 64, True, True),
    ([(200, [(1, 300), (1, 200), (1, 201), (1, 50), (0, 300), (1, 0), (4, 203), (1, 260)])], [], 4, 1, 128, 16, False, True),
    ([(200, [(1, 300), (1, 200), (1, 199), (3, 10)])], [], 4, 1, 128, 16, True, False),     # not causal: 200 keys are the prefix itself
    ([after(600, (5, 5), (5, 80), (2, 700), (5, 300))], [], 12, 2, 128, 16, False, True),   # 30 rows
    ([after(600, (5, 5), (5, 80), (2, 700), (5, 300))], [], 12, 2, 64, 32, True, True),
    ([after(900, (1, 1), (40, 300), (1, 20), (130, 130), (1, 60))], [], 4, 2, 128, 16, False, True),  # and chunks
    ([after(333, (100, 613), (1, 64), (50, 50)), after(80, (3, 3), (60, 90))], [(33, 900), (1, 100)], 8, 2, 128, 32, True, True),
    ([after(450, (64, 257), (5, 9))], [], 40, 2, 64, 64, False, True),                # groups of heads wider than a tile
    ([after(450, (1, 2000), (1, 300), (1, 9))], [], 48, 1, 64, 16, True, True),
    ([after(5000, (1, 1), (1, 1), (1, 3000))], [], 8, 2, 128, 16, False, True),       # many chunks, own keys split
    ([after(4097, (20, 2000), (1, 1))], [], 8, 4, 128, 16, False, True),
    ([after(130, *[(1, 1 + i % 50) for i in range(130)])], [(1, 1 + 9 * i) for i in range(70)], 4, 2, 64, 16, True, True),
    ([after(64 + i, (1, 1 + i % 5), (1, 3)) for i in range(90)], [], 4, 2, 64, 16, False, True),      # more than 64 groups
    ([after(64, *[(17, 20 + i) for i in range(70)])], [], 4, 2, 64, 16, False, True),  # many chunks
    ([after(256, (2, 2), (2, 2))], [], 32, 2, 128, 256, False, True),                 # 32 rows, whole pages
    ([after(230, (1, 2), (1, 140), (1, 33))], [(1, 50)], 24, 1, 128, 16, True, True),  # single tokens of 24 rows
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(v) for v in c).replace(" ", "")[-70:])
def test_groups(m, case):
    groups, tail, hq, hkv, d, page, fp8, causal = case
    b = Batch(m, gen(hq + d + len(groups)), groups, hq, hkv, d, page, fp8, tail)
    lens = [L for _, L in b.seqs]
    assert m.mlora_validate_pages(b.cache, b.table, b.cu, lens, b.T, b.mq, b.mk) == (m.MLORA_OK, 0)
    lse = torch.full((b.T, hq), 7.0, device="cuda")
    out = b.run(causal, lse)
    b.check(out, causal, lse)


MANY = [
    # more sequences and groups than a workgroup lists at a time
    ([after(40 + i, (1, 1 + i % 7), (1, 2), (2, 5)) for i in range(120)], [(1, 30)], 4, 2, 64, 16, True, True),
    ([after(90, *[(1, 1 + i % 9) for i in range(300)])], [], 4, 1, 128, 16, False, True),
    ([after(90, *[(1, 1 + i % 9) for i in range(255)]), after(33, (1, 2), (1, 40))], [], 2, 2, 64, 32, False, True),
    ([after(256, *[(1, 1 + i % 9) for i in range(100)] + [(70, 100)] + [(1, 1 + i % 9) for i in range(100)])], [], 8, 2, 64, 16,
     True, True),                                                                     # rows of one that shares nothing between
]


@pytest.mark.parametrize("case", MANY, ids=lambda c: "-".join(str(v) for v in c).replace(" ", "")[-40:])
def test_many_sequences(m, case):
    test_groups(m, case)


FEW = [
    ([after(5, (1, 1), (1, 3))], [], 4, 2, 128, 16, False),
    ([after(130, (1, 2), (1, 60), (1, 200)), after(64, (1, 1), (1, 5))], [(1, 90)], 8, 2, 128, 32, False),
    ([after(130, (1, 2), (1, 60), (1, 200)), after(64, (1, 1), (1, 5))], [(1, 90)], 16, 1, 64, 16, True),
    ([after(300, (3, 60), (4, 130), (1, 20))], [], 8, 2, 64, 16, False),
    ([after(40, *[(1, 1 + i % 30) for i in range(50)])], [], 4, 1, 128, 16, True),
    ([after(90, (1, 70), (100, 300), (1, 4))], [], 6, 2, 128, 16, False),          # beside a chunk
]


@pytest.mark.parametrize("case", FEW, ids=lambda c: "-".join(str(v) for v in c).replace(" ", "")[-50:])
def test_few_rows_round_only_the_result(m, case):
    """Sequences of up to 16 rows (queries x heads of a group) keep a probability in two bf16 parts, of shared keys and of
    their own: the second part is at most 2^-7 of it and rounded to bf16."""
    groups, tail, hq, hkv, d, page, fp8 = case
    b = Batch(m, gen(13 * hq + d), groups, hq, hkv, d, page, fp8, tail)
    out = b.run()
    at = 0
    for (n, L), (k, v) in zip(b.seqs, b.vals):
        if 0 < n * (hq // hkv) <= 16:
            ref, _, mag, big = ref_attention(b.q[at:at + n].double(), k, v, True, 0, d ** -0.5)
            err = (2 * 2.0 ** -23 * (big[..., None] + 16) * 4 + 2.0 ** -7 * BF) * mag
            bad = ~((out[at:at + n].cpu().double() - ref).abs() <= BF * ref.abs() + (1 + BF) * err + 1e-30)
            assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} at {(n, L)}"
        at += n


@pytest.mark.parametrize("d", [64, 128])
def test_an_infinite_value_stays_infinite(m, d):
    """An infinity in V, of a shared token (of a whole tile and of the last one) or an own one, gives the same infinity."""
    b = Batch(m, gen(d + 2), [after(150, (1, 5), (2, 40), (1, 100))], 4, 2, d, 16, False)
    row_seq = [i for i, (n, _) in enumerate(b.seqs) for _ in range(n)]
    pos = torch.tensor([L - n + i for n, L in b.seqs for i in range(n)])
    for of, key in ((0, 3), (0, 70), (0, 143), (1, 160), (2, 249)):
        pg, at = int(b.table[of, key // 16]), key % 16
        holds = torch.tensor([int(b.table[s, key // 16]) == pg and b.seqs[s][1] > key for s in row_seq])
        seen = holds & (pos >= key)
        for value in (math.inf, -math.inf):
            keep = b.cache.v[pg, :, at, 9].clone()
            b.cache.v[pg, :, at, 9] = value
            got = b.run().cpu()
            b.cache.v[pg, :, at, 9] = keep
            assert seen.any() and (got[seen][..., 9] == value).all()
            assert got[~seen].isfinite().all()
            assert got[..., [i for i in range(d) if i != 9]].isfinite().all()


@pytest.mark.parametrize("seed", range(40))
def test_random_groups(m, seed):
    r = random.Random(seed)
    hkv = r.choice([1, 2, 3])
    hq = hkv * r.choice([1, 2, 4, 7])
    news = r.choice([[1], [1], [1, 0], [1, 2, 5], [1, 3, 60]])
    groups = []
    for _ in range(r.randint(1, 5)):
        p = r.choice([0, 1, 63, 64, 65, 128, r.randint(1, 700), r.randint(1, 2500)])
        members = []
        for i in range(r.choice([0, 1, 2, 3, 9])):
            n = r.choice(news)
            own = n + r.choice([0, 1, r.randint(0, 60), r.randint(0, 900)])
            if i and r.random() < 0.1:
                members.append((n, r.randint(0, p + n)))
            else:
                members.append((n, p + own))
        groups.append((p, members))
    tail = [(r.choice(news), r.randint(1, 300)) for _ in range(r.choice([0, 1, 4]))] + [(1, 5)]
    b = Batch(m, gen(seed), groups, hq, hkv, r.choice([64, 128]), r.choice([16, 32, 256]), r.random() < 0.5, tail)
    causal = r.random() < 0.85
    lse = torch.full((b.T, hq), 7.0, device="cuda")
    out = b.run(causal, lse)
    b.check(out, causal, lse)


def test_bounds_above_the_sizes(m):
    """max_q, max_kv and max_prefix are bounds; a smaller max_prefix shares fewer keys."""
    b = Batch(m, gen(3), [after(700, *[(1, 1 + 40 * i) for i in range(9)])], 8, 2, 128, 16, False)
    for kw in (dict(max_prefix=100000, max_kv=100000), dict(max_prefix=100), dict(max_prefix=0), dict(max_prefix=699)):
        a = {**b.args(), **kw}
        ws = m.prefix_workspace(b.T, 9, 1, 8, 2, 128, 5, a["max_kv"], a["max_prefix"])
        ws.fill_(255)
        out = torch.full((b.T, 8, 128), 7.0, device="cuda", dtype=torch.bfloat16)
        m.mlora_prefix_attention(**{**a, "max_q": 5}, out=out, ws=ws)
        torch.cuda.synchronize()
        b.check(out)
    out = b.run(group_start=ints(0), prefix_len=ints())          # no group at all
    b.check(out)


def test_no_keys_and_no_table(m):
    """A batch whose sequences hold nothing yet, with a table of no columns: zeros and -inf."""
    k, v = [torch.zeros(2, 2, 16, 64, device="cuda", dtype=torch.bfloat16) for _ in range(2)]
    for n, w in ((3, 1), (2, 70)):
        T = n * w
        q = randn(gen(n), T, 4, 64).cuda()
        out, lse = torch.full_like(q, 7.0), torch.full((T, 4), 7.0, device="cuda")
        table = torch.empty(n, 0, device="cuda", dtype=torch.int32)
        for causal in (True, False):
            m.mlora_prefix_attention(q, m.Cache(k, v), table, ints(*range(0, T + 1, w)), ints(*[0] * n), ints(0, n), ints(40), out,
                                     w, 100, 60, causal=causal, lse=lse, ws=m.prefix_workspace(T, n, 1, 4, 2, 64, w, 100, 60))
            torch.cuda.synchronize()
            assert (out == 0).all() and (lse == -math.inf).all()
            out.fill_(7.0)


def test_unanswered_and_padding_rows_are_left(m):
    """Sequences of more queries than max_q and rows past the last sequence keep what was there."""
    b = Batch(m, gen(4), [after(200, (1, 4), (9, 30), (1, 1))], 4, 2, 64, 16, False)
    pad = torch.cat([b.q, b.q[:3]])
    out = torch.full((b.T + 3, 4, 64), 7.0, device="cuda", dtype=torch.bfloat16)
    ws = m.prefix_workspace(b.T + 3, 3, 1, 4, 2, 64, 1, b.mk, b.mp)
    m.mlora_prefix_attention(**{**b.args(), "q": pad.cuda(), "max_q": 1}, out=out, ws=ws)
    torch.cuda.synchronize()
    full = b.run()
    kept = torch.ones(b.T + 3, dtype=torch.bool)
    kept[[0, 10]] = False
    assert (out.cpu()[kept] == 7.0).all()
    b.check(full)
    for t in (0, 10):
        # other launches, other parts: equal up to their roundings
        assert (out[t].float() - full[t].float()).abs().max() <= 2.0 ** -6 * full[t].float().abs().max()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("d", [64, 128])
def test_bad_values_reach_only_who_sees_them(m, d, fp8):
    """NaN in a shared token reaches every row of the group, in a sequence's own token only the rows that see it."""
    seqs = [(1, 5), (3, 40), (1, 300), (40, 50)]
    b = Batch(m, gen(d), [after(333, *seqs), after(90, (1, 4), (1, 2))], 4, 2, d, 16, fp8, [(1, 30)])
    good = b.run().cpu()
    row_seq = [i for i, (n, _) in enumerate(b.seqs) for _ in range(n)]
    pos = torch.tensor([L - n + i for n, L in b.seqs for i in range(n)])
    seq = torch.tensor(row_seq)
    for of, key in ((0, 0), (0, 100), (0, 319), (1, 334), (1, 370), (2, 400), (3, 335), (3, 382), (4, 12), (6, 20)):
        pg, at = int(b.table[of, key // 16]), key % 16
        old = [t.clone() for t in (b.cache.k, b.cache.v)]
        for t in (b.cache.k, b.cache.v):
            if fp8:
                t.view(torch.uint8)[pg, :, at, 7] = 0x7f
            else:
                t[pg, :, at, 7] = math.nan
        got = b.run().cpu()
        for t, o in zip((b.cache.k, b.cache.v), old):
            t.copy_(o)
        holds = torch.tensor([int(b.table[s, key // 16]) == pg and b.seqs[s][1] > key for s in row_seq])
        seen = holds & (pos >= key)
        assert seen.any()
        assert torch.equal(good[~seen], got[~seen])
        assert got[seen].isnan().any(-1).all()


def test_pages_past_32_bits(m):
    """Pages whose bytes lie past 4 GiB from the start of the cache, in both operators; a workspace that starts anywhere."""
    hkv, page, d, pages = 8, 64, 128, 40000                       # 2.6 billion values, 5.2 GB each of K and V
    b = Batch(m, gen(6), [after(150, (1, 4), (1, 90), (5, 20))], 16, hkv, d, page, False)
    k, v = [torch.empty(pages, hkv, page, d, device="cuda", dtype=torch.bfloat16) for _ in range(2)]
    n = b.cache.n_pages
    k[pages - n:], v[pages - n:] = b.cache.k, b.cache.v
    table = torch.where(b.table < n, b.table + (pages - n), b.table).cuda()
    cache = m.Cache(k, v)
    ws = b.workspace()[8:]
    out = torch.empty(b.T, 16, d, device="cuda", dtype=torch.bfloat16)
    m.mlora_prefix_attention(**{**b.args(), "cache": cache, "page_table": table}, out=out, ws=ws)
    torch.cuda.synchronize()
    b.check(out)
    a = b.args()
    outs = []
    for c, t in ((b.cache, b.table.cuda()), (cache, table)):
        o = torch.empty_like(out)
        m.mlora_paged_attention(a["q"], c, t, a["cu_q"], a["kv_len"], o, b.mq, b.mk, window=40, sinks=3,
                                ws=m.paged_workspace(b.T, 3, 16, hkv, d, b.mq, b.mk))
        outs.append(o)
    torch.cuda.synchronize()
    assert torch.equal(*outs)


def test_strided_rows_and_scale(m):
    """Queries and outputs as parts of wider rows, a scale of its own."""
    b = Batch(m, gen(8), [after(260, (1, 4), (2, 30), (1, 150))], 4, 2, 128, 16, True)
    wide = torch.full((b.T, 5, 256), 7.0, device="cuda", dtype=torch.bfloat16).view(b.T, 1280)
    q = wide[:, 8:8 + 512].unflatten(1, (4, 128))
    q.copy_(b.q)
    o = torch.full((b.T, 1280), 7.0, device="cuda", dtype=torch.bfloat16)
    out = o[:, 256:768].unflatten(1, (4, 128))
    m.mlora_prefix_attention(**{**b.args(), "q": q}, out=out, scale=0.31, ws=b.workspace())
    torch.cuda.synchronize()
    at = 0
    for (n, L), (k, v) in zip(b.seqs, b.vals):
        ref, _, mag, big = ref_attention(b.q[at:at + n].double(), k, v, True, 0, 0.31)
        check(out[at:at + n], ref, mag, big)
        at += n
    assert (o[:, :256] == 7.0).all() and (o[:, 768:] == 7.0).all()


def test_captured_and_two_at_once(m):
    """In a graph, replayed with other groups and lengths; and two calls at once on streams and workspaces of their
    own: the eager bits."""
    b = Batch(m, gen(11), [after(800, *[(1, 1 + 70 * i) for i in range(12)]), after(300, (1, 2), (1, 400))], 8, 2, 128, 16,
              True, [(1, 90)])
    a = b.args()
    ws, ws2 = b.workspace(), b.workspace()
    out, out2 = [torch.empty(b.T, 8, 128, device="cuda", dtype=torch.bfloat16) for _ in range(2)]
    call = lambda o, w: m.mlora_prefix_attention(**a, out=o, ws=w)  # noqa: E731
    whole = (a["group_start"].clone(), a["prefix_len"].clone(), a["kv_len"].clone())
    fewer = (ints(0, 5, 14), ints(790, 0), a["kv_len"] - (a["kv_len"] > 810).int() * 3)
    eager = []
    for s in (whole, fewer):
        for t, v in zip((a["group_start"], a["prefix_len"], a["kv_len"]), s):
            t.copy_(v)
        call(out, ws)
        torch.cuda.synchronize()
        eager.append(out.clone())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(out, ws)
    for i in (0, 1, 1, 0, 0):
        for t, v in zip((a["group_start"], a["prefix_len"], a["kv_len"]), (whole, fewer)[i]):
            t.copy_(v)
        out.fill_(3.0)
        ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager[i])
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, o, w in zip(streams, (out, out2), (ws, ws2)):
            with torch.cuda.stream(s):
                call(o, w)
    torch.cuda.synchronize()
    assert torch.equal(out, eager[0]) and torch.equal(out2, eager[0])


def test_binding_refusals(m):
    b = Batch(m, gen(1), [after(20, (1, 4), (1, 3))], 4, 2, 64, 16, False)
    a = {**b.args(), "out": torch.empty(2, 4, 64, device="cuda", dtype=torch.bfloat16), "ws": b.workspace()}
    m.mlora_prefix_attention(**a)
    for change, error in ((dict(prefix_len=ints(20, 3)), ValueError), (dict(group_start=ints(0, 2).long()), ValueError),
                          (dict(prefix_len=ints(20).cpu()), ValueError), (dict(kv_len=ints(24)), ValueError),
                          (dict(page_table=ints(0)), ValueError), (dict(q=a["q"].float()), ValueError),
                          (dict(max_prefix="3"), TypeError), (dict(max_prefix=-1), m.MloraError), (dict(ws=None), m.MloraError),
                          (dict(max_prefix=1 << 30), m.MloraError), (dict(scale=-1.0), m.MloraError)):
        with pytest.raises(error):
            m.mlora_prefix_attention(**{**a, **change})
    torch.cuda.synchronize()
