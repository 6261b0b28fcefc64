"""Where a probability is kept in two bf16 parts with a window and first tokens, and over shared prefixes: nothing but the
result is rounded to bf16 then.

Tolerance as in test_gpu_attention_few_rows: scores, exponentials and sums in fp32; a probability (over an e4m3 cache: times
its value's scale, as the matrix cores take it) is a part and a rest of at most 2^-7 of it, which is rounded to bf16; then
the result's rounding.
"""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

from tests.test_gpu_attention import BF, gen, m, paged_batch, randn, ref_attention  # noqa: E402, F401  (m: a fixture)
from tests.test_gpu_attention_prefix import Batch, after  # noqa: E402
from tests.test_gpu_attention_sinks import reference  # noqa: E402


def check(got, ref, mag, big, what):
    err = (2 * 2.0 ** -23 * (big[..., None] + 16) * 4 + 2.0 ** -7 * BF) * mag
    bad = ~((got.cpu().double() - ref).abs() <= BF * ref.abs() + (1 + BF) * err + 1e-30)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} at {what}"


def windowed(m, seqs, hq, hkv, d, page, fp8, window, sinks):  # noqa: F811
    g = gen(3 * hq + d + window)
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
        ref, _, mag, big = reference(q[at:at + n].double(), k, v, True, window, sinks, d ** -0.5)
        check(out[at:at + n], ref, mag, big, (n, L))
        at += n


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("window,sinks", [(1, 1), (5, 2), (30, 1), (64, 4), (64, 70)])
def test_short_windows_of_a_few_tokens_a_sequence(m, d, window, sinks, fp8):  # noqa: F811
    """Windows of up to 64 keys where max_q gives 17 to 32 rows (queries x heads of a kv head's group)."""
    windowed(m, [(5, 300), (5, 5), (1, 40), (8, 1500), (3, 90)], 8, 2, d, 16, fp8, window, sinks)


E4M3 = [
    # (queries, keys) of the sequences, hq, hkv, d, page, window, sinks
    ([(5, 700), (5, 5), (1, 300), (8, 1500)], 8, 2, 128, 32, 300, 4),                  # 17 to 32 rows
    ([(5, 700), (2, 130), (4, 65)], 12, 2, 64, 16, 70, 1),
    ([(300, 900)], 4, 2, 128, 32, 300, 1),                                             # a chunk, cut into pieces
    ([(70, 70), (90, 400)], 8, 2, 64, 16, 100, 2),
    ([(1, 700), (70, 300), (1, 20), (2, 90)], 4, 2, 128, 16, 65, 4),                   # single tokens beside chunks
    ([(1, 50 + 7 * i) for i in range(40)] + [(200, 600)], 8, 2, 64, 64, 200, 130),
    ([(40, 60 + 9 * i) for i in range(70)] + [(1, 9)], 4, 1, 64, 16, 90, 3),           # more row blocks than workgroups at first
]


@pytest.mark.parametrize("case", E4M3, ids=lambda c: "-".join(str(v) for v in c).replace(" ", "")[-50:])
def test_first_tokens_over_an_e4m3_cache(m, case):  # noqa: F811
    """The matrix cores take a probability times its value's scale: of few keys with most of the weight one rounding to bf16
    would be in all of a row's results."""
    seqs, hq, hkv, d, page, window, sinks = case
    windowed(m, seqs, hq, hkv, d, page, True, window, sinks)


FEW = [
    # groups, sequences of no group, hq, hkv, d, page, fp8: 17 to 32 rows a sequence, and fewer
    ([after(20, (5, 5), (5, 80), (2, 300), (5, 33))], [], 8, 2, 128, 16, False),
    ([after(20, (5, 5), (5, 80), (2, 300), (5, 33))], [], 8, 2, 64, 32, True),
    ([after(600, (5, 5), (5, 80), (2, 700), (1, 3))], [(5, 40)], 12, 2, 128, 32, True),
    ([after(65, (3, 3), (3, 1500)), after(130, (3, 20), (2, 9), (1, 1))], [(3, 400), (3, 2)], 10, 1, 64, 16, False),
    ([after(90, (8, 8), (8, 300)), (0, [(8, 70)])], [(8, 8)], 4, 1, 128, 16, False),
    ([after(40, *[(5, 5 + 7 * i % 90) for i in range(70)])], [], 8, 2, 128, 16, True),
]


@pytest.mark.parametrize("case", FEW, ids=lambda c: "-".join(str(v) for v in c).replace(" ", "")[-50:])
def test_a_few_tokens_a_sequence_behind_prefixes(m, case):  # noqa: F811
    """Where max_q gives 17 to 32 rows, of shared keys and of their own."""
    groups, tail, hq, hkv, d, page, fp8 = case
    b = Batch(m, gen(17 * hq + d), groups, hq, hkv, d, page, fp8, tail)
    out = b.run()
    at = 0
    for (n, L), (k, v) in zip(b.seqs, b.vals):
        ref, _, mag, big = ref_attention(b.q[at:at + n].double(), k, v, True, 0, d ** -0.5)
        check(out[at:at + n], ref, mag, big, (n, L))
        at += n


CHUNKS = [
    # groups, sequences of no group, hq, hkv, d, page: chunks of up to 256 rows, which share, and of more, which do not
    ([after(200, (100, 300), (1, 5), (60, 60))], [(33, 900)], 8, 2, 128, 16),
    ([after(65, (64, 64), (40, 700), (2, 2)), after(300, (1, 9), (90, 90))], [(70, 70)], 4, 1, 64, 32),
    ([after(130, *[(40, 40 + 9 * i) for i in range(40)])], [(1, 300)], 4, 2, 64, 16),    # more row blocks than workgroups
]


@pytest.mark.parametrize("case", CHUNKS, ids=lambda c: "-".join(str(v) for v in c).replace(" ", "")[-50:])
def test_chunks_behind_prefixes_of_an_e4m3_cache(m, case):  # noqa: F811
    groups, tail, hq, hkv, d, page = case
    b = Batch(m, gen(19 * hq + d), groups, hq, hkv, d, page, True, tail)
    out = b.run()
    at = 0
    for (n, L), (k, v) in zip(b.seqs, b.vals):
        ref, _, mag, big = ref_attention(b.q[at:at + n].double(), k, v, True, 0, d ** -0.5)
        check(out[at:at + n], ref, mag, big, (n, L))
        at += n
