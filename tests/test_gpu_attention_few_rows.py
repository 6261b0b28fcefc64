"""Single and few tokens over the cache on the GPU: sequences of up to 16 rows (queries x heads of a group) keep their
probabilities in two bf16 parts, so nothing but the result is rounded to bf16."""
import math

import pytest

from tests.test_gpu_attention import BF, gen, m, paged_batch, randn, ref_attention  # noqa: F401  (m: a fixture)

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

FEW = [
    # (queries, keys) of the sequences, hq, hkv, d, page, fp8, window
    ([(1, 2), (1, 1), (1, 37), (1, 300), (1, 64)], 4, 2, 128, 16, False, 0),
    ([(1, 5), (1, 41), (1, 150), (1, 299)], 8, 1, 64, 32, True, 0),
    ([(1, 90), (1, 33), (1, 7)], 6, 2, 128, 16, True, 30),
    ([(3, 60), (4, 130), (1, 20)], 8, 2, 64, 16, False, 0),
    ([(4, 200), (2, 90), (3, 31)], 4, 1, 128, 32, False, 0),
    ([(1, 140), (1, 8), (1, 61)], 16, 1, 64, 16, True, 0),
    ([(1, 100), (1, 61)], 11, 1, 128, 16, False, 0),
    ([(1, 900), (1, 50)], 8, 2, 128, 16, False, 0),                  # split over keys
    ([(4, 900)], 4, 1, 64, 16, True, 0),
    ([(1, 70), (1, 300), (40, 90), (2, 33)], 4, 2, 128, 16, False, 0),     # beside a chunk
    ([(1, 70), (1, 300), (40, 90), (2, 33)], 4, 2, 64, 16, True, 0),
]


@pytest.mark.parametrize("case", FEW, ids=lambda c: "-".join(str(v) for v in c).replace(" ", ""))
def test_few_rows_round_only_the_result(m, case):  # noqa: F811
    seqs, hq, hkv, d, page, fp8, window = case
    g = gen(11 * sum(L for _, L in seqs) + hq + d)
    c, table, vals = paged_batch(m, g, seqs, hkv, d, page, fp8)
    T, dev = sum(n for n, _ in seqs), "cuda"
    q = randn(g, T, hq, d)
    cu = torch.tensor([sum(n for n, _ in seqs[:i]) for i in range(len(seqs) + 1)], dtype=torch.int32)
    lens = torch.tensor([L for _, L in seqs], dtype=torch.int32)
    mq, mk = max(n for n, _ in seqs), max(L for _, L in seqs)
    out = torch.full((T, hq, d), 7.0, device=dev, dtype=torch.bfloat16)
    m.mlora_paged_attention(q.to(dev), c, table.to(dev), cu.to(dev), lens.to(dev), out, mq, mk, window=window,
                            ws=m.paged_workspace(T, len(seqs), hq, hkv, d, mq, mk))
    torch.cuda.synchronize()
    at = 0
    for (n, L), (k, v) in zip(seqs, vals):
        if n * (hq // hkv) <= 16:           # (a chunk's own rows aside)
            ref, _, mag, big = ref_attention(q[at:at + n].double(), k, v, True, window, d ** -0.5)
            # scores, exponentials and sums in fp32 (d products a score, a scaling to a power of two; exponentials to
            # 2^-21); a probability's second part is at most 2^-7 of it and rounded to bf16; then the result's rounding
            err = (2 * 2.0 ** -23 * (big[..., None] + 16) * 4 + 2.0 ** -7 * BF) * mag
            got = out[at:at + n].cpu().double()
            bad = ~((got - ref).abs() <= BF * ref.abs() + (1 + BF) * err + 1e-30)
            assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} at {(n, L)}"
        at += n


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [1, 4, 7])
def test_an_infinite_value_stays_infinite(m, n, d):  # noqa: F811
    """An infinity in V gives the same infinity to every row that sees it, of whole tiles and of the last ones."""
    hq, hkv, page, L, dev = 4, 1, 16, 300, "cuda"
    g = gen(n + d)
    c, table, _ = paged_batch(m, g, [(n, L)], hkv, d, page, False)
    q = randn(g, n, hq, d).to(dev)
    ints = lambda *v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    ws = m.paged_workspace(n, 1, hq, hkv, d, n, L)
    for key in (3, 150, L - n, L - 2):
        for value in (math.inf, -math.inf):
            pg, at = int(table[0, key // page]), key % page
            keep = c.v[pg, :, at, 9].clone()
            c.v[pg, :, at, 9] = value
            out = torch.empty(n, hq, d, device=dev, dtype=torch.bfloat16)
            m.mlora_paged_attention(q, c, table.to(dev), ints(0, n), ints(L), out, n, L, ws=ws)
            torch.cuda.synchronize()
            c.v[pg, :, at, 9] = keep
            seen = torch.arange(L - n, L) >= key
            got = out.cpu()
            assert (got[seen][..., 9] == value).all()
            assert got[~seen].isfinite().all()
            assert got[..., [i for i in range(d) if i != 9]].isfinite().all()
