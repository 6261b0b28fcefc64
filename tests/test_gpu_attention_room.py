"""Calls with a short window and few first tokens over long contexts: what nobody sees is not cut into parts, so they need less
workspace than the same batch without a window, and single and few tokens none."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

from tests.test_gpu_attention import check, gen, m, paged_batch, randn  # noqa: E402, F401  (m: a fixture)
from tests.test_gpu_attention_sinks import reference  # noqa: E402

CASES = [
    # (queries, keys) of the sequences, hq, hkv, d, page, fp8, window, sinks.  The chunks' 128 rows see the window, their own 64
    # or 32 tokens and one more, and room is kept for two units of 128 keys around the first ones: 351 and 319 keys here,
    # two pieces of 256
    ([(1, 5000), (1, 40), (1, 3000)], 4, 2, 128, 16, False, 100, 4),
    ([(1, 4200), (1, 900)], 8, 1, 64, 32, True, 200, 1),
    ([(5, 4100), (2, 1700)], 8, 2, 128, 16, False, 60, 128),            # 20 rows
    ([(40, 4300)], 4, 2, 64, 16, False, 30, 2),                         # a chunk
    ([(1, 4000), (33, 2500), (1, 7)], 4, 1, 128, 64, True, 30, 3),      # beside single tokens
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(v) for v in c).replace(" ", "")[-50:])
def test_a_short_window_needs_less_workspace(m, case):  # noqa: F811
    seqs, hq, hkv, d, page, fp8, window, sinks = case
    g = gen(hq + d + window)
    c, table, vals = paged_batch(m, g, seqs, hkv, d, page, fp8)
    T = sum(n for n, _ in seqs)
    q = randn(g, T, hq, d)
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    mq, mk = max(n for n, _ in seqs), max(L for _, L in seqs)
    out = torch.full((T, hq, d), 7.0, device="cuda", dtype=torch.bfloat16)
    args = (q.cuda(), c, table.cuda(), ints([sum(n for n, _ in seqs[:i]) for i in range(len(seqs) + 1)]),
            ints([L for _, L in seqs]), out, mq, mk)
    # two fp32 parts of every row, outputs and (maximum, sum), each from a multiple of 256 bytes on
    room = 2 * T * hq * (4 * d + 8) + 3 * 256 if mq * (hq // hkv) > 32 else 0
    ws = torch.full((room,), 255, device="cuda", dtype=torch.uint8) if room else None
    for kw in (dict(), dict(window=3000, sinks=sinks), dict(window=window, sinks=3000)):
        with pytest.raises(m.MloraError):
            m.mlora_paged_attention(*args, ws=ws, **kw)
    assert (out == 7.0).all()
    m.mlora_paged_attention(*args, ws=ws, window=window, sinks=sinks)
    torch.cuda.synchronize()
    at = 0
    for (n, L), (k, v) in zip(seqs, vals):
        ref, _, mag, big = reference(q[at:at + n].double(), k, v, True, window, sinks, d ** -0.5)
        check(out[at:at + n], ref, mag, big)
        at += n
