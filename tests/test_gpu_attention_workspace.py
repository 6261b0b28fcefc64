"""One workspace, made for the largest step, on the GPU."""
import pytest

from tests.test_gpu_attention import gen, m, paged_batch, randn  # noqa: F401  (m: a fixture)

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.mark.parametrize("hq,hkv,d,fp8", [(32, 8, 128, False), (8, 1, 64, True)])
def test_one_workspace_for_all_steps(m, hq, hkv, d, fp8):  # noqa: F811
    """A workspace of the sizes of the largest batch serves every smaller one, with the same bits."""
    g = gen(hq)
    most, dev = [(1, 1 + 7 * i) for i in range(256)] + [(600, 3000)], "cuda"
    c, table, _ = paged_batch(m, g, most, hkv, d, 16, fp8)
    table = table.clamp(0, c.n_pages - 1).to(dev)
    q = randn(g, 856, hq, d).to(dev)
    sizes = lambda seqs: (sum(n for n, _ in seqs), len(seqs), hq, hkv, d, max(n for n, _ in seqs),  # noqa: E731
                          max(L for _, L in seqs))
    one = m.paged_workspace(*sizes(most))

    def run(seqs, ws):
        T, n, _, _, _, mq, mk = sizes(seqs)
        ints = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
        out = torch.empty(T, hq, d, device=dev, dtype=torch.bfloat16)
        ws.fill_(255)
        m.mlora_paged_attention(q[:T], c, table[:n].contiguous(), ints([sum(k for k, _ in seqs[:i]) for i in range(n + 1)]),
                                ints([L for _, L in seqs]), out, mq, mk, ws=ws)
        return out

    for seqs in (most, [(1, 3000)], [(1, 700)] * 30, [(512, 3000)], [(64, 2999)] * 2, [(3, 1000)] * 5, [(40, 40)],
                 [(17, 3000)] + [(1, 1024)] * 31, [(1, 900)] * 256):
        a = run(seqs, one)
        b = run(seqs, m.paged_workspace(*sizes(seqs)))
        torch.cuda.synchronize()
        assert torch.equal(a, b)
        assert a.isfinite().all()
