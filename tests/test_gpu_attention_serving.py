"""The attention operators together, as a server uses them: a system prompt prefilled once into the cache, requests that
share its pages and bring their own tokens, then single tokens; one layer that sees everything (shared prefix) and
one with a window and first tokens that stay visible.  Every output against a plain implementation in 64 bits over the
cache's own contents; the last step also captured in a graph.
"""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

from tests.test_gpu_attention import check, gen, randn  # noqa: E402
from tests.test_gpu_attention_sinks import reference  # noqa: E402

HQ, HKV, D, PAGE, WINDOW, SINKS = 8, 2, 128, 16, 70, 4


@pytest.fixture(scope="module")
def m():
    from lora_serving_amd import mlora
    return mlora


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("fp8", [False, True])
def test_shared_prompt_then_tokens(m, fp8):
    g = gen(77)
    shared, own = 200, [3, 40, 17, 66, 1]
    n = len(own)
    kind = torch.float8_e4m3fn if fp8 else torch.bfloat16
    pages = 100
    shape = (pages, HKV, PAGE, D)
    layers = []
    for _ in range(2):
        k, v = [torch.zeros(shape, device="cuda", dtype=torch.bfloat16).to(kind) for _ in range(2)]
        ks, vs = [torch.ones(shape[:3], device="cuda") if fp8 else None for _ in range(2)]
        layers.append(m.Cache(k, v, ks, vs))
    free = list(torch.randperm(pages, generator=g).numpy())
    whole = shared // PAGE
    common = [int(free.pop()) for _ in range(whole)]
    table = torch.full((n, 24), -1, dtype=torch.int32)
    for b in range(n):
        table[b, :whole] = torch.tensor(common, dtype=torch.int32)
        for p in range(whole, 20):
            table[b, p] = int(free.pop())
    rope = m.Rope(m.mlora_rope_turns(D).cuda(), D)
    lens = [0] * n
    ws = m.prefix_workspace(400, n, 1, HQ, HKV, D, 400, 400, 400)
    ws2 = m.paged_workspace(400, n, HQ, HKV, D, 400, 400)

    def slots(b, lo, hi):
        return [int(table[b, j // PAGE]) * PAGE + j % PAGE for j in range(lo, hi)]

    def store(cache, rows, pos, slot):
        """Norm-free rotation and cache write of merged rows; the queries."""
        q = torch.empty(rows.shape[0], HQ, D, device="cuda", dtype=torch.bfloat16)
        m.mlora_qk_rope(rows, HQ, HKV, D, ints(pos), rope, q, cache=cache, slot=ints(slot))
        return q

    def content(cache, b, L):
        k, v = [torch.empty(L, HKV, D, device="cuda", dtype=torch.bfloat16) for _ in range(2)]
        m.mlora_cache_read(cache, ints(slots(b, 0, L)), k, v)
        return k.cpu().double(), v.cpu().double()

    def attend(cache, q, new, layer):
        cu = ints([sum(new[:i]) for i in range(n + 1)])
        out = torch.empty_like(q)
        if layer == 0:
            m.mlora_prefix_attention(q, cache, table.cuda(), cu, ints(lens), ints([0, n]), ints([shared]), out, max_q=max(new),
                                     max_kv=max(lens), max_prefix=shared, ws=ws)
        else:
            m.mlora_paged_attention(q, cache, table.cuda(), cu, ints(lens), out, max(new), max(lens), window=WINDOW, sinks=SINKS,
                                    ws=ws2)
        return out

    def verify(cache, q, out, new, layer):
        torch.cuda.synchronize()
        at = 0
        for b in range(n):
            k, v = content(cache, b, lens[b])
            args = (WINDOW, SINKS) if layer else (0, 0)
            ref, _, mag, big = reference(q[at:at + new[b]].cpu().double(), k, v, True, *args, D ** -0.5)
            # (the e4m3 values read back are rounded to bf16 once: 2^-8 of K in the scores, of V in the results)
            slack = 2.0 ** -8 if fp8 else 0.0
            if fp8:
                tol = (3 * 2.0 ** -8 + 2 * slack * big[..., None]) * mag + 2.0 ** -7 * ref.abs()
                assert ((out[at:at + new[b]].cpu().double() - ref).abs() <= tol).all()
            else:
                check(out[at:at + new[b]], ref, mag, big)
            at += new[b]

    for layer, cache in enumerate(layers):
        # the system prompt: all of its tokens into the first request's pages, and the others' copies of the last page's
        rows = randn(g, shared, (HQ + 2 * HKV) * D).cuda()
        q = store(cache, rows, range(shared), slots(0, 0, shared))
        for b in range(1, n):
            rest = range(whole * PAGE, shared)
            store(cache, rows[whole * PAGE:], rest, slots(b, whole * PAGE, shared))
        if not fp8:        # its own outputs, packed
            k, v = [torch.empty(shared, HKV, D, device="cuda", dtype=torch.bfloat16) for _ in range(2)]
            m.mlora_cache_read(cache, ints(slots(0, 0, shared)), k, v)
            out = torch.empty_like(q)
            kw = dict(window=WINDOW, sinks=SINKS) if layer else {}
            m.mlora_attention(q, k, v, ints([0, shared]), out, max_q=shared, **kw)
            torch.cuda.synchronize()
            ref, _, mag, big = reference(q.cpu().double(), k.cpu().double(), v.cpu().double(), True, *((WINDOW, SINKS) if layer else (0, 0)),
                                         D ** -0.5)
            check(out, ref, mag, big)
        # the requests' own tokens, then steps of one token
        lens[:] = [shared] * n
        for new in (own, [1] * n, [1] * n):
            T = sum(new)
            rows = randn(g, T, (HQ + 2 * HKV) * D).cuda()
            pos = [p for b in range(n) for p in range(lens[b], lens[b] + new[b])]
            slot = [s for b in range(n) for s in slots(b, lens[b], lens[b] + new[b])]
            q = store(cache, rows, pos, slot)
            lens[:] = [a + c for a, c in zip(lens, new)]
            out = attend(cache, q, new, layer)
            verify(cache, q, out, new, layer)
        eager = out.clone()
        cu, ln, tb, gs, pl = ints(list(range(n + 1))), ints(lens), table.cuda(), ints([0, n]), ints([shared])
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            if layer == 0:
                m.mlora_prefix_attention(q, cache, tb, cu, ln, gs, pl, out, max_q=1, max_kv=max(lens), max_prefix=shared, ws=ws)
            else:
                m.mlora_paged_attention(q, cache, tb, cu, ln, out, 1, max(lens), window=WINDOW, sinks=SINKS, ws=ws2)
        for _ in range(3):
            out.fill_(5.0)
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, eager)
            ws.fill_(255)
            ws2.fill_(255)
