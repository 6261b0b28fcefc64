"""The attention step's operators together: prompts, then captured decode steps over the paged cache."""
import math
import os
import sys

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

BF = 2.0 ** -8


def reference(q, k, v, scale):
    """One query [hq, d] over keys and values [L, hkv, d], 64 bits: output, sum p |v|, largest sum |scale q k|."""
    r = q.shape[0] // k.shape[1]
    kk, vv = k.repeat_interleave(r, 1), v.repeat_interleave(r, 1)
    s = (kk * q).sum(-1) * scale
    big = ((kk * q).abs().sum(-1) * scale).amax(0)
    w = torch.softmax(s, 0)
    return (w[..., None] * vv).sum(0), (w[..., None] * vv.abs()).sum(0), big


@pytest.mark.parametrize("e4m3", [False, True])
def test_prompts_then_tokens(e4m3):
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    try:
        import attention_step as ex
    finally:
        sys.path.pop(0)
    from lora_serving_amd import mlora
    g = torch.Generator()
    g.manual_seed(5)
    prompts, steps = [1, 37, 130, 16], 20
    layer = ex.AttentionLayer(8, 2, 64, slots=3, rank=8, tokens=4 * (130 + 21 + 16), e4m3=e4m3)
    batch = ex.Requests(layer, [-1, 0, 2, 1], prompts, steps + 1)
    T = sum(prompts)
    x = torch.randn(T, layer.n_in, generator=g).to(torch.bfloat16).cuda()
    out = batch.prefill(x)
    last = (torch.tensor(prompts).cumsum(0) - 1).cuda()
    nxt = out.view(T, -1)[last].contiguous()
    inputs = []
    graph = batch.decoder(nxt)
    scale = layer.d ** -0.5
    for i in range(steps):
        inputs.append(nxt.clone())
        graph.replay()
        torch.cuda.synchronize()
        assert batch.kv_len.tolist() == [n + i + 1 for n in prompts]
        if i not in (0, 15, steps - 1):
            continue
        for b, n in enumerate(prompts):         # the cache as it is read back, attended in 64 bits
            j = torch.arange(n + i + 1)
            slot = (batch.table_host[b, j // layer.page].long() * layer.page + j % layer.page).to(torch.int32).cuda()
            k, v = [torch.empty(n + i + 1, layer.hkv, layer.d, device="cuda", dtype=torch.bfloat16) for _ in range(2)]
            mlora.mlora_cache_read(layer.cache, slot, k, v)
            ref, mag, big = reference(batch.q[b].cpu().double(), k.cpu().double(), v.cpu().double(), scale)
            # probabilities and result rounded to bf16; from an e4m3 cache the values read back are rounded once
            # more, which moves a score by up to 2^-8 of its terms and a value by 2^-8
            extra = (torch.expm1(2 * BF * big)[:, None] + BF) * mag if e4m3 else 0.0
            tol = (BF + 2.0 ** -18) * mag + BF * ref.abs() + BF * BF * mag + extra + 1e-30
            assert ((batch.out[b].cpu().double() - ref).abs() <= tol).all()
    if e4m3:
        return
    # the same tokens as whole prompts: the layer's other kernels may round y the other way (2^-8 of a value each for
    # q, k and v), no more
    whole = ex.Requests(layer, [-1, 0, 2, 1], [n + steps for n in prompts], 1)
    parts, at = [], 0
    for b, n in enumerate(prompts):
        parts += [x[at:at + n], torch.stack([t[b] for t in inputs])]
        at += n
    full = whole.prefill(torch.cat(parts))
    torch.cuda.synchronize()
    at = -1
    for b, n in enumerate(prompts):
        at += n + steps
        j = torch.arange(n + steps)
        slot = (whole.table_host[b, j // layer.page].long() * layer.page + j % layer.page).to(torch.int32).cuda()
        k, v = [torch.empty(n + steps, layer.hkv, layer.d, device="cuda", dtype=torch.bfloat16) for _ in range(2)]
        mlora.mlora_cache_read(layer.cache, slot, k, v)
        _, mag, big = reference(batch.q[b].cpu().double(), k.cpu().double(), v.cpu().double(), scale)
        tol = (torch.expm1(2 * 4 * BF * big)[:, None] + 4 * BF) * mag
        diff = (batch.out[b].cpu().double() - full[at].cpu().double()).abs()
        assert (diff <= tol).all() and math.isfinite(float(diff.max()))
