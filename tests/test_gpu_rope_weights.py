"""Norm weights that are not finite, on the GPU: they reach the values that the formula gives them."""
import math

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.mark.parametrize("bad", [math.inf, math.nan])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("d,rot", [(64, 32), (128, 16), (64, 0)])
def test_weight_of_a_value_that_does_not_turn(d, rot, inter, bad):
    """A weight past the rotated part reaches its own value only."""
    from lora_serving_amd import mlora as m
    g = torch.Generator()
    g.manual_seed(d + rot)
    T, hq, hkv = 9, 4, 2
    qkv = torch.randn(T, (hq + 2 * hkv) * d, generator=g).to(torch.bfloat16).cuda()
    pos = torch.arange(T, dtype=torch.int32, device="cuda") * 7 + 1
    r = m.Rope(m.mlora_rope_turns(rot).cuda() if rot else None, rot, interleaved=inter)
    at = rot + 5
    w = torch.linspace(0.5, 1.5, d).to(torch.bfloat16).cuda()
    outs = []
    for value in (w[at].item(), bad):
        wb = w.clone()
        wb[at] = value
        q, k = [torch.empty(T, h, d, device="cuda", dtype=torch.bfloat16) for h in (hq, hkv)]
        m.mlora_qk_rope(qkv, hq, hkv, d, pos, r, q, k_out=k, q_weight=wb, k_weight=wb)
        torch.cuda.synchronize()
        outs.append(torch.cat([q, k], 1).cpu())
    good, got = outs
    rest = [i for i in range(d) if i != at]
    assert torch.equal(good[..., rest], got[..., rest])
    x = qkv.cpu()[:, :(hq + hkv) * d].view(T, hq + hkv, d)[..., at].float()
    want = x * bad
    assert torch.equal(got[..., at].float().nan_to_num(nan=7.0), want.nan_to_num(nan=7.0))
