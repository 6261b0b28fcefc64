"""The binding of the attention step's calls: what a call does besides its arguments."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def m():
    from lora_serving_amd import mlora
    return mlora


def new(*s, t=torch.bfloat16):
    return torch.zeros(s, device="cuda", dtype=t)


def ints(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def test_an_argument_that_fails_launches_nothing(m):
    class Unknown:
        def __bool__(self):
            raise RuntimeError("neither")

    q, k, cu = new(5, 4, 64), new(5, 2, 64), ints(0, 5)
    out = torch.full((5, 4, 64), 7.0, device="cuda", dtype=torch.bfloat16)
    with pytest.raises(RuntimeError, match="neither"):
        m.mlora_attention(q, k, k, cu, out, causal=Unknown())
    c = m.Cache(new(2, 2, 16, 64), new(2, 2, 16, 64))
    with pytest.raises(RuntimeError, match="neither"):
        m.mlora_paged_attention(q, c, ints(0)[None], cu, ints(5), out, 5, 16, causal=Unknown(),
                                ws=m.paged_workspace(5, 1, 4, 2, 64, 5, 16))
    torch.cuda.synchronize()
    assert (out == 7.0).all()
