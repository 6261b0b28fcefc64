"""The binding of the attention step's calls: what a call does besides its arguments."""
import sys
import threading
import time

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


def test_other_threads_run_during_a_call(m):
    """The interpreter's lock is free while a call launches.  Nothing else here gives it up: the interval after which
    a thread has to is set past the test's length, and the other thread sleeps after each count."""
    c, slot, k = m.Cache(new(2, 2, 16, 64), new(2, 2, 16, 64)), ints(0, 1, 2, 3), new(4, 2, 64)
    q, cu, out = new(4, 4, 64), ints(0, 4), new(4, 4, 64)
    qkv, ws = new(4, 512), m.paged_workspace(4, 1, 4, 2, 64, 4, 16)
    table, length, rope = ints(0)[None], ints(4), m.Rope(m.mlora_rope_turns(64).cuda(), 64)
    calls = [lambda: m.mlora_cache_read(c, slot, k, None), lambda: m.mlora_qk_rope(qkv, 4, 2, 64, slot, rope, q),
             lambda: m.mlora_attention(q, k, k, cu, out),
             lambda: m.mlora_paged_attention(q, c, table, cu, length, out, 4, 16, ws=ws)]
    for f in calls:
        f()
    torch.cuda.synchronize()
    count, stop, interval = [0], threading.Event(), sys.getswitchinterval()

    def other():
        while not stop.is_set():
            count[0] += 1
            time.sleep(0)

    t = threading.Thread(target=other)
    sys.setswitchinterval(1000)
    try:
        t.start()
        time.sleep(0.05)
        for f in calls:
            before = count[0]
            for _ in range(4000):
                f()
            assert count[0] > before
    finally:
        stop.set()
        sys.setswitchinterval(interval)
        t.join()
    torch.cuda.synchronize()
