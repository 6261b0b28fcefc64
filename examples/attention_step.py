"""Serving one layer's attention with adapters: prompts, then tokens one at a time.

Every request names its own adapter.  A prompt batch runs the merged QKV layer (mlora_linear), the
norms, the rotation and the cache write (mlora_qk_rope) and attention over the packed prompts
(mlora_attention); each decode step runs the same layer on one token a request and attention over
the paged cache (mlora_paged_attention), as replays of one captured HIP graph.  A request's next
input is its attention output, so that the layer feeds itself; weights are random.

    python examples/attention_step.py [--requests 32] [--prompt 500] [--steps 64] [--e4m3]
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from lora_serving_amd import mlora  # noqa: E402

EPS = 1e-6


class AttentionLayer:
    """A merged QKV layer with adapter slots and the paged cache of its requests."""

    def __init__(self, hq, hkv, head_dim, slots, rank, tokens, page=16, e4m3=False, seed=0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        self.hq, self.hkv, self.d, self.page = hq, hkv, head_dim, page
        self.n_in, self.n_out = hq * head_dim, (hq + 2 * hkv) * head_dim
        bf = torch.bfloat16
        self.W = (rand(self.n_out, self.n_in) * self.n_in ** -0.5).to(bf)
        A = (rand(slots, 3, rank, self.n_in) * self.n_in ** -0.5).to(bf)
        B = (rand(slots, self.n_out, rank) * rank ** -0.5).to(bf)
        q, k = hq * head_dim, hkv * head_dim
        self.slots = mlora.Slots(A, B, torch.full((slots,), 0.5, device="cuda"), slice_start=[0, q, q + k, q + 2 * k])
        self.qw, self.kw = [(1 + 0.1 * rand(head_dim)).to(bf) for _ in range(2)]
        self.rope = mlora.Rope(mlora.mlora_rope_turns(head_dim, 500000.0).cuda(), head_dim)
        pages = (tokens + page - 1) // page
        shape = (pages, hkv, page, head_dim)
        zeros = lambda: torch.zeros(shape, device="cuda", dtype=bf)  # noqa: E731
        if e4m3:
            kind = torch.float8_e4m3fn
            self.cache = mlora.Cache(zeros().to(kind), zeros().to(kind), torch.zeros(shape[:3], device="cuda"),
                                     torch.zeros(shape[:3], device="cuda"))
        else:
            self.cache = mlora.Cache(zeros(), zeros())

    def buffers(self, T):
        """What a step of T tokens writes: y, q, out, and the layer's workspace."""
        bf = torch.bfloat16
        return (torch.empty(T, self.n_out, device="cuda", dtype=bf),
                torch.empty(T, self.hq, self.d, device="cuda", dtype=bf),
                torch.empty(T, self.hq, self.d, device="cuda", dtype=bf),
                mlora.workspace(T, 1, self.n_in, self.n_out, self.slots, "cuda"))

    def qkv(self, x, idx, pos, slot, y, q, ws):
        """The merged layer on x [T][n_in], then queries to q, keys and values to the cache (and, rotated, to y)."""
        mlora.mlora_linear(x, self.W, self.slots, idx, None, y, ws=ws)
        heads = y.view(-1, self.hq + 2 * self.hkv, self.d)
        mlora.mlora_qk_rope(y, self.hq, self.hkv, self.d, pos, self.rope, q, k_out=heads[:, self.hq:self.hq + self.hkv],
                            q_weight=self.qw, k_weight=self.kw, eps=EPS, cache=self.cache, slot=slot)
        return heads


class Requests:
    """A batch of requests: adapters, lengths and page tables, on the GPU."""

    def __init__(self, layer, adapters, prompts, room):
        self.layer, self.n, self.prompts = layer, len(prompts), list(prompts)
        page = layer.page
        per = (max(prompts) + room + page - 1) // page
        order = torch.randperm(self.n * per)
        self.table_host = order.view(self.n, per).to(torch.int32)
        self.table = self.table_host.cuda()
        self.adapter = torch.tensor(adapters, dtype=torch.int32)
        self.kv_len = torch.tensor(prompts, dtype=torch.int32, device="cuda")
        self.cu = torch.arange(self.n + 1, dtype=torch.int32, device="cuda")
        self.max_len = max(prompts) + room

    def prefill(self, x):
        """All prompts in one packed step: x [sum of the lengths][n_in] -> attention outputs."""
        layer = self.layer
        T = sum(self.prompts)
        pos = torch.cat([torch.arange(n) for n in self.prompts])
        req = torch.repeat_interleave(torch.arange(self.n), torch.tensor(self.prompts))
        slot = self.table_host[req, pos // layer.page].long() * layer.page + pos % layer.page
        cu = torch.zeros(self.n + 1, dtype=torch.int32)
        cu[1:] = torch.tensor(self.prompts).cumsum(0)
        y, q, out, ws = layer.buffers(T)
        i32 = lambda t: t.to(torch.int32).cuda()  # noqa: E731
        heads = layer.qkv(x, i32(self.adapter[req])[:, None].contiguous(), i32(pos), i32(slot), y, q, ws)
        hq, hkv = layer.hq, layer.hkv
        mlora.mlora_attention(q, heads[:, hq:hq + hkv], heads[:, hq + hkv:], cu.cuda(), out, max_q=max(self.prompts))
        return out

    def decoder(self, x):
        """A captured step of one token a request: reads x [n][n_in], appends the token to the cache and leaves the
        attention outputs in .out and, as the next step's input, in x."""
        layer = self.layer
        page = layer.page
        self.y, self.q, self.out, ws = layer.buffers(self.n)
        idx = self.adapter.cuda()[:, None].contiguous()
        paged_ws = mlora.paged_workspace(self.n, self.n, layer.hq, layer.hkv, layer.d, 1, self.max_len)
        rows = torch.arange(self.n, device="cuda")
        # a replay reads and writes these at their addresses, so they live as long as the graph's owner does
        self.held = (x, idx, rows, ws, paged_ws)

        def step():
            pos = self.kv_len.clone()
            slot = self.table[rows, (pos // page).long()] * page + pos % page
            self.kv_len.add_(1)
            layer.qkv(x, idx, pos, slot, self.y, self.q, ws)
            mlora.mlora_paged_attention(self.q, layer.cache, self.table, self.cu, self.kv_len, self.out, 1, self.max_len,
                                        ws=paged_ws)
            x.copy_(self.out.view(self.n, -1))

        keep = self.kv_len.clone(), x.clone()
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            step()                              # first uses happen outside the capture
        torch.cuda.current_stream().wait_stream(s)
        self.kv_len.copy_(keep[0])
        x.copy_(keep[1])
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        return graph


def main(argv=None):
    ap = argparse.ArgumentParser()
    ap.add_argument("--requests", type=int, default=32)
    ap.add_argument("--prompt", type=int, default=500, help="longest prompt")
    ap.add_argument("--steps", type=int, default=64)
    ap.add_argument("--e4m3", action="store_true", help="8-bit cache")
    a = ap.parse_args(argv)
    g = torch.Generator()
    g.manual_seed(1)
    prompts = torch.randint(1, a.prompt + 1, (a.requests,), generator=g).tolist()
    room = a.steps + 1
    layer = AttentionLayer(32, 8, 128, slots=8, rank=16, tokens=a.requests * (max(prompts) + room + 16), e4m3=a.e4m3)
    batch = Requests(layer, torch.randint(-1, 8, (a.requests,), generator=g).tolist(), prompts, room)
    x = torch.randn(sum(prompts), layer.n_in, generator=g).to(torch.bfloat16).cuda()
    out = batch.prefill(x)
    torch.cuda.synchronize()
    last = torch.tensor(prompts).cumsum(0) - 1
    nxt = out.view(sum(prompts), -1)[last.cuda()].contiguous()
    graph = batch.decoder(nxt)
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    for _ in range(a.steps):
        graph.replay()
    torch.cuda.synchronize()
    ms = (time.perf_counter() - t0) / a.steps * 1e3
    print(f"{a.requests} requests, prompts of 1 to {max(prompts)} tokens, {a.steps} steps: {ms:.3f} ms a step, "
          f"{a.requests / ms * 1e3:.0f} tokens/s of one layer's attention, contexts now up to {int(batch.kv_len.max())}")


if __name__ == "__main__":
    main()
