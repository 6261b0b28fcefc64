"""The attention step after the merged QKV layer: which calls are timed, their plain forms and
their definition in 64 bits.

Operators: mlora_qk_rope (norms of queries and keys per head, rotation by position, K and V
written to the paged cache), mlora_cache_read (cached tokens back as bf16), mlora_attention
(packed prompts) and mlora_paged_attention (new tokens over a paged cache).
"""
import math
import random

import torch

own = False

EPS = 1e-6
E4M3_MAX = 448.0
TINY = 2.0 ** -90          # smallest amax a scale is made from
SCORES = 1 << 28           # scores that the plain form holds at once


# ---- cases -------------------------------------------------------------------------------------
def listed():
    return [
        # 64 requests, one new token each: what a decode step does between the QKV layer and attention
        dict(name="rope_decode64", op="rope", T=64, hq=32, hkv=8, d=128, rot=128, inter=False, norm=True,
             factor=1.0, far=8192, fp8=False, page=16, pad=3),
        # a prefill batch of 16384 tokens, positions scaled by parts for long contexts
        dict(name="rope_prefill16384", op="rope", T=16384, hq=32, hkv=8, d=128, rot=128, inter=False, norm=True,
             factor=8.0, far=131072, fp8=False, page=64, pad=0),
        # 256 decode tokens and a 2048-token segment into an 8-bit cache, half of each head rotated, and the
        # written tokens read back (as when a finished prefill is moved to another pool)
        dict(name="rope_fp8_mixed2304", op="rope", T=2304, hq=32, hkv=8, d=128, rot=64, inter=True, norm=False,
             factor=1.0, far=40000, fp8=True, page=16, pad=0),
        # one short prefix copied out of the cache
        dict(name="read_short333", op="read", T=333, hkv=8, d=128, fp8=False, page=16),
        # prefixes of a batch copied out of an 8-bit cache
        dict(name="read_fp8_32768", op="read", T=32768, hkv=8, d=128, fp8=True, page=32),
        # a handful of short prompts of uneven lengths, narrow heads, sliding window
        dict(name="prompt_ragged_short", op="prompt", lens="1,17,129,300,65,511,2", hq=16, hkv=4, d=64, causal=True,
             window=128),
        # the prefill batch: 8 prompts of 2048 tokens
        dict(name="prompt_8x2048", op="prompt", lens=",".join(["2048"] * 8), hq=32, hkv=8, d=128, causal=True,
             window=0),
        # one long document
        dict(name="prompt_16384", op="prompt", lens="16384", hq=32, hkv=8, d=128, causal=True, window=0),
        # one user, one token
        dict(name="paged_decode1", op="paged", new="1x1", lo=1003, hi=1003, spread=1, hq=32, hkv=8, d=128, fp8=False,
             page=16, window=0),
        # a decode batch of 64 with contexts of 1 to 8192
        dict(name="paged_decode64", op="paged", new="64x1", lo=1, hi=8192, spread=2, hq=32, hkv=8, d=128, fp8=False,
             page=16, window=0),
        # a decode batch of 256 over an 8-bit cache
        dict(name="paged_decode256_fp8", op="paged", new="256x1", lo=128, hi=4096, spread=3, hq=32, hkv=8, d=128,
             fp8=True, page=32, window=0),
        # the mixed batch: 256 decode tokens and one 2048-token chunk of a long prompt
        dict(name="paged_mixed2304", op="paged", new="256x1,1x2048", lo=64, hi=2048, chunk_before=6000, spread=4,
             hq=32, hkv=8, d=128, fp8=False, page=16, window=0),
    ]


def log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "read", "prompt", "prompt", "paged", "paged", "paged"])
    hkv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 3, 4, 7, 8]) if hkv < 8 else rng.choice([1, 2, 4])
    d = rng.choice([64, 128])
    page = rng.choice([16, 32, 64])
    fp8 = rng.random() < 0.4
    if op == "rope":
        return dict(op=op, T=log_int(rng, 1, 16384), hq=hkv * group, hkv=hkv, d=d, rot=rng.choice([16, 32, d // 2, d]),
                    inter=rng.random() < 0.5, norm=rng.random() < 0.6, factor=rng.choice([1.0, 1.0, 4.0, 32.0]),
                    far=log_int(rng, 100, 1000000), fp8=fp8, page=page, pad=rng.choice([0, 0, 1]))
    if op == "read":
        return dict(op=op, T=log_int(rng, 1, 32768), hkv=hkv, d=d, fp8=fp8, page=page)
    if op == "prompt":
        n = rng.randint(1, 9)
        most = 11000 // n
        lens = ",".join(str(log_int(rng, 1, most)) for _ in range(n))
        return dict(op=op, lens=lens, hq=hkv * group, hkv=hkv, d=d, causal=rng.random() < 0.8,
                    window=rng.choice([0, 0, 0, log_int(rng, 1, 4096)]))
    hi = log_int(rng, 16, 8192)
    new = "%dx%d" % (log_int(rng, 1, min(256, 1 + 200000 // hi)), rng.choice([1, 1, 1, 1, 2, 5]))
    if rng.random() < 0.35:
        new += ",1x%d" % log_int(rng, 2, 2048)
    return dict(op=op, new=new, lo=1, hi=hi, chunk_before=log_int(rng, 1, 6000), spread=rng.randrange(1 << 30),
                hq=hkv * group, hkv=hkv, d=d, fp8=fp8, page=page, window=rng.choice([0, 0, 0, log_int(rng, 1, 2048)]))


def prompt_lens(case):
    return [int(v) for v in case["lens"].split(",")]


def paged_lens(case):
    """(new tokens, keys with them) of every sequence: a group AxB is A sequences of B new tokens; in a group
    of one sequence with more than one new token the keys before them are chunk_before."""
    r = random.Random(case["spread"])
    out = []
    for part in case["new"].split(","):
        a, b = (int(v) for v in part.split("x"))
        for _ in range(a):
            before = case.get("chunk_before", 0) if (a == 1 and b > 1) else r.randint(case["lo"], case["hi"]) - 1
            out.append((b, before + b))
    return out


def visible(case, new, keys):
    """Pairs of a query and a key it sees, and the keys that any query sees."""
    causal, window = case.get("causal", True), case["window"]
    pairs, first = 0, keys
    for i in range(new):
        p = keys - new + i
        hi = p + 1 if causal else keys
        lo = max(0, p - window + 1) if window else 0
        if hi > lo:
            pairs += hi - lo
            first = min(first, lo)
    return pairs, keys - first


def work(case):
    op, hkv, d = case["op"], case["hkv"], case["d"]
    if op == "rope":
        T, hq = case["T"], case["hq"]
        size = T * (hq + 2 * hkv) * d * 2 + T * hq * d * 2
        if case["fp8"]:
            size += T * 2 * hkv * (d + 4) + T * 2 * hkv * d * 2
        else:
            size += T * 2 * hkv * d * 2
        return {"bytes": size, "flops": T * (hq + hkv) * (3 * case["rot"] + (4 * d if case["norm"] else 0))}
    if op == "read":
        per = d + 4 if case["fp8"] else 2 * d
        return {"bytes": case["T"] * 2 * hkv * (per + 2 * d), "flops": case["T"] * 2 * hkv * d}
    if op == "prompt":
        seqs = [(n, n) for n in prompt_lens(case)]
        per = 2 * d
    else:
        seqs = paged_lens(case)
        per = d + 4 if case["fp8"] else 2 * d
    size, pairs = 0, 0
    for new, keys in seqs:
        p, k = visible(case, new, keys)
        pairs += p
        size += new * case["hq"] * d * 2 * 2 + k * 2 * hkv * per
    return {"bytes": size, "flops": 4 * d * case["hq"] * pairs}


# ---- inputs ------------------------------------------------------------------------------------
def turns_per_position(case):
    """Turns of the circle per position of every rotated pair, in 64 bits; factor above 1 scales by parts: slow
    pairs (under one turn in the original length of 4096) are stretched by the factor, fast ones (over 32
    turns) stay, between them a linear ramp."""
    rot, factor = case["rot"], case["factor"]
    out = []
    for i in range(rot // 2):
        f = 500000.0 ** (-2.0 * i / rot) / (2.0 * math.pi)
        if factor != 1.0:
            turns = 4096 * f
            keep = min(1.0, max(0.0, (turns - 1.0) / (32.0 - 1.0)))
            f = f * keep + f / factor * (1.0 - keep)
        out.append(f)
    return out


def magnitude(case):
    return 0.1 * math.log(case["factor"]) + 1.0


def to_e4m3(x):
    """fp32 [..., d] as e4m3 codes and one fp32 scale for each vector."""
    scale = x.abs().amax(-1, keepdim=True).clamp_min(TINY) / E4M3_MAX
    return (x / scale).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn), scale.squeeze(-1)


def filled_cache(case, pages, g):
    dev = "cuda"
    shape = (pages, case["hkv"], case["page"], case["d"])
    s = {}
    for n in ("k", "v"):
        x = torch.randn(shape, generator=g, device=dev, dtype=torch.bfloat16)
        if case["fp8"]:
            # tokens differ in size, as keys and values do
            x = x.float() * (0.25 + 2 * torch.rand(shape[:3] + (1,), generator=g, device=dev))
            s[n], s[n + "s"] = to_e4m3(x)
        else:
            s[n], s[n + "s"] = x, None
        del x
    return s


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed * 7919 + 11)
    s = {"case": case}
    op, hkv, d = case["op"], case["hkv"], case["d"]
    bf, i32 = torch.bfloat16, torch.int32
    if op == "rope":
        T, hq = case["T"], case["hq"]
        s["qkv"] = torch.randn(T, (hq + 2 * hkv) * d, generator=g, device=dev, dtype=bf)
        s["pos"] = torch.randint(0, case["far"], (T,), generator=g, device=dev, dtype=i32)
        s["qw"] = s["kw"] = None
        if case["norm"]:
            s["qw"] = (1 + 0.2 * torch.randn(d, generator=g, device=dev)).to(bf)
            s["kw"] = (1 + 0.2 * torch.randn(d, generator=g, device=dev)).to(bf)
        pages = (T + case["page"] - 1) // case["page"] + 2
        shape = (pages, hkv, case["page"], d)
        kind = torch.float8_e4m3fn if case["fp8"] else bf
        s["k"] = torch.zeros(shape, device=dev, dtype=bf).to(kind)
        s["v"] = torch.zeros(shape, device=dev, dtype=bf).to(kind)
        s["ks"] = s["vs"] = None
        if case["fp8"]:
            s["ks"] = torch.zeros(shape[:3], device=dev)
            s["vs"] = torch.zeros(shape[:3], device=dev)
            s["kb"] = torch.empty(T, hkv, d, device=dev, dtype=bf)
            s["vb"] = torch.empty(T, hkv, d, device=dev, dtype=bf)
        # tokens fill shuffled pages in order; padding tokens are stored nowhere
        order = torch.randperm(pages, generator=g, device=dev)
        t = torch.arange(T, device=dev)
        slot = order[t // case["page"]] * case["page"] + t % case["page"]
        if case["pad"] and T > case["pad"]:
            slot[T - case["pad"]:] = -1
        s["slot"] = slot.to(i32)
        s["q"] = torch.empty(T, hq, d, device=dev, dtype=bf)
    elif op == "read":
        T = case["T"]
        pages = (T + case["page"] - 1) // case["page"] + 2
        s.update(filled_cache(case, pages, g))
        order = torch.randperm(pages, generator=g, device=dev)
        t = torch.arange(T, device=dev)
        s["slot"] = (order[t // case["page"]] * case["page"] + t % case["page"]).to(i32)
        s["kb"] = torch.empty(T, hkv, d, device=dev, dtype=bf)
        s["vb"] = torch.empty(T, hkv, d, device=dev, dtype=bf)
    elif op == "prompt":
        lens = prompt_lens(case)
        T, hq = sum(lens), case["hq"]
        # q, k and v lie in the merged layer's rows
        s["qkv"] = torch.randn(T, (hq + 2 * hkv) * d, generator=g, device=dev, dtype=bf)
        s["cu"] = torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], device=dev, dtype=i32)
        s["lens"] = lens
        s["out"] = torch.empty(T, hq, d, device=dev, dtype=bf)
    else:
        seqs = paged_lens(case)
        T, hq = sum(n for n, _ in seqs), case["hq"]
        need = [(n + case["page"] - 1) // case["page"] for _, n in seqs]
        pages = sum(need) + 3
        s.update(filled_cache(case, pages, g))
        order = torch.randperm(pages, generator=g, device=dev).cpu()
        table = torch.zeros(len(seqs), max(need) + 1, dtype=i32)
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = order[at:at + n]
            at += n
        s["table"] = table.to(dev)
        s["q"] = torch.randn(T, hq, d, generator=g, device=dev, dtype=bf)
        new = [n for n, _ in seqs]
        s["cu"] = torch.tensor([sum(new[:i]) for i in range(len(new) + 1)], device=dev, dtype=i32)
        s["len"] = torch.tensor([n for _, n in seqs], device=dev, dtype=i32)
        s["seqs"] = seqs
        s["out"] = torch.empty(T, hq, d, device=dev, dtype=bf)
    if own:
        from lora_serving_amd import mlora
        if "k" in s:
            s["cache"] = mlora.Cache(s["k"], s["v"], s["ks"], s["vs"])
        if op == "rope":
            if case["factor"] == 1.0:
                turns = mlora.mlora_rope_turns(case["rot"], 500000.0)
            else:
                turns = mlora.mlora_rope_turns(case["rot"], 500000.0, scaling=mlora.MLORA_ROPE_PARTS,
                                               factor=case["factor"], orig_len=4096, fast=32.0, slow=1.0)
            s["rope"] = mlora.Rope(turns.to(dev), case["rot"], interleaved=case["inter"], magnitude=magnitude(case))
        if op == "paged":
            s["max_new"] = max(n for n, _ in seqs)
            s["max_len"] = max(n for _, n in seqs)
            s["ws"] = mlora.paged_workspace(T, len(seqs), hq, hkv, d, s["max_new"], s["max_len"])
        if op == "prompt":
            s["max_len"] = max(lens)
    return s


# ---- plain forms -------------------------------------------------------------------------------
def rotate(x, case, cos, sin):
    rot = case["rot"]
    y = x.clone()
    if case["inter"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2] = a * cos - b * sin
        y[..., 1:rot:2] = b * cos + a * sin
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y[..., :rot // 2] = a * cos - b * sin
        y[..., rot // 2:rot] = b * cos + a * sin
    return y


def plain_rope(s):
    case = s["case"]
    T, hq, hkv, d = case["T"], case["hq"], case["hkv"], case["d"]
    x = s["qkv"].view(T, hq + 2 * hkv, d).float()
    q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    if case["norm"]:
        q = q * torch.rsqrt(q.square().mean(-1, keepdim=True) + EPS) * s["qw"].float()
        k = k * torch.rsqrt(k.square().mean(-1, keepdim=True) + EPS) * s["kw"].float()
    f = torch.tensor(turns_per_position(case), device=x.device, dtype=torch.float64)
    a = (s["pos"].double()[:, None] * f).frac() * (2 * math.pi)
    cos = (a.cos() * magnitude(case)).float()[:, None]
    sin = (a.sin() * magnitude(case)).float()[:, None]
    q, k = rotate(q, case, cos, sin), rotate(k, case, cos, sin)
    s["q"].copy_(q)
    keep = (s["slot"] >= 0).nonzero().squeeze(1)
    slot = s["slot"][keep].long()
    page, off = slot // case["page"], slot % case["page"]
    if not case["fp8"]:
        s["k"][page, :, off] = k[keep].to(torch.bfloat16)
        s["v"][page, :, off] = v[keep].to(torch.bfloat16)
        return s["q"], s["k"], s["v"]
    for name, val in (("k", k), ("v", v)):
        code, scale = to_e4m3(val[keep])
        s[name].view(torch.uint8)[page, :, off] = code.view(torch.uint8)
        s[name + "s"][page, :, off] = scale
    plain_read(s)
    return s["q"], s["kb"], s["vb"]


def cached(s, name, slot):
    """Tokens of the cache in 32 bits, [n, heads, d]."""
    case = s["case"]
    slot = slot.long()
    page, off = slot // case["page"], slot % case["page"]
    if not case["fp8"]:
        return s[name][page, :, off].float()
    code = s[name].view(torch.uint8)[page, :, off].view(torch.float8_e4m3fn).float()
    return code * s[name + "s"][page, :, off][..., None]


def plain_read(s):
    none = (s["slot"] < 0)[:, None, None]
    for name in ("k", "v"):
        s[name + "b"].copy_(cached(s, name, s["slot"].clamp_min(0)).masked_fill(none, 0.0))
    return s["kb"], s["vb"]


def plain_sequence(case, q, k, v, out):
    """One sequence: q [n, hq, d], k and v [L, hkv, d] in 32 bits, out bf16."""
    n, hq, d = q.shape
    L, hkv = k.shape[0], k.shape[1]
    group = hq // hkv
    kt, vt = k.permute(1, 2, 0).contiguous(), v.permute(1, 0, 2).contiguous()
    step = max(1, SCORES // (hq * L))
    for i in range(0, n, step):
        m = min(step, n - i)
        p = torch.arange(L - n + i, L - n + i + m, device=q.device)[:, None]
        j = torch.arange(L, device=q.device)[None]
        off = torch.zeros(m, L, dtype=torch.bool, device=q.device)
        if case.get("causal", True):
            off |= j > p
        if case["window"]:
            off |= j <= p - case["window"]
        qs = q[i:i + m].reshape(m, hkv, group, d).permute(1, 2, 0, 3).reshape(hkv, group * m, d)
        sc = torch.bmm(qs, kt).view(hkv, group, m, L) / math.sqrt(d)
        sc.masked_fill_(off, -math.inf)
        top = sc.amax(-1, keepdim=True)
        e = (sc - top.masked_fill(top == -math.inf, 0.0)).exp_()
        total = e.sum(-1, keepdim=True)
        o = torch.bmm(e.view(hkv, group * m, L), vt).view(hkv, group, m, d)
        o = o / total.masked_fill(total == 0, 1.0)
        out[i:i + m] = o.permute(2, 0, 1, 3).reshape(m, hq, d).to(torch.bfloat16)


def plain_prompt(s):
    case = s["case"]
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    x = s["qkv"].view(-1, hq + 2 * hkv, d)
    at = 0
    for n in s["lens"]:
        part = x[at:at + n].float()
        plain_sequence(case, part[:, :hq], part[:, hq:hq + hkv], part[:, hq + hkv:], s["out"][at:at + n])
        at += n
    return s["out"]


def plain_paged(s):
    case = s["case"]
    at = 0
    for b, (n, L) in enumerate(s["seqs"]):
        j = torch.arange(L, device=s["q"].device)
        slot = s["table"][b].long()[j // case["page"]] * case["page"] + j % case["page"]
        plain_sequence(case, s["q"][at:at + n].float(), cached(s, "k", slot), cached(s, "v", slot),
                       s["out"][at:at + n])
        at += n
    return s["out"]


def run(s):
    case = s["case"]
    op, hq, hkv, d = case["op"], case.get("hq"), case["hkv"], case["d"]
    if not own:
        return {"rope": plain_rope, "read": plain_read, "prompt": plain_prompt, "paged": plain_paged}[op](s)
    from lora_serving_amd import mlora
    if op == "rope":
        mlora.mlora_qk_rope(s["qkv"], hq, hkv, d, s["pos"], s["rope"], s["q"], q_weight=s["qw"], k_weight=s["kw"],
                            eps=EPS, cache=s["cache"], slot=s["slot"])
        if not case["fp8"]:
            return s["q"], s["k"], s["v"]
        mlora.mlora_cache_read(s["cache"], s["slot"], s["kb"], s["vb"])
        return s["q"], s["kb"], s["vb"]
    if op == "read":
        mlora.mlora_cache_read(s["cache"], s["slot"], s["kb"], s["vb"])
        return s["kb"], s["vb"]
    if op == "prompt":
        x = s["qkv"].view(-1, hq + 2 * hkv, d)
        mlora.mlora_attention(x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], s["cu"], s["out"], max_q=s["max_len"],
                              causal=case["causal"], window=case["window"])
    else:
        mlora.mlora_paged_attention(s["q"], s["cache"], s["table"], s["cu"], s["len"], s["out"], max_q=s["max_new"],
                                    max_kv=s["max_len"], window=case["window"], ws=s["ws"])
    return s["out"]


# ---- the definition in 64 bits -----------------------------------------------------------------
def nearest_e4m3(x):
    """The e4m3 value nearest to each (ties to the even one), in 64 bits."""
    a = x.abs().clamp_max(E4M3_MAX)
    e = torch.floor(torch.log2(a.clamp_min(2.0 ** -30))).clamp_min(-6.0)
    step = torch.pow(torch.full_like(e, 2.0), e - 3.0)
    return torch.sign(x) * torch.round(a / step) * step


def exact_attention(case, q, k, v):
    """[n, hq, d] from q [n, hq, d], k and v [L, hkv, d], all in 64 bits, one head at a time."""
    n, hq, d = q.shape
    L, hkv = k.shape[0], k.shape[1]
    out = torch.zeros_like(q)
    pos = torch.arange(n, device=q.device) + (L - n)
    key = torch.arange(L, device=q.device)
    rows = max(1, (1 << 27) // L)
    for i in range(0, n, rows):
        p = pos[i:i + rows, None]
        see = key[None] >= 0
        if case.get("causal", True):
            see = see & (key[None] <= p)
        if case["window"]:
            see = see & (key[None] > p - case["window"])
        see = see.expand(p.shape[0], L)
        for h in range(hq):
            kv = h * hkv // hq
            sc = (q[i:i + rows, h] @ k[:, kv].t().contiguous()) * (d ** -0.5)
            w = torch.where(see, sc, torch.full_like(sc, -math.inf))
            w = torch.softmax(w, -1)
            w = torch.where(see, w, torch.zeros_like(w))  # a row that sees nothing is zero
            out[i:i + rows, h] = w @ v[:, kv].contiguous()
    return out


def exact(case, seed):
    op, hkv, d = case["op"], case["hkv"], case["d"]
    s = prepare(case, seed)

    def values(name, slot):
        page, off = torch.div(slot, case["page"], rounding_mode="floor"), slot % case["page"]
        x = s[name].double().permute(0, 2, 1, 3)[page, off]
        if case["fp8"]:
            x = x * s[name + "s"].double().permute(0, 2, 1)[page, off].unsqueeze(-1)
        return x

    if op == "read":
        return values("k", s["slot"].long()), values("v", s["slot"].long())
    if op == "rope":
        T, hq, rot = case["T"], case["hq"], case["rot"]
        x = s["qkv"].double().reshape(T, hq + 2 * hkv, d)
        rows = []
        angle = s["pos"].double().unsqueeze(1) * torch.tensor(turns_per_position(case), dtype=torch.float64,
                                                              device=x.device)
        turn = torch.polar(torch.full_like(angle, magnitude(case)), 2 * math.pi * (angle - angle.floor()))
        for part, weight in ((x[:, :hq], s["qw"]), (x[:, hq:hq + hkv], s["kw"])):
            if weight is not None:
                part = part / (part.pow(2).sum(-1, keepdim=True) / d + EPS).sqrt() * weight.double()
            head = part[..., :rot]
            # pairs as complex numbers, turned
            pairs = head.unflatten(-1, (rot // 2, 2)) if case["inter"] else head.unflatten(-1, (2, rot // 2)).transpose(-1, -2)
            z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn.unsqueeze(1))
            z = z.flatten(-2) if case["inter"] else z.transpose(-1, -2).flatten(-2)
            rows.append(torch.cat([z, part[..., rot:]], -1))
        q, k, v = rows[0], rows[1], x[:, hq + hkv:]
        kept = (s["slot"] >= 0)
        if case["fp8"]:
            back = []
            for val in (k, v):
                scale = val.abs().amax(-1, keepdim=True).clamp_min(TINY) / E4M3_MAX
                back.append(nearest_e4m3(val / scale) * scale * kept[:, None, None])
            return q, back[0], back[1]
        out = []
        slot = s["slot"].long()[kept]
        for name, val in (("k", k), ("v", v)):
            c = s[name].double().permute(0, 2, 1, 3).reshape(-1, hkv, d).contiguous()
            c[slot] = val[kept]
            out.append(c.view(-1, case["page"], hkv, d).permute(0, 2, 1, 3).contiguous())
        return q, out[0], out[1]
    hq = case["hq"]
    outs = []
    at = 0
    if op == "prompt":
        x = s["qkv"].double().view(-1, hq + 2 * hkv, d)
        for n in s["lens"]:
            y = x[at:at + n]
            outs.append(exact_attention(case, y[:, :hq], y[:, hq:hq + hkv], y[:, hq + hkv:]))
            at += n
        return torch.cat(outs)
    for b, (n, L) in enumerate(s["seqs"]):
        j = torch.arange(L, device=s["q"].device)
        slot = s["table"].long()[b, torch.div(j, case["page"], rounding_mode="floor")] * case["page"] + j % case["page"]
        page, off = torch.div(slot, case["page"], rounding_mode="floor"), slot % case["page"]
        kv = []
        for name in ("k", "v"):
            y = s[name].transpose(1, 2)
            y = (y.contiguous().view(torch.uint8)[page, off].view(y.dtype) if case["fp8"] else y[page, off]).double()
            if case["fp8"]:
                y = y * s[name + "s"].transpose(1, 2)[page, off].double().unsqueeze(-1)
            kv.append(y)
        outs.append(exact_attention(case, s["q"][at:at + n].double(), kv[0], kv[1]))
        at += n
    return torch.cat(outs)
