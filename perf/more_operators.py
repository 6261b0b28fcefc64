"""Attention that reads less of a paged cache: which calls are timed, their plain forms and their definition
in 64 bits.

Operators: attention with a sliding window and a few first tokens that stay visible (sinks), over packed
prompts (mlora_attention) and over pages (mlora_paged_attention), and attention of a batch whose sequences
share long prefixes (mlora_prefix_attention).
"""
import math
import random

import torch

own = False

E4M3_MAX = 448.0
TINY = 2.0 ** -90          # smallest amax a scale is made from
SCORES = 1 << 28           # scores that the plain form holds at once


# ---- cases -------------------------------------------------------------------------------------
def listed():
    wide = dict(hq=32, hkv=8, d=128)
    return [
        # a handful of short prompts of uneven lengths, narrow heads
        dict(name="sink_prompt_short", op="prompt", lens="1,17,129,300,65,511,2", hq=16, hkv=4, d=64, window=64,
             sinks=4),
        # a prefill batch of 8 prompts of 2048 tokens
        dict(name="sink_prompt_8x2048", op="prompt", lens=",".join(["2048"] * 8), window=512, sinks=4, **wide),
        # one long document
        dict(name="sink_prompt_16384", op="prompt", lens="16384", window=4096, sinks=16, **wide),
        # one user, one token of a long conversation
        dict(name="sink_decode1", op="paged", new="1x1", lo=10007, hi=10007, spread=1, fp8=False, page=16, window=1020,
             sinks=4, **wide),
        # a decode batch of 64, some contexts shorter than the window
        dict(name="sink_decode64", op="paged", new="64x1", lo=1, hi=16384, spread=2, fp8=False, page=16, window=2048,
             sinks=4, **wide),
        # a decode batch of 256 over an 8-bit cache
        dict(name="sink_decode256_fp8", op="paged", new="256x1", lo=128, hi=8192, spread=3, fp8=True, page=32,
             window=1024, sinks=8, **wide),
        # 256 decode tokens and a 2048-token chunk of a long prompt
        dict(name="sink_mixed2304", op="paged", new="256x1,1x2048", lo=64, hi=4096, chunk_before=6000, spread=4,
             fp8=False, page=16, window=2048, sinks=4, **wide),
        # a few requests with one short system prompt
        dict(name="prefix_decode8", op="prefix", groups="8x1000", alone=0, new=1, chunk=0, lo=1, hi=60, spread=5,
             fp8=False, page=16, **wide),
        # a decode batch of 64 with one long system prompt
        dict(name="prefix_decode64", op="prefix", groups="64x4096", alone=0, new=1, chunk=0, lo=1, hi=1024, spread=6,
             fp8=False, page=16, **wide),
        # a decode batch of 256 over an 8-bit cache: four system prompts, one for each of four adapters, and
        # requests that share nothing
        dict(name="prefix_decode256_fp8", op="prefix", groups="100x2000,61x517,64x4099,23x1500", alone=8, new=1,
             chunk=0, lo=1, hi=700, spread=7, fp8=True, page=32, **wide),
        # drafted tokens: five new ones a sequence, two long prefixes, narrow heads
        dict(name="prefix_draft160", op="prefix", groups="20x8192,12x6001", alone=0, new=5, chunk=0, lo=5, hi=600,
             spread=8, hq=16, hkv=4, d=64, fp8=False, page=16),
        # 128 decode tokens behind a long prefix, and a request's first 1024 own tokens behind the same one
        dict(name="prefix_mixed1152", op="prefix", groups="129x8000", alone=0, new=1, chunk=1024, lo=1, hi=1000,
             spread=9, fp8=False, page=16, **wide),
    ]


def log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prompt", "paged", "paged", "prefix", "prefix", "prefix"])
    hkv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 3, 4, 7, 8]) if hkv < 8 else rng.choice([1, 2, 4])
    d = rng.choice([64, 128])
    heads = dict(hq=hkv * group, hkv=hkv, d=d)
    if op == "prompt":
        n = rng.randint(1, 9)
        lens = ",".join(str(log_int(rng, 1, 11000 // n)) for _ in range(n))
        return dict(op=op, lens=lens, window=log_int(rng, 1, 4096), sinks=log_int(rng, 1, 256), **heads)
    page = rng.choice([16, 32, 64])
    fp8 = rng.random() < 0.4
    hi = log_int(rng, 16, 16384)
    if op == "paged":
        new = "%dx%d" % (log_int(rng, 1, min(256, 1 + 400000 // hi)), rng.choice([1, 1, 1, 1, 2, 5]))
        if rng.random() < 0.35:
            new += ",1x%d" % log_int(rng, 2, 2048)
        return dict(op=op, new=new, lo=1, hi=hi, chunk_before=log_int(rng, 1, 6000), spread=rng.randrange(1 << 30),
                    fp8=fp8, page=page, window=log_int(rng, 1, 4096), sinks=log_int(rng, 1, 256), **heads)
    groups = []
    left = log_int(rng, 2, 128)
    for _ in range(rng.randint(1, 4)):
        n = rng.randint(1, max(1, left))
        groups.append("%dx%d" % (n, log_int(rng, 1, 8192)))
        left -= n
        if left <= 0:
            break
    new = rng.choice([1, 1, 1, 2, 5])
    chunk = log_int(rng, 2, 1024) if rng.random() < 0.25 else 0
    return dict(op=op, groups=",".join(groups), alone=rng.choice([0, 0, 3, 9]), new=new, chunk=chunk, lo=new,
                hi=max(new, log_int(rng, 8, 1024)), spread=rng.randrange(1 << 30), fp8=fp8, page=page, **heads)


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


def prefix_groups(case):
    """(sequences, shared tokens) of every group; the requests that share nothing are the last one."""
    out = [tuple(int(v) for v in part.split("x")) for part in case["groups"].split(",")]
    return out + ([(case["alone"], 0)] if case["alone"] else [])


def prefix_lens(case):
    """(new tokens, shared keys, keys) of every sequence, group after group; with a chunk, the first group's last
    sequence brings that many new tokens.  Requests of no group have longer contexts of their own."""
    r = random.Random(case["spread"])
    out = []
    for g, (count, shared) in enumerate(prefix_groups(case)):
        for i in range(count):
            new = case["new"]
            own_keys = r.randint(case["lo"], case["hi"])
            if g == 0 and i == count - 1 and case["chunk"]:
                new = own_keys = case["chunk"]
            out.append((new, shared, shared + own_keys * (1 if shared else 3)))
    return out


def seen(case, new, keys):
    """Pairs of a query and a key it sees, and the keys that any query sees (causal, window and sinks)."""
    window, sinks = case["window"], case["sinks"]
    pairs, first, last_sink = 0, keys, 0
    for i in range(new):
        p = keys - new + i
        lo = max(0, p - window + 1)
        pairs += max(0, p + 1 - lo) + max(0, min(sinks, lo, p + 1))
        if p >= 0:
            first = min(first, lo)
            last_sink = min(sinks, p + 1)
    return pairs, keys - first + min(last_sink, first)


def work(case):
    op, hkv, d = case["op"], case["hkv"], case["d"]
    per = d + 4 if case.get("fp8") else 2 * d
    size, pairs = 0, 0
    if op == "prefix":
        for new, shared, keys in prefix_lens(case):
            pairs += new * keys - new * (new - 1) // 2
            size += new * case["hq"] * d * 4 + (keys - shared) * 2 * hkv * per
        size += sum(shared for _, shared in prefix_groups(case)) * 2 * hkv * per
    else:
        for new, keys in ([(n, n) for n in prompt_lens(case)] if op == "prompt" else paged_lens(case)):
            p, k = seen(case, new, keys)
            pairs += p
            size += new * case["hq"] * d * 4 + k * 2 * hkv * per
    return {"bytes": size, "flops": 4 * d * case["hq"] * pairs}


# ---- inputs ------------------------------------------------------------------------------------
def to_e4m3(x):
    """fp32 [..., d] as e4m3 codes and one fp32 scale for each vector."""
    scale = x.abs().amax(-1, keepdim=True).clamp_min(TINY) / E4M3_MAX
    return (x / scale).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn), scale.squeeze(-1)


def filled_cache(case, pages, g, sink_rows=None, toward=None):
    """Keys and values of every page; keys at sink_rows (page, offset) lean toward the queries, as first tokens'
    keys do."""
    dev = "cuda"
    shape = (pages, case["hkv"], case["page"], case["d"])
    s = {}
    for n in ("k", "v"):
        x = torch.randn(shape, generator=g, device=dev, dtype=torch.bfloat16)
        if n == "k" and sink_rows is not None:
            page, off = sink_rows
            x[page, :, off] = (x[page, :, off] + 4 * toward).to(torch.bfloat16)
        if case["fp8"]:
            # tokens differ in size, as keys and values do
            x = x.float() * (0.25 + 2 * torch.rand(shape[:3] + (1,), generator=g, device=dev))
            s[n], s[n + "s"] = to_e4m3(x)
        else:
            s[n], s[n + "s"] = x, None
        del x
    return s


def starts(lens):
    out = [0]
    for n in lens:
        out.append(out[-1] + n)
    return out


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed * 7919 + 13)
    s = {"case": case}
    op, hq, hkv, d = case["op"], case["hq"], case["hkv"], case["d"]
    bf, i32 = torch.bfloat16, torch.int32
    # a direction that the queries share a little of
    toward = torch.randn(d, generator=g, device=dev)
    toward /= toward.square().mean().sqrt() * math.sqrt(d) / 4

    def queries(T):
        return (torch.randn(T, hq, d, generator=g, device=dev) + toward).to(bf)

    if op == "prompt":
        lens = prompt_lens(case)
        T = sum(lens)
        # q, k and v lie in the merged layer's rows
        s["qkv"] = torch.randn(T, (hq + 2 * hkv) * d, generator=g, device=dev, dtype=bf)
        x = s["qkv"].view(T, hq + 2 * hkv, d)
        for i in range(0, T, 1024):
            x[i:i + 1024, :hq] = (x[i:i + 1024, :hq] + toward).to(bf)
        s["lens"] = lens
        at = starts(lens)
        for i, n in zip(at, lens):
            n = min(n, case["sinks"])
            x[i:i + n, hq:hq + hkv] = (x[i:i + n, hq:hq + hkv] + 4 * toward).to(bf)
        s["cu"] = torch.tensor(at, device=dev, dtype=i32)
        s["out"] = torch.empty(T, hq, d, device=dev, dtype=bf)
        s["max_len"] = max(lens)
        return s
    page = case["page"]
    if op == "paged":
        seqs = paged_lens(case)
        need = [(n + page - 1) // page for _, n in seqs]
        pages = sum(need) + 3
        order = torch.randperm(pages, generator=g, device=dev).cpu()
        table = torch.zeros(len(seqs), max(need) + 1, dtype=i32)
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = order[at:at + n]
            at += n
        sink = [(int(table[b, j // page]), j % page) for b, (_, n) in enumerate(seqs) for j in range(min(n, case["sinks"]))]
        rows = torch.tensor(sink, device=dev)
        s.update(filled_cache(case, pages, g, (rows[:, 0], rows[:, 1]), toward))
        s["seqs"] = seqs
    else:
        lens = prefix_lens(case)
        groups = prefix_groups(case)
        # a group's sequences share the whole pages of the prefix and copy its last, part filled one
        need = [(n + page - 1) // page for _, _, n in lens]
        pages = sum(n - shared // page for n, (_, shared, _) in zip(need, lens)) + sum(p // page for _, p in groups) + 3
        order = torch.randperm(pages, generator=g, device=dev).cpu()
        table = torch.zeros(len(lens), max(need) + 1, dtype=i32)
        copies = []
        at = b = 0
        for count, shared in groups:
            whole = shared // page
            common = order[at:at + whole]
            at += whole
            for i in range(count):
                table[b, :whole] = common
                table[b, whole:need[b]] = order[at:at + need[b] - whole]
                if i and shared % page:
                    copies.append((int(table[b - i, whole]), int(table[b, whole]), shared % page))
                at += need[b] - whole
                b += 1
        s.update(filled_cache(case, pages, g))
        for n in ("k", "v"):
            for a, b, count in copies:
                x = s[n].view(torch.uint8) if case["fp8"] else s[n]
                x[b, :, :count] = x[a, :, :count]
                if case["fp8"]:
                    s[n + "s"][b, :, :count] = s[n + "s"][a, :, :count]
        s["seqs"] = [(n, keys) for n, _, keys in lens]
        s["group_start"] = torch.tensor(starts([n for n, _ in groups]), device=dev, dtype=i32)
        s["prefix_len"] = torch.tensor([p for _, p in groups], device=dev, dtype=i32)
        s["max_prefix"] = max(p for _, p in groups)
    new = [n for n, _ in s["seqs"]]
    T = sum(new)
    s["table"] = table.to(dev)
    s["q"] = queries(T)
    s["cu"] = torch.tensor(starts(new), device=dev, dtype=i32)
    s["len"] = torch.tensor([n for _, n in s["seqs"]], device=dev, dtype=i32)
    s["out"] = torch.empty(T, hq, d, device=dev, dtype=bf)
    s["max_new"] = max(new)
    s["max_len"] = max(n for _, n in s["seqs"])
    if own:
        from lora_serving_amd import mlora
        s["cache"] = mlora.Cache(s["k"], s["v"], s["ks"], s["vs"])
        n = len(new)
        if op == "paged":
            s["ws"] = mlora.paged_workspace(T, n, hq, hkv, d, s["max_new"], s["max_len"])
        else:
            s["ws"] = mlora.prefix_workspace(T, n, len(s["prefix_len"]), hq, hkv, d, s["max_new"], s["max_len"],
                                             s["max_prefix"])
    return s


# ---- plain forms -------------------------------------------------------------------------------
def plain_rows(q, k, v, off):
    """q [m, hq, d], k and v [L, hkv, d] in 32 bits, off [m, L]: true where a query does not see a key."""
    m, hq, d = q.shape
    L, hkv = k.shape[0], k.shape[1]
    group = hq // hkv
    kt, vt = k.permute(1, 2, 0).contiguous(), v.permute(1, 0, 2).contiguous()
    qs = q.reshape(m, hkv, group, d).permute(1, 2, 0, 3).reshape(hkv, group * m, d)
    sc = torch.bmm(qs, kt).view(hkv, group, m, L) / math.sqrt(d)
    sc.masked_fill_(off, -math.inf)
    top = sc.amax(-1, keepdim=True)
    e = (sc - top.masked_fill(top == -math.inf, 0.0)).exp_()
    total = e.sum(-1, keepdim=True)
    o = torch.bmm(e.view(hkv, group * m, L), vt).view(hkv, group, m, d)
    o = o / total.masked_fill(total == 0, 1.0)
    return o.permute(2, 0, 1, 3).reshape(m, hq, d)


def plain_sequence(case, q, L, keys, out):
    """One sequence: q [n, hq, d] in 32 bits, its L keys, of which keys(j) gives K and V at j, out bf16.  Only keys
    that some of the queries at hand see are taken."""
    n, hq, _ = q.shape
    window, sinks = case.get("window", 0), case.get("sinks", 0)
    span = min(L, window + sinks) if window else L
    step = max(1, SCORES // (hq * span), span // 2) if window else max(1, SCORES // (hq * L))
    while window and step > 1 and hq * step * (span + step) > SCORES:
        step = (step + 1) // 2
    for i in range(0, n, step):
        m = min(step, n - i)
        p = torch.arange(L - n + i, L - n + i + m, device=q.device)[:, None]
        lo = max(0, L - n + i - window + 1) if window else 0
        j = torch.arange(lo, L - n + i + m, device=q.device)
        if min(sinks, lo) > 0:
            j = torch.cat([torch.arange(0, min(sinks, lo), device=q.device), j])
        off = j[None] > p
        if window:
            off |= (j[None] <= p - window) & (j[None] >= sinks)
        k, v = keys(j)
        out[i:i + m] = plain_rows(q[i:i + m], k, v, off).to(torch.bfloat16)


def plain_prompt(s):
    case = s["case"]
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    x = s["qkv"].view(-1, hq + 2 * hkv, d)
    at = 0
    for n in s["lens"]:
        y = x[at:at + n].float()
        plain_sequence(case, y[:, :hq], n, lambda j: (y[j, hq:hq + hkv], y[j, hq + hkv:]), s["out"][at:at + n])
        at += n
    return s["out"]


def cached(s, name, slot):
    """Tokens of the cache in 32 bits, [n, heads, d]."""
    case = s["case"]
    page, off = slot // case["page"], slot % case["page"]
    if not case["fp8"]:
        return s[name][page, :, off].float()
    code = s[name].view(torch.uint8)[page, :, off].view(torch.float8_e4m3fn).float()
    return code * s[name + "s"][page, :, off][..., None]


def plain_paged(s):
    case = s["case"]
    at = 0
    for b, (n, L) in enumerate(s["seqs"]):
        def keys(j):
            slot = s["table"][b].long()[j // case["page"]] * case["page"] + j % case["page"]
            return cached(s, "k", slot), cached(s, "v", slot)
        plain_sequence(case, s["q"][at:at + n].float(), L, keys, s["out"][at:at + n])
        at += n
    return s["out"]


def run(s):
    case = s["case"]
    op, hq, hkv, d = case["op"], case["hq"], case["hkv"], case["d"]
    if not own:
        return plain_prompt(s) if op == "prompt" else plain_paged(s)
    from lora_serving_amd import mlora
    if op == "prompt":
        x = s["qkv"].view(-1, hq + 2 * hkv, d)
        mlora.mlora_attention(x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], s["cu"], s["out"], max_q=s["max_len"],
                              window=case["window"], sinks=case["sinks"])
    elif op == "paged":
        mlora.mlora_paged_attention(s["q"], s["cache"], s["table"], s["cu"], s["len"], s["out"], max_q=s["max_new"],
                                    max_kv=s["max_len"], window=case["window"], sinks=case["sinks"], ws=s["ws"])
    else:
        mlora.mlora_prefix_attention(s["q"], s["cache"], s["table"], s["cu"], s["len"], s["group_start"],
                                     s["prefix_len"], s["out"], max_q=s["max_new"], max_kv=s["max_len"],
                                     max_prefix=s["max_prefix"], ws=s["ws"])
    return s["out"]


# ---- the definition in 64 bits -----------------------------------------------------------------
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
        see = key[None] <= p
        if case["op"] != "prefix":
            see = see & ((key[None] + case["window"] > p) | (key[None] < case["sinks"]))
        for h in range(hq):
            kv = h * hkv // hq
            sc = (q[i:i + rows, h] @ k[:, kv].t().contiguous()) * (d ** -0.5)
            w = torch.softmax(torch.where(see, sc, torch.full_like(sc, -math.inf)), -1)
            out[i:i + rows, h] = torch.where(see, w, torch.zeros_like(w)) @ v[:, kv].contiguous()
    return out


def exact(case, seed):
    s = prepare(case, seed)
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    outs = []
    at = 0
    if case["op"] == "prompt":
        x = s["qkv"].double().view(-1, hq + 2 * hkv, d)
        for n in s["lens"]:
            y = x[at:at + n]
            outs.append(exact_attention(case, y[:, :hq], y[:, hq:hq + hkv], y[:, hq + hkv:]))
            at += n
        return torch.cat(outs)
    for b, (n, L) in enumerate(s["seqs"]):
        # whole pages, [tokens, heads, d]
        page = s["table"][b, :(L + case["page"] - 1) // case["page"]].long()
        kv = []
        for name in ("k", "v"):
            y = s[name].view(torch.uint8)[page].view(s[name].dtype).double()
            if case["fp8"]:
                y = y * s[name + "s"][page].double().unsqueeze(-1)
            kv.append(y.transpose(1, 2).reshape(-1, hkv, d)[:L])
        outs.append(exact_attention(case, s["q"][at:at + n].double(), kv[0], kv[1]))
        at += n
    return torch.cat(outs)
