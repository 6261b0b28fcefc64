"""The attention step on the GPU against plain implementations in 64 bits on the CPU.

Tolerances count roundings: bf16 is off by at most 2^-8 of the value and e4m3 by 2^-4 (half a step
relative to the value, torch.finfo(t).eps / 2), sums and exponentials are fp32.
"""
import math

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

BF = 2.0 ** -8
E4M3 = 2.0 ** -4
# sine and cosine of a turn: the fraction of a turn is kept to 2^-25 relative (2 pi 2^-26 of the circle), the
# instruction's own error is below 2^-18
TRIG = 2.0 ** -17


@pytest.fixture(scope="module")
def m():
    from lora_serving_amd import mlora
    return mlora


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def randn(g, *shape):
    return torch.randn(*shape, generator=g).to(torch.bfloat16)


# ---- norm, rotation, cache ---------------------------------------------------------------------
def e4m3_values(x, scale):
    """Nearest e4m3 value of x / scale (64 bits)."""
    a = (x / scale).abs().clamp_max(448.0)
    step = torch.exp2(torch.floor(torch.log2(a.clamp_min(2.0 ** -20))).clamp_min(-6.0) - 3.0)
    return torch.sign(x) * torch.round(a / step) * step


def ref_rope(x, weight, eps, pos, turns, rot, inter, mag):
    """x [T, heads, d] fp64 -> (rotated, a bound of its fp32 error)."""
    if weight is not None:
        x = x * (x.square().mean(-1, keepdim=True) + eps).rsqrt() * weight
    # the table's integers, exactly: 2^64 = one turn
    frac = torch.tensor([[((int(p) * (int(t) % 2 ** 64)) % 2 ** 64) / 2.0 ** 64 for t in turns] for p in pos],
                        dtype=torch.float64).reshape(len(pos), -1)
    cos, sin = [mag * f(2 * math.pi * frac)[:, None] for f in (torch.cos, torch.sin)]
    y, err = x.clone(), 2.0 ** -20 * x.abs()
    if rot:
        ia = torch.arange(0, rot, 2) if inter else torch.arange(rot // 2)
        ib = ia + 1 if inter else ia + rot // 2
        a, b = x[..., ia], x[..., ib]
        y[..., ia] = a * cos - b * sin
        y[..., ib] = b * cos + a * sin
        for i in (ia, ib):
            err[..., i] = (TRIG + 2.0 ** -20) * mag * (a.abs() + b.abs())
    return y, err


ROPE_CASES = [
    # T, hq, hkv, d, rot, inter, norm, fp8, page, far, magnitude
    (1, 1, 1, 64, 64, False, True, False, 16, 10, 1.0),
    (5, 4, 2, 128, 128, False, True, False, 16, 1000, 1.0),
    (67, 7, 7, 64, 32, False, False, False, 32, 100000, 1.2),
    (33, 6, 2, 128, 96, False, True, True, 64, 2 ** 31 - 1, 1.0),
    (40, 5, 1, 128, 64, True, True, True, 16, 1000000, 0.7),
    (130, 8, 8, 64, 16, True, False, True, 256, 5000, 1.0),
    (21, 3, 3, 64, 0, False, True, False, 16, 100, 1.0),
    (300, 32, 8, 128, 128, True, False, False, 128, 30000, 1.0),
]


@pytest.mark.parametrize("case", ROPE_CASES, ids=lambda c: "-".join(str(v) for v in c))
def test_qk_rope_and_cache(m, case):
    T, hq, hkv, d, rot, inter, norm, fp8, page, far, mag = case
    g = gen(T * 31 + d)
    width = (hq + 2 * hkv) * d
    qkv = randn(g, T, width + 8)                      # rows lie apart
    pos = torch.randint(-5, far, (T,), generator=g, dtype=torch.int64).to(torch.int32)
    qw, kw = (1 + 0.3 * randn(g, d).float()).to(torch.bfloat16), (1 + 0.3 * randn(g, d).float()).to(torch.bfloat16)
    if not norm:
        qw = kw = None
    pages = (T + page - 1) // page + 2
    slot = torch.randperm(pages * page, generator=g)[:T].to(torch.int32)
    if T > 4:
        slot[1], slot[3] = -1, pages * page           # stored nowhere
    turns = m.mlora_rope_turns(max(rot, 2), 10000.0)
    dev = "cuda"
    r = m.Rope(turns.to(dev) if rot else None, rot, interleaved=inter, magnitude=mag)
    kind = torch.float8_e4m3fn if fp8 else torch.bfloat16
    shape = (pages, hkv, page, d)
    fill = 1.5
    kc, vc = [torch.full(shape, fill, device=dev, dtype=torch.bfloat16).to(kind) for _ in range(2)]
    ks, vs = [torch.full(shape[:3], 2.0, device=dev) if fp8 else None for _ in range(2)]
    c = m.Cache(kc, vc, ks, vs)
    q = torch.empty(T, hq, d, device=dev, dtype=torch.bfloat16)
    k = torch.empty(T, hkv, d, device=dev, dtype=torch.bfloat16)
    dq = qkv.to(dev)
    up = lambda w: None if w is None else w.to(dev)  # noqa: E731
    m.mlora_qk_rope(dq[:, :width], hq, hkv, d, pos.to(dev), r, q, k_out=k, q_weight=up(qw), k_weight=up(kw), eps=1e-5,
                    cache=c, slot=slot.to(dev))
    kb, vb = torch.empty_like(k), torch.empty_like(k)
    m.mlora_cache_read(c, slot.to(dev), kb, vb)
    # again without a cache, in place
    dq2 = qkv.to(dev)
    rows = dq2[:, :width].unflatten(1, (hq + 2 * hkv, d))
    m.mlora_qk_rope(dq2[:, :width], hq, hkv, d, pos.to(dev), r, rows[:, :hq], k_out=rows[:, hq:hq + hkv],
                    q_weight=up(qw), k_weight=up(kw), eps=1e-5)
    torch.cuda.synchronize()
    assert torch.equal(rows[:, :hq], q) and torch.equal(rows[:, hq:hq + hkv], k)
    assert torch.equal(rows[:, hq + hkv:].cpu(), qkv[:, :width].unflatten(1, (-1, d))[:, hq + hkv:])

    x = qkv[:, :width].double().unflatten(1, (hq + 2 * hkv, d))
    wq, wk = (None, None) if not norm else (qw.double(), kw.double())
    rq, eq = ref_rope(x[:, :hq], wq, 1e-5, pos, turns, rot, inter, mag)
    rk, ek = ref_rope(x[:, hq:hq + hkv], wk, 1e-5, pos, turns, rot, inter, mag)
    rv = x[:, hq + hkv:]
    for got, ref, err in ((q, rq, eq), (k, rk, ek)):
        assert ((got.cpu().double() - ref).abs() <= BF * ref.abs() + (1 + BF) * err + 1e-30).all()
    stored = (slot >= 0) & (slot < pages * page)
    assert (kb.cpu()[~stored] == 0).all() and (vb.cpu()[~stored] == 0).all()
    if fp8:
        for got, ref, err in ((kb, rk, ek), (vb, rv, torch.zeros_like(rv))):
            ref, err, got = ref[stored], err[stored], got.cpu().double()[stored]
            scale = ref.abs().amax(-1, keepdim=True) / 448.0
            tol = (E4M3 + 2 * BF) * (ref.abs() + err) + err + 2.0 ** -10 * scale * (1 + BF)
            assert ((got - ref).abs() <= tol).all()
        # values are not rotated: away from a tie the code is the nearest one
        scale = (rv[stored].abs().amax(-1, keepdim=True) / 448.0).float().double()
        near = e4m3_values(rv[stored], scale * (1 + 2.0 ** -20))
        same = near == e4m3_values(rv[stored], scale * (1 - 2.0 ** -20))
        want = (near * scale).to(torch.bfloat16)
        diff = (want.double() - vb.cpu()[stored].double()).abs()
        assert (diff[same] <= BF * want[same].double().abs()).all()
    else:
        assert torch.equal(kb.cpu()[stored], k.cpu()[stored])
        assert torch.equal(vb.cpu()[stored], qkv[:, :width].unflatten(1, (-1, d))[:, hq + hkv:][stored])
    # slots that no token names keep what they held
    untouched = torch.ones(pages * page, dtype=torch.bool)
    untouched[slot[stored].long()] = False
    flat = kc.float().cpu().permute(0, 2, 1, 3).reshape(pages * page, hkv, d)
    assert (flat[untouched] == torch.tensor(fill)).all()


def test_rope_is_exact_at_far_positions(m):
    """Position p + 1 from p by one more turn of each pair: the angle does not lose bits with p."""
    d, dev = 64, "cuda"
    turns = m.mlora_rope_turns(d, 10000.0)
    x = torch.ones(4, 3 * d, dtype=torch.bfloat16)
    pos = torch.tensor([3, 2 ** 20 + 7, 2 ** 30 + 1, 2 ** 31 - 1], dtype=torch.int32)
    q = torch.empty(4, 1, d, device=dev, dtype=torch.bfloat16)
    m.mlora_qk_rope(x.to(dev), 1, 1, d, pos.to(dev), m.Rope(turns.to(dev), d), q)
    ref, err = ref_rope(torch.ones(4, 1, d, dtype=torch.float64), None, 0.0, pos, turns, d, False, 1.0)
    assert ((q.cpu().double() - ref).abs() <= BF * ref.abs() + err * (1 + BF)).all()


def test_e4m3_cache_of_zeros_and_extremes(m):
    """A zero vector comes back as zeros; tiny and huge vectors keep their size."""
    d, dev = 64, "cuda"
    v = torch.zeros(4, d, dtype=torch.bfloat16)
    v[1] = torch.linspace(-1, 1, d).to(torch.bfloat16) * 2.0 ** -80
    v[2] = torch.linspace(-1, 1, d).to(torch.bfloat16) * 2.0 ** 120
    v[3, 5] = 1.0
    qkv = torch.cat([torch.zeros(4, d, dtype=torch.bfloat16), v, v], 1).to(dev)
    z = lambda: torch.zeros(1, 1, 16, d, device=dev, dtype=torch.bfloat16).to(torch.float8_e4m3fn)  # noqa: E731
    c = m.Cache(z(), z(), torch.zeros(1, 1, 16, device=dev), torch.zeros(1, 1, 16, device=dev))
    slot = torch.arange(4, dtype=torch.int32, device=dev)
    q = torch.empty(4, 1, d, device=dev, dtype=torch.bfloat16)
    m.mlora_qk_rope(qkv, 1, 1, d, slot, m.Rope(None, 0), q, cache=c, slot=slot)
    kb, vb = torch.empty_like(q), torch.empty_like(q)
    m.mlora_cache_read(c, slot, kb, vb)
    ref = v.double()[:, None]
    tol = (E4M3 + 2 * BF) * ref.abs() + 2.0 ** -10 * ref.abs().amax(-1, keepdim=True) / 448
    for got in (kb, vb):
        assert ((got.cpu().double() - ref).abs() <= tol).all()


# ---- attention ---------------------------------------------------------------------------------
def ref_attention(q, k, v, causal, window, scale):
    """q [n, hq, d], k, v [L, hkv, d] fp64 -> out, lse, sum p |v|, largest sum of |scale q k|.  What is masked
    is left out of the sums, not multiplied by zero."""
    n, hq, d = q.shape
    L, hkv = k.shape[:2]
    out, mag = torch.zeros_like(q), torch.zeros_like(q)
    lse = torch.full((n, hq), -math.inf, dtype=torch.float64)
    big = torch.zeros(n, hq, dtype=torch.float64)
    for i in range(n):
        p = L - n + i
        hi = min(L, p + 1) if causal else L
        lo = max(0, p - window + 1) if window else 0
        if hi <= lo:
            continue
        kk = k[lo:hi].repeat_interleave(hq // hkv, 1)
        vv = v[lo:hi].repeat_interleave(hq // hkv, 1)
        s = (kk * q[i]).sum(-1) * scale                       # [keys, hq]
        big[i] = ((kk * q[i]).abs().sum(-1) * scale).amax(0)
        lse[i] = torch.logsumexp(s, 0)
        w = torch.exp(s - lse[i])
        out[i] = (w[..., None] * vv).sum(0)
        mag[i] = (w[..., None] * vv.abs()).sum(0)
    return out, lse, mag, big


def check(got, ref, mag, big):
    """Probabilities rounded to bf16, the result rounded to bf16; scores in fp32 (d products each, and the
    scaling to a power of two), exponentials to 2^-21."""
    rel = 2 * 2.0 ** -23 * (big[..., None] + 16) * 4
    tol = (BF + rel) * mag + BF * ref.abs() + BF * BF * mag + 1e-30
    bad = ~((got.cpu().double() - ref).abs() <= tol)        # (a NaN is bad)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()}, worst " \
                          f"{float(((got.cpu().double() - ref).abs() / tol).max()):.2f} of the tolerance"


def check_lse(got, ref, big):
    empty = ref == -math.inf
    assert torch.equal(got.cpu() == -math.inf, empty)
    tol = 2.0 ** -20 * (4 + big + ref.abs())
    assert ((got.cpu().double() - ref).abs()[~empty] <= tol[~empty]).all()


PROMPTS = [
    # lens of queries, lens of keys (None: the same), hq, hkv, d, causal, window
    ([1], None, 1, 1, 64, True, 0),
    ([1, 0, 2, 63, 64, 65], None, 4, 2, 64, True, 0),
    ([127, 129, 5], None, 4, 1, 128, True, 0),
    ([300], None, 6, 2, 128, False, 0),
    ([200, 31], None, 14, 2, 64, True, 17),
    ([150], None, 8, 8, 128, True, 64),
    ([90, 40], None, 2, 1, 64, False, 33),
    ([5, 100, 70], [0, 160, 30], 4, 2, 128, True, 0),      # no keys, more keys, fewer keys than queries
    ([100, 3], [400, 131], 3, 1, 64, False, 0),
    ([70, 9], [200, 64], 4, 4, 128, True, 1),
    ([40], None, 35, 5, 64, True, 0),
    ([257], None, 16, 1, 128, True, 100),
]


@pytest.mark.parametrize("case", PROMPTS, ids=lambda c: "-".join(str(v) for v in c).replace(" ", ""))
def test_prompts(m, case):
    lq, lk, hq, hkv, d, causal, window = case
    lk = lq if lk is None else lk
    g = gen(sum(lq) + 7 * hq + d)
    Tq, Tk = sum(lq), sum(lk)
    q = randn(g, Tq, hq * d + 16)[:, 8:8 + hq * d].unflatten(1, (hq, d))     # rows lie apart
    kv = randn(g, Tk, 2 * hkv, d)
    cu = lambda n: torch.tensor([sum(n[:i]) for i in range(len(n) + 1)], dtype=torch.int32)  # noqa: E731
    scale = 0.17
    dev = "cuda"
    dkv = kv.to(dev)
    base = torch.empty(Tq, hq * d + 16, device=dev, dtype=torch.bfloat16)
    base[:, 8:8 + hq * d] = q.reshape(Tq, -1).to(dev)
    dq = base[:, 8:8 + hq * d].unflatten(1, (hq, d))
    out = torch.full((Tq, hq, d), 7.0, device=dev, dtype=torch.bfloat16)
    lse = torch.full((Tq, hq), 7.0, device=dev)
    m.mlora_attention(dq, dkv[:, :hkv], dkv[:, hkv:], cu(lq).to(dev), out, cu_k=cu(lk).to(dev), max_q=max(lq),
                      causal=causal, window=window, scale=scale, lse=lse)
    torch.cuda.synchronize()
    a = c = 0
    for n, L in zip(lq, lk):
        ref, rl, mag, big = ref_attention(q[a:a + n].double(), kv[c:c + L, :hkv].double(), kv[c:c + L, hkv:].double(),
                                          causal, window, scale)
        if n:
            check(out[a:a + n], ref, mag, big)
            check_lse(lse[a:a + n], rl, big)
        a, c = a + n, c + L


def paged_batch(m, g, seqs, hkv, d, page, fp8, poison=False):
    """Random cache pages for sequences of (queries, keys): the cache, the table, and the K, V values of each
    sequence in 64 bits."""
    dev = "cuda"
    need = [(L + page - 1) // page for _, L in seqs]
    pages = sum(need) + 2
    shape = (pages, hkv, page, d)
    raw = [torch.randn(shape, generator=g) * (0.3 + torch.rand(shape[:3] + (1,), generator=g)) for _ in range(2)]
    order = torch.randperm(pages, generator=g)
    table = torch.full((len(seqs), max(need + [0]) + 2), 10 ** 6, dtype=torch.int32)    # unreached: out of range
    at, vals, live = 0, [], torch.zeros(pages, page, dtype=torch.bool)
    for b, (n, (_, L)) in enumerate(zip(need, seqs)):
        table[b, :n] = order[at:at + n]
        at += n
        j = torch.arange(L)
        live[table[b, j // page].long(), j % page] = True
    if fp8:
        store = [x.to(torch.float8_e4m3fn) for x in raw]
        sc = [0.1 + torch.rand(shape[:3], generator=g) for _ in range(2)]
        value = [x.double() * s[..., None].double() for x, s in zip(store, sc)]
    else:
        store, sc = [x.to(torch.bfloat16) for x in raw], [None, None]
        value = [x.double() for x in store]
    if poison:      # slots that no token fills hold anything
        for i in range(2):
            bad = (~live)[:, None, :, None].expand(shape)
            x = store[i].float()
            x[bad] = math.nan
            store[i] = x.to(store[i].dtype)
            if fp8:
                sc[i][(~live)[:, None].expand(shape[:3])] = math.nan
    for b, (_, L) in enumerate(seqs):
        j = torch.arange(L)
        pg = table[b, j // page].long()
        vals.append([x[pg, :, j % page] for x in value])
    up = lambda t: None if t is None else t.to(dev)  # noqa: E731
    return m.Cache(up(store[0]), up(store[1]), up(sc[0]), up(sc[1])), table, vals


PAGED = [
    # (queries, keys) of the sequences, hq, hkv, d, page, fp8, causal, window
    ([(1, 1)], 1, 1, 64, 16, False, True, 0),
    ([(1, 1), (1, 0), (1, 17), (1, 333), (0, 5), (1, 32)], 4, 2, 128, 16, False, True, 0),
    ([(1, 1000), (1, 31), (1, 512)], 8, 1, 64, 32, True, True, 0),
    ([(1, 700), (1, 129), (1, 64)], 4, 4, 128, 64, True, True, 50),
    ([(1, 600), (1, 4)], 6, 2, 64, 16, False, True, 100),
    ([(4, 300), (3, 3), (4, 2), (1, 77)], 8, 2, 128, 16, False, True, 0),      # 16 rows; fewer keys than queries
    ([(5, 200), (2, 90)], 12, 2, 128, 32, True, True, 0),                     # 30 rows
    ([(8, 140), (8, 8)], 4, 1, 64, 256, False, True, 9),
    ([(5, 100)], 4, 1, 64, 16, False, False, 0),
    ([(1, 500), (40, 300), (1, 20), (130, 130)], 4, 2, 128, 16, False, True, 0),       # decode and chunks
    ([(33, 900), (1, 100), (70, 70)], 8, 2, 128, 32, True, True, 0),
    ([(100, 613), (1, 64)], 3, 1, 64, 16, False, True, 75),
    ([(64, 257), (5, 0)], 40, 2, 64, 64, True, True, 0),                      # groups wider than a tile
    ([(1, 3000)], 8, 2, 128, 16, False, True, 0),                             # split over keys
    ([(1, 2500), (1, 40)], 16, 1, 64, 16, True, True, 700),
    ([(20, 2000)], 8, 4, 128, 16, False, True, 0),
    ([(50, 1500)], 4, 1, 64, 32, True, True, 600),
]


@pytest.mark.parametrize("poison", [False, True], ids=["", "poison"])
@pytest.mark.parametrize("case", PAGED, ids=lambda c: "-".join(str(v) for v in c).replace(" ", ""))
def test_paged(m, case, poison):
    seqs, hq, hkv, d, page, fp8, causal, window = case
    g = gen(sum(L for _, L in seqs) + 13 * hq + d)
    c, table, vals = paged_batch(m, g, seqs, hkv, d, page, fp8, poison)
    T = sum(n for n, _ in seqs)
    dev = "cuda"
    q = randn(g, T, hq, d)
    cu = torch.tensor([sum(n for n, _ in seqs[:i]) for i in range(len(seqs) + 1)], dtype=torch.int32)
    lens = torch.tensor([L for _, L in seqs], dtype=torch.int32)
    mq, mk = max(n for n, _ in seqs), max(L for _, L in seqs)
    assert m.mlora_validate_pages(c, table, cu, lens, T, mq, mk) == (m.MLORA_OK, 0)
    out = torch.full((T, hq, d), 7.0, device=dev, dtype=torch.bfloat16)
    lse = torch.full((T, hq), 7.0, device=dev)
    ws = m.paged_workspace(T, len(seqs), hq, hkv, d, mq, mk)
    ws.fill_(255)                                      # NaN in every word
    m.mlora_paged_attention(q.to(dev), c, table.to(dev), cu.to(dev), lens.to(dev), out, mq, mk, causal=causal,
                            window=window, lse=lse, ws=ws)
    torch.cuda.synchronize()
    at = 0
    for (n, L), (k, v) in zip(seqs, vals):
        ref, rl, mag, big = ref_attention(q[at:at + n].double(), k, v, causal, window, d ** -0.5)
        if n:
            check(out[at:at + n], ref, mag, big)
            check_lse(lse[at:at + n], rl, big)
        at += n


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_unseen_values_have_no_effect(m, d, bad):
    """An infinity or NaN in the K or V of a key reaches only the queries that see the key."""
    g = gen(d)
    n, hq, hkv, dev = 150, 4, 2, "cuda"
    q, k, v = randn(g, n, hq, d), randn(g, n, hkv, d), randn(g, n, hkv, d)
    at = 77
    cu = torch.tensor([0, n], dtype=torch.int32, device=dev)
    outs = []
    for poison in (False, True):
        kk, vv = k.clone(), v.clone()
        if poison:
            vv[at, :, 3] = bad
            kk[at, :, 5] = bad
        out = torch.empty(n, hq, d, device=dev, dtype=torch.bfloat16)
        m.mlora_attention(q.to(dev), kk.to(dev), vv.to(dev), cu, out)
        win = torch.empty_like(out)
        m.mlora_attention(q.to(dev), kk.to(dev), vv.to(dev), cu, win, window=20)
        # the same keys as a cache, the queries in chunks of 4 (decode) and of 50
        page = 16
        pages = (n + page - 1) // page
        kc, vc = [torch.zeros(pages * page, hkv, d, dtype=torch.bfloat16) for _ in range(2)]
        kc[:n], vc[:n] = kk, vv
        c = m.Cache(*[x.view(pages, page, hkv, d).permute(0, 2, 1, 3).contiguous().to(dev) for x in (kc, vc)])
        table = torch.arange(pages, dtype=torch.int32, device=dev)[None]
        parts = []
        for step in (4, 50):
            for i in range(0, 100, step):
                o = torch.empty(step, hq, d, device=dev, dtype=torch.bfloat16)
                m.mlora_paged_attention(q[i:i + step].to(dev), c, table,
                                        torch.tensor([0, step], dtype=torch.int32, device=dev),
                                        torch.tensor([i + step], dtype=torch.int32, device=dev), o, step, i + step,
                                        ws=m.paged_workspace(step, 1, hq, hkv, d, step, i + step))
                parts.append(o)
        torch.cuda.synchronize()
        outs.append([out.cpu(), win.cpu(), torch.cat(parts).cpu()])
    (a, aw, ap), (b, bw, bp) = outs
    seen = torch.arange(n) >= at
    assert torch.equal(a[~seen], b[~seen]) and b[seen].isnan().any(-1).all()
    seen_w = seen & (torch.arange(n) < at + 20)
    assert torch.equal(aw[~seen_w], bw[~seen_w]) and bw[seen_w].isnan().any(-1).all()
    seen_p = torch.cat([torch.arange(100), torch.arange(100)]) >= at
    assert torch.equal(ap[~seen_p], bp[~seen_p]) and bp[seen_p].isnan().any(-1).all()


LONG_PROMPTS = [
    # lens of queries, lens of keys (None: the same), hq, hkv, d, causal, window
    ([700], None, 4, 2, 128, True, 0),                # several tiles seen in full, one and two rows blocks at the edge
    ([390], None, 3, 3, 64, True, 0),
    ([33], [1000], 8, 2, 128, False, 0),
    ([300], None, 2, 1, 128, True, 150),              # full tiles between two edges
    ([130], [600], 2, 2, 64, False, 400),
    ([4] * 70 + [150], None, 2, 1, 64, True, 0),      # more than 64 sequences
    ([1, 260, 3], [5, 900, 2], 2, 1, 128, True, 2 ** 31 - 1),   # a window wider than any sequence
]


@pytest.mark.parametrize("case", LONG_PROMPTS, ids=lambda c: "-".join(str(v) for v in c).replace(" ", "")[:60])
def test_long_prompts(m, case):
    test_prompts(m, case)


LONG_PAGED = [
    # (queries, keys) of the sequences, hq, hkv, d, page, fp8, causal, window
    ([(1, 1 + 61 * i % 1500) for i in range(70)], 2, 1, 64, 16, False, True, 0),       # more than 64 sequences
    ([(1, 40 * i) for i in range(130)], 2, 2, 64, 32, True, True, 0),
    ([(1, 1200), (0, 0), (3, 0), (1, 5000), (2, 1), (4, 4)], 8, 2, 128, 16, False, True, 0),
    ([(1, 3000), (1, 1)], 8, 2, 128, 64, True, True, 2 ** 31 - 1),
    ([(3, 2), (1, 700)], 4, 2, 128, 16, False, True, 2 ** 31 - 1),                     # fewer keys than queries
    ([(7, 1500), (8, 900)], 8, 2, 128, 16, False, True, 0),                           # 32 rows, split
    ([(6, 1000)], 4, 1, 128, 32, True, False, 300),
    ([(150, 1300), (1, 900), (1, 30)], 4, 2, 128, 16, False, True, 0),                # chunks split too
    ([(140, 900)], 6, 2, 128, 32, True, True, 260),
    ([(129, 700)], 2, 2, 64, 64, True, False, 0),
    ([(1, 2000)] * 3, 48, 1, 64, 16, False, True, 0),                                  # a group of 48
]


@pytest.mark.parametrize("poison", [False, True], ids=["", "poison"])
@pytest.mark.parametrize("case", LONG_PAGED, ids=lambda c: "-".join(str(v) for v in c).replace(" ", "")[:60])
def test_long_paged(m, case, poison):
    test_paged(m, case, poison)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n,window", [(1, 0), (1, 100), (3, 0), (5, 90), (60, 0), (60, 130)])
def test_unseen_values_in_pages(m, n, window, d, fp8):
    """NaN in K, V and the scales of single keys reaches only the queries that see them, split or not."""
    g = gen(n + d + window)
    hq, hkv, page, dev, L = 4, 2, 16, "cuda", 900
    c, table, _ = paged_batch(m, g, [(n, L)], hkv, d, page, fp8)
    q = randn(g, n, hq, d).to(dev)
    ints = lambda *v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    ws = m.paged_workspace(n, 1, hq, hkv, d, n, L)
    pos = torch.arange(L - n, L)
    for key in (0, 100, L - window - 2, L - window, L - 33, L - 3, L - 2, L - 1):
        if not 0 <= key < L:
            continue
        outs = []
        old = [t.clone() for t in (c.k, c.v) + ((c.k_scale, c.v_scale) if fp8 else ())]
        for poison in (False, True):
            if poison:
                pg, at = int(table[0, key // page]), key % page
                for t in (c.k, c.v):
                    if fp8:
                        t.view(torch.uint8)[pg, :, at, 7] = 0x7f
                    else:
                        t[pg, :, at, 7] = math.nan
                if fp8:
                    c.k_scale[pg, :, at] = math.nan
                    c.v_scale[pg, :, at] = math.inf
            o = torch.empty(n, hq, d, device=dev, dtype=torch.bfloat16)
            m.mlora_paged_attention(q, c, table.to(dev), ints(0, n), ints(L), o, n, L, window=window, ws=ws)
            torch.cuda.synchronize()
            outs.append(o.cpu())
        for t, v in zip((c.k, c.v) + ((c.k_scale, c.v_scale) if fp8 else ()), old):
            t.copy_(v)
        seen = (pos >= key) & ((pos - window < key) if window else torch.ones(n, dtype=torch.bool))
        assert torch.equal(outs[0][~seen], outs[1][~seen])
        assert outs[1][seen].isnan().any(-1).all()


@pytest.mark.parametrize("window", [0, 200])
@pytest.mark.parametrize("d", [64, 128])
def test_unseen_values_in_long_prompts(m, d, window):
    """The same where a row block has tiles that it sees in full."""
    g = gen(d + window)
    n, hq, hkv, dev = 600, 2, 1, "cuda"
    q, k, v = randn(g, n, hq, d).to(dev), randn(g, n, hkv, d).to(dev), randn(g, n, hkv, d).to(dev)
    cu = torch.tensor([0, n], dtype=torch.int32, device=dev)
    good = torch.empty(n, hq, d, device=dev, dtype=torch.bfloat16)
    m.mlora_attention(q, k, v, cu, good, window=window)
    pos = torch.arange(n)
    for key in (0, 63, 64, 255, 300, 511, 599):
        kk, vv = k.clone(), v.clone()
        vv[key, 0, 11] = math.inf
        kk[key, 0, 2] = math.nan
        out = torch.empty_like(good)
        m.mlora_attention(q, kk, vv, cu, out, window=window)
        torch.cuda.synchronize()
        seen = (pos >= key) & ((pos - window < key) if window else torch.ones(n, dtype=torch.bool))
        assert torch.equal(out.cpu()[~seen], good.cpu()[~seen])
        assert out.cpu()[seen].isnan().any(-1).all()


def test_large_scores(m):
    """Scores of hundreds: the maximum is taken off before the exponential."""
    g = gen(3)
    n, hq, d, dev = 100, 2, 64, "cuda"
    q, k, v = randn(g, n, hq, d) * 8, randn(g, n, 1, d) * 8, randn(g, n, 1, d)
    cu = torch.tensor([0, n], dtype=torch.int32, device=dev)
    out = torch.empty(n, hq, d, device=dev, dtype=torch.bfloat16)
    lse = torch.empty(n, hq, device=dev)
    m.mlora_attention(q.to(dev), k.to(dev), v.to(dev), cu, out, lse=lse)
    ref, rl, mag, big = ref_attention(q.double(), k.double(), v.double(), True, 0, d ** -0.5)
    check(out, ref, mag, big)
    check_lse(lse, rl, big)


def test_pages_outside_the_cache_do_not_fault(m):
    """A page number outside the cache is read as the nearest page; the other sequences are answered."""
    g = gen(9)
    seqs, hq, hkv, d, page = [(1, 50), (1, 60), (40, 200)], 4, 2, 64, 16
    c, table, vals = paged_batch(m, g, seqs, hkv, d, page, False)
    table[1, 1], table[1, 2] = -7, 2 ** 31 - 1
    q = randn(g, 42, hq, d)
    cu = torch.tensor([0, 1, 2, 42], dtype=torch.int32)
    lens = torch.tensor([50, 60, 200], dtype=torch.int32)
    assert m.mlora_validate_pages(c, table, cu, lens, 42, 40, 200) == (m.MLORA_ERR_INDEX, -7)
    out = torch.empty(42, hq, d, device="cuda", dtype=torch.bfloat16)
    m.mlora_paged_attention(q.cuda(), c, table.cuda(), cu.cuda(), lens.cuda(), out, 40, 200,
                            ws=m.paged_workspace(42, 3, hq, hkv, d, 40, 200))
    torch.cuda.synchronize()
    for b, (lo, hi) in ((0, (0, 1)), (2, (2, 42))):
        ref, _, mag, big = ref_attention(q[lo:hi].double(), vals[b][0], vals[b][1], True, 0, d ** -0.5)
        check(out[lo:hi], ref, mag, big)


def test_binding_refusals(m):
    """Tensors of another shape, dtype, layout or device raise before anything is launched."""
    dev, bf = "cuda", torch.bfloat16
    new = lambda *s, t=bf: torch.zeros(s, device=dev, dtype=t)  # noqa: E731
    ints = lambda *v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    x, k, cu, out = new(5, 4, 64), new(5, 2, 64), ints(0, 5), new(5, 4, 64)
    c = m.Cache(new(2, 2, 16, 64), new(2, 2, 16, 64))
    rope = m.Rope(m.mlora_rope_turns(64).to(dev), 64)
    ws = m.paged_workspace(5, 1, 4, 2, 64, 5, 16)
    pos = ints(0, 1, 2, 3, 4)
    attend = lambda **a: m.mlora_attention(**{**dict(q=x, k=k, v=k, cu_q=cu, out=out), **a})  # noqa: E731
    paged = lambda **a: m.mlora_paged_attention(**{**dict(q=x, cache=c, page_table=ints(0)[None], cu_q=cu,  # noqa: E731
                                                          kv_len=ints(5), out=out, max_q=5, max_kv=16, ws=ws), **a})
    rotate = lambda **a: m.mlora_qk_rope(**{**dict(qkv=new(5, 512), n_q_heads=4, n_kv_heads=2, head_dim=64,  # noqa: E731
                                                   pos=pos, rope=rope, q_out=out), **a})
    read = lambda **a: m.mlora_cache_read(**{**dict(cache=c, slot=pos, k=k, v=k.clone()), **a})  # noqa: E731
    for call in (attend, paged, rotate, read):
        call()
    bad = [(attend, dict(q=x.float())), (attend, dict(q=x.cpu())), (attend, dict(q=x[0])), (attend, dict(q=None)),
           (attend, dict(q=new(5, 64, 4).transpose(1, 2))), (attend, dict(v=new(4, 2, 64))), (attend, dict(out=new(5, 4, 128))),
           (attend, dict(k=new(5, 2, 128), v=new(5, 2, 128))), (attend, dict(cu_q=cu.long())), (attend, dict(cu_k=ints(0, 2, 5))),
           (attend, dict(lse=new(5, 4))), (attend, dict(lse=new(5, 2, t=torch.float32))), (attend, dict(window=2 ** 31)),
           (paged, dict(kv_len=ints(5, 5))), (paged, dict(page_table=ints(0))), (paged, dict(q=new(5, 4, 128), out=new(5, 4, 128))),
           (paged, dict(ws=ws.cpu())), (paged, dict(cu_q=ints(0, 2, 5))),
           (rotate, dict(qkv=new(5, 500))), (rotate, dict(qkv=new(512, 5).t())), (rotate, dict(pos=ints(0, 1))),
           (rotate, dict(q_weight=new(128))), (rotate, dict(k_weight=new(64, t=torch.float32))), (rotate, dict(q_out=new(4, 4, 64))),
           (rotate, dict(k_out=new(5, 4, 64))), (rotate, dict(cache=c, slot=pos.long())),
           (read, dict(slot=pos.long())), (read, dict(k=new(5, 2, 32))), (read, dict(v=k.transpose(0, 1)))]
    for call, change in bad:
        with pytest.raises(ValueError):
            call(**change)
    for call, change in ((attend, dict(scale=-1.0)), (attend, dict(k=new(5, 3, 64), v=new(5, 3, 64))), (rotate, dict(cache=c))):
        with pytest.raises(m.MloraError):
            call(**change)
    with pytest.raises(TypeError):
        attend(max_q="5")
    torch.cuda.synchronize()


def test_streams_and_graph(m):
    """On a stream of its own and captured in a graph, replayed with eager work between: the eager bits."""
    g = gen(21)
    seqs, hq, hkv, d, page = [(1, 900), (1, 40), (1, 2000)], 8, 2, 128, 16
    c, table, _ = paged_batch(m, g, seqs, hkv, d, page, True)
    dev = "cuda"
    qkv = randn(g, 3, (hq + 2 * hkv) * d).to(dev)
    cu = torch.arange(4, dtype=torch.int32, device=dev)
    lens = torch.tensor([L for _, L in seqs], dtype=torch.int32, device=dev)
    pos = lens - 1
    slot = torch.tensor([int(table[b, (L - 1) // page]) * page + (L - 1) % page for b, (_, L) in enumerate(seqs)],
                        dtype=torch.int32, device=dev)
    r = m.Rope(m.mlora_rope_turns(d).to(dev), d)
    ws = m.paged_workspace(3, 3, hq, hkv, d, 1, 2000)
    dt = table.to(dev)
    q, out, outp = [torch.empty(3, hq, d, device=dev, dtype=torch.bfloat16) for _ in range(3)]
    kb, vb = [torch.empty(3, hkv, d, device=dev, dtype=torch.bfloat16) for _ in range(2)]

    def step():
        m.mlora_qk_rope(qkv, hq, hkv, d, pos, r, q, cache=c, slot=slot)
        m.mlora_cache_read(c, slot, kb, vb)
        m.mlora_paged_attention(q, c, dt, cu, lens, out, 1, 2000, ws=ws)
        m.mlora_attention(q, kb, vb, cu, outp, max_q=1)
        return [t.clone() for t in (q, kb, vb, out, outp)]

    eager = step()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        other = step()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(eager, other))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for _ in range(4):
        for t in (q, out, outp, kb, vb):
            t.fill_(3.0)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(eager, held))
        ws.fill_(255)
        torch.cuda.synchronize()


WHOLE_OR_SHARED = [
    # contexts of 5 to 9 units of 128 keys, with fewer (sequence, kv head) pairs than CUs and with as many; odd head
    # counts, for the heads' order turns with the sequence
    ([(1, 1 + 97 * i % 1024) for i in range(63)] + [(1, 1024)], 4, 4, 64, 16, False, True, 0),      # 256, whole
    ([(1, 1 + 97 * i % 1024) for i in range(84)] + [(1, 1024)], 3, 3, 64, 16, True, True, 0),       # 255, shared
    ([(1, 1 + 97 * i % 1024) for i in range(63)] + [(1, 1025)], 8, 4, 128, 16, True, True, 0),      # 256, 9 units
    ([(2, 2 + 61 * i % 900) for i in range(52)], 10, 5, 128, 32, False, True, 700),                 # 260, whole
    ([(1, 1280)] * 7, 14, 7, 128, 64, False, True, 0),                                              # equal, shared
    ([(1, 640)] * 40 + [(200, 900)], 14, 7, 64, 16, True, True, 0),                                 # and a chunk
]


@pytest.mark.parametrize("poison", [False, True], ids=["", "poison"])
@pytest.mark.parametrize("case", WHOLE_OR_SHARED, ids=lambda c: "-".join(str(v) for v in c).replace(" ", "")[-60:])
def test_paged_whole_or_shared(m, case, poison):
    test_paged(m, case, poison)


MANY_ITEMS = [
    # more row blocks than workgroups launched for them: 100 sequences of 5 tokens among 300 of one (in one kernel),
    # their keys cut into chunks or not, and with windows
    ([(1, 1 + i % 50) for i in range(300)] + [(5, 5 + i % 60) for i in range(100)], 64, 16, 64, 16, False, True, 0),
    ([(1, 1 + i % 50) for i in range(300)] + [(5, 5 + i % 60) for i in range(100)], 64, 16, 64, 16, True, True, 0),
    ([(17, 17 + 3 * i) if i % 5 == 0 else (1, 1 + i % 40) for i in range(200)], 32, 32, 128, 32, False, True, 0),
    ([(17, 17 + 7 * i % 400) if i % 9 == 4 else (1, 900) for i in range(170)], 24, 24, 64, 16, False, True, 150),
    ([(130, 300), (0, 0), (1, 40)] + [(1, 1 + i) for i in range(90)] + [(260, 260), (1, 7)], 8, 2, 128, 16, True, True, 0),
]


@pytest.mark.parametrize("poison", [False, True], ids=["", "poison"])
@pytest.mark.parametrize("case", MANY_ITEMS, ids=lambda c: "-".join(str(v) for v in c).replace(" ", "")[-60:])
def test_paged_many_items(m, case, poison):
    test_paged(m, case, poison)


def test_many_prompts(m):
    """More than 64 x 64 sequences: a lane counts more than one wave's worth."""
    test_prompts(m, ([1 + i % 3 for i in range(4200)] + [140], None, 1, 1, 64, True, 0))
