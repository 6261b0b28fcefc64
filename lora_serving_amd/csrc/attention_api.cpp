// C ABI of the attention step: argument checks, launch plans and dispatch.  Declarations and the
// contract of every entry point are in include/mlora.h.
#include <algorithm>
#include <cmath>
#include <cstring>

#include "abi.h"
#include "attention.h"
#include "kernels.h"

using namespace mlora;

namespace {

constexpr int64_t MAX_ROWS = INT64_C(1) << 31;   // query rows x heads: 32-bit row numbers
constexpr int64_t MAX_KEYS = INT64_C(1) << 30;   // tokens: positions and windows add up within 32 bits
constexpr int64_t MAX_STRIDE = INT64_C(1) << 24; // K and V rows: 64 of them within a 32-bit byte offset

bool head_dim_ok(int32_t d) { return d == 64 || d == 128; }

mlora_status check_heads(int32_t hq, int32_t hkv, int32_t d)
{
    if (hq < 1 || hkv < 1)
        return MLORA_ERR_ARG;
    if (hq > MLORA_MAX_HEADS || !head_dim_ok(d))
        return MLORA_ERR_UNSUPPORTED;
    return hq % hkv ? MLORA_ERR_SHAPE : MLORA_OK;
}

mlora_status check_cache_sizes(int64_t n_pages, int32_t hkv, int32_t page_size, int32_t d, int32_t dtype)
{
    if (n_pages < 1 || hkv < 1)
        return MLORA_ERR_ARG;
    if (page_size < 16 || page_size > MLORA_MAX_PAGE || (page_size & (page_size - 1)) || !head_dim_ok(d) ||
        hkv > MLORA_MAX_HEADS || (dtype != MLORA_CACHE_BF16 && dtype != MLORA_CACHE_E4M3) ||
        n_pages >= MAX_ROWS / page_size)
        return MLORA_ERR_UNSUPPORTED;
    return MLORA_OK;
}

mlora_status check_cache(const mlora_cache *c, CacheGeom *g)
{
    if (c == nullptr)
        return MLORA_ERR_ARG;
    const mlora_status st = check_cache_sizes(c->n_pages, c->n_kv_heads, c->page_size, c->head_dim, c->dtype);
    if (st != MLORA_OK)
        return st;
    if (c->k == nullptr || c->v == nullptr || !aligned16(c->k) || !aligned16(c->v))
        return MLORA_ERR_ARG;
    const bool fp8 = c->dtype == MLORA_CACHE_E4M3;
    if (fp8 && (c->k_scale == nullptr || c->v_scale == nullptr || !aligned16(c->k_scale) ||
                !aligned16(c->v_scale)))
        return MLORA_ERR_ARG;
    g->k = (uint8_t *)c->k;
    g->v = (uint8_t *)c->v;
    g->k_scale = c->k_scale;
    g->v_scale = c->v_scale;
    g->n_pages = c->n_pages;
    g->hkv = c->n_kv_heads;
    g->ps = 0;
    while ((1 << g->ps) < c->page_size)
        ++g->ps;
    g->fp8 = fp8;
    return MLORA_OK;
}

// Sizes of a paged call (none negative) that the plan and the kernels hold in 32 bits.
bool paged_sizes_ok(int64_t T, int32_t n_seqs, int32_t hq, int32_t hkv, int64_t max_kv)
{
    return T < MAX_KEYS && T * hq < MAX_ROWS && max_kv < MAX_KEYS && (int64_t)n_seqs * hkv < MAX_ROWS &&
           (int64_t)n_seqs * hkv * (max_kv / DECODE_UNIT + 1) < MAX_ROWS;
}

// And of a call over shared prefixes, whose shares are made of smaller units (64 lanes count the groups in equal runs).
bool prefix_sizes_ok(int32_t n_seqs, int32_t n_groups, int32_t hkv, int64_t max_kv, int64_t max_prefix)
{
    return max_prefix < MAX_KEYS && n_groups < MAX_KEYS && (int64_t)n_seqs * hkv * (max_kv / OWN_UNIT + 1) < MAX_ROWS;
}

bool rows_ok(int64_t stride, int64_t width) { return stride >= width && stride % 8 == 0; }

// A window that no sequence is longer than hides nothing (and is left out, so that positions minus the window
// stay within 32 bits).
int32_t seen_window(int32_t window, int64_t max_keys) { return window >= max_keys ? 0 : window; }

// First keys beside a window (as seen_window gives it): none where nothing is hidden, at most all.
int32_t seen_sinks(int32_t sinks, int32_t window, int64_t max_keys)
{
    return window > 0 ? (int32_t)std::min<int64_t>(sinks, max_keys) : 0;
}

size_t align_up(size_t v) { return (v + 255) & ~(size_t)255; }

// Bytes of the parts of the decode kernel: two slots of `rows` rows a share.
void decode_parts(int64_t shares, int64_t rows, int32_t d, size_t *o, size_t *ml)
{
    const size_t slots = (size_t)shares * 2 * rows;
    *o = align_up(slots * d * 4);
    *ml = align_up(slots * 8);
}

// And of the wide kernel's: one row a token, head and chunk of keys.
void wide_parts(int64_t T, int32_t hq, int64_t chunks, int32_t d, size_t *o, size_t *ml)
{
    const size_t slots = (size_t)T * hq * chunks;
    *o = align_up(slots * d * 4);
    *ml = align_up(slots * 8);
}

// Chunks of keys of the wide kernel: as many as make WIDE_WANT workgroups, of WIDE_LEAST keys or more; not cut from
// WIDE_WHOLE workgroups on.
constexpr int64_t WIDE_WHOLE = 192, WIDE_WANT = 512, WIDE_LEAST = 256;
int64_t wide_cuts(int64_t items, int64_t max_kv)
{
    return std::max<int64_t>(1, std::min((WIDE_WANT + items - 1) / items, (max_kv + WIDE_LEAST - 1) / WIDE_LEAST));
}

// How a paged call is cut: which kernels run, and the chunks of keys that give each enough
// workgroups.  Made from the sizes alone, so that the workspace can be sized before the call.
struct PagedPlan {
    int nq = 1, shares = 0;              // column tiles and workgroups of the decode kernel
    bool split = false;
    int64_t dec_rows = 0;                // sequences of up to this many rows go to it (0: none can)
    bool wide = false;                   // some sequence may have more
    int64_t wide_chunk = 0, wide_chunks = 0;
    size_t dec_o = 0, dec_ml = 0, wide_o = 0, wide_ml = 0;   // bytes
    size_t total() const { return dec_o + dec_ml + wide_o + wide_ml; }
};

// (window, sinks: 0, or both as the kernels get them.  A cut is then made of the keys that a sequence's queries or
// those of a row block may see, never into more than without them.)
PagedPlan paged_plan(int64_t T, int32_t n_seqs, int32_t hq, int32_t hkv, int32_t d, int64_t max_q, int64_t max_kv,
                     int64_t window, int64_t sinks)
{
    PagedPlan p;
    const int64_t group = hq / hkv, most = max_q * group;
    max_kv = std::max<int64_t>(max_kv, 1);
    const auto seen = [&](int64_t queries) {
        const int64_t first = (sinks + DECODE_UNIT) / DECODE_UNIT * DECODE_UNIT;
        return sinks > 0 ? std::min(max_kv, window + queries + first + DECODE_UNIT) : max_kv;
    };
    if (most <= 32) {
        p.dec_rows = most;
        p.nq = most <= 16 ? 1 : 2;
    } else {
        p.wide = true;
        p.dec_rows = std::min<int64_t>(16, T * group);
        if (group > 16)
            p.dec_rows = 0;
    }
    if (p.dec_rows > 0) {
        // Equal shares of all keys, one for each workgroup that the card holds (64 contexts of 1 to 8192 tokens,
        // 314332 together: 230 us, whole 274).  Contexts of up to 4 units are not split, for they are answered
        // sooner than parts are joined (8 of 300 tokens: 8.6 us, so split 10.6), nor those of up to 8 units where
        // they give every CU one (32 of 600: 17 us, split 22; 256 of 1 to 1024, 136636 together: 110, split 126, of
        // an e4m3 cache 64 and 87; but 16 of 1 to 1024, 7644 together, are split: 15, whole 18).
        const int64_t items = (int64_t)n_seqs * hkv, keys = seen(std::min<int64_t>(max_q, 32));
        const int64_t units = (keys + DECODE_UNIT - 1) / DECODE_UNIT;
        p.split = units > (items >= CUS ? 8 : 4);
        // (With sinks and chunks, one a CU beside a chunk's workgroups: 47 batches of 16 to 1000 tokens and a chunk of 33 to 2048
        // 3% faster in the mean, 13% slower at the most; 256 tokens and a chunk of 2048, window 2048, 393 us, so 347.)
        const int64_t slots = p.wide && sinks > 0 ? 1 : decode_slots(d, p.nq);
        p.shares = (int)(p.split ? std::min(items * units, slots * CUS) : items);
        if (p.split)
            decode_parts(p.shares, p.dec_rows, d, &p.dec_o, &p.dec_ml);
    }
    if (p.wide) {
        // row blocks: as many as the rows fill, or one a sequence where there are rows enough for all of them to
        // come here (100 sequences of 40 rows over 1500 keys: 94 us in chunks, 67 whole)
        const bool all = T * group > n_seqs * p.dec_rows;
        const int64_t items = std::max<int64_t>((T * group + WIDE_ROWS - 1) / WIDE_ROWS, all ? n_seqs : 0) * hkv;
        const int64_t n = items >= WIDE_WHOLE ? 1 : wide_cuts(items, seen(WIDE_ROWS / group + 1));
        p.wide_chunk = ((max_kv + n - 1) / n + 127) & ~INT64_C(127);
        p.wide_chunks = sinks > 0 ? n : (max_kv + p.wide_chunk - 1) / p.wide_chunk;
        if (p.wide_chunks > 1)
            wide_parts(T, hq, p.wide_chunks, d, &p.wide_o, &p.wide_ml);
    }
    return p;
}

// The most that paged_plan asks for over all T, n_seqs, max_q and max_kv up to these: a larger batch is cut less, and
// needs fewer parts, so that the plan's own bytes fall here and there as a size rises.
size_t paged_room(int64_t T, int32_t n_seqs, int32_t hq, int32_t hkv, int32_t d, int64_t max_q, int64_t max_kv)
{
    const int64_t group = hq / hkv, most = max_q * group, units = (max_kv + DECODE_UNIT - 1) / DECODE_UNIT;
    size_t dec = 0, wide = 0, o, ml;
    for (int nq = 1; nq <= 2 && units > 4; ++nq) {
        if (nq == 2 && most <= 16)
            break;
        decode_parts(std::min((int64_t)n_seqs * hkv * units, (int64_t)decode_slots(d, nq) * CUS),
                     std::min<int64_t>(most, 16 * nq), d, &o, &ml);
        dec = std::max(dec, o + ml);
    }
    // r row blocks: the tokens that fill them, cut the finer the fewer they are
    for (int64_t r = 1; most > 32 && r * hkv < WIDE_WHOLE && (r - 1) * WIDE_ROWS < T * group; ++r) {
        const int64_t cuts = wide_cuts(r * hkv, max_kv);
        if (cuts > 1) {
            wide_parts(std::min(T, r * WIDE_ROWS / group), hq, cuts, d, &o, &ml);
            wide = std::max(wide, o + ml);
        }
    }
    return dec + wide;
}

// How a call over shared prefixes is cut: the kernels as in paged_plan, but always with parts, for the join takes a row's own
// keys as one of them; a sequence of more than ALONE_ROWS rows shares nothing (it reads the prefix for rows enough, and
// answers them without parts).
constexpr int32_t ALONE_ROWS = 256;

// Chunks of keys for `items` row blocks of `keys` keys at the most, up to `limit`, in us: a tile takes 1.2 in a workgroup alone
// on its CU and 1.95 in two, in rounds of 512, and a part of 128 rows 0.08 to write and to read again.  shared: probabilities
// are two bf16 parts there, a quarter more a tile, and one chunk leaves a part, too.
int64_t prefix_cuts(int64_t items, int64_t keys, int64_t limit, bool shared)
{
    const int64_t tiles = (keys + 63) / 64;
    int64_t best = 1;
    double least = 0.;
    for (int64_t n = 1; n <= limit && (n == 1 || n * items <= 8 * CUS); ++n) {
        const int64_t groups = items * n, each = (tiles + n - 1) / n;
        const double tile_us = groups <= CUS ? 1.2 : 1.95 * ((groups + 2 * CUS - 1) / (2 * CUS));
        const double us = tile_us * each * (shared ? 1.25 : 1.) + (shared || n > 1 ? 0.08 * groups : 0.);
        if (n == 1 || us < least) {
            best = n;
            least = us;
        }
    }
    return best;
}

// The limit of the cuts of a batch of these row blocks: every row has room for a part of each.
int64_t most_prefix_cuts(int64_t items, int64_t keys)
{
    return std::max<int64_t>(1, std::min<int64_t>(std::min<int64_t>(64, 8 * CUS / items), (keys + 63) / 64 / 2));
}

struct PrefixPlan {
    PagedPlan own;
    int64_t chunk = 0, chunks = 0;
    int64_t share_slots = 0, row_parts = 0;     // parts of the decode kernel's shares, and of each row
    size_t o = 0, ml = 0, cuts = 0;             // bytes
    size_t total() const { return o + ml + cuts; }
};

size_t cut_bytes(int64_t n_seqs, int32_t hkv) { return align_up((size_t)n_seqs * hkv * 16); }

// Workgroups of the decode kernel, of four shares each.
int64_t own_workgroups(int32_t n_seqs, int32_t hkv, int64_t max_kv)
{
    const int64_t units = (std::max<int64_t>(max_kv, 1) + OWN_UNIT - 1) / OWN_UNIT;
    return std::min(((int64_t)n_seqs * hkv * units + 3) / 4, 2 * CUS);
}

PrefixPlan prefix_plan(int64_t T, int32_t n_seqs, int32_t n_groups, int32_t hq, int32_t hkv, int32_t d, int64_t max_q,
                       int64_t max_kv, int64_t max_prefix)
{
    PrefixPlan p;
    p.own = paged_plan(T, n_seqs, hq, hkv, d, max_q, max_kv, 0, 0);
    // The rows of sequences that share nothing, if those of more than one token are alike, and the others'.
    const int64_t group = hq / hkv, all = T * group, items = (all + WIDE_ROWS - 1) / WIDE_ROWS * hkv;
    const int64_t chunks = std::max<int64_t>(T - n_seqs, 0) / std::max<int64_t>(max_q - 1, 1);
    const int64_t alone = max_q * group > ALONE_ROWS ? std::min(T, chunks * max_q) * group : 0;
    const auto blocks = [&](int64_t rows) { return std::max<int64_t>(1, (rows + WIDE_ROWS - 1) / WIDE_ROWS) * hkv; };
    // (half of the groups' last row blocks are taken to be more)
    const int64_t shared = blocks(all - alone) + std::min<int64_t>(n_groups / 2, T) * hkv;
    int64_t n = prefix_cuts(shared, max_prefix, most_prefix_cuts(items, max_prefix), true);
    p.chunk = ((max_prefix + n - 1) / n + 63) & ~INT64_C(63);
    p.chunks = (max_prefix + p.chunk - 1) / p.chunk;
    // The card holds 512 workgroups: those of the shares start beside the others', one of which a CU has at the most.  Where
    // sequences have many keys of their own, they outlast the others, and as many on every CU are faster than a second one on
    // some (128 tokens behind 4000 keys, 500 to 3000 of their own: 384 209 us, 256 182; 64 behind 4096, 1 to 1024: 384 39, 256
    // 45).  The host knows bounds alone: their difference is what a sequence of the longest prefix may have, more than 1536
    // keys here, but sequences of no group or of a shorter prefix may have more (8 of 1 to 9200 beside 64 behind 8192: both 84
    // us; 64 of 1 to 9000 beside 128 behind 8000: 362, with 256 301), and one long one may stand for none of the others (one
    // of 8000 beside 64 behind 2000: 384 43, 256 45; beside 128: 90 and 82).
    const int64_t beside = std::min(shared * p.chunks, CUS);
    int64_t groups = 2 * CUS - beside;
    if (max_kv - max_prefix > 1536)
        groups = beside < CUS / 2 ? 2 * CUS : CUS;
    p.own.shares = p.own.dec_rows > 0 ? (int)std::min(own_workgroups(n_seqs, hkv, max_kv), groups) : 0;
    p.share_slots = 2 * 4 * (int64_t)p.own.shares * p.own.dec_rows;
    if (p.own.wide) {
        const int64_t keys = std::max<int64_t>(max_kv, 1);
        n = prefix_cuts(blocks(alone > 0 ? alone : all), keys, most_prefix_cuts(items, keys), false);
        p.own.wide_chunk = ((keys + n - 1) / n + 127) & ~INT64_C(127);
        p.own.wide_chunks = (keys + p.own.wide_chunk - 1) / p.own.wide_chunk;
    }
    p.row_parts = p.chunks + std::max<int64_t>(p.own.wide_chunks, 1);
    const size_t slots = (size_t)p.share_slots + (size_t)T * hq * p.row_parts;
    p.o = align_up(slots * d * 4);
    p.ml = align_up(slots * 8);
    p.cuts = cut_bytes(n_seqs, hkv);
    return p;
}

// The most that prefix_plan asks for over all sizes up to these (see paged_room).
size_t prefix_room(int64_t T, int32_t n_seqs, int32_t hq, int32_t hkv, int32_t d, int64_t max_q, int64_t max_kv,
                   int64_t max_prefix)
{
    const int64_t group = hq / hkv, most = max_q * group;
    const size_t shares = 8 * (size_t)own_workgroups(n_seqs, hkv, max_kv) * std::min<int64_t>(most, 32);
    size_t rows = (size_t)T * hq * 2;
    for (int64_t r = 1; r * hkv <= 8 * CUS && (r - 1) * WIDE_ROWS < T * group; ++r) {
        const int64_t wide = most > 32 ? most_prefix_cuts(r * hkv, std::max<int64_t>(max_kv, 1)) : 1;
        rows = std::max(rows, (size_t)std::min(T, r * WIDE_ROWS / group) * hq * (most_prefix_cuts(r * hkv, max_prefix) + wide));
    }
    return align_up((shares + rows) * d * 4) + align_up((shares + rows) * 8) + cut_bytes(n_seqs, hkv);
}

mlora_status attention(const void *q, int64_t q_stride, const void *k, int64_t k_stride, const void *v,
                       int64_t v_stride, int64_t T_q, int64_t T_k, int32_t n_seqs, const int32_t *cu_q,
                       const int32_t *cu_k, int32_t n_q_heads, int32_t n_kv_heads, int32_t head_dim, int64_t max_q,
                       int32_t causal, int32_t window, int32_t sinks, float scale, void *out, int64_t out_stride,
                       float *lse, hipStream_t stream)
{
    if (T_q < 0 || T_k < 0 || n_seqs < 0 || max_q < 0 || window < 0 || sinks < 0 || !(scale >= 0.f) ||
        std::isinf(scale))
        return MLORA_ERR_ARG;
    const mlora_status st = check_heads(n_q_heads, n_kv_heads, head_dim);
    if (st != MLORA_OK)
        return st;
    const int64_t qw = (int64_t)n_q_heads * head_dim, kw = (int64_t)n_kv_heads * head_dim;
    if (!rows_ok(q_stride, qw) || !rows_ok(out_stride, qw) || !rows_ok(k_stride, kw) || !rows_ok(v_stride, kw) ||
        (cu_k == nullptr && T_k != T_q))
        return MLORA_ERR_SHAPE;
    if (T_q >= MAX_KEYS || T_k >= MAX_KEYS || T_q * n_q_heads >= MAX_ROWS || k_stride >= MAX_STRIDE ||
        v_stride >= MAX_STRIDE)
        return MLORA_ERR_UNSUPPORTED;
    if (T_q == 0 || n_seqs == 0 || max_q == 0)
        return MLORA_OK;
    if (q == nullptr || out == nullptr || cu_q == nullptr || !aligned16(q) || !aligned16(k) || !aligned16(v) ||
        !aligned16(out) || (T_k > 0 && (k == nullptr || v == nullptr)))
        return MLORA_ERR_ARG;
    AttnArgs a{};
    a.q = (const uint16_t *)q;
    a.k = (const uint16_t *)k;
    a.v = (const uint16_t *)v;
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.out_stride = out_stride;
    a.T = T_q;
    a.Tk = T_k;
    a.n_seqs = n_seqs;
    a.hq = n_q_heads;
    a.hkv = n_kv_heads;
    a.group = n_q_heads / n_kv_heads;
    a.cu_q = cu_q;
    a.cu_k = cu_k;
    a.max_q = std::min(max_q, T_q);
    a.causal = causal;
    a.window = seen_window(window, T_k);
    a.sinks = seen_sinks(sinks, a.window, T_k);
    a.scale = scale == 0.f ? (float)(1.0 / std::sqrt((double)head_dim)) : scale;
    a.out = (uint16_t *)out;
    a.lse = lse;
    a.chunk = 1 << 30;
    a.n_chunks = 1;
    a.max_rows = 0x7fffffff;
    trace_mark(stream, true);
    const hipError_t e = launch_attn_wide(a, head_dim, false, stream);
    trace_mark(stream, false);
    return hip_status(e);
}

// A paged call that has passed its checks (nothing: there is nothing to do).
struct PagedCall {
    AttnArgs a{};
    int32_t d = 0;
    bool nothing = false;
};

mlora_status paged_call(PagedCall *c, const void *q, int64_t q_stride, int64_t T, int32_t n_q_heads, const mlora_cache *cache,
                        const int32_t *page_table, int64_t table_stride, int32_t n_seqs, const int32_t *cu_q,
                        const int32_t *kv_len, int64_t max_q, int64_t max_kv, int32_t causal, int32_t window,
                        int32_t sinks, float scale, void *out, int64_t out_stride, float *lse)
{
    if (T < 0 || n_seqs < 0 || max_q < 0 || max_kv < 0 || table_stride < 0 || window < 0 || sinks < 0 || !(scale >= 0.f) ||
        std::isinf(scale))
        return MLORA_ERR_ARG;
    AttnArgs &a = c->a;
    mlora_status st = check_cache(cache, &a.cache);
    if (st != MLORA_OK)
        return st;
    const int32_t d = c->d = cache->head_dim;
    st = check_heads(n_q_heads, cache->n_kv_heads, d);
    if (st != MLORA_OK)
        return st;
    if (!rows_ok(q_stride, (int64_t)n_q_heads * d) || !rows_ok(out_stride, (int64_t)n_q_heads * d))
        return MLORA_ERR_SHAPE;
    if (!paged_sizes_ok(T, n_seqs, n_q_heads, cache->n_kv_heads, max_kv) || table_stride >= MAX_ROWS)
        return MLORA_ERR_UNSUPPORTED;
    c->nothing = T == 0 || n_seqs == 0 || max_q == 0;
    if (c->nothing)
        return MLORA_OK;
    if (q == nullptr || out == nullptr || cu_q == nullptr || kv_len == nullptr || !aligned16(q) || !aligned16(out) ||
        (max_kv > 0 && table_stride > 0 && page_table == nullptr))
        return MLORA_ERR_ARG;
    a.q = (const uint16_t *)q;
    a.q_stride = q_stride;
    a.out_stride = out_stride;
    a.T = T;
    a.n_seqs = n_seqs;
    a.hq = n_q_heads;
    a.hkv = cache->n_kv_heads;
    a.group = n_q_heads / cache->n_kv_heads;
    a.cu_q = cu_q;
    a.kv_len = kv_len;
    a.table = page_table;
    a.table_stride = table_stride;
    a.max_q = std::min(max_q, T);
    a.max_kv = max_kv;
    a.causal = causal;
    a.window = seen_window(window, max_kv);
    a.sinks = seen_sinks(sinks, a.window, max_kv);
    a.scale = scale == 0.f ? (float)(1.0 / std::sqrt((double)d)) : scale;
    a.out = (uint16_t *)out;
    a.lse = lse;
    return MLORA_OK;
}

// The aligned start of a workspace, or NULL where it has not `need` bytes from there.
uint8_t *workspace(void *ws, size_t ws_bytes, size_t need)
{
    uint8_t *const base = (uint8_t *)(((uintptr_t)ws + 255) & ~(uintptr_t)255);
    return ws != nullptr && ws_bytes >= need + (size_t)(base - (uint8_t *)ws) ? base : nullptr;
}

mlora_status run_paged(const PagedCall &c, void *ws, size_t ws_bytes, hipStream_t stream)
{
    AttnArgs a = c.a;
    const int32_t d = c.d;
    const PagedPlan p = paged_plan(a.T, a.n_seqs, a.hq, a.hkv, d, a.max_q, a.max_kv, a.window, a.sinks);
    if (p.wide_chunks > 65535)
        return MLORA_ERR_UNSUPPORTED;
    uint8_t *const base = workspace(ws, ws_bytes, p.total());
    if (p.total() > 0 && base == nullptr)
        return MLORA_ERR_WORKSPACE;
    AttnArgs w = a;                     // the wide part
    w.min_rows = (int32_t)p.dec_rows + 1;
    w.max_rows = 0x7fffffff;
    w.chunk = (int32_t)p.wide_chunk;
    w.n_chunks = (int32_t)p.wide_chunks;
    w.part_o = (float *)(base + p.dec_o + p.dec_ml);
    w.part_ml = (float *)(base + p.dec_o + p.dec_ml + p.wide_o);
    a.max_rows = (int32_t)p.dec_rows;   // and the decode rows
    a.part_o = p.split ? (float *)base : nullptr;
    a.part_ml = p.split ? (float *)(base + p.dec_o) : nullptr;
    trace_mark(stream, true);
    hipError_t e;
    if (p.wide && p.dec_rows > 0)
        e = launch_attn_mixed(w, a, d, p.shares, stream);
    else if (p.wide)
        e = launch_attn_wide(w, d, true, stream);
    else
        e = launch_attn_decode(a, d, p.nq, p.shares, stream);
    if (e == hipSuccess && p.wide_chunks > 1)
        e = launch_attn_wide_combine(w, d, stream);
    if (e == hipSuccess && p.split)
        e = launch_attn_combine(a, d, p.shares, stream);
    trace_mark(stream, false);
    return hip_status(e);
}

mlora_status paged_attention(const void *q, int64_t q_stride, int64_t T, int32_t n_q_heads, const mlora_cache *cache,
                             const int32_t *page_table, int64_t table_stride, int32_t n_seqs, const int32_t *cu_q,
                             const int32_t *kv_len, int64_t max_q, int64_t max_kv, int32_t causal, int32_t window,
                             int32_t sinks, float scale, void *out, int64_t out_stride, float *lse, void *ws,
                             size_t ws_bytes, hipStream_t stream)
{
    PagedCall c;
    const mlora_status st = paged_call(&c, q, q_stride, T, n_q_heads, cache, page_table, table_stride, n_seqs, cu_q, kv_len,
                                       max_q, max_kv, causal, window, sinks, scale, out, out_stride, lse);
    return st != MLORA_OK || c.nothing ? st : run_paged(c, ws, ws_bytes, stream);
}

mlora_status validate_pages(const mlora_cache *cache, const int32_t *page_table, int64_t table_stride, int32_t n_seqs,
                            const int32_t *cu_q, const int32_t *kv_len, int64_t T, int64_t max_q, int64_t max_kv,
                            int32_t window, int32_t sinks, int64_t *bad_value)
{
    if (cache == nullptr || n_seqs < 0 || T < 0 || table_stride < 0 || max_q < 0 || max_kv < 0 ||
        window < 0 || sinks < 0)
        return MLORA_ERR_ARG;
    const mlora_status st =
        check_cache_sizes(cache->n_pages, cache->n_kv_heads, cache->page_size, cache->head_dim, cache->dtype);
    if (st != MLORA_OK)
        return st;
    if (table_stride >= MAX_ROWS)
        return MLORA_ERR_UNSUPPORTED;
    if (cu_q == nullptr || (n_seqs > 0 && kv_len == nullptr))
        return MLORA_ERR_ARG;
    const auto bad = [bad_value](mlora_status s, int64_t v) {
        if (bad_value)
            *bad_value = v;
        return s;
    };
    if (cu_q[0] != 0)
        return bad(MLORA_ERR_SHAPE, cu_q[0]);
    for (int32_t b = 0; b < n_seqs; ++b) {
        const int64_t n = (int64_t)cu_q[b + 1] - cu_q[b];
        if (n < 0 || n > max_q)
            return bad(MLORA_ERR_SHAPE, n);
        if (kv_len[b] < 0 || kv_len[b] > max_kv || kv_len[b] > table_stride * cache->page_size)
            return bad(MLORA_ERR_SHAPE, kv_len[b]);
        if (kv_len[b] > 0 && page_table == nullptr)
            return MLORA_ERR_ARG;
        const int64_t pages = ((int64_t)kv_len[b] + cache->page_size - 1) / cache->page_size;
        // the queries see keys [0, first) and [lo, kv_len[b]) (without a window every page is looked at)
        const int64_t lo = window <= 0 ? 0 : n > 0 ? std::max<int64_t>(0, kv_len[b] - n - window + 1) : kv_len[b];
        const int64_t first = n > 0 ? sinks : 0;
        for (int64_t i = 0; i < pages; ++i) {
            if (window > 0 && i * cache->page_size >= first && (n == 0 || (i + 1) * cache->page_size <= lo))
                continue;
            const int32_t p = page_table[b * table_stride + i];
            if (p < 0 || p >= cache->n_pages)
                return bad(MLORA_ERR_INDEX, p);
        }
    }
    if (cu_q[n_seqs] != T)
        return bad(MLORA_ERR_SHAPE, cu_q[n_seqs]);
    return MLORA_OK;
}

}  // namespace

extern "C" {

mlora_status mlora_rope_turns(int32_t rot_dim, double base, int32_t scaling, double factor, int64_t orig_len,
                              double fast, double slow, uint64_t *turns)
{
    if (turns == nullptr || rot_dim < 2 || rot_dim % 2 || !(base > 1.0) || !(factor >= 1.0) ||
        !std::isfinite(base) || !std::isfinite(factor))
        return MLORA_ERR_ARG;
    if (scaling != MLORA_ROPE_PLAIN && scaling != MLORA_ROPE_LINEAR && scaling != MLORA_ROPE_PARTS)
        return MLORA_ERR_ARG;
    if (scaling == MLORA_ROPE_PARTS && (orig_len < 1 || !(fast > slow) || !(slow >= 0.0)))
        return MLORA_ERR_ARG;
    const long double two_pi = 6.283185307179586476925286766559005768L;
    for (int32_t i = 0; i < rot_dim / 2; ++i) {
        long double f = std::pow((long double)base, -2.0L * i / rot_dim) / two_pi;
        if (scaling == MLORA_ROPE_LINEAR) {
            f /= (long double)factor;
        } else if (scaling == MLORA_ROPE_PARTS) {
            const long double keep = std::min(1.0L, std::max(0.0L, (orig_len * f - (long double)slow) /
                                                                       ((long double)fast - (long double)slow)));
            f = f * keep + f / (long double)factor * (1.0L - keep);
        }
        turns[i] = (uint64_t)std::llround(f * 0x1p64L);   // f < 1/4: fits
    }
    return MLORA_OK;
}

int64_t mlora_cache_bytes(int64_t n_pages, int32_t n_kv_heads, int32_t page_size, int32_t head_dim, int32_t dtype)
{
    if (check_cache_sizes(n_pages, n_kv_heads, page_size, head_dim, dtype) != MLORA_OK)
        return -1;
    const int64_t vectors = 2 * n_pages * n_kv_heads * page_size;
    return dtype == MLORA_CACHE_E4M3 ? vectors * (head_dim + 4) : vectors * head_dim * 2;
}

mlora_status mlora_qk_rope(const void *qkv, int64_t T, int64_t row_stride, int32_t n_q_heads, int32_t n_kv_heads,
                           int32_t head_dim, const int32_t *pos, const mlora_rope *rope, const void *q_weight,
                           const void *k_weight, float eps, void *q_out, int64_t q_stride, void *k_out,
                           int64_t k_stride, const mlora_cache *cache, const int32_t *slot, hipStream_t stream)
{
    if (T < 0 || rope == nullptr)
        return MLORA_ERR_ARG;
    mlora_status st = check_heads(n_q_heads, n_kv_heads, head_dim);
    if (st != MLORA_OK)
        return st;
    if (rope->rot_dim < 0 || rope->rot_dim > head_dim || rope->rot_dim % 16)
        return MLORA_ERR_SHAPE;
    if (!rows_ok(row_stride, (int64_t)(n_q_heads + 2 * n_kv_heads) * head_dim) ||
        !rows_ok(q_stride, (int64_t)n_q_heads * head_dim) ||
        (k_out != nullptr && !rows_ok(k_stride, (int64_t)n_kv_heads * head_dim)))
        return MLORA_ERR_SHAPE;
    if (!(eps >= 0.f) || (cache == nullptr) != (slot == nullptr))
        return MLORA_ERR_ARG;
    RopeArgs a{};
    if (cache != nullptr) {
        st = check_cache(cache, &a.cache);
        if (st != MLORA_OK)
            return st;
        if (cache->n_kv_heads != n_kv_heads || cache->head_dim != head_dim)
            return MLORA_ERR_SHAPE;
    }
    if (T >= MAX_ROWS)
        return MLORA_ERR_UNSUPPORTED;
    if (T == 0)
        return MLORA_OK;
    if (qkv == nullptr || q_out == nullptr || pos == nullptr || !aligned16(qkv) || !aligned16(q_out) ||
        !aligned16(k_out) || !aligned16(q_weight) || !aligned16(k_weight) ||
        (rope->rot_dim > 0 && rope->turns == nullptr))
        return MLORA_ERR_ARG;
    a.qkv = (const uint16_t *)qkv;
    a.T = T;
    a.row_stride = row_stride;
    a.hq = n_q_heads;
    a.hkv = n_kv_heads;
    a.pos = pos;
    a.turns = rope->turns;
    a.rot = rope->rot_dim;
    a.interleaved = rope->interleaved;
    a.magnitude = rope->magnitude;
    a.qw = (const uint16_t *)q_weight;
    a.kw = (const uint16_t *)k_weight;
    a.eps = eps;
    a.q_out = (uint16_t *)q_out;
    a.k_out = (uint16_t *)k_out;
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.slot = slot;
    trace_mark(stream, true);
    const hipError_t e = launch_qk_rope(a, head_dim, stream);
    trace_mark(stream, false);
    return hip_status(e);
}

mlora_status mlora_cache_read(const mlora_cache *cache, const int32_t *slot, int64_t T, void *k, void *v,
                              hipStream_t stream)
{
    if (T < 0)
        return MLORA_ERR_ARG;
    CacheGeom g;
    const mlora_status st = check_cache(cache, &g);
    if (st != MLORA_OK)
        return st;
    if (T >= MAX_ROWS)
        return MLORA_ERR_UNSUPPORTED;
    if (T == 0 || (k == nullptr && v == nullptr))
        return MLORA_OK;
    if (slot == nullptr || !aligned16(k) || !aligned16(v))
        return MLORA_ERR_ARG;
    trace_mark(stream, true);
    const hipError_t e = launch_cache_read(g, cache->head_dim, slot, T, (uint16_t *)k, (uint16_t *)v, stream);
    trace_mark(stream, false);
    return hip_status(e);
}

mlora_status mlora_attention(const void *q, int64_t q_stride, const void *k, int64_t k_stride, const void *v,
                             int64_t v_stride, int64_t T_q, int64_t T_k, int32_t n_seqs, const int32_t *cu_q,
                             const int32_t *cu_k, int32_t n_q_heads, int32_t n_kv_heads, int32_t head_dim,
                             int64_t max_q, int32_t causal, int32_t window, float scale, void *out,
                             int64_t out_stride, float *lse, hipStream_t stream)
{
    return attention(q, q_stride, k, k_stride, v, v_stride, T_q, T_k, n_seqs, cu_q, cu_k, n_q_heads, n_kv_heads,
                     head_dim, max_q, causal, window, 0, scale, out, out_stride, lse, stream);
}

mlora_status mlora_attention_sinks(const void *q, int64_t q_stride, const void *k, int64_t k_stride, const void *v,
                                   int64_t v_stride, int64_t T_q, int64_t T_k, int32_t n_seqs, const int32_t *cu_q,
                                   const int32_t *cu_k, int32_t n_q_heads, int32_t n_kv_heads, int32_t head_dim,
                                   int64_t max_q, int32_t causal, int32_t window, int32_t sinks, float scale,
                                   void *out, int64_t out_stride, float *lse, hipStream_t stream)
{
    return attention(q, q_stride, k, k_stride, v, v_stride, T_q, T_k, n_seqs, cu_q, cu_k, n_q_heads, n_kv_heads,
                     head_dim, max_q, causal, window, sinks, scale, out, out_stride, lse, stream);
}

size_t mlora_paged_workspace_size(int64_t T, int32_t n_seqs, int32_t n_q_heads, int32_t n_kv_heads,
                                  int32_t head_dim, int64_t max_q, int64_t max_kv)
{
    if (T < 0 || n_seqs < 0 || max_q < 0 || max_kv < 0 ||
        check_heads(n_q_heads, n_kv_heads, head_dim) != MLORA_OK ||
        !paged_sizes_ok(T, n_seqs, n_q_heads, n_kv_heads, max_kv))
        return 0;
    return paged_room(T, n_seqs, n_q_heads, n_kv_heads, head_dim, std::min(max_q, T), max_kv) + 256;
}

mlora_status mlora_paged_attention(const void *q, int64_t q_stride, int64_t T, int32_t n_q_heads,
                                   const mlora_cache *cache, const int32_t *page_table, int64_t table_stride,
                                   int32_t n_seqs, const int32_t *cu_q, const int32_t *kv_len, int64_t max_q,
                                   int64_t max_kv, int32_t causal, int32_t window, float scale, void *out,
                                   int64_t out_stride, float *lse, void *ws, size_t ws_bytes, hipStream_t stream)
{
    return paged_attention(q, q_stride, T, n_q_heads, cache, page_table, table_stride, n_seqs, cu_q, kv_len, max_q, max_kv,
                           causal, window, 0, scale, out, out_stride, lse, ws, ws_bytes, stream);
}

mlora_status mlora_paged_attention_sinks(const void *q, int64_t q_stride, int64_t T, int32_t n_q_heads,
                                         const mlora_cache *cache, const int32_t *page_table, int64_t table_stride,
                                         int32_t n_seqs, const int32_t *cu_q, const int32_t *kv_len, int64_t max_q,
                                         int64_t max_kv, int32_t causal, int32_t window, int32_t sinks, float scale,
                                         void *out, int64_t out_stride, float *lse, void *ws, size_t ws_bytes,
                                         hipStream_t stream)
{
    return paged_attention(q, q_stride, T, n_q_heads, cache, page_table, table_stride, n_seqs, cu_q, kv_len, max_q, max_kv,
                           causal, window, sinks, scale, out, out_stride, lse, ws, ws_bytes, stream);
}

size_t mlora_prefix_workspace_size(int64_t T, int32_t n_seqs, int32_t n_groups, int32_t n_q_heads, int32_t n_kv_heads,
                                   int32_t head_dim, int64_t max_q, int64_t max_kv, int64_t max_prefix)
{
    if (n_groups < 0 || max_prefix < 0)
        return 0;
    const size_t paged = mlora_paged_workspace_size(T, n_seqs, n_q_heads, n_kv_heads, head_dim, max_q, max_kv);
    if (paged > 0 && !prefix_sizes_ok(n_seqs, n_groups, n_kv_heads, max_kv, max_prefix))
        return 0;
    if (paged == 0 || n_groups == 0 || max_prefix == 0)
        return paged;
    return std::max(paged, prefix_room(T, n_seqs, n_q_heads, n_kv_heads, head_dim, std::min(max_q, T), max_kv, max_prefix) + 256);
}

mlora_status mlora_prefix_attention(const void *q, int64_t q_stride, int64_t T, int32_t n_q_heads,
                                    const mlora_cache *cache, const int32_t *page_table, int64_t table_stride,
                                    int32_t n_seqs, const int32_t *cu_q, const int32_t *kv_len, int32_t n_groups,
                                    const int32_t *group_start, const int32_t *prefix_len, int64_t max_q,
                                    int64_t max_kv, int64_t max_prefix, int32_t causal, float scale, void *out,
                                    int64_t out_stride, float *lse, void *ws, size_t ws_bytes, hipStream_t stream)
{
    if (n_groups < 0 || max_prefix < 0)
        return MLORA_ERR_ARG;
    PagedCall c;
    const mlora_status st = paged_call(&c, q, q_stride, T, n_q_heads, cache, page_table, table_stride, n_seqs, cu_q, kv_len,
                                       max_q, max_kv, causal, 0, 0, scale, out, out_stride, lse);
    if (st != MLORA_OK)
        return st;
    if (!prefix_sizes_ok(n_seqs, n_groups, c.a.hkv, max_kv, max_prefix))
        return MLORA_ERR_UNSUPPORTED;
    if (c.nothing)
        return MLORA_OK;
    if (n_groups > 0 && (group_start == nullptr || prefix_len == nullptr))
        return MLORA_ERR_ARG;
    max_prefix = std::min(max_prefix, max_kv);
    if (n_groups == 0 || max_prefix == 0)
        return run_paged(c, ws, ws_bytes, stream);
    const AttnArgs &a = c.a;
    const PrefixPlan p = prefix_plan(a.T, a.n_seqs, n_groups, a.hq, a.hkv, c.d, a.max_q, a.max_kv, max_prefix);
    if (p.own.wide_chunks > 65535)
        return MLORA_ERR_UNSUPPORTED;
    uint8_t *const base = workspace(ws, ws_bytes, p.total());
    if (base == nullptr)
        return MLORA_ERR_WORKSPACE;
    AttnArgs d = a;                     // the decode rows' own keys
    d.max_rows = (int32_t)p.own.dec_rows;
    d.part_o = (float *)base;
    d.part_ml = (float *)(base + p.o);
    d.group_start = group_start;
    d.prefix_len = prefix_len;
    d.n_groups = n_groups;
    d.max_prefix = max_prefix;
    d.row_slot = p.share_slots;
    d.row_parts = (int32_t)p.row_parts;
    d.row_first = (int32_t)p.chunks;
    d.cuts = (int32_t *)(base + p.o + p.ml);
    d.alone_rows = ALONE_ROWS;
    AttnArgs w = d;                     // the wide ones'
    w.min_rows = d.max_rows + 1;
    w.max_rows = 0x7fffffff;
    w.chunk = (int32_t)p.own.wide_chunk;
    w.n_chunks = (int32_t)std::max<int64_t>(p.own.wide_chunks, 1);
    AttnArgs s = d;                     // and the shared ones
    s.max_q = a.T;
    s.chunk = (int32_t)p.chunk;
    s.n_chunks = (int32_t)p.chunks;
    s.row_first = 0;
    s.max_rows = (int32_t)std::min<int64_t>(a.max_q * a.group, 0x7fffffff);
    trace_mark(stream, true);
    hipError_t e = launch_attn_prefix(s, w, d, c.d, p.own.wide, p.own.nq, p.own.shares, stream);
    if (e == hipSuccess)
        e = launch_attn_prefix_join(s, w, d, c.d, stream);
    trace_mark(stream, false);
    return hip_status(e);
}

mlora_status mlora_validate_prefixes(const mlora_cache *cache, int64_t table_stride, int32_t n_seqs,
                                     const int32_t *kv_len, int32_t n_groups, const int32_t *group_start,
                                     const int32_t *prefix_len, int64_t max_prefix, int64_t *bad_value)
{
    if (cache == nullptr || table_stride < 0 || n_seqs < 0 || n_groups < 0 || max_prefix < 0)
        return MLORA_ERR_ARG;
    const mlora_status st =
        check_cache_sizes(cache->n_pages, cache->n_kv_heads, cache->page_size, cache->head_dim, cache->dtype);
    if (st != MLORA_OK)
        return st;
    if (table_stride >= MAX_ROWS)
        return MLORA_ERR_UNSUPPORTED;
    if (n_groups == 0)
        return MLORA_OK;
    if (group_start == nullptr || prefix_len == nullptr || (n_seqs > 0 && kv_len == nullptr))
        return MLORA_ERR_ARG;
    const auto bad = [bad_value](int64_t v) {
        if (bad_value)
            *bad_value = v;
        return MLORA_ERR_SHAPE;
    };
    if (group_start[0] != 0)
        return bad(group_start[0]);
    for (int32_t g = 0; g < n_groups; ++g) {
        const int32_t b0 = group_start[g], b1 = group_start[g + 1];
        if (b1 < b0 || b1 > n_seqs)
            return bad(b1);
        const int64_t keys = prefix_len[g];
        if (keys < 0 || keys > max_prefix || keys > table_stride * cache->page_size || (b1 > b0 && keys > kv_len[b0]))
            return bad(keys);
    }
    return MLORA_OK;
}

mlora_status mlora_validate_pages(const mlora_cache *cache, const int32_t *page_table, int64_t table_stride,
                                  int32_t n_seqs, const int32_t *cu_q, const int32_t *kv_len, int64_t T,
                                  int64_t max_q, int64_t max_kv, int64_t *bad_value)
{
    return validate_pages(cache, page_table, table_stride, n_seqs, cu_q, kv_len, T, max_q, max_kv, 0, 0, bad_value);
}

mlora_status mlora_validate_pages_sinks(const mlora_cache *cache, const int32_t *page_table, int64_t table_stride,
                                        int32_t n_seqs, const int32_t *cu_q, const int32_t *kv_len, int64_t T,
                                        int64_t max_q, int64_t max_kv, int32_t window, int32_t sinks,
                                        int64_t *bad_value)
{
    return validate_pages(cache, page_table, table_stride, n_seqs, cu_q, kv_len, T, max_q, max_kv, window, sinks, bad_value);
}

}  // extern "C"
