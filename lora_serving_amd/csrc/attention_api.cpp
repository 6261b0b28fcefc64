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

bool rows_ok(int64_t stride, int64_t width) { return stride >= width && stride % 8 == 0; }

// A window that no sequence is longer than hides nothing (and is left out, so that positions minus the window
// stay within 32 bits).
int32_t seen_window(int32_t window, int64_t max_keys) { return window >= max_keys ? 0 : window; }

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

PagedPlan paged_plan(int64_t T, int32_t n_seqs, int32_t hq, int32_t hkv, int32_t d, int64_t max_q, int64_t max_kv)
{
    PagedPlan p;
    const int64_t group = hq / hkv, most = max_q * group;
    max_kv = std::max<int64_t>(max_kv, 1);
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
        const int64_t items = (int64_t)n_seqs * hkv, units = (max_kv + DECODE_UNIT - 1) / DECODE_UNIT;
        p.split = units > (items >= CUS ? 8 : 4);
        p.shares = (int)(p.split ? std::min(items * units, (int64_t)decode_slots(d, p.nq) * CUS) : items);
        if (p.split)
            decode_parts(p.shares, p.dec_rows, d, &p.dec_o, &p.dec_ml);
    }
    if (p.wide) {
        // row blocks: as many as the rows fill, or one a sequence where there are rows enough for all of them to
        // come here (100 sequences of 40 rows over 1500 keys: 94 us in chunks, 67 whole)
        const bool all = T * group > n_seqs * p.dec_rows;
        const int64_t items = std::max<int64_t>((T * group + WIDE_ROWS - 1) / WIDE_ROWS, all ? n_seqs : 0) * hkv;
        const int64_t n = items >= WIDE_WHOLE ? 1 : wide_cuts(items, max_kv);
        p.wide_chunk = ((max_kv + n - 1) / n + 127) & ~INT64_C(127);
        p.wide_chunks = (max_kv + p.wide_chunk - 1) / p.wide_chunk;
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
    if (T_q < 0 || T_k < 0 || n_seqs < 0 || max_q < 0 || window < 0 || !(scale >= 0.f) ||
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
    if (T < 0 || n_seqs < 0 || max_q < 0 || max_kv < 0 || table_stride < 0 || window < 0 || !(scale >= 0.f) ||
        std::isinf(scale))
        return MLORA_ERR_ARG;
    AttnArgs a{};
    mlora_status st = check_cache(cache, &a.cache);
    if (st != MLORA_OK)
        return st;
    const int32_t d = cache->head_dim;
    st = check_heads(n_q_heads, cache->n_kv_heads, d);
    if (st != MLORA_OK)
        return st;
    if (!rows_ok(q_stride, (int64_t)n_q_heads * d) || !rows_ok(out_stride, (int64_t)n_q_heads * d))
        return MLORA_ERR_SHAPE;
    if (!paged_sizes_ok(T, n_seqs, n_q_heads, cache->n_kv_heads, max_kv) || table_stride >= MAX_ROWS)
        return MLORA_ERR_UNSUPPORTED;
    if (T == 0 || n_seqs == 0 || max_q == 0)
        return MLORA_OK;
    if (q == nullptr || out == nullptr || cu_q == nullptr || kv_len == nullptr || !aligned16(q) || !aligned16(out) ||
        (max_kv > 0 && table_stride > 0 && page_table == nullptr))
        return MLORA_ERR_ARG;
    max_q = std::min(max_q, T);
    const PagedPlan p = paged_plan(T, n_seqs, n_q_heads, cache->n_kv_heads, d, max_q, max_kv);
    if (p.wide_chunks > 65535)
        return MLORA_ERR_UNSUPPORTED;
    uint8_t *base = (uint8_t *)(((uintptr_t)ws + 255) & ~(uintptr_t)255);
    if (p.total() > 0 && (ws == nullptr || ws_bytes < p.total() + (size_t)(base - (uint8_t *)ws)))
        return MLORA_ERR_WORKSPACE;
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
    a.max_q = max_q;
    a.max_kv = max_kv;
    a.causal = causal;
    a.window = seen_window(window, max_kv);
    a.scale = scale == 0.f ? (float)(1.0 / std::sqrt((double)d)) : scale;
    a.out = (uint16_t *)out;
    a.lse = lse;
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

mlora_status mlora_validate_pages(const mlora_cache *cache, const int32_t *page_table, int64_t table_stride,
                                  int32_t n_seqs, const int32_t *cu_q, const int32_t *kv_len, int64_t T,
                                  int64_t max_q, int64_t max_kv, int64_t *bad_value)
{
    if (cache == nullptr || n_seqs < 0 || T < 0 || table_stride < 0 || max_q < 0 || max_kv < 0)
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
        for (int64_t i = 0; i < pages; ++i) {
            const int32_t p = page_table[b * table_stride + i];
            if (p < 0 || p >= cache->n_pages)
                return bad(MLORA_ERR_INDEX, p);
        }
    }
    if (cu_q[n_seqs] != T)
        return bad(MLORA_ERR_SHAPE, cu_q[n_seqs]);
    return MLORA_OK;
}

}  // extern "C"
