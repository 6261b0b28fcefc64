// Host-side launchers of the attention step's kernels, called by attention_api.cpp.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mlora {

// A paged cache by value (include/mlora.h's mlora_cache; page_size = 1 << ps).
struct CacheGeom {
    uint8_t *k, *v;
    float *k_scale, *v_scale;
    int32_t n_pages, hkv, ps;
    bool fp8;
};

// ---- qk_rope.hip ---------------------------------------------------------------------------
struct RopeArgs {
    const uint16_t *qkv;
    int64_t T, row_stride;
    int32_t hq, hkv;
    const int32_t *pos;
    const uint64_t *turns;
    int32_t rot, interleaved;
    float magnitude;
    const uint16_t *qw, *kw;
    float eps;
    uint16_t *q_out, *k_out;
    int64_t q_stride, k_stride;
    CacheGeom cache;          // cache.k == nullptr: no cache
    const int32_t *slot;
};
hipError_t launch_qk_rope(const RopeArgs &a, int head_dim, hipStream_t stream);
hipError_t launch_cache_read(const CacheGeom &c, int head_dim, const int32_t *slot, int64_t T,
                             uint16_t *k, uint16_t *v, hipStream_t stream);

// ---- attention over rows or pages ----------------------------------------------------------
struct AttnArgs {
    const uint16_t *q, *k, *v;     // k, v: rows (whole prompts) only
    int64_t q_stride, k_stride, v_stride, out_stride;
    int64_t T, Tk;                 // query rows; key rows (whole prompts)
    int32_t n_seqs, hq, hkv, group;
    const int32_t *cu_q, *cu_k;    // cu_k: whole prompts
    const int32_t *kv_len, *table; // pages
    int64_t table_stride, max_q, max_kv;
    CacheGeom cache;
    int32_t causal, window;
    float scale;
    uint16_t *out;
    float *lse;
    // split over keys: parts as fp32 rows and their maxima and sums, which a second kernel joins.  Wide: chunks of
    // `chunk` keys (a multiple of 64), [token][head][n_chunks]; decode: two slots of max_rows rows a share
    // (part_o == nullptr: no split).
    int32_t chunk, n_chunks;
    float *part_o, *part_ml;       // [..][head_dim], [..][2]
    int32_t min_rows, max_rows;    // sequences this launch answers: rows = queries * group
};
// Whole prompts (cache unused) or, with pages, chunks of new tokens.
hipError_t launch_attn_wide(const AttnArgs &a, int head_dim, bool pages, hipStream_t stream);
constexpr int64_t CUS = 256;      // of an MI355X
constexpr int WIDE_ROWS = 128;    // rows (queries x heads of a group) of one workgroup
// Row blocks that a launch may have: each sequence's last one may be part empty, at most one more a sequence.
inline int64_t wide_items(const AttnArgs &a)
{
    const int64_t least = a.min_rows > a.group ? a.min_rows : a.group, seqs = a.T * a.group / least;
    const int64_t most = (a.max_q * a.group + WIDE_ROWS - 1) / WIDE_ROWS * a.n_seqs;
    const int64_t fill = a.T * a.group / WIDE_ROWS + (seqs < a.n_seqs ? seqs : a.n_seqs);
    return most < fill ? most : fill;
}
// Row blocks that workgroups are launched for over pages (a workgroup takes further ones where there are more): those
// that the rows fill and two workgroups a CU, unless all sequences may be wide.
inline int64_t wide_launched(const AttnArgs &a)
{
    const int64_t items = wide_items(a), card = 2 * CUS / ((int64_t)a.hkv * a.n_chunks);
    const int64_t few = (a.T * a.group + WIDE_ROWS - 1) / WIDE_ROWS + (card > 1 ? card : 1);
    return a.T * a.group > (int64_t)a.n_seqs * (a.min_rows - 1) || items < few ? items : few;
}
hipError_t launch_attn_wide_combine(const AttnArgs &a, int head_dim, hipStream_t stream);
// Sequences of up to 16 * nq rows (nq 1 or 2) over pages, their keys cut into `shares` equal shares, or (part_o ==
// nullptr) one workgroup a sequence and kv head, then shares = n_seqs * hkv.
constexpr int DECODE_UNIT = 128;  // keys: the unit that shares are made of
// Workgroups that a CU holds at a time.
constexpr int decode_slots(int head_dim, int nq) { return head_dim == 64 && nq == 1 ? 3 : 2; }
hipError_t launch_attn_decode(const AttnArgs &a, int head_dim, int nq, int shares, hipStream_t stream);
hipError_t launch_attn_combine(const AttnArgs &a, int head_dim, int shares, hipStream_t stream);
// Both kinds of sequences over pages in one launch: w as for launch_attn_wide, d as for launch_attn_decode (nq 1).
hipError_t launch_attn_mixed(const AttnArgs &w, const AttnArgs &d, int head_dim, int shares, hipStream_t stream);

}  // namespace mlora
