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
    // split over keys: sequences of more than one chunk leave fp32 partial rows that
    // launch_attn_combine joins
    int32_t chunk, n_chunks;       // keys per chunk (a multiple of 64), chunks a launch covers
    float *part_o, *part_ml;       // [rows][n_chunks][head_dim], [rows][n_chunks][2]
    int32_t min_rows, max_rows;    // sequences this launch answers: rows = queries * group
};
// Whole prompts (cache unused) or, with pages, chunks of new tokens.
hipError_t launch_attn_wide(const AttnArgs &a, int head_dim, bool pages, hipStream_t stream);
constexpr int WIDE_ROWS = 128;    // rows (queries x heads of a group) of one workgroup
hipError_t launch_attn_wide_combine(const AttnArgs &a, int head_dim, hipStream_t stream);
// Sequences of up to 16 * nq rows (nq 1 or 2) over pages.
hipError_t launch_attn_decode(const AttnArgs &a, int head_dim, int nq, int waves, hipStream_t stream);
hipError_t launch_attn_combine(const AttnArgs &a, int head_dim, hipStream_t stream);

}  // namespace mlora
