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
    int32_t sinks;                 // first keys that stay visible behind the window (0, or a window is set)
    // Sequences that share first keys: group g is the sequences [group_start[g], group_start[g + 1]), of which
    // prefix_len[g] keys are shared.  Parts of a row in row_parts slots of its own from slot row_slot on ([token][head]
    // [row_parts]), this launch's from number row_first on; cuts: where the decode kernel left a sequence and head.
    const int32_t *group_start, *prefix_len;
    int32_t n_groups, row_first, row_parts;
    int32_t alone_rows;            // sequences of more rows share nothing
    int64_t max_prefix, row_slot;
    int32_t *cuts;                 // [n_seqs][hkv][4]: first share (-1: a slot of the row), last share, shared keys
};
// Which keys a kernel's queries see, besides the causal limit: all or a window of them; a window and the first ones;
// those that a group's sequences share (the group's rows are one sequence's); a sequence's others.
enum { KEYS_PLAIN = 0, KEYS_SINKS = 1, KEYS_SHARED = 2, KEYS_OWN = 3 };
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
constexpr int OWN_UNIT = 32;      // of KEYS_OWN, whose shares are a wave's
// Workgroups that a CU holds at a time.
constexpr int decode_slots(int head_dim, int nq) { return head_dim == 64 && nq == 1 ? 3 : 2; }
hipError_t launch_attn_decode(const AttnArgs &a, int head_dim, int nq, int shares, hipStream_t stream);
hipError_t launch_attn_combine(const AttnArgs &a, int head_dim, int shares, hipStream_t stream);
// With a window of up to 64 keys a few keys share a row's weight, and the roundings of their probabilities even out the least
// (up to 1.5 times the error of a result that is rounded alone): both kernels take them in two bf16 parts.  Such calls are
// short (8 prompts of 2048, windows of 32 and 64: 111 and 105 us, with two parts 121 and 116; one of 16384: 98 and 100, 107 and
// 108).  The decode kernel's two column tiles spill 56 registers for them at D = 128 (27 with one part; 32 x 5 tokens, window 64:
// 14.6 us, with two parts 17.9, e4m3 11.9 and 13.6, D = 64 7.5 and 7.8; 256 x 8 81 and 101).
inline bool few_keys(const AttnArgs &a) { return a.sinks > 0 && a.window <= 64; }
// And over an e4m3 cache, whatever the window, and behind shared prefixes: there the matrix cores take a probability times its
// value's scale, so that the largest one, exactly 1, is rounded as well, and where a few first keys hold most of the weight one
// rounding is in all of a row's results (windows of 70 to 300: up to 2.1 times the rms error of a result that is rounded alone,
// with two parts 1.0; in bf16 1.1 at the most).  D = 128: a chunk of 2048 over 8048 keys, window 2048, 101 us, with two parts
// 127; beside 256 tokens 256 and 268; 32 x 5 tokens, window 2048, 57 and 62; 256 x 5, window 1024, 188 and 207; a chunk of D =
// 64 52 and 58.  Chunks behind a prefix: 2.05 times that error; 128 tokens and a chunk of 1024 behind 8000 keys 277 and 322, 32
// and 300 behind 4000 82 and 99.
template <int KEYS, bool FP8, int PARTS> constexpr int key_parts = KEYS != KEYS_PLAIN && FP8 ? 2 : PARTS;
// Both kinds of sequences over pages in one launch: w as for launch_attn_wide, d as for launch_attn_decode (nq 1).
hipError_t launch_attn_mixed(const AttnArgs &w, const AttnArgs &d, int head_dim, int shares, hipStream_t stream);

// Sequences that share first keys: s (wide: the shared keys, n_chunks chunks), w and d (their own ones; as for
// launch_attn_mixed, but `wide` = false: no sequence has more rows than 16 nq) in one launch, and the join of all parts.
hipError_t launch_attn_prefix(const AttnArgs &s, const AttnArgs &w, const AttnArgs &d, int head_dim, bool wide, int nq,
                              int shares, hipStream_t stream);
hipError_t launch_attn_prefix_join(const AttnArgs &s, const AttnArgs &w, const AttnArgs &d, int head_dim,
                                   hipStream_t stream);

}  // namespace mlora
