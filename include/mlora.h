/*
 * mlora: multi-LoRA adapted linear layer for AMD Instinct MI355X (gfx950).
 *
 * Computes, for a batch of T tokens in which every token carries its own K adapter slots,
 *
 *   y[t] = W x[t] + sum_{j : a = idx[t][j] != -1}  s[t][j] * f[a] * B[a] (A[a] x[t])
 *
 * with f[a] = alpha_a / r_a, or alpha_a / sqrt(r_a) for rsLoRA adapters.
 *
 * Sources (web pages):
 *  - "Multi-LoRA Serving Explained" (sevydevy.com): the LoRA layer W x + B(A x) scaled by
 *    alpha/r (B is out x rank, A is rank x in); one shared base product for the whole batch plus
 *    a per-token side path found through the token's slot id, -1 meaning base model only (the
 *    six-token batching script); stacked zero-padded slot buffers of width max_lora_rank
 *    (section "Why max-lora-rank costs memory even for small adapters"); sorting tokens by slot
 *    before shrink/expand and skipping the LoRA kernels when no token uses an adapter.
 *  - "[RFC]: Per-request activation of multiple LoRA adapters with static scales" (vLLM issue
 *    51940), Proposed Change: k slots per token with sentinel fill, per-adapter static scales,
 *    the slots iterated inside the kernels.
 *  - vLLM learning book, chapter "04. LoRA Serving", section 6 (PunicaWrapper): add_lora_linear,
 *    add_shrink (scaled x A, rank-wide intermediate) and add_expand (y += intermediate B).
 *  - "[vLLM] LoRA" (blog.secrett2633.cloud), PEFTHelper section: the rsLoRA factor.
 *
 * Conventions shared by every entry point:
 *  - Device pointers unless marked "host".  bf16 buffers are passed as void* holding bfloat16
 *    bits.  Everything is row-major and contiguous; base pointers must be 16-byte aligned.
 *  - The caller owns every buffer.  The library allocates no device memory on these calls:
 *    scratch space comes in through (ws, ws_bytes), sized by mlora_workspace_size(); its
 *    contents need no preparation and carry nothing from one call to the next.
 *  - Calls enqueue work on `stream` and return; the status reports only the synchronous
 *    argument checks and launch errors (MLORA_ERR_HIP).  No exception crosses the ABI.
 *  - Calls on one stream are ordered; two calls that share a workspace must not overlap.
 *  - Indices outside [-1, S) are undefined behaviour on the fast path; mlora_validate() checks
 *    them (and the ranks) synchronously.
 *  - Results are deterministic: the same inputs give the same output bits on every run.
 */
#ifndef MLORA_H
#define MLORA_H

#include <stddef.h>
#include <stdint.h>

#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    MLORA_OK = 0,
    MLORA_ERR_ARG = 1,         /* null pointer, negative size, misaligned pointer            */
    MLORA_ERR_SHAPE = 2,       /* inconsistent sizes (slice table, n_in not a multiple of 8) */
    MLORA_ERR_RANK = 3,        /* an adapter rank outside [1, R]                             */
    MLORA_ERR_INDEX = 4,       /* a slot index outside [-1, S)                               */
    MLORA_ERR_WORKSPACE = 5,   /* workspace missing or smaller than mlora_workspace_size()   */
    MLORA_ERR_HIP = 6,         /* a HIP call or kernel launch failed                         */
    MLORA_ERR_UNSUPPORTED = 7  /* outside the supported limits below                         */
} mlora_status;

/* Supported limits. */
#define MLORA_MAX_SLICES 4        /* output slices of a merged layer (QKV = 3)                 */
#define MLORA_MAX_RANK 512        /* slot width R: a power of two from 8 to 512                */
#define MLORA_MAX_SLOTS 16384     /* S                                                         */
#define MLORA_MAX_K 8             /* adapter slots per token                                   */

/* flags of mlora_linear */
#define MLORA_NO_ADAPTERS 1u      /* host hint: no token uses an adapter; run the base only    */
#define MLORA_PATH_DECODE 2u      /* force the decode kernels (token chunks of 64)             */
#define MLORA_PATH_TILED 4u       /* force the tiled prefill kernels (256-token tiles)         */
#define MLORA_W_PACKED 8u         /* W is in the packed layout of mlora_pack_weight            */
#define MLORA_PATH_GROUPED 16u    /* force the grouped decode: decode base, LoRA per adapter   */

/*
 * The adapter slot set of ONE layer: S slots, each R wide (R = max_lora_rank), an adapter of
 * rank r < R sitting zero-padded in the first r rows of A and first r columns of B.
 * A merged layer (e.g. QKV) has n_slices output slices: slice s owns output rows
 * [slice_start[s], slice_start[s+1]) and has its own down matrix A[a][s].
 */
typedef struct {
    const void *A;          /* bf16 [S][n_slices][R][n_in]; rows >= rank[a] must be zero     */
    const void *B;          /* bf16 [S][n_out][R];          cols >= rank[a] must be zero     */
    const float *factor;    /* fp32 [S]: alpha/r or alpha/sqrt(r) (see mlora_factor)         */
    int32_t S;              /* number of slots, 1..MLORA_MAX_SLOTS                           */
    int32_t R;              /* slot width, a power of two, 8 <= R <= MLORA_MAX_RANK          */
    int32_t n_slices;       /* 1..MLORA_MAX_SLICES                                           */
    int32_t slice_start[MLORA_MAX_SLICES + 1]; /* host values: 0 = s_0 < s_1 < .. = n_out.
                                                  With n_slices == 1 it may be all zero,
                                                  meaning {0, n_out}.                        */
    const int32_t *rank;    /* int32 [S] device: each slot's true rank r <= R, or NULL (= R).
                               With it the kernels skip the zero padding beyond r (same
                               results: the skipped products are exact zeros).  Values must be
                               in [1, R] (mlora_validate); larger ones are read as R.        */
} mlora_slots;

/* Text for a status code (static storage). */
const char *mlora_status_string(mlora_status status);

/* Text of the last HIP failure seen by this thread (the call that failed and HIP's message),
 * or "" if none; valid until the next failing call on the same thread. */
const char *mlora_last_error(void);

/*
 * Host helper: the scale factor of one adapter, alpha/r, or alpha/sqrt(r) when use_rslora is
 * non-zero ("[vLLM] LoRA", PEFTHelper section).  r is the adapter's true rank, not R.
 * Computed in double and rounded once to float.  Returns NaN for r < 1.
 */
float mlora_factor(float alpha, int32_t r, int32_t use_rslora);

/*
 * Host helper: bytes of one layer's slot buffers, S * (n_slices*R*n_in + n_out*R) * 2
 * ("Multi-LoRA Serving Explained", memory script: rank x (in + out) 16-bit numbers per adapted
 * layer, slots sized at max_lora_rank).  Returns -1 on negative arguments.
 */
int64_t mlora_slot_bytes(int32_t S, int32_t R, int64_t n_in, int64_t n_out, int32_t n_slices);

/*
 * Bytes of workspace that mlora_plan / mlora_shrink / mlora_linear need for these sizes
 * (an upper bound over every index map of this shape).  Returns 0 on invalid arguments.
 * The largest part is the tiled path's V blocks, about T x n_slices x 4 R x min(256 K, S)
 * bytes (T up to 1,048,576 tokens a launch): each 256-token tile's block is sized for a tile
 * that holds min(256 K, S) adapters, since a tile with too many adapters for the extra
 * k-steps takes the per-adapter route only while its fp32 sums fit the 64 MiB kept for them
 * (else the extra k-steps).  The rest: at most 64 MiB each of those fp32 sums and of the
 * shrink's partial blocks, and the decode kernels' split partials (16 n_out bytes a token of a
 * launch of up to 512).  For example 605 MiB at T = 16384, 4096 -> 11008, S = 100, R = 64;
 * 36 MiB for the 64-token decode batch at 4096 -> 4096; 3.2 GiB for a merged QKV layer with
 * S = 1000, R = 64 at T = 16384 (the size is linear in T: such callers can split the batch).
 */
size_t mlora_workspace_size(int64_t T, int32_t K, int64_t n_in, int64_t n_out,
                            const mlora_slots *slots);

/*
 * Slot activation ("Multi-LoRA Serving Explained": slots sized for max_lora_rank R, an adapter
 * of rank r < R zero-padded in its slot; an adapter whose rank exceeds R is rejected).  Loads
 * one adapter into slot `slot` of a slot set whose device buffers are A, B and factor (the
 * same buffers and layout as mlora_slots: A bf16 [S][n_slices][R][n_in], B bf16 [S][n_out][R],
 * factor fp32 [S]):
 *   A_src  bf16 [n_slices][r][n_in]   the adapter's down matrices (host or device memory)
 *   B_src  bf16 [n_out][r]            its up matrix (host or device memory)
 *   r      its true rank, 1 <= r <= R, else MLORA_ERR_RANK
 *   f      its scale factor (mlora_factor), written to factor[slot]
 * Rows r..R-1 of the slot's A and columns r..R-1 of its B are set to zero.  Everything is
 * enqueued on `stream` (asynchronous copies, then one kernel; no memset): host sources must
 * stay valid until the stream reaches the call, and are copied asynchronously only when
 * pinned.  The slot must not be in use by work in flight on other streams.  MLORA_ERR_ARG on
 * a NULL pointer, slot outside [0, S) or sizes below 1; MLORA_ERR_UNSUPPORTED outside the
 * limits above (S, R, n_slices).
 */
mlora_status mlora_slot_load(void *A, void *B, float *factor, int32_t S, int32_t R,
                             int32_t n_slices, int64_t n_in, int64_t n_out, int32_t slot,
                             const void *A_src, const void *B_src, int32_t r, float f,
                             hipStream_t stream);

/*
 * Packed base weight (a relayout for the matrix cores, done once when a weight is loaded; not
 * from the pages): the layer's W bf16 [n_out][n_in] rearranged so that each 16-row x 32-column
 * block is 1 KB contiguous in the order the v_mfma_f32_16x16x32_bf16 A operand takes it
 * (lane l: row l % 16, columns 8 (l / 16) .. +8), blocks ordered by row group, then column
 * block; zero padded to 16 rows and 32 columns:
 *   Wp[rg][kb][l][e] = W[16 rg + l % 16][32 kb + 8 (l / 16) + e]
 * mlora_packed_weight_bytes returns its size (0 on invalid sizes); mlora_pack_weight writes it
 * (one kernel on `stream`; W and Wp device, 16-byte aligned, not overlapping).  mlora_linear
 * with MLORA_W_PACKED then takes Wp in place of W and gives the same output bits: the
 * kernels read whole cache lines of W per load instruction.  MLORA_ERR_ARG on NULL or
 * misaligned pointers or sizes below 1, MLORA_ERR_SHAPE if n_in is not a multiple of 8.
 */
int64_t mlora_packed_weight_bytes(int64_t n_out, int64_t n_in);
mlora_status mlora_pack_weight(const void *W, int64_t n_out, int64_t n_in, void *Wp,
                               hipStream_t stream);

/*
 * Synchronous check of an index map and of the adapter ranks (blocks on `stream`).
 *   idx   int32 [T][K] device
 *   rank  int32 [S] host, true adapter ranks (may be NULL to skip the rank check)
 * Returns MLORA_ERR_INDEX if some idx is outside [-1, S), MLORA_ERR_RANK if some rank is
 * outside [1, R] ("Multi-LoRA Serving Explained": an adapter whose rank exceeds max_lora_rank
 * is rejected); the offending value is written to *bad_value (may be NULL).
 */
mlora_status mlora_validate(const int32_t *idx, int64_t T, int32_t K, const mlora_slots *slots,
                            const int32_t *rank, int64_t *bad_value, hipStream_t stream);

/*
 * Token-mapping plan ("Multi-LoRA Serving Explained": tokens sorted by slot, one group per
 * adapter; six-token script's stable argsort).  The flat pairs p = t*K + j are sorted by slot
 * idx[p] ascending, ties in ascending p; pairs holding -1 are dropped.
 * Outputs (device):
 *   perm       int32 [T*K]  first n_pairs entries: sorted pair indices
 *   seg_slot   int32 [S]    first n_seg entries: slot of each segment, ascending
 *   seg_start  int32 [S]    first position of the segment in perm
 *   seg_len    int32 [S]    its length
 *   counts     int32 [2]    {n_seg, n_pairs}
 * Exactly one result is correct, so the outputs are bit-exact.  T = 0 writes counts {0, 0}.
 * ws: at least the plan's part of mlora_workspace_size for T, K and S (MLORA_ERR_WORKSPACE
 * otherwise; maps of up to 8192 pairs over up to 1000 slots are sorted in one launch that
 * leaves it untouched).
 */
mlora_status mlora_plan(const int32_t *idx, int64_t T, int32_t K, int32_t S, int32_t *perm,
                        int32_t *seg_slot, int32_t *seg_start, int32_t *seg_len,
                        int32_t *counts, void *ws, size_t ws_bytes, hipStream_t stream);

/*
 * Shrink (learning book section 6, add_shrink; RFC stage 4: the K slots in one pass):
 *   v[j][t][s*R + rho] = scale[t][j] * factor[a] * sum_i A[a][s][rho][i] x[t][i],  a = idx[t][j]
 * and v[j][t][:] = 0 where idx[t][j] == -1.
 *   x      bf16 [T][n_in]
 *   idx    int32 [T][K]
 *   scale  fp32 [T][K], or NULL for all ones
 *   v      fp32 [K][T][n_slices*R]   (output, overwritten)
 */
mlora_status mlora_shrink(const void *x, int64_t T, int64_t n_in, const mlora_slots *slots,
                          const int32_t *idx, int32_t K, const float *scale, float *v, void *ws,
                          size_t ws_bytes, hipStream_t stream);

/*
 * Expand (learning book section 6, add_expand):
 *   y[t][n] = bf16( y[t][n] + sum_j [idx[t][j] != -1] sum_rho B[a][n][rho] v[j][t][s(n)*R+rho] )
 * where s(n) is the slice owning row n.  Rows whose slots are all -1 are left untouched.
 *   v  fp32 [K][T][n_slices*R]   (as written by mlora_shrink)
 *   y  bf16 [T][n_out]           (in/out; one rounding of the sum)
 */
mlora_status mlora_expand(const float *v, int64_t T, int64_t n_out, const mlora_slots *slots,
                          const int32_t *idx, int32_t K, void *y, hipStream_t stream);

/*
 * The whole layer, one rounding of each output:
 *   y[t] = bf16( W x[t] + sum_j [idx[t][j] != -1] scale[t][j] factor[a] B[a] (A[a] x[t]) )
 *   x  bf16 [T][n_in];  W  bf16 [n_out][n_in] (row n is output n);  y  bf16 [T][n_out] (out)
 *   idx, scale as in mlora_shrink.  slots may be NULL only with MLORA_NO_ADAPTERS.
 * With flags & MLORA_NO_ADAPTERS no LoRA kernel is launched (y = bf16(W x)); without it, an
 * all-sentinel map gives the same values.  T = 0 is a no-op.  By default the library picks
 * the decode kernels or the tiled kernels, whichever a host-side model of their measured
 * rates estimates faster for the sizes (the tiled kernels from about 1536 tokens at 4096 ->
 * 4096, 768 at 4096 -> 11008, 256 at vocabulary-wide outputs).  Where the decode kernels
 * are picked, a batch of 128 or more tokens whose per-token adapter reads (each (token, slot)
 * pair's A rows and B columns) would exceed both four times W's bytes and 200 MB
 * takes the grouped decode ("Multi-LoRA Serving Explained", the segmented method: tokens
 * sorted by adapter so that each adapter is read once per group): the decode kernels' base
 * product, the LoRA terms computed per adapter over its tokens.  The decode kernels compute
 * the shrink inside the GEMM pass, or, where 64 output rows would get 4 or more (token, slot)
 * pairs of a 64-token chunk (narrow outputs), with the per-pair shrink kernel ahead of a GEMM
 * of the base alone.  MLORA_PATH_DECODE /
 * MLORA_PATH_TILED / MLORA_PATH_GROUPED force one (more than one set: MLORA_ERR_ARG;
 * MLORA_PATH_GROUPED where the fp32 sums of one launch's up to 512 tokens exceed what the
 * grouped expand keeps, 64 MiB or one 256-token tile: MLORA_ERR_UNSUPPORTED).
 * mlora_workspace_size() covers every path.  With
 * MLORA_W_PACKED, W points to the packed layout written by mlora_pack_weight (same output
 * bits).
 */
mlora_status mlora_linear(const void *x, const void *W, int64_t T, int64_t n_in, int64_t n_out,
                          const mlora_slots *slots, const int32_t *idx, int32_t K,
                          const float *scale, void *y, uint32_t flags, void *ws, size_t ws_bytes,
                          hipStream_t stream);

/*
 * Which kernels mlora_linear runs for these sizes, slots and flags: MLORA_PATH_DECODE,
 * MLORA_PATH_TILED or MLORA_PATH_GROUPED (the choice is made on the host from the shapes and
 * flags alone, as described above; idx is not read).  Host only, no GPU call; slots' data
 * pointers are not checked.  Returns 0 where mlora_linear would fail its checks on these
 * arguments (sizes, slot geometry, conflicting flags, MLORA_PATH_GROUPED that does not fit).
 */
uint32_t mlora_linear_path(int64_t T, int64_t n_in, int64_t n_out, const mlora_slots *slots,
                           int32_t K, uint32_t flags);

/*
 * mlora_linear for callers that cannot allocate device memory (code under HIP graph capture,
 * tight serving loops, harnesses that forbid hipMalloc): the same computation, kernels and
 * output bits as mlora_linear with the same arguments, but its scratch space is a fixed array
 * of MLORA_NOALLOC_SCRATCH_BYTES inside the library (one per GPU, held until the process ends)
 * instead of a caller-provided workspace.  The caller still passes inputs and outputs.  It
 * calls no hipMalloc, hipFree or allocating routine.  A call whose path needs more scratch than
 * the fixed size (e.g. large tiled batches, very wide outputs) returns MLORA_ERR_WORKSPACE
 * before launching anything, with the needed size in mlora_last_error().  All calls on one GPU
 * share its array: calls that may overlap on one GPU (other streams, other threads) race and
 * must not be issued.  The array belongs to the device of `stream` (the current device for the
 * null stream).
 */
#define MLORA_NOALLOC_SCRATCH_BYTES (64u << 20)
mlora_status mlora_linear_noalloc(const void *x, const void *W, int64_t T, int64_t n_in,
                                  int64_t n_out, const mlora_slots *slots, const int32_t *idx,
                                  int32_t K, const float *scale, void *y, uint32_t flags,
                                  hipStream_t stream);

/*
 * ---- The attention step after a merged QKV layer -------------------------------------------
 *
 * A serving step runs mlora_linear on the merged layer, mlora_qk_rope on its rows (norms,
 * rotation, K and V into the paged cache), then mlora_attention (whole prompts) or
 * mlora_paged_attention (new tokens over the cache: one token a sequence when decoding).
 * head_dim is 64 or 128; query head i reads kv head i / (n_q_heads / n_kv_heads).
 */

/* Limits of the attention entry points. */
#define MLORA_CACHE_BF16 0        /* dtype of mlora_cache: bfloat16 values                     */
#define MLORA_CACHE_E4M3 1        /* 8-bit e4m3 codes with an fp32 scale per token and head    */
#define MLORA_MAX_PAGE 256        /* page_size: a power of two from 16 to 256                  */
#define MLORA_MAX_HEADS 1024      /* query heads                                               */

/* scaling of mlora_rope_turns */
#define MLORA_ROPE_PLAIN 0
#define MLORA_ROPE_LINEAR 1       /* every pair slowed down by factor                          */
#define MLORA_ROPE_PARTS 2        /* slow pairs by factor, fast ones kept, a ramp between      */

/*
 * A paged cache of one layer's keys and values.  Token `slot` sits in page slot / page_size at
 * offset slot % page_size; one kv head of a page is contiguous.  In e4m3 a vector is
 * code * scale, scale = max(amax, 2^-90) / 448 of the vector.
 */
typedef struct {
    void *k, *v;              /* bf16 or e4m3 [n_pages][n_kv_heads][page_size][head_dim]       */
    float *k_scale, *v_scale; /* fp32 [n_pages][n_kv_heads][page_size]; e4m3 only, else NULL   */
    int32_t n_pages, n_kv_heads, page_size, head_dim;
    int32_t dtype;            /* MLORA_CACHE_BF16 or MLORA_CACHE_E4M3                          */
} mlora_cache;

/*
 * Rotation by position of the first rot_dim values of a head (rot_dim a multiple of 16, at most
 * head_dim; 0: none, turns unused).  Pair i turns by frac(pos * turns[i] / 2^64) of a circle:
 * integer arithmetic modulo 2^64, exact at any position, so no table over positions is kept.
 * Pairs are (i, i + rot_dim / 2), or (2 i, 2 i + 1) when `interleaved` is non-zero; cosine and
 * sine are multiplied by `magnitude` (1, or what the scaling for long contexts asks for).
 */
typedef struct {
    const uint64_t *turns;    /* uint64 [rot_dim / 2] device (mlora_rope_turns)                */
    int32_t rot_dim;
    int32_t interleaved;
    float magnitude;
} mlora_rope;

/*
 * Host helper: turns[i] (host, rot_dim / 2 values) = 2^64 * f_i, f_i = base^(-2 i / rot_dim) /
 * (2 pi) turns per position, computed in long double.  MLORA_ROPE_LINEAR divides f_i by factor.
 * MLORA_ROPE_PARTS keeps pairs with at least `fast` turns in orig_len positions, divides those
 * with at most `slow` by factor, and ramps linearly in the number of turns between.
 * (The ramp is over turns.  Models that ramp over the pair's number have other frequencies: they
 * fill turns themselves.)
 * MLORA_ERR_ARG on NULL, rot_dim not a positive even number, base <= 1, factor < 1, unknown
 * scaling, or (PARTS) orig_len < 1 or fast <= slow.
 */
mlora_status mlora_rope_turns(int32_t rot_dim, double base, int32_t scaling, double factor,
                              int64_t orig_len, double fast, double slow, uint64_t *turns);

/* Host helper: bytes of a cache's k and v buffers (and scales) together; -1 on arguments outside
 * the limits above. */
int64_t mlora_cache_bytes(int64_t n_pages, int32_t n_kv_heads, int32_t page_size,
                          int32_t head_dim, int32_t dtype);

/*
 * Norm, rotation and cache write of T rows of a merged QKV layer.  Row t holds n_q_heads query
 * heads, then n_kv_heads key heads, then n_kv_heads value heads of head_dim values:
 *   n = x * (mean(x^2) + eps)^(-1/2) * weight   (queries and keys with a weight; else n = x)
 *   o = n rotated by pos[t]
 * in fp32, rounded once: queries to q_out, keys to k_out and to the cache, values (unchanged) to
 * the cache.
 *   qkv      bf16 [T] rows, row_stride elements apart
 *   pos      int32 [T]
 *   q_weight, k_weight  bf16 [head_dim], each may be NULL (no norm)
 *   q_out    bf16 [T][n_q_heads * head_dim], rows q_stride elements apart
 *   k_out    bf16 [T][n_kv_heads * head_dim], rows k_stride elements apart, or NULL
 *   cache, slot  where K and V go: slot int32 [T], a token whose slot is outside
 *            [0, n_pages * page_size) (-1: padding) is not stored; both NULL: no cache.  Two
 *            tokens of one call must not name the same slot.
 * q_out and k_out may be the rows' own query and key parts (in place) but overlap qkv in no
 * other way.  Strides are multiples of 8.  T = 0 is a no-op.
 */
mlora_status mlora_qk_rope(const void *qkv, int64_t T, int64_t row_stride, int32_t n_q_heads,
                           int32_t n_kv_heads, int32_t head_dim, const int32_t *pos,
                           const mlora_rope *rope, const void *q_weight, const void *k_weight,
                           float eps, void *q_out, int64_t q_stride, void *k_out,
                           int64_t k_stride, const mlora_cache *cache, const int32_t *slot,
                           hipStream_t stream);

/*
 * Cached tokens back as bf16 (e4m3: code * scale, rounded once):
 *   k, v  bf16 [T][n_kv_heads][head_dim] (either may be NULL);  slot int32 [T], tokens whose
 *   slot is outside [0, n_pages * page_size) give zeros.
 */
mlora_status mlora_cache_read(const mlora_cache *cache, const int32_t *slot, int64_t T, void *k,
                              void *v, hipStream_t stream);

/*
 * Attention over whole prompts, packed: sequence b owns query rows [cu_q[b], cu_q[b+1]) and key
 * rows [cu_k[b], cu_k[b+1]) (cu_k NULL: the same as cu_q).  With n queries and L keys, query i
 * stands at p = L - n + i and sees key j when j < L, j <= p (if causal) and j > p - window (if
 * window > 0):
 *   out = sum_j softmax_j(scale q . k_j) v_j    over the keys it sees, fp32 softmax
 *   lse = ln sum_j exp(scale q . k_j)
 * A query that sees no key gives zeros and lse = -inf; what it does not see has no effect on it,
 * infinities and NaN included.  Probabilities are rounded to bf16 for the product with V.
 *   q   bf16 [T_q][n_q_heads * head_dim], rows q_stride elements apart (k, v: T_k rows of
 *       n_kv_heads * head_dim; strides multiples of 8, so views of a merged row will do)
 *   out bf16 like q, rows out_stride apart;  lse fp32 [T_q][n_q_heads], or NULL
 *   cu_q, cu_k  int32 [n_seqs + 1] device, ascending from 0; entries beyond the T given are read
 *       as T.  max_q: an upper bound of the sequences' query counts (host; sizes the launch).
 *   scale  of the scores, finite and not negative; 0 means head_dim^(-1/2)
 * T_q and T_k are below 2^30, T_q * n_q_heads below 2^31, k_stride and v_stride below 2^24.
 */
mlora_status mlora_attention(const void *q, int64_t q_stride, const void *k, int64_t k_stride,
                             const void *v, int64_t v_stride, int64_t T_q, int64_t T_k,
                             int32_t n_seqs, const int32_t *cu_q, const int32_t *cu_k,
                             int32_t n_q_heads, int32_t n_kv_heads, int32_t head_dim,
                             int64_t max_q, int32_t causal, int32_t window, float scale,
                             void *out, int64_t out_stride, float *lse, hipStream_t stream);

/*
 * mlora_attention with a few first keys of each sequence that stay visible behind the window: with window > 0, query i
 * sees key j when j < L, j <= p (if causal) and j > p - window or j < sinks.  sinks >= 0; without a window it hides and
 * shows nothing.  All else as mlora_attention, which answers calls with sinks = 0 or a window of T_k (over pages: max_kv) or
 * more; in others a window of up to 64 keys, or any over an e4m3 cache, keeps 2^-15 of a probability.
 */
mlora_status mlora_attention_sinks(const void *q, int64_t q_stride, const void *k, int64_t k_stride,
                                   const void *v, int64_t v_stride, int64_t T_q, int64_t T_k,
                                   int32_t n_seqs, const int32_t *cu_q, const int32_t *cu_k,
                                   int32_t n_q_heads, int32_t n_kv_heads, int32_t head_dim,
                                   int64_t max_q, int32_t causal, int32_t window, int32_t sinks,
                                   float scale, void *out, int64_t out_stride, float *lse,
                                   hipStream_t stream);

/*
 * Attention of new tokens over a paged cache that already holds them (mlora_qk_rope first):
 * sequence b owns query rows [cu_q[b], cu_q[b+1]) and kv_len[b] cached tokens, token j in page
 * page_table[b][j / page_size].  Semantics as mlora_attention with L = kv_len[b]; decode is one
 * query row a sequence, and decode rows and prefill chunks may share a call.  Sequences of up to 16
 * rows (queries x heads of a kv head's group) keep 2^-15 of a probability instead of bf16's 2^-8,
 * but in calls whose max_q gives 17 to 32 rows.
 *   page_table int32 [n_seqs][table_stride] device; kv_len int32 [n_seqs] device, read as at
 *       most table_stride * page_size and max_kv
 *   max_q, max_kv  host upper bounds of the query counts and of kv_len (they size the launch;
 *       sequences with more queries than max_q are left unanswered)
 *   ws  mlora_paged_workspace_size() bytes for the same sizes, or for larger ones of the same heads: the
 *       size never falls as T, n_seqs, max_q or max_kv rises, so one workspace made for a server's
 *       largest step serves every other
 * max_kv and T are below 2^30, T * n_q_heads, n_seqs * n_kv_heads * (max_kv / 128 + 1) and table_stride
 * below 2^31; mlora_paged_workspace_size gives 0 where the call would refuse its sizes.
 * A page number outside the cache is read as its nearest valid page (no fault; such sequences'
 * results are meaningless): mlora_validate_pages checks a batch's tables on the host.
 */
size_t mlora_paged_workspace_size(int64_t T, int32_t n_seqs, int32_t n_q_heads,
                                  int32_t n_kv_heads, int32_t head_dim, int64_t max_q,
                                  int64_t max_kv);
mlora_status mlora_paged_attention(const void *q, int64_t q_stride, int64_t T, int32_t n_q_heads,
                                   const mlora_cache *cache, const int32_t *page_table,
                                   int64_t table_stride, int32_t n_seqs, const int32_t *cu_q,
                                   const int32_t *kv_len, int64_t max_q, int64_t max_kv,
                                   int32_t causal, int32_t window, float scale, void *out,
                                   int64_t out_stride, float *lse, void *ws, size_t ws_bytes,
                                   hipStream_t stream);

/*
 * mlora_paged_attention with a few first tokens of each sequence that stay visible behind the window (see
 * mlora_attention_sinks); the workspace is the same.  Pages that hold no token which a query sees may have been given
 * up: their entries in page_table may be any number, and what they hold has no effect.
 */
mlora_status mlora_paged_attention_sinks(const void *q, int64_t q_stride, int64_t T, int32_t n_q_heads,
                                         const mlora_cache *cache, const int32_t *page_table,
                                         int64_t table_stride, int32_t n_seqs, const int32_t *cu_q,
                                         const int32_t *kv_len, int64_t max_q, int64_t max_kv,
                                         int32_t causal, int32_t window, int32_t sinks, float scale,
                                         void *out, int64_t out_stride, float *lse, void *ws,
                                         size_t ws_bytes, hipStream_t stream);

/*
 * Host check of a paged batch before its arrays are copied to the GPU (all pointers host):
 * cu_q ascending from 0 to T, 0 <= kv_len[b] <= min(table_stride * page_size, max_kv), query
 * counts at most max_q, and every page that a sequence's kv_len reaches in [0, n_pages).
 * MLORA_ERR_SHAPE for the lengths, MLORA_ERR_INDEX for a page; the offending value in *bad_value
 * (may be NULL).
 */
mlora_status mlora_validate_pages(const mlora_cache *cache, const int32_t *page_table,
                                  int64_t table_stride, int32_t n_seqs, const int32_t *cu_q,
                                  const int32_t *kv_len, int64_t T, int64_t max_q,
                                  int64_t max_kv, int64_t *bad_value);

/*
 * The same for mlora_paged_attention_sinks: pages without a token that some query of the sequence sees are not looked
 * at (window 0: all pages are).
 */
mlora_status mlora_validate_pages_sinks(const mlora_cache *cache, const int32_t *page_table,
                                        int64_t table_stride, int32_t n_seqs, const int32_t *cu_q,
                                        const int32_t *kv_len, int64_t T, int64_t max_q,
                                        int64_t max_kv, int32_t window, int32_t sinks,
                                        int64_t *bad_value);

/*
 * mlora_paged_attention (without a window) of a batch whose sequences share first tokens: sequences
 * [group_start[g], group_start[g + 1]) hold the same first prefix_len[g] tokens in the cache, and these are read once for
 * the group, from the pages of its first sequence, instead of once a sequence.
 *   group_start int32 [n_groups + 1] device, ascending from 0 (read as at most n_seqs; sequences from the last entry on
 *       are in no group);  prefix_len int32 [n_groups] device, read as at most max_prefix and table_stride * page_size.
 *       A group may be empty, of one sequence, or share nothing.
 *   max_prefix  host upper bound of prefix_len
 * page_table and kv_len are mlora_paged_attention's, with all tokens of every sequence; a sequence whose queries do not
 * all see the whole prefix (kv_len less its queries, if causal, is below prefix_len) is answered from its own pages.
 * A group's first sequence must hold the whole prefix.  Probabilities of shared keys keep 2^-15, and so do those of other
 * keys of sequences of up to 16 rows, or 32 where max_q gives no more, and of all over an e4m3 cache; else 2^-8 (and as in
 * mlora_paged_attention, which answers the call, where n_groups or max_prefix is 0).  Sequences of more than 256 rows
 * (queries x heads of a kv head's group) read the prefix for themselves, for they fill the matrix cores without others.  It
 * pays where enough keys and values need not be read again (sequences x shared tokens x a token's bytes): over a bf16 cache
 * from 16 to 50 MB on for up to 16 sequences, from 30 to 130 MB on for more (64 sequences of 32 heads on 8, head_dim 128:
 * 370 tokens); over an e4m3 cache from 40 to 130 MB on, for fewer than 16 sequences from 100 MB on or not at all.  With less
 * mlora_paged_attention is faster, by up to 10 us.
 *   ws  mlora_prefix_workspace_size() bytes for the same sizes, or for larger ones of the same heads; the size
 *       never falls as any of them rises (0 where the call would refuse them).  It holds fp32 parts of every row, at least
 *       2 T n_q_heads (4 head_dim + 8) bytes, rows of long chunks too, though few calls write those (16384 tokens of 32 heads,
 *       head_dim 128, at once: 613 MB, mlora_paged_workspace_size 62)
 * n_groups and max_prefix are below 2^30, n_seqs * n_kv_heads * (max_kv / 32 + 1) below 2^31, other sizes as in
 * mlora_paged_attention.
 * mlora_validate_prefixes checks the groups on the host (all pointers host): group_start, 0 <= prefix_len <= max_prefix,
 * and that the table and each first sequence's kv_len reach that far; MLORA_ERR_SHAPE and the value where not.
 */
size_t mlora_prefix_workspace_size(int64_t T, int32_t n_seqs, int32_t n_groups, int32_t n_q_heads,
                                   int32_t n_kv_heads, int32_t head_dim, int64_t max_q,
                                   int64_t max_kv, int64_t max_prefix);
mlora_status mlora_prefix_attention(const void *q, int64_t q_stride, int64_t T, int32_t n_q_heads,
                                    const mlora_cache *cache, const int32_t *page_table,
                                    int64_t table_stride, int32_t n_seqs, const int32_t *cu_q,
                                    const int32_t *kv_len, int32_t n_groups,
                                    const int32_t *group_start, const int32_t *prefix_len,
                                    int64_t max_q, int64_t max_kv, int64_t max_prefix, int32_t causal,
                                    float scale, void *out, int64_t out_stride, float *lse, void *ws,
                                    size_t ws_bytes, hipStream_t stream);
mlora_status mlora_validate_prefixes(const mlora_cache *cache, int64_t table_stride, int32_t n_seqs,
                                     const int32_t *kv_len, int32_t n_groups,
                                     const int32_t *group_start, const int32_t *prefix_len,
                                     int64_t max_prefix, int64_t *bad_value);

/*
 * Profiling hook (not part of the computation).  mlora_trace_start creates 2*capacity HIP
 * events (no device memory); from then on every mlora_linear call records one event on its
 * stream right before and one right after each launch of its main product kernel (the decode
 * GEMM or the tiled GEMM), every mlora_shrink / mlora_expand call around its one kernel, and
 * every mlora_plan call around its kernels (one duration for the one or three), and the calls
 * of the attention step around theirs (one duration a call), for the first `capacity`
 * launches.
 * mlora_trace_stop waits for the recorded events, writes the duration of launch i in
 * milliseconds to ms[i] (host array of `capacity` floats; NULL discards them), releases the
 * events and returns the number of durations written (-1 on a HIP error).
 * Process-wide state, guarded by a lock; start returns MLORA_ERR_ARG unless
 * 1 <= capacity <= 2^20 and MLORA_ERR_HIP if an event cannot be created.
 */
mlora_status mlora_trace_start(int32_t capacity);
int32_t mlora_trace_stop(float *ms, int32_t capacity);

#ifdef __cplusplus
}
#endif

#endif /* MLORA_H */
