// Attention of a batch whose sequences share long prefixes: a group's rows (queries x heads, of all its sequences) are
// multiplied with the prefix together, so that it is read once, and each sequence's rows with its own further keys;
// what both leave of a row, fp32 outputs o with their maximum m and sum l, is joined:
//   M = max m_c,  out = sum_c 2^(m_c - M) o_c / sum_c 2^(m_c - M) l_c
// The shared part is the wide kernel's (attn_wide_body.h: the group as one sequence of queries that see every key),
// cut into chunks of keys; the own part is the mixed batch's (attn_mixed.hip).  All of them in one launch, for the former
// is bound by the matrix cores and the latter by memory.  Measured (D = 128, 32 heads on 8, both kernels): 64 tokens behind 4096
// keys, 1 to 1024 of their own, 46 to 47 us (3.3 TB/s of what has to be read), 256 of an e4m3 cache in four groups 82 us (2.8),
// 32 x 5 of D = 64 behind 8192 and 6001 25.5 us, 128 tokens and a chunk of 1024 behind 8000 215 to 217 us (745 TFLOP/s), 8 tokens
// behind 1000 keys 14 us; in a graph of calls on three inputs 48, 84, 29, 216 and 16 us, where mlora_paged_attention takes 155,
// 196, 51, 586 and 19.  Bound by the own keys' reads and, as long as both run, by what the two kinds cost each other; the join
// is 5 to 11 us.
#include "attn_decode_body.h"
#include "attn_mixed.h"
#include "attn_wide_body.h"

namespace mlora {

template <int D, int NQ, bool FP8, bool WIDE>
__global__ __launch_bounds__(256, 2) void attn_prefix_kernel(AttnArgs s, AttnArgs w, AttnArgs d, uint32_t shared_x,
                                                             uint32_t wide_x, uint32_t shares)
{
    constexpr int SRC = FP8 ? AW_PAGES_E4M3 : AW_PAGES;
    constexpr int LDS_D = decode_lds<D, NQ, KEYS_OWN>, LDS_W = wide_lds<D, SRC, 1, KEYS_OWN>, LDS = LDS_W > LDS_D ? LDS_W : LDS_D;
    __shared__ __attribute__((aligned(16))) uint8_t smem[LDS];
    uint32_t i = blockIdx.x;
    const uint32_t shared = shared_x * s.n_chunks;
    if (!mixed_place(shared + (WIDE ? wide_x * w.n_chunks : 0), shares, &i)) {
        attn_decode_body<D, NQ, FP8, KEYS_OWN>(d, i, shares, smem);
    } else if (WIDE && i < wide_x * w.n_chunks) {
        // (the longer ones: over a bf16 cache one bf16 part of a probability, as in chunks of mlora_paged_attention: up to 1.36
        // times the rms error of a result that is rounded alone; two parts 1.0, but 128 tokens and a chunk of 1024 behind 8000
        // keys 272 us, so 227.  e4m3: see key_parts; 277 us with one part, with two 322)
        attn_wide_pages<D, SRC, KEYS_OWN, key_parts<KEYS_OWN, FP8, 1>>(w, (int)(i % wide_x), (int)(i / wide_x), (int)wide_x,
                                                                       smem);
    } else {
        if (WIDE)
            i -= wide_x * w.n_chunks;
        attn_wide_body<D, SRC, 1, false, KEYS_SHARED>(s, (int)(i % shared_x), (int)(i / shared_x), smem);
    }
}

// The parts of a row, joined by D / 4 lanes (`lane` of them; a row's lanes are in step): parts [0, n) at slot(c).  (join_parts
// takes a wave a row; here every row has parts, and a wave's loads of 16 bytes a lane serve 2 or 4 rows.)
template <int D, class Slot>
__device__ __forceinline__ void join_row(const AttnArgs &a, int n, Slot slot, int64_t t, int hd, int lane)
{
    constexpr int LPR = D / 4, AHEAD = 8;
    auto largest = [](float v) {
#pragma unroll
        for (int off = LPR / 2; off >= 1; off >>= 1)
            v = fmaxf(v, __shfl_xor(v, off, 64));
        return v;
    };
    auto load_ml = [&](int c) { return c < n ? *(const f32x2 *)(a.part_ml + 2 * slot(c)) : f32x2{ATTN_LOWEST, 0.f}; };
    const f32x2 first = load_ml(lane);
    float mx = first[0];
    for (int c = lane + LPR; c < n; c += LPR)
        mx = fmaxf(mx, load_ml(c)[0]);
    mx = largest(fmaxf(mx, ATTN_LOWEST));
    float sum = 0.f;
    f32x4 acc = {0.f, 0.f, 0.f, 0.f};
    for (int c0 = 0; c0 < n; c0 += LPR) {
        const f32x2 ml = c0 ? load_ml(c0 + lane) : first;
        const float f = c0 + lane < n ? __builtin_amdgcn_exp2f(ml[0] - mx) : 0.f;       // this lane's part
        sum += f * ml[1];
        const int m = min(LPR, n - c0);
        for (int i = 0; i < m; i += AHEAD) {
            f32x4 x[AHEAD];
#pragma unroll
            for (int j = 0; j < AHEAD; ++j)
                x[j] = *(const f32x4 *)(a.part_o + slot(c0 + min(i + j, m - 1)) * D + 4 * lane);
#pragma unroll
            for (int j = 0; j < AHEAD; ++j) {
                const float w = __shfl(f, i + j, LPR);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    acc[e] += i + j < m ? w * x[j][e] : 0.f;
            }
        }
    }
#pragma unroll
    for (int off = LPR / 2; off >= 1; off >>= 1)
        sum += __shfl_xor(sum, off, 64);
    const float inv = sum > 0.f ? 1.f / sum : sum == 0.f ? 0.f : sum;
    *(u32x2 *)(a.out + t * a.out_stride + (int64_t)hd * D + 4 * lane) =
        u32x2{cvt_bf16x2(acc[0] * inv, acc[1] * inv), cvt_bf16x2(acc[2] * inv, acc[3] * inv)};
    if (a.lse && lane == 0)
        a.lse[t * a.hq + hd] = sum == 0.f ? -INFINITY : (mx + __builtin_amdgcn_logf(sum)) * (1.f / ATTN_LOG2E);
}

// The join, D / 4 lanes a (token, head): the chunks of the shared keys, and what its own keys left: a slot of the row, or
// (decode) the parts of the shares that it was cut between, or (wide) its chunks.  A wave takes `heads` heads of a token.
template <int D>
__global__ __launch_bounds__(256) void attn_prefix_join_kernel(AttnArgs s, AttnArgs w, AttnArgs d, int heads)
{
    const uint32_t item = blockIdx.x * 4 + (threadIdx.x >> 6), pieces = (uint32_t)(d.hq + heads - 1) / heads;
    const int t = uniform((int)(item / pieces)), h0 = uniform((int)(item - t * pieces)) * heads;
    const int lane = threadIdx.x & 63;
    if (t >= d.T)
        return;
    // the token's sequence: as in a batch of single tokens, or searched for, 256 sequences a trip to memory
    int b = min(t, d.n_seqs - 1), q0 = d.cu_q[b], q1 = d.cu_q[b + 1];
    if (t < q0 || t >= q1) {
        b = -1;
        for (int s0 = 0; s0 < d.n_seqs && b < 0; s0 += 256) {
            int from[4], to[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int i = min(s0 + 64 * j + lane, d.n_seqs - 1);
                from[j] = d.cu_q[i];
                to[j] = d.cu_q[i + 1];
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint64_t hit = ballot64(from[j] <= t && t < to[j]);
                if (b < 0 && hit) {
                    const int src = __ffsll((unsigned long long)hit) - 1;
                    b = min(s0 + 64 * j + src, d.n_seqs - 1);
                    q0 = __builtin_amdgcn_readlane(from[j], src);
                    q1 = __builtin_amdgcn_readlane(to[j], src);
                }
            }
        }
        if (b < 0)
            return;
    }
    q0 = max(q0, 0);
    const int n = (int)min((int64_t)q1, d.T) - q0;
    if (n > d.max_q)
        return;
    constexpr int LPR = D / 4;
    const int64_t rows = (int64_t)n * d.group;
    const int end = min(h0 + heads, d.hq), l = lane & (LPR - 1);
    if (rows <= d.max_rows) {
        for (int hd = h0 + lane / LPR; hd < end; hd += 64 / LPR) {
            const int h = hd / d.group, row = (t - q0) * d.group + hd - h * d.group;
            const u32x4 c = *(const u32x4 *)(d.cuts + 4 * ((int64_t)b * d.hkv + h));
            const int w0 = (int)c[0], w1 = (int)c[1], keys = (int)c[2], chunks = (keys + s.chunk - 1) / s.chunk;
            if (w0 < 0 && keys == 0)        // answered whole
                continue;
            join_row<D>(d, chunks + (w0 < 0 ? 1 : w1 - w0 + 1), [&](int i) {
                return i < chunks ? row_slot(s, t, hd, i)
                       : w0 < 0   ? row_slot(d, t, hd, 0)
                                  : part_slot(d, w0 + i - chunks, i > chunks, row);
            }, t, hd, l);
        }
    } else {
        const int L = (int)min((int64_t)max(d.kv_len[b], 0), min(d.max_kv, d.table_stride << d.cache.ps));
        const int keys = shared_keys(d, b, n, L), chunks = (keys + s.chunk - 1) / s.chunk;
        if (w.n_chunks == 1 && keys == 0)
            return;
        const int hi = w.causal ? min(L, L - n + t - q0 + 1) : L, from = keys & ~(AW_BN - 1);
        const int own = hi > keys ? (hi - 1 - from) / w.chunk + 1 : 1;
        for (int hd = h0 + lane / LPR; hd < end; hd += 64 / LPR)
            join_row<D>(d, chunks + own, [&](int i) {
                return i < chunks ? row_slot(s, t, hd, i) : row_slot(w, t, hd, i - chunks);
            }, t, hd, l);
    }
}

hipError_t launch_attn_prefix(const AttnArgs &s, const AttnArgs &w, const AttnArgs &d, int head_dim, bool wide, int nq,
                              int shares, hipStream_t stream)
{
    // row blocks of the groups: each one's last may be part empty
    const int64_t all = s.T * s.group, shared_x = (all / WIDE_ROWS + (all < s.n_groups ? all : s.n_groups)) * s.hkv;
    const int64_t wide_x = wide ? wide_launched(w) * w.hkv : 0;
    const int64_t blocks = shared_x * s.n_chunks + wide_x * w.n_chunks + shares;
    if (blocks > 0x7fffffff)
        return hipErrorInvalidValue;
    const dim3 grid((unsigned)blocks);
    const uint32_t x[3] = {(uint32_t)shared_x, (uint32_t)wide_x, (uint32_t)shares};
#define PRE(D, NQ, F, W) attn_prefix_kernel<D, NQ, F, W><<<grid, dim3(256), 0, stream>>>(s, w, d, x[0], x[1], x[2])
#define PRE_W(D, F) (wide ? PRE(D, 1, F, true) : nq == 1 ? PRE(D, 1, F, false) : PRE(D, 2, F, false))
#define PRE_F(D) (d.cache.fp8 ? PRE_W(D, true) : PRE_W(D, false))
    head_dim == 64 ? PRE_F(64) : PRE_F(128);
#undef PRE_F
#undef PRE_W
#undef PRE
    return hipGetLastError();
}

hipError_t launch_attn_prefix_join(const AttnArgs &s, const AttnArgs &w, const AttnArgs &d, int head_dim, hipStream_t stream)
{
    // a wave's lanes full, and more heads a wave where there are rows enough to fill the card with waves
    const int least = 256 / head_dim;
    int heads = least;
    while (heads < 8 && d.T * d.hq >= 2 * heads * INT64_C(8192))
        heads *= 2;
    const int64_t waves = d.T * ((d.hq + heads - 1) / heads);
    if (waves > INT64_C(0x7fffffff))
        return hipErrorInvalidValue;
    const unsigned blocks = (unsigned)((waves + 3) / 4);
    if (head_dim == 64)
        attn_prefix_join_kernel<64><<<blocks, 256, 0, stream>>>(s, w, d, heads);
    else
        attn_prefix_join_kernel<128><<<blocks, 256, 0, stream>>>(s, w, d, heads);
    return hipGetLastError();
}

}  // namespace mlora
