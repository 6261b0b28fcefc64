// Attention of few query rows over a paged cache (decode), and the join of split rows.
//
// The rows of one sequence and kv head (queries x heads of the group, up to 16 NQ) are the
// columns of 16x16x32 MFMA tiles, so K and V are read once for all of them.  A workgroup takes
// one (sequence, kv head, chunk of keys); its four waves take steps of 32 keys in turn, each with
// its own running maximum, sums and accumulators, joined in LDS at the end.  K goes from memory
// straight into the fragments; V through a wave's own piece of LDS, written by rows and read
// transposed, so the loop has no barrier.  The next step's loads are issued while this one's
// softmax and second product run.  Bound by HBM (or, for a short batch, by latency).
#include <algorithm>

#include "attention.h"
#include "attention_device.h"

namespace mlora {

// Chunks of a sequence: keys [lo, L) that its queries can see, cut at multiples of `chunk`.
struct SeqChunks {
    int q0, n, L, lo, c0, count;
};

__device__ __forceinline__ SeqChunks seq_chunks(const AttnArgs &a, int b)
{
    SeqChunks s;
    s.q0 = (int)min((int64_t)max(a.cu_q[b], 0), a.T);
    s.n = (int)min((int64_t)max(a.cu_q[b + 1], 0), a.T) - s.q0;
    s.L = (int)min((int64_t)max(a.kv_len[b], 0),
                   min(a.max_kv, a.table_stride << a.cache.ps));
    s.lo = a.window > 0 ? max(0, s.L - s.n - a.window + 1) : 0;
    s.c0 = s.lo / a.chunk;
    s.count = s.L > s.lo ? (s.L - 1) / a.chunk - s.c0 + 1 : 1;
    return s;
}

__device__ __forceinline__ bool answers(const AttnArgs &a, const SeqChunks &s)
{
    return s.n > 0 && s.n <= a.max_q && (int64_t)s.n * a.group >= a.min_rows &&
           (int64_t)s.n * a.group <= a.max_rows;
}

template <int D, int NQ, bool FP8>
__global__ __launch_bounds__(256) void attn_decode_kernel(AttnArgs a)
{
    constexpr int KS = D / 32;          // k-steps of the first product
    constexpr int DB = D / 16;          // row blocks of the second
    constexpr int LD = FP8 ? D / 64 : D / 32;   // 16-byte loads per lane and 16-key block
    constexpr int OS = D + 4;           // row stride of the joined accumulators in LDS
    constexpr int VW = 32 * D;          // a wave's V rows in LDS
    __shared__ __attribute__((aligned(16))) uint16_t lds[4 * (VW > 32 * OS ? VW : 32 * OS)];
    __shared__ float ml[4][16][2];

    const int b = (int)(blockIdx.x / a.hkv), h = (int)(blockIdx.x - (unsigned)b * a.hkv);
    const SeqChunks sq = seq_chunks(a, b);
    const int c = blockIdx.y;
    if (!answers(a, sq) || c >= sq.count)
        return;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lane = threadIdx.x & 63, col = lane & 15, g = lane >> 4;
    const int rows = sq.n * a.group, L = sq.L;
    const int k0 = max((sq.c0 + c) * a.chunk, sq.lo & ~31), k1 = min(L, (sq.c0 + c + 1) * a.chunk);
    const int32_t *__restrict__ table = a.table + (int64_t)b * a.table_stride;
    const int ps = a.cache.ps, pm = (1 << ps) - 1;
    uint16_t *vl = lds + wave * VW;

    // Q as B operand: column = row of the sequence, 8 values a k-step; its position
    u32x4 qf[NQ][KS];
    int pos[NQ];
#pragma unroll
    for (int j = 0; j < NQ; ++j) {
        const int r = min(16 * j + col, rows - 1), i = r / a.group, hd = h * a.group + r - i * a.group;
        pos[j] = L - sq.n + i;
        const uint16_t *qr = a.q + (sq.q0 + i) * a.q_stride + (int64_t)hd * D;
#pragma unroll
        for (int s = 0; s < KS; ++s)   // e4m3 K comes 16 values a lane: two k-steps side by side
            qf[j][s] = *(const u32x4 *)(qr + (FP8 ? 64 * (s >> 1) + 16 * g + 8 * (s & 1) : 32 * s + 8 * g));
    }
    const float cs = a.scale * ATTN_LOG2E;

    f32x4 o[NQ][DB];
    float m[NQ], l[NQ];
#pragma unroll
    for (int j = 0; j < NQ; ++j) {
        m[j] = ATTN_LOWEST;
        l[j] = 0.f;
#pragma unroll
        for (int d = 0; d < DB; ++d)
            o[j][d] = f32x4{0.f, 0.f, 0.f, 0.f};
    }

    u32x4 kr[2][LD], vr[2][LD];
    f32x4 ks[2], vs[2];
    int pg[2];
    // pages of the two 16-key blocks of the step at kb (blocks past the end: the last key's page)
    auto lookup = [&](int kb) {
#pragma unroll
        for (int u = 0; u < 2; ++u)
            pg[u] = clamp_page(table[min(kb + 16 * u, L - 1) >> ps], a.cache.n_pages);
    };
    auto load = [&](int kb) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int64_t at = (((int64_t)pg[u] * a.cache.hkv + h) << ps) + (min(kb + 16 * u, (L - 1) & ~15) & pm);
            const int esz = FP8 ? 1 : 2;
            const uint8_t *kp = a.cache.k + (at + col) * D * esz + 16 * g;
            const uint8_t *vp = a.cache.v + (at + col) * D * esz + 16 * g;
#pragma unroll
            for (int s = 0; s < LD; ++s)
                kr[u][s] = *(const u32x4 *)(kp + 64 * s);
#pragma unroll
            for (int s = 0; s < LD; ++s)
                vr[u][s] = *(const u32x4 *)(vp + 64 * s);
            if (FP8) {
                ks[u] = *(const f32x4 *)(a.cache.k_scale + at + 4 * g);
                vs[u] = *(const f32x4 *)(a.cache.v_scale + at + 4 * g);
            }
        }
    };

    int kb = k0 + 32 * wave;
    if (kb < k1) {
        lookup(kb);
        load(kb);
        if (kb + 128 < k1)
            lookup(kb + 128);
    }
    for (; kb < k1; kb += 128) {
        // a step whose keys some query of the sequence does not see
        const bool edge = kb + 32 > L - sq.n + 1 || (a.window > 0 && kb <= L - 1 - a.window);
        // S^T: rows = keys 16 u + 4 g + i, column = query
        f32x4 st[NQ][2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
#pragma unroll
            for (int j = 0; j < NQ; ++j)
                st[j][u] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int s = 0; s < KS; ++s) {
                bf16x8 kf;
                if (FP8)
                    kf = as_bf16x8(e4m3_to_bf16x8(kr[u][s >> 1][2 * (s & 1)], kr[u][s >> 1][2 * (s & 1) + 1]));
                else
                    kf = as_bf16x8(kr[u][FP8 ? 0 : s]);
#pragma unroll
                for (int j = 0; j < NQ; ++j)
                    st[j][u] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kf, as_bf16x8(qf[j][s]), st[j][u], 0, 0, 0);
            }
        }
        // V rows into LDS ([key][D], 16-byte pieces swizzled by key); rows outside [lo, L) as zeros
        uint32_t bad = 0;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int key = 16 * u + col;
            const bool in = kb + key < L && kb + key >= sq.lo;
#pragma unroll
            for (int s = 0; s < LD; ++s) {
                u32x4 w[2];
                if (FP8) {
                    w[0] = e4m3_to_bf16x8(vr[u][s][0], vr[u][s][1]);
                    w[1] = e4m3_to_bf16x8(vr[u][s][2], vr[u][s][3]);
                } else {
                    w[0] = vr[u][s];
                }
#pragma unroll
                for (int e = 0; e < (FP8 ? 2 : 1); ++e) {
                    if (edge) {
                        w[e] = in ? w[e] : u32x4{0, 0, 0, 0};
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            bad = not_finite(bad, w[e][i]);
                    }
                    const int piece = FP8 ? 8 * s + 2 * g + e : 4 * s + g;   // D = 64: 8 pieces a row
                    *(u32x4 *)(vl + key * D + 8 * (piece ^ (key & (D / 8 - 1)))) = w[e];
                }
            }
        }
        f32x4 kss[2], vss[2];
        if (FP8) {
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                kss[u] = ks[u];
                vss[u] = vs[u];
            }
        }
        // the next step's loads
        if (kb + 128 < k1) {
            load(kb + 128);
            if (kb + 256 < k1)
                lookup(kb + 256);
        }
        u32x4 pf[NQ];
#pragma unroll
        for (int j = 0; j < NQ; ++j) {
            float mx = -INFINITY;
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float s = st[j][u][i] * cs;
                    if (FP8)
                        s *= kss[u][i];
                    if (edge) {
                        const int key = kb + 16 * u + 4 * g + i;
                        const bool see = key < L && (!a.causal || key <= pos[j]) &&
                                         (a.window <= 0 || key > pos[j] - a.window);
                        s = see ? s : -INFINITY;
                    }
                    st[j][u][i] = s;
                    mx = fmaxf(mx, s);
                }
            if (__any(mx > m[j] + ATTN_SLACK)) {
                mx = fmaxf(mx, __shfl_xor(mx, 16, 64));
                mx = fmaxf(mx, __shfl_xor(mx, 32, 64));
                // (each column on its own: a row's bits do not depend on its neighbours)
                const float mn = mx > m[j] + ATTN_SLACK ? mx : m[j], f = __builtin_amdgcn_exp2f(m[j] - mn);
                m[j] = mn;
                l[j] *= f;
#pragma unroll
                for (int d = 0; d < DB; ++d)
                    o[j][d] *= f;
            }
            float p[8];
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float e = __builtin_amdgcn_exp2f(st[j][u][i] - m[j]);
                    l[j] += e;
                    // (a masked key's scale may be anything)
                    p[4 * u + i] = !FP8 ? e : edge && st[j][u][i] == -INFINITY ? 0.f : e * vss[u][i];
                }
#pragma unroll
            for (int i = 0; i < 4; ++i)
                pf[j][i] = cvt_bf16x2(p[2 * i], p[2 * i + 1]);
        }
        // O^T += V^T P^T; k index (g, e) is key 16 (e / 4) + 4 g + e % 4
        auto vfrag = [&](int d) {
            u32x4 f;
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int key = 16 * u + 4 * g + (col >> 2), piece = 2 * d + ((col & 3) >> 1);
                const u32x2 w = lds_read_tr(vl + key * D + 8 * (piece ^ (key & (D / 8 - 1))) + 4 * (col & 1));
                f[2 * u] = w[0];
                f[2 * u + 1] = w[1];
            }
            return f;
        };
        if (!(edge && __any((bad & 0x80008000u) != 0))) {
#pragma unroll
            for (int d = 0; d < DB; ++d) {
                const bf16x8 vf = as_bf16x8(vfrag(d));
#pragma unroll
                for (int j = 0; j < NQ; ++j)
                    o[j][d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vf, as_bf16x8(pf[j]), o[j][d], 0, 0, 0);
            }
        } else {
            // V holds an infinity or NaN where some query must not see it (0 x NaN is NaN): one key at a
            // time, kept only by the queries that see it
#pragma unroll 1
            for (int key = 0; key < 32; ++key) {
                const bool mine = g == ((key & 15) >> 2);
                const int e = 4 * (key >> 4) + (key & 3);
                const uint32_t half = (e & 1) ? 0xffff0000u : 0xffffu;
                const int ka = kb + key;
#pragma unroll
                for (int d = 0; d < DB; ++d) {
                    u32x4 f = vfrag(d);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        f[i] = mine && i == (e >> 1) ? f[i] & half : 0u;
#pragma unroll
                    for (int j = 0; j < NQ; ++j) {
                        const f32x4 t = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(f), as_bf16x8(pf[j]), o[j][d], 0, 0, 0);
                        const bool see = ka < L && (!a.causal || ka <= pos[j]) &&
                                         (a.window <= 0 || ka > pos[j] - a.window);
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            o[j][d][i] = see ? t[i] : o[j][d][i];
                    }
                }
            }
        }
    }

    // join the four waves, 16 rows at a time
    float *of = (float *)lds;
#pragma unroll
    for (int j = 0; j < NQ; ++j) {
        if (j > 0 && 16 * j >= rows)
            break;
        float lj = l[j] + __shfl_xor(l[j], 16, 64);
        lj += __shfl_xor(lj, 32, 64);
        __syncthreads();
#pragma unroll
        for (int d = 0; d < DB; ++d)
            *(f32x4 *)(of + (wave * 16 + col) * OS + 16 * d + 4 * g) = o[j][d];
        if (g == 0) {
            ml[wave][col][0] = m[j];
            ml[wave][col][1] = lj;
        }
        __syncthreads();
        const int r = threadIdx.x >> 4, part = threadIdx.x & 15;
        const int row = 16 * j + r;
        if (row < rows) {
            float mx = ml[0][r][0];
#pragma unroll
            for (int w = 1; w < 4; ++w)
                mx = fmaxf(mx, ml[w][r][0]);
            float f[4], sum = 0.f;
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                f[w] = __builtin_amdgcn_exp2f(ml[w][r][0] - mx);
                sum += f[w] * ml[w][r][1];
            }
            constexpr int VPT = D / 16;   // values a thread
            float acc[VPT];
#pragma unroll
            for (int e = 0; e < VPT; ++e) {
                acc[e] = 0.f;
#pragma unroll
                for (int w = 0; w < 4; ++w)
                    acc[e] += f[w] * of[(w * 16 + r) * OS + part * VPT + e];
            }
            const int i = row / a.group, hd = h * a.group + row - i * a.group;
            if (sq.count == 1) {
                const float inv = sum > 0.f ? 1.f / sum : sum == 0.f ? 0.f : sum;
                uint16_t *dst = a.out + (sq.q0 + i) * a.out_stride + (int64_t)hd * D + part * VPT;
#pragma unroll
                for (int e = 0; e < VPT; e += 4) {
                    const u32x2 w = {cvt_bf16x2(acc[e] * inv, acc[e + 1] * inv),
                                     cvt_bf16x2(acc[e + 2] * inv, acc[e + 3] * inv)};
                    *(u32x2 *)(dst + e) = w;
                }
                if (a.lse && part == 0)
                    a.lse[(int64_t)(sq.q0 + i) * a.hq + hd] =
                        sum == 0.f ? -INFINITY : (mx + __builtin_amdgcn_logf(sum)) * (1.f / ATTN_LOG2E);
            } else {
                const int64_t slot = (((int64_t)b * a.hkv + h) * a.max_rows + row) * a.n_chunks + c;
                float *dst = a.part_o + slot * D + part * VPT;
#pragma unroll
                for (int e = 0; e < VPT; e += 4)
                    *(f32x4 *)(dst + e) = f32x4{acc[e], acc[e + 1], acc[e + 2], acc[e + 3]};
                if (part == 0)
                    *(f32x2 *)(a.part_ml + 2 * slot) = f32x2{mx, sum};
            }
        }
    }
}

// One wave a row: the row's chunks joined by their maxima and sums.  Rows of one chunk were
// written whole.  Slots are numbered by (sequence, kv head, row).
template <int D>
__global__ __launch_bounds__(256) void attn_combine_kernel(AttnArgs a)
{
    constexpr int VPT = D / 64;
    const int b = (int)(blockIdx.x / a.hkv), h = (int)(blockIdx.x - (unsigned)b * a.hkv);
    const SeqChunks sq = seq_chunks(a, b);
    const int row = (int)blockIdx.y * 4 + (threadIdx.x >> 6), lane = threadIdx.x & 63;
    if (!answers(a, sq) || sq.count <= 1 || row >= sq.n * a.group)
        return;
    const int64_t slot = (((int64_t)b * a.hkv + h) * a.max_rows + row) * a.n_chunks;
    float mx = ATTN_LOWEST, sum = 0.f, acc[VPT];
    for (int c = 0; c < sq.count; ++c)
        mx = fmaxf(mx, a.part_ml[2 * (slot + c)]);
#pragma unroll
    for (int e = 0; e < VPT; ++e)
        acc[e] = 0.f;
    for (int c = 0; c < sq.count; ++c) {
        const float f = __builtin_amdgcn_exp2f(a.part_ml[2 * (slot + c)] - mx);
        sum += f * a.part_ml[2 * (slot + c) + 1];
#pragma unroll
        for (int e = 0; e < VPT; ++e)
            acc[e] += f * a.part_o[(slot + c) * D + lane * VPT + e];
    }
    const float inv = sum > 0.f ? 1.f / sum : sum == 0.f ? 0.f : sum;
    const int i = row / a.group, hd = h * a.group + row - i * a.group;
    uint16_t *dst = a.out + (sq.q0 + i) * a.out_stride + (int64_t)hd * D + lane * VPT;
#pragma unroll
    for (int e = 0; e < VPT; ++e)
        dst[e] = f32_to_bf16(acc[e] * inv);
    if (a.lse && lane == 0)
        a.lse[(int64_t)(sq.q0 + i) * a.hq + hd] =
            sum == 0.f ? -INFINITY : (mx + __builtin_amdgcn_logf(sum)) * (1.f / ATTN_LOG2E);
}

hipError_t launch_attn_decode(const AttnArgs &a, int head_dim, int nq, hipStream_t stream)
{
    const dim3 grid((unsigned)(a.n_seqs * (int64_t)a.hkv), (unsigned)a.n_chunks);
#define DEC(D, NQ, F) attn_decode_kernel<D, NQ, F><<<grid, dim3(256), 0, stream>>>(a)
#define DEC_F(D, NQ) (a.cache.fp8 ? DEC(D, NQ, true) : DEC(D, NQ, false))
#define DEC_Q(D) (nq == 1 ? DEC_F(D, 1) : DEC_F(D, 2))
    head_dim == 64 ? DEC_Q(64) : DEC_Q(128);
#undef DEC_Q
#undef DEC_F
#undef DEC
    return hipGetLastError();
}

hipError_t launch_attn_combine(const AttnArgs &a, int head_dim, hipStream_t stream)
{
    const dim3 grid((unsigned)(a.n_seqs * (int64_t)a.hkv), (unsigned)((a.max_rows + 3) / 4));
    if (head_dim == 64)
        attn_combine_kernel<64><<<grid, dim3(256), 0, stream>>>(a);
    else
        attn_combine_kernel<128><<<grid, dim3(256), 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace mlora
