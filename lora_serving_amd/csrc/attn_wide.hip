// Attention of many query rows: whole prompts (rows of packed sequences) and chunks of new tokens
// over a paged cache.
//
// Rows are (query, head of the kv head's group) pairs of one sequence, so that the heads of a group
// share each tile of K and V and a workgroup's causal edge is only its 256 / group queries wide.  A
// wave owns 32 rows as the columns of 32x32x16 MFMA tiles (S^T = K Q^T, O^T = V^T P^T, see
// attention_device.h); all waves of the workgroup share 64-key tiles of K and V in LDS, double
// buffered: the next tile is copied straight into LDS while this one is computed, one barrier a
// tile.  e4m3 tiles are converted to bf16 (exactly) on their way into LDS, their scales applied to
// the scores and the probabilities.  Bound by the matrix cores together with the exponentials.
#include <algorithm>

#include "attention.h"
#include "attention_device.h"

namespace mlora {

constexpr int AW_BN = 64;      // keys a tile
enum { AW_ROWS = 0, AW_PAGES = 1, AW_PAGES_E4M3 = 2 };

// One 16-byte copy per lane from global memory straight into LDS (64 lanes: 1 KB at lds).
__device__ __forceinline__ void aw_dma(const void *g, uint16_t *lds)
{
    __builtin_amdgcn_global_load_lds(g, (void __attribute__((address_space(3))) *)lds, 16, 0, 0);
}

template <int D, int NW, int SRC>
__global__ __launch_bounds__(NW * 64, 2) void attn_wide_kernel(AttnArgs a)
{
    constexpr bool FP8 = SRC == AW_PAGES_E4M3;
    constexpr int BM = NW * 32, BN = AW_BN;
    constexpr int KS = D / 16;              // k-steps of the first product
    constexpr int DB = D / 32;              // row blocks of the second
    constexpr int CPR = D / 8;              // 16-byte pieces of a bf16 row
    constexpr int LPR = FP8 ? D / 16 : CPR; // lanes a row of the copy
    constexpr int RPI = 64 / LPR;           // rows a copy instruction
    constexpr int IPW = BN / RPI / NW > 0 ? BN / RPI / NW : 1;  // copies a wave, for K and for V each
    constexpr int COPIERS = BN / RPI / IPW; // waves that copy
    __shared__ __attribute__((aligned(1024))) uint16_t kl[2][BN * D];
    __shared__ __attribute__((aligned(1024))) uint16_t vl[2][BN * D];
    __shared__ __attribute__((aligned(16))) float sc[FP8 ? 2 : 1][2][FP8 ? BN : 4];

    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lane = threadIdx.x & 63, col = lane & 31, hh = lane >> 5;
    const int item = (int)(blockIdx.x / a.hkv), h = (int)(blockIdx.x - (unsigned)item * a.hkv);

    // the item's sequence and row block
    int b = -1, rb = 0;
    for (int s0 = 0, base = 0; s0 < a.n_seqs; s0 += 64) {
        const int s = s0 + lane;
        int nb = 0;
        if (s < a.n_seqs) {
            const int64_t lo = min((int64_t)max(a.cu_q[s], 0), a.T), hi = min((int64_t)max(a.cu_q[s + 1], 0), a.T);
            const int64_t rows = (hi - lo) * a.group;
            if (hi > lo && hi - lo <= a.max_q && rows >= a.min_rows && rows <= a.max_rows)
                nb = (int)((rows + BM - 1) / BM);
        }
        int total;
        const int ex = wave_exclusive_scan(nb, &total);
        if (item < base + total) {
            const uint64_t hit = ballot64(item >= base + ex && item < base + ex + nb);
            const int src = __ffsll((unsigned long long)hit) - 1;
            b = s0 + src;
            rb = __shfl(nb, src, 64) - 1 - (item - base - __shfl(ex, src, 64));   // the longest rows first
            break;
        }
        base += total;
    }
    if (b < 0)
        return;
    b = __builtin_amdgcn_readfirstlane(b);
    rb = __builtin_amdgcn_readfirstlane(rb);
    const int q0 = (int)min((int64_t)max(a.cu_q[b], 0), a.T);
    const int n = (int)min((int64_t)max(a.cu_q[b + 1], 0), a.T) - q0;
    int L;
    int64_t key0 = 0;
    if (SRC == AW_ROWS) {
        const int32_t *cu = a.cu_k ? a.cu_k : a.cu_q;
        key0 = min((int64_t)max(cu[b], 0), a.Tk);
        L = (int)max(min((int64_t)max(cu[b + 1], 0), a.Tk) - key0, (int64_t)0);
    } else {
        L = (int)min((int64_t)max(a.kv_len[b], 0), min(a.max_kv, a.table_stride << a.cache.ps));
    }
    const int rows = n * a.group;

    // this lane's row, and the keys that the workgroup's and the wave's rows see
    const int row = rb * BM + wave * 32 + col;
    const int ri = min(row, rows - 1) / a.group, hd = h * a.group + min(row, rows - 1) - ri * a.group;
    const int pos = L - n + ri;
    auto first_key = [&](int r) { return a.window > 0 ? max(0, L - n + min(r, rows - 1) / a.group - a.window + 1) : 0; };
    auto end_key = [&](int r) { return a.causal ? min(L, L - n + min(r, rows - 1) / a.group + 1) : L; };
    const int c0 = (int)blockIdx.y * a.chunk;
    const int kmin = max(first_key(rb * BM), c0);
    const int kmax = (int)min((int64_t)end_key(rb * BM + BM - 1), (int64_t)c0 + a.chunk);
    if (blockIdx.y > 0 && kmin >= kmax)
        return;
    const int wrow = rb * BM + wave * 32;
    const int wmin = first_key(wrow), wmax = wrow < rows ? end_key(wrow + 31) : 0;
    // keys from wfull on, and before wfree, are seen by some of the wave's rows only
    const int wfull = end_key(wrow), wfree = first_key(wrow + 31);
    const int t0 = kmin / BN, t1 = kmax > kmin ? (kmax + BN - 1) / BN : t0;

    u32x4 qf[KS];
    {
        const uint16_t *qr = a.q + (int64_t)(q0 + ri) * a.q_stride + (int64_t)hd * D;
#pragma unroll
        for (int s = 0; s < KS; ++s)
            qf[s] = *(const u32x4 *)(qr + 16 * s + 8 * hh);
    }
    const float cs = a.scale * ATTN_LOG2E;
    f32x16 o[DB];
#pragma unroll
    for (int d = 0; d < DB; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i)
            o[d][i] = 0.f;
    float m = ATTN_LOWEST, l = 0.f;

    // copies of a tile: K and V rows [key][D], the 16-byte pieces of a row swizzled by the key
    const int crow = lane / LPR, cpiece = lane % LPR;
    const int32_t *__restrict__ table = SRC == AW_ROWS ? nullptr : a.table + (int64_t)b * a.table_stride;
    const int ps = a.cache.ps, pm = (1 << ps) - 1;
    int pg[IPW];
    u32x4 kr[IPW], vr[IPW];
    float scr = 0.f;
    // pages of the tile's rows that this wave copies (a copy's rows lie in one page)
    auto lookup = [&](int t) {
        if (SRC == AW_ROWS)
            return;
#pragma unroll
        for (int i = 0; i < IPW; ++i)
            pg[i] = clamp_page(table[min(t * BN + (wave * IPW + i) * RPI, L - 1) >> ps], a.cache.n_pages);
    };
    auto stage = [&](int t, int buf) {
        if (wave >= COPIERS)
            return;
#pragma unroll
        for (int i = 0; i < IPW; ++i) {
            const int r0 = (wave * IPW + i) * RPI, r = r0 + crow;
            const int key = min(t * BN + r, L - 1);     // rows past the end: the last key again
            if (SRC == AW_ROWS) {
                const int64_t at = key0 + key;
                const int piece = 8 * (cpiece ^ (r & (CPR - 1)));
                aw_dma(a.k + at * a.k_stride + (int64_t)h * D + piece, kl[buf] + r0 * D);
                aw_dma(a.v + at * a.v_stride + (int64_t)h * D + piece, vl[buf] + r0 * D);
            } else {
                const int64_t at = (((int64_t)pg[i] * a.cache.hkv + h) << ps) + (key & pm);
                if (!FP8) {
                    const int piece = 16 * (cpiece ^ (r & (CPR - 1)));
                    aw_dma(a.cache.k + at * D * 2 + piece, kl[buf] + r0 * D);
                    aw_dma(a.cache.v + at * D * 2 + piece, vl[buf] + r0 * D);
                } else {
                    kr[i] = *(const u32x4 *)(a.cache.k + at * D + 16 * cpiece);
                    vr[i] = *(const u32x4 *)(a.cache.v + at * D + 16 * cpiece);
                }
            }
        }
        if (FP8 && threadIdx.x < 2 * BN) {
            const int key = min(t * BN + (int)(threadIdx.x & (BN - 1)), L - 1);
            const int page = clamp_page(table[key >> ps], a.cache.n_pages);
            const float *src = threadIdx.x < BN ? a.cache.k_scale : a.cache.v_scale;
            scr = src[(((int64_t)page * a.cache.hkv + h) << ps) + (key & pm)];
        }
    };
    // e4m3: the loaded tile into LDS
    auto deposit = [&](int buf) {
        if (!FP8)
            return;
        if (wave < COPIERS)
#pragma unroll
            for (int i = 0; i < IPW; ++i) {
                const int r = (wave * IPW + i) * RPI + crow;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int piece = 8 * ((2 * cpiece + e) ^ (r & (CPR - 1)));
                    *(u32x4 *)(kl[buf] + r * D + piece) = e4m3_to_bf16x8(kr[i][2 * e], kr[i][2 * e + 1]);
                    *(u32x4 *)(vl[buf] + r * D + piece) = e4m3_to_bf16x8(vr[i][2 * e], vr[i][2 * e + 1]);
                }
            }
        if (threadIdx.x < 2 * BN)
            sc[FP8 ? buf : 0][threadIdx.x / BN][FP8 ? threadIdx.x & (BN - 1) : 0] = scr;
    };

    if (t0 < t1) {
        lookup(t0);
        stage(t0, 0);
        deposit(0);
        if (t0 + 1 < t1)
            lookup(t0 + 1);
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    for (int t = t0; t < t1; ++t) {
        const int buf = (t - t0) & 1, kb = t * BN;
        if (t + 1 < t1) {
            stage(t + 1, buf ^ 1);
            if (t + 2 < t1)
                lookup(t + 2);
        }
        if (kb < wmax && kb + BN > wmin) {
            const uint16_t *kt = kl[buf], *vt = vl[buf];
            const bool edge = kb + BN > wfull || kb < wfree;
            // S^T: rows = keys 32 u + 8 (i / 4) + 4 hh + i % 4, column = query
            f32x16 st[2];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    st[u][i] = 0.f;
#pragma unroll
                for (int s = 0; s < KS; ++s) {
                    const int key = 32 * u + col;
                    const u32x4 kf = *(const u32x4 *)(kt + key * D + 8 * ((2 * s + hh) ^ (key & (CPR - 1))));
                    st[u] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(as_bf16x8(kf), as_bf16x8(qf[s]), st[u], 0, 0, 0);
                }
            }
            if (FP8) {
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const f32x4 k4 = *(const f32x4 *)(&sc[buf][0][32 * u + 8 * i + 4 * hh]);
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            st[u][4 * i + e] *= k4[e];
                    }
            }
            if (edge) {
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const int key = kb + 32 * u + 8 * (i / 4) + 4 * hh + i % 4;
                        const bool see = key < L && (!a.causal || key <= pos) &&
                                         (a.window <= 0 || key > pos - a.window);
                        st[u][i] = see ? st[u][i] : -INFINITY;
                    }
            }
            float mx = st[0][0];
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    mx = fmaxf(mx, st[u][i]);
            mx *= cs;
            if (__any(mx > m + ATTN_SLACK)) {
                mx = fmaxf(mx, __shfl_xor(mx, 32, 64));
                // (each column on its own: a row's bits do not depend on its neighbours)
                const float mn = mx > m + ATTN_SLACK ? mx : m, f = __builtin_amdgcn_exp2f(m - mn);
                m = mn;
                l *= f;
#pragma unroll
                for (int d = 0; d < DB; ++d)
                    o[d] *= f;
            }
            // P^T: rounding to bf16 (2^-9 relative) for the matrix cores; the sum keeps fp32
            u32x4 pf[4];
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    f32x4 p, v4;
                    if (FP8)
                        v4 = *(const f32x4 *)(&sc[FP8 ? buf : 0][1][FP8 ? 32 * u + 8 * i + 4 * hh : 0]);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float s = st[u][4 * i + e];
                        const float x = __builtin_amdgcn_exp2f(fmaf(s, cs, -m));
                        l += x;
                        // (a masked key's scale may be anything)
                        p[e] = !FP8 ? x : edge && s == -INFINITY ? 0.f : x * v4[e];
                    }
                    pf[2 * u + i / 2][2 * (i & 1)] = cvt_bf16x2(p[0], p[1]);
                    pf[2 * u + i / 2][2 * (i & 1) + 1] = cvt_bf16x2(p[2], p[3]);
                }
            // O^T += V^T P^T; k index (hh, e) of step s is key 16 s + 8 (e / 4) + 4 hh + e % 4
            const int vi = lane & 15, vd = (lane >> 4) & 1;
            auto vfrag = [&](int s, int d) {
                u32x4 f;
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int key = 16 * s + 8 * u + 4 * hh + (vi >> 2);
                    const int piece = 4 * d + 2 * vd + ((vi & 3) >> 1);
                    const u32x2 w = lds_read_tr(vt + key * D + 8 * (piece ^ (key & (CPR - 1))) + 4 * (vi & 1));
                    f[2 * u] = w[0];
                    f[2 * u + 1] = w[1];
                }
                return f;
            };
            uint32_t bad = 0;
            if (edge) {
#pragma unroll
                for (int s = 0; s < 4; ++s)
#pragma unroll
                    for (int d = 0; d < DB; ++d) {
                        const u32x4 f = vfrag(s, d);
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            bad = not_finite(bad, f[i]);
                    }
            }
            if (!__any((bad & 0x80008000u) != 0)) {
#pragma unroll
                for (int s = 0; s < 4; ++s)
#pragma unroll
                    for (int d = 0; d < DB; ++d)
                        o[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(as_bf16x8(vfrag(s, d)), as_bf16x8(pf[s]), o[d], 0, 0, 0);
            } else {
                // V holds an infinity or NaN where some row must not see it (0 x NaN is NaN): one key at
                // a time, kept only by the rows that see it
#pragma unroll
                for (int s = 0; s < 4; ++s)
#pragma unroll 1
                    for (int k = 0; k < 16; ++k) {
                        const int key = kb + 16 * s + k, e = 4 * (k >> 3) + (k & 3);
                        const bool mine = hh == ((k >> 2) & 1);
                        const bool see = key < L && (!a.causal || key <= pos) &&
                                         (a.window <= 0 || key > pos - a.window);
                        const uint32_t half = (e & 1) ? 0xffff0000u : 0xffffu;
#pragma unroll
                        for (int d = 0; d < DB; ++d) {
                            u32x4 f = vfrag(s, d);
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                f[i] = mine && i == (e >> 1) ? f[i] & half : 0u;
                            const f32x16 x = __builtin_amdgcn_mfma_f32_32x32x16_bf16(as_bf16x8(f), as_bf16x8(pf[s]), o[d], 0, 0, 0);
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                o[d][i] = see ? x[i] : o[d][i];
                        }
                    }
            }
        }
        if (t + 1 < t1)
            deposit(buf ^ 1);
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        __syncthreads();
    }

    l += __shfl_xor(l, 32, 64);
    if (row >= rows)
        return;
    if (a.n_chunks == 1) {
        const float inv = l > 0.f ? 1.f / l : l == 0.f ? 0.f : l;
        uint16_t *dst = a.out + (int64_t)(q0 + ri) * a.out_stride + (int64_t)hd * D + 4 * hh;
#pragma unroll
        for (int d = 0; d < DB; ++d)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                *(u32x2 *)(dst + 32 * d + 8 * i) =
                    u32x2{cvt_bf16x2(o[d][4 * i] * inv, o[d][4 * i + 1] * inv),
                          cvt_bf16x2(o[d][4 * i + 2] * inv, o[d][4 * i + 3] * inv)};
        if (a.lse && hh == 0)
            a.lse[(int64_t)(q0 + ri) * a.hq + hd] =
                l == 0.f ? -INFINITY : (m + __builtin_amdgcn_logf(l)) * (1.f / ATTN_LOG2E);
    } else {
        const int64_t slot = ((int64_t)(q0 + ri) * a.hq + hd) * a.n_chunks + blockIdx.y;
#pragma unroll
        for (int d = 0; d < DB; ++d)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                *(f32x4 *)(a.part_o + slot * D + 32 * d + 8 * i + 4 * hh) =
                    f32x4{o[d][4 * i], o[d][4 * i + 1], o[d][4 * i + 2], o[d][4 * i + 3]};
        if (hh == 0)
            *(f32x2 *)(a.part_ml + 2 * slot) = f32x2{m, l};
    }
}

// One wave a (token, head): the chunks that hold keys it sees, joined.
template <int D>
__global__ __launch_bounds__(256) void attn_wide_combine_kernel(AttnArgs a)
{
    constexpr int VPT = D / 64;
    const int64_t th = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    const int lane = threadIdx.x & 63;
    if (th >= a.T * a.hq)
        return;
    const int t = (int)(th / a.hq), hd = (int)(th - (int64_t)t * a.hq);
    int b = -1;
    for (int s0 = 0; s0 < a.n_seqs; s0 += 64) {
        const int s = s0 + lane;
        const uint64_t hit = ballot64(s < a.n_seqs && a.cu_q[s] <= t && t < a.cu_q[s + 1]);
        if (hit) {
            b = s0 + __ffsll((unsigned long long)hit) - 1;
            break;
        }
    }
    if (b < 0)
        return;
    const int q0 = max(a.cu_q[b], 0), n = (int)min((int64_t)a.cu_q[b + 1], a.T) - q0;
    const int64_t rows = (int64_t)n * a.group;
    if (n > a.max_q || rows < a.min_rows || rows > a.max_rows)
        return;
    const int L = (int)min((int64_t)max(a.kv_len[b], 0), min(a.max_kv, a.table_stride << a.cache.ps));
    const int pos = L - n + t - q0;
    const int lo = a.window > 0 ? max(0, pos - a.window + 1) : 0, hi = a.causal ? min(L, pos + 1) : L;
    const int64_t slot = th * a.n_chunks;
    const int ca = lo / a.chunk, cb = hi > lo ? (hi - 1) / a.chunk + 1 : ca;
    float mx = ATTN_LOWEST, sum = 0.f, acc[VPT];
    for (int c = ca; c < cb; ++c)
        mx = fmaxf(mx, a.part_ml[2 * (slot + c)]);
#pragma unroll
    for (int e = 0; e < VPT; ++e)
        acc[e] = 0.f;
    for (int c = ca; c < cb; ++c) {
        const float f = __builtin_amdgcn_exp2f(a.part_ml[2 * (slot + c)] - mx);
        sum += f * a.part_ml[2 * (slot + c) + 1];
#pragma unroll
        for (int e = 0; e < VPT; ++e)
            acc[e] += f * a.part_o[(slot + c) * D + lane * VPT + e];
    }
    const float inv = sum > 0.f ? 1.f / sum : sum == 0.f ? 0.f : sum;
    uint16_t *dst = a.out + (int64_t)t * a.out_stride + (int64_t)hd * D + lane * VPT;
#pragma unroll
    for (int e = 0; e < VPT; ++e)
        dst[e] = f32_to_bf16(acc[e] * inv);
    if (a.lse && lane == 0)
        a.lse[th] = sum == 0.f ? -INFINITY : (mx + __builtin_amdgcn_logf(sum)) * (1.f / ATTN_LOG2E);
}

int wide_rows(int64_t T, int32_t hq, int32_t group)
{
    (void)group;
    return T * hq >= 256 * 256 ? 256 : 128;
}

hipError_t launch_attn_wide(const AttnArgs &a, int head_dim, bool pages, hipStream_t stream)
{
    const int bm = wide_rows(a.T, a.hq, a.group);
    // each sequence's last row block may be part empty: at most one more block a sequence
    const int64_t items = std::min(a.T * a.group / bm + a.n_seqs,
                                   a.n_seqs * ((a.max_q * a.group + bm - 1) / bm));
    if (items * a.hkv > 0x7fffffff)
        return hipErrorInvalidValue;
    const dim3 grid((unsigned)(items * a.hkv), (unsigned)a.n_chunks);
#define AW(D, NW, SRC) attn_wide_kernel<D, NW, SRC><<<grid, dim3(NW * 64), 0, stream>>>(a)
#define AW_S(D, NW) (!pages ? AW(D, NW, AW_ROWS) : a.cache.fp8 ? AW(D, NW, AW_PAGES_E4M3) : AW(D, NW, AW_PAGES))
#define AW_N(D) (bm == 256 ? AW_S(D, 8) : AW_S(D, 4))
    head_dim == 64 ? AW_N(64) : AW_N(128);
#undef AW_N
#undef AW_S
#undef AW
    return hipGetLastError();
}

hipError_t launch_attn_wide_combine(const AttnArgs &a, int head_dim, hipStream_t stream)
{
    const unsigned blocks = (unsigned)((a.T * a.hq + 3) / 4);
    if (head_dim == 64)
        attn_wide_combine_kernel<64><<<blocks, 256, 0, stream>>>(a);
    else
        attn_wide_combine_kernel<128><<<blocks, 256, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace mlora
