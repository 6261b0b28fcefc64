// Attention of many query rows: whole prompts (rows of packed sequences) and chunks of new tokens
// over a paged cache.
//
// Rows are (query, head of the kv head's group) pairs of one sequence, so that the heads of a group
// share each tile of K and V and a workgroup's causal edge is only its 128 / group queries wide.  A
// wave owns 32 rows as the columns of 32x32x16 MFMA tiles (S^T = K Q^T, O^T = V^T P^T, see
// attention_device.h); the four waves of a workgroup share 64-key tiles of K and V in LDS, double
// buffered: the next tile is copied straight into LDS while this one is computed, one barrier a
// tile.  e4m3 tiles are converted to bf16 (exactly) on their way into LDS, their scales applied to
// the scores and the probabilities.
//
// Two workgroups of 128 rows a CU, which wait at barriers of their own, rather than one of 256 rows
// (8 causal prompts of 2048, 32 heads of 128 on 8: 338 us against 357 when that was chosen).  Bound by
// the issue of products and exponentials together: on a prompt of 16384 tokens a SIMD's matrix core
// is busy for 61 to 63% of the cycles and its vector unit for 53 to 54%, at 1.7 to 1.8 GHz.  Measured
// (D = 128, 32 heads on 8): 8 prompts of 2048 308 to 317 us (870 to 890 TFLOP/s), one of 16384 1.91 to 1.97 ms
// (1120 to 1150), 2048 tokens over 8192 keys in bf16 pages 228 to 234 us (1030 to 1050), in e4m3 pages 273 to
// 282 us (850 to 880: conversions and scales take the issue), D = 64 148 to 153 us (780 to 810: the same
// exponentials for half the products).
#pragma once

#include <type_traits>

#include "attention.h"
#include "attention_device.h"

namespace mlora {

constexpr int AW_BN = 64;      // keys a tile
enum { AW_ROWS = 0, AW_PAGES = 1, AW_PAGES_E4M3 = 2 };

// One 16-byte copy a lane from global memory (a scalar base and a byte offset of the lane) straight into
// LDS: 64 lanes fill 1 KB at byte `to` + `more` of it.  In asm, so that the compiler does not drain the
// copies in flight before each LDS read (it cannot tell the buffers apart); every copy is waited for by
// hand.  The compiler keeps no value in m0 but sets it before each use of its own: naming it orders the
// statement against those (clang 22 of ROCm 7.2 warns of the name as of any reserved register).
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void aw_dma(const void *base, uint32_t off, uint32_t to, int more)
{
    asm volatile("s_add_u32 m0, %2, %3\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1"
                 :: "v"(off), "s"(base), "s"(to), "i"(more) : "memory", "scc", "m0");
}
#pragma clang diagnostic pop

// Swizzle of the 16-byte pieces of a row by its key, a bijection for reads of one piece over 16 keys
// (K, ds_read_b128) that also spreads a transposing read's 4 keys x 64 bytes (V) over all banks.
template <int D>
__device__ __forceinline__ int aw_swz(int key)
{
    return D == 128 ? ((key & 3) << 2) | ((key >> 2) & 3) : (((key >> 1) & 1) << 2) | ((key >> 2) & 3);
}

// A workgroup's work: row block `block` of a sequence's query rows [q0, q0 + n), its L keys (rows: from key0 on).
struct WideItem {
    int seq, block, q0, n, key0, L;
    int total;              // items of all sequences
};

// The sequence and row block of an item: the longest row blocks (the last ones of a causal prompt) first, of
// all sequences up to 64 of them (they start first, so that the launch ends on short ones: 8 prompts of 2048
// tokens), in each sequence where there are more (short prompts, or one chunk among many single tokens).
template <bool ROWS>
__device__ __forceinline__ bool aw_item(const AttnArgs &a, int item, int lane, WideItem *w)
{
    int q0 = 0, q1 = 0, k0 = 0, k1 = 0;
    auto load = [&](int s) {
        q0 = q1 = k0 = k1 = 0;
        if (s < a.n_seqs) {
            const int32_t *cu = ROWS && a.cu_k ? a.cu_k : a.cu_q;
            const int32_t qa = a.cu_q[s], qb = a.cu_q[s + 1], ka = ROWS ? cu[s] : 0, kb = ROWS ? cu[s + 1] : a.kv_len[s];
            q0 = (int)min((int64_t)max(qa, 0), a.T);
            q1 = (int)min((int64_t)max(qb, 0), a.T);
            k0 = (int)min((int64_t)max(ka, 0), a.Tk);
            k1 = (int)min((int64_t)max(kb, 0), ROWS ? a.Tk : min(a.max_kv, a.table_stride << a.cache.ps));
        }
        const int64_t rows = (int64_t)(q1 - q0) * a.group;
        const bool mine = q1 > q0 && q1 - q0 <= a.max_q && rows >= a.min_rows && rows <= a.max_rows;
        return mine ? (int)((rows + WIDE_ROWS - 1) / WIDE_ROWS) : 0;
    };
    auto take = [&](int s0, int src, int block) {
        w->seq = s0 + src;
        w->block = block;
        w->q0 = __builtin_amdgcn_readlane(q0, src);
        w->n = __builtin_amdgcn_readlane(q1, src) - w->q0;
        w->key0 = __builtin_amdgcn_readlane(k0, src);
        w->L = max(__builtin_amdgcn_readlane(k1, src) - w->key0, 0);
    };
    if (a.n_seqs <= 64) {
        const int nb = load(lane);
        // items of block numbers >= r
        auto count = [&](int r) { return wave_total(max(nb - r, 0)); };
        w->total = count(0);
        if (item >= w->total)
            return false;
        // count(lo) > item >= count(hi)
        int lo = 0, hi = (int)((a.max_q * a.group + WIDE_ROWS - 1) / WIDE_ROWS);
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (count(mid) > item)
                lo = mid;
            else
                hi = mid;
        }
        const int nth = item - count(hi);       // among the sequences of more than lo blocks
        const uint64_t have = ballot64(nb > lo);
        const int rank = __popcll(have & ((UINT64_C(1) << lane) - 1));
        take(0, uniform(__ffsll((unsigned long long)ballot64(nb > lo && rank == nth)) - 1), lo);
        return true;
    }
    // a lane counts `per` consecutive sequences; then those of the lane that has the item, a lane each
    const int per = (a.n_seqs + 63) / 64;
    int mine = 0;
#pragma unroll 4
    for (int i = 0; i < per; ++i)
        mine += load(lane * per + i);
    const int upto = wave_prefix(mine);
    w->total = __builtin_amdgcn_readlane(upto, 63);
    if (item >= w->total)
        return false;
    const int owner = uniform(__ffsll((unsigned long long)ballot64(item < upto)) - 1);
    int rest = item - (__builtin_amdgcn_readlane(upto, owner) - __builtin_amdgcn_readlane(mine, owner));
    for (int s0 = owner * per;; s0 += 64) {
        const int nb = s0 + lane < owner * per + per ? load(s0 + lane) : 0;
        const int up = wave_prefix(nb), total = __builtin_amdgcn_readlane(up, 63);
        if (rest < total) {
            const int src = uniform(__ffsll((unsigned long long)ballot64(rest < up)) - 1);
            take(s0, src, __builtin_amdgcn_readlane(up, src) - 1 - rest);
            return true;
        }
        rest -= total;
    }
}

template <int D, int SRC, int KG>
constexpr int wide_lds = KG * 4 * AW_BN * D * 2 + (SRC == AW_PAGES_E4M3 ? 4 * 2 * AW_BN * 4 : 0) + (KG > 1 ? 4 * 64 * 2 * 4 : 0);

// Item and kv head bx, and chunk of keys by; smem: wide_lds bytes.  Returns how many items there are.  (MORE: called
// for several items.)
template <int D, int SRC, int KG, bool MORE = false>
__device__ __forceinline__ int attn_wide_body(const AttnArgs &a, int bx, int by, uint8_t *smem)
{
    constexpr bool FP8 = SRC == AW_PAGES_E4M3;
    constexpr int NW = 4, BM = WIDE_ROWS, BN = AW_BN;
    constexpr int KS = D / 16;              // k-steps of the first product
    constexpr int DB = D / 32;              // row blocks of the second
    constexpr int CPR = D / 8;              // 16-byte pieces of a bf16 row
    constexpr int LPR = FP8 ? D / 16 : CPR; // lanes a row of the copy
    constexpr int RPI = 64 / LPR;           // rows a copy instruction
    constexpr int IPW = BN / RPI / NW;      // copies a wave, for K and for V each
    constexpr int TILE = BN * D;
    constexpr int GROUP = 4 * TILE;         // two tiles of K, two of V
    uint16_t *const lds = (uint16_t *)smem;
    float (*const sc)[2][BN] = (float (*)[2][BN])(smem + KG * GROUP * 2);           // e4m3: scales of 4 tiles
    float (*const joint)[64][2] = (float (*)[64][2])(smem + KG * GROUP * 2);        // KG = 2: maxima and sums

    static_assert(KG == 1 || !FP8, "one set of scales");
    int thread = threadIdx.x;
    if (MORE)           // (opaque: what the items of a workgroup have in common is not kept, and spilled, between)
        asm volatile("" : "+v"(thread));
    const int kg = KG > 1 ? uniform(thread >> 8) : 0, wave = uniform((thread >> 6) & 3);
    uint16_t *const kl = lds + kg * GROUP, *const vl = kl + 2 * TILE;
    const int lane = thread & 63, col = lane & 31, hh = lane >> 5;
    const int item = (int)((unsigned)bx / a.hkv), h = (int)((unsigned)bx - (unsigned)item * a.hkv);

    WideItem it;
    if (!aw_item<SRC == AW_ROWS>(a, item, lane, &it))
        return it.total;
    const int b = it.seq, rb = it.block, q0 = it.q0, n = it.n, L = it.L, key0 = it.key0;
    const int rows = n * a.group;

    // this lane's row, and the keys that the workgroup's and the wave's rows see
    const int row = rb * BM + wave * 32 + col;
    const int ri = min(row, rows - 1) / a.group, hd = h * a.group + min(row, rows - 1) - ri * a.group;
    const int pos = L - n + ri;
    auto first_key = [&](int r) { return a.window > 0 ? max(0, L - n + min(r, rows - 1) / a.group - a.window + 1) : 0; };
    auto end_key = [&](int r) { return a.causal ? min(L, L - n + min(r, rows - 1) / a.group + 1) : L; };
    const int c0 = by * a.chunk;
    const int kmin = max(first_key(rb * BM), c0);
    const int kmax = (int)min((int64_t)end_key(rb * BM + BM - 1), (int64_t)c0 + a.chunk);
    if (by > 0 && kmin >= kmax)
        return it.total;
    const int wrow = rb * BM + wave * 32;
    const int wmin = first_key(wrow), wmax = wrow < rows ? end_key(wrow + 31) : 0;
    // the tiles, or this half's of them
    const int ta = kmin / BN, tb = kmax > kmin ? (kmax + BN - 1) / BN : ta, tm = KG > 1 ? ta + (tb - ta + 1) / 2 : tb;
    const int t0 = kg ? tm : ta, t1 = kg ? tb : tm;
    // tiles [f0, f1): every row of the workgroup sees every key
    const int f0 = max(t0, (first_key(rb * BM + BM - 1) + BN - 1) / BN);
    const int f1 = max(min(t1, min(kmax, end_key(rb * BM)) / BN), f0);

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

    // Copies of a tile: K and V rows [key][D], the 16-byte pieces of a row swizzled by the key.  A wave copies 16
    // rows, which lie in one page, from a scalar base with constant 32-bit offsets.  Rows past the end of a sequence
    // are the last key again, or in a page whatever it holds: they are masked.
    const int w16 = 16 * wave, crow = lane / LPR, cpiece = lane % LPR;
    const int32_t *__restrict__ table = SRC == AW_ROWS ? nullptr : a.table + (int64_t)b * a.table_stride;
    const int ps = a.cache.ps, pm = (1 << ps) - 1;
    uint32_t off_k[IPW], off_v[IPW], piece[IPW];
#pragma unroll
    for (int i = 0; i < IPW; ++i) {
        const int r = RPI * i + crow;
        piece[i] = 16 * (FP8 ? cpiece : cpiece ^ aw_swz<D>(r));
        off_k[i] = piece[i] + (SRC == AW_ROWS ? (uint32_t)(w16 + r) * (uint32_t)(2 * a.k_stride)
                                              : (uint32_t)r * D * (FP8 ? 1 : 2));
        off_v[i] = SRC == AW_ROWS ? piece[i] + (uint32_t)(w16 + r) * (uint32_t)(2 * a.v_stride) : off_k[i];
    }
    const uint16_t *kp = a.k + ((int64_t)key0 + (int64_t)t0 * BN) * a.k_stride + (int64_t)h * D;   // rows: the next tile
    const uint16_t *vp = a.v + ((int64_t)key0 + (int64_t)t0 * BN) * a.v_stride + (int64_t)h * D;
    int pgs = 0, pgk = 0, pgv = 0;
    u32x4 kr[IPW], vr[IPW];
    float scr = 0.f;
    // pages of this wave's rows of the 64 tiles around t, one a lane: a scalar load a tile comes late when memory is
    // busy, and its wait drains the reads of LDS with it (256 single tokens and a chunk of 2048 392 us, so 367; a
    // chunk split into pieces of a few tiles waits longer for its first: 100 tokens over 8192 39.4 us, so 40.1)
    auto lookup = [&](int t) {
        if (SRC != AW_ROWS)
            pgs = table[min(((t & ~63) + lane) * BN + w16, L - 1) >> ps];
    };
    // (to: where the tile goes, bytes of LDS, this wave's rows)
    auto copy = [&](int t, const uint16_t *&rows, int64_t stride, const uint8_t *pages, int pg, const uint32_t (&off)[IPW],
                    uint32_t to, u32x4 (&regs)[IPW]) __attribute__((always_inline)) {
        if (SRC == AW_ROWS) {
            if (t * BN + BN <= L) {
#pragma unroll
                for (int i = 0; i < IPW; ++i)
                    aw_dma(rows, off[i], to, RPI * i * D * 2);
            } else {
#pragma unroll
                for (int i = 0; i < IPW; ++i)
                    aw_dma(rows, (uint32_t)min(w16 + RPI * i + crow, L - 1 - t * BN) * (uint32_t)(2 * stride) + piece[i],
                           to, RPI * i * D * 2);
            }
            rows += BN * stride;
        } else {
            const int64_t at = (((int64_t)uniform(pg) * a.cache.hkv + h) << ps) + ((t * BN + w16) & pm);
            const uint8_t *base = pages + at * D * (FP8 ? 1 : 2);
#pragma unroll
            for (int i = 0; i < IPW; ++i)
                if (!FP8)
                    aw_dma(base, off[i], to, RPI * i * D * 2);
                else
                    regs[i] = *(const u32x4 *)(base + off[i]);
        }
    };
    const uint32_t to_k = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint16_t *)lds +
                          (uint32_t)(kg * GROUP + w16 * D) * 2, to_v = to_k + 4 * TILE;
    // K of tile t + 1 on its way (pgk: its page), and V of tile t (pgv: its page); K first
    auto issue_k = [&](int t) __attribute__((always_inline)) {
        if (t + 1 < t1) {
            if (SRC != AW_ROWS)
                pgk = clamp_page(__builtin_amdgcn_readlane(pgs, (t + 1) & 63), a.cache.n_pages);
            copy(t + 1, kp, a.k_stride, a.cache.k, pgk, off_k, to_k + ((t + 1) & 1) * (2 * TILE), kr);
            if (FP8 && lane < 32)       // scales of K and of V, both of tile t + 1 (this wave's rows)
                scr = (lane < 16 ? a.cache.k_scale : a.cache.v_scale)[(((int64_t)pgk * a.cache.hkv + h) << ps) +
                                                                      (((t + 1) * BN + w16 + (lane & 15)) & pm)];
        }
    };
    auto issue_v = [&](int t) __attribute__((always_inline)) {
        if (t >= t0)
            copy(t, vp, a.v_stride, a.cache.v, pgv, off_v, to_v + (t & 1) * (2 * TILE), vr);
        if (SRC != AW_ROWS) {
            pgv = pgk;
            if (t + 2 < t1 && ((t + 2) & 63) == 0)
                lookup(t + 2);
        }
    };
    auto issue = [&](int t) __attribute__((always_inline)) {
        issue_k(t);
        issue_v(t);
    };
    // what issue(t) started has arrived in LDS (this wave's part; a barrier makes it the workgroup's)
    auto land = [&](int t) {
        if (FP8) {
            const int nb = (t + 1) & 1;
#pragma unroll
            for (int i = 0; i < IPW; ++i) {
                const int r = w16 + RPI * i + crow;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int p = 8 * ((2 * cpiece + e) ^ aw_swz<D>(r));
                    if (t + 1 < t1)
                        *(u32x4 *)(kl + nb * TILE + r * D + p) = e4m3_to_bf16x8(kr[i][2 * e], kr[i][2 * e + 1]);
                    if (t >= t0)
                        *(u32x4 *)(vl + (nb ^ 1) * TILE + r * D + p) = e4m3_to_bf16x8(vr[i][2 * e], vr[i][2 * e + 1]);
                }
            }
            if (lane < 32)
                sc[(t + 1) & 3][lane >> 4][w16 + (lane & 15)] = scr;
            asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
        } else {
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        }
    };
    auto phase_end = [] {
        __builtin_amdgcn_sched_barrier(0);
        asm volatile("s_barrier" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
    };

    // (opaque to the compiler, which would otherwise keep every address of both buffers in registers and spill)
    auto tile_at = [](uint32_t at, int t) {
        at ^= (t & 1) * TILE * 2;
        asm volatile("" : "+v"(at));
        return at;
    };

    f32x16 sa[2], sb[2], zero;
#pragma unroll
    for (int i = 0; i < 16; ++i)
        zero[i] = 0.f;
    u32x4 pf[4];
    // S^T: rows = keys 32 u + 8 (i / 4) + 4 hh + i % 4, column = query
    const uint32_t klane = kg * GROUP * 2 + col * D * 2 + 16 * (hh ^ aw_swz<D>(col));
    auto kfrag = [&](uint32_t at, int s, int u) {
        return *(const u32x4 *)((const uint8_t *)lds + (at ^ (32 * s)) + 64 * u * D);
    };
    auto scores = [&](int t, f32x16 (&st)[2]) {
        const uint32_t at = tile_at(klane, t);
#pragma unroll
        for (int s = 0; s < KS; ++s)
#pragma unroll
            for (int u = 0; u < 2; ++u)
                st[u] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(as_bf16x8(kfrag(at, s, u)), as_bf16x8(qf[s]),
                                                                s ? st[u] : zero, 0, 0, 0);
    };
    // e4m3: the keys' scales (of 4 scores)
    auto scaled = [&](int t, int u, int i, f32x16 (&st)[2]) {
        if (FP8) {
            const f32x4 k4 = *(const f32x4 *)(&sc[t & 3][0][32 * u + 8 * i + 4 * hh]);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                st[u][4 * i + e] *= k4[e];
        }
    };
    auto all_scaled = [&](int t, f32x16 (&st)[2]) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            scaled(t, i >> 2, i & 3, st);
    };
    auto hide = [&](int t, f32x16 (&st)[2]) {
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int key = t * BN + 32 * u + 8 * (i / 4) + 4 * hh + i % 4;
                const bool see = key < L && (!a.causal || key <= pos) && (a.window <= 0 || key > pos - a.window);
                st[u][i] = see ? st[u][i] : -INFINITY;
            }
    };
    auto largest = [&](const f32x16 &s, int i0, int i1, float mx) {
#pragma unroll
        for (int i = i0; i < i1; ++i)
            mx = fmaxf(mx, s[i]);
        return mx;
    };
    // the running maximum follows the largest score of a tile, and what was summed before with it
    auto raise = [&](float mx) {
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
    };
    // 2 scores to probabilities (k: 0 .. 15), P^T rounded to bf16 (half a step: 2^-8 relative) for the matrix cores;
    // the sum keeps fp32
    auto powers = [&](int t, int k, const f32x16 (&st)[2], auto edge) {
        const int u = k >> 3, i = 2 * (k & 7);
        float p[2];
        f32x2 v2;
        if (FP8)
            v2 = *(const f32x2 *)(&sc[t & 3][1][32 * u + 8 * (i >> 2) + 4 * hh + (i & 3)]);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const float s = st[u][i + e];
            const float x = __builtin_amdgcn_exp2f(fmaf(s, cs, -m));
            l += x;
            // (a masked key's scale may be anything)
            p[e] = !FP8 ? x : edge && s == -INFINITY ? 0.f : x * v2[e];
        }
        pf[k >> 2][k & 3] = cvt_bf16x2(p[0], p[1]);
    };
    auto all_powers = [&](int t, const f32x16 (&st)[2], auto edge) {
#pragma unroll
        for (int k = 0; k < 16; ++k)
            powers(t, k, st, edge);
    };
    // O^T += V^T P^T; k index (hh, e) of step s is key 16 s + 8 (e / 4) + 4 hh + e % 4
    const int vi = lane & 15, vd = (lane >> 4) & 1, vk = 4 * hh + (vi >> 2);
    const uint32_t vlane = kg * GROUP * 2 + vk * D * 2 + 16 * ((2 * vd + ((vi & 3) >> 1)) ^ aw_swz<D>(vk)) + 8 * (vi & 1);
    auto vfrag = [&](uint32_t at, int s, int d) {
        u32x4 f;
#pragma unroll
        for (int u = 0; u < 2; ++u) {       // keys 16 s + 8 u + vk, values 32 d ..
            const uint8_t *v = (const uint8_t *)(lds + 2 * TILE) + (at ^ (64 * d + 32 * u)) + (16 * u + 32 * s) * D;
            const u32x2 w = lds_read_tr((const uint16_t *)v);
            f[2 * u] = w[0];
            f[2 * u + 1] = w[1];
        }
        return f;
    };
    auto outputs = [&](int t) {
        const uint32_t at = tile_at(vlane, t);
#pragma unroll
        for (int s = 0; s < 4; ++s)
#pragma unroll
            for (int d = 0; d < DB; ++d)
                o[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(as_bf16x8(vfrag(at, s, d)), as_bf16x8(pf[s]), o[d], 0, 0, 0);
    };
    // Scores of tile t + 1 (into nx), powers of tile t (from st) and its outputs, in steps of two products: the
    // fragments are read AHEAD steps before their use, the powers of a step's keys come before it, and the next
    // tile's largest score after its last; the fences keep the compiler to that order.  Copies of rows are issued
    // between the first products (10000 tokens of one head: 115 us against 123), those of pages, whose
    // addresses take longer, before them (2048 tokens over 8192: 232 us against 239).
    auto body = [&](int t, const f32x16 (&st)[2], f32x16 (&nx)[2]) __attribute__((always_inline)) {
        constexpr int N = KS + 2 * DB, AHEAD = FP8 ? 2 : 4;     // (e4m3: as the registers allow)
        if (SRC != AW_ROWS)
            issue(t + 1);
        const uint32_t ka = tile_at(klane, t + 1), va = tile_at(vlane, t);
        u32x4 f[AHEAD][2];
        auto read = [&](int i) {
#pragma unroll
            for (int e = 0; e < 2; ++e)
                f[i % AHEAD][e] = i < KS ? kfrag(ka, i, e) : vfrag(va, 2 * (i - KS) / DB, 2 * (i - KS) % DB + e);
        };
        // powers that are done after step i
        auto done = [](int i) {
            return D == 128 ? (i < 8 ? (i + 1) / 2 * 2 : i < 12 ? 2 * i - 6 : 16)
                            : (i < 4 ? 2 * i + 2 : i < 6 ? 4 * i - 4 : 16);
        };
#pragma unroll
        for (int i = 0; i < AHEAD; ++i)
            read(i);
        __builtin_amdgcn_sched_barrier(0);
        float mx = -INFINITY;
#pragma unroll
        for (int i = 0; i < N; ++i) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const bf16x8 x = as_bf16x8(f[i % AHEAD][e]);
                const int d = (2 * (i - KS) % DB + e) & (DB - 1), s = 2 * (i - KS) / DB;
                if (i < KS)
                    nx[e] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(x, as_bf16x8(qf[i < KS ? i : 0]), i ? nx[e] : zero, 0, 0, 0);
                else
                    o[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(x, as_bf16x8(pf[i < KS ? 0 : s]), o[d], 0, 0, 0);
            }
            if (i + AHEAD < N)
                read(i + AHEAD);
#pragma unroll
            for (int k = i ? done(i - 1) : 0; k < done(i); ++k)
                powers(t, k, st, std::false_type());
            if (i >= N - 2) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    scaled(t + 1, i - (N - 2), j, nx);
                mx = largest(nx[i - (N - 2)], 0, 16, mx);
            }
            __builtin_amdgcn_sched_barrier(0);
            if (SRC == AW_ROWS && i == 0)
                issue_k(t + 1);
            if (SRC == AW_ROWS && i == KS / 2)
                issue_v(t + 1);
            if (SRC == AW_ROWS && (i == 0 || i == KS / 2))
                __builtin_amdgcn_sched_barrier(0);
        }
        raise(mx);
        land(t + 1);
        phase_end();
    };
    // the same for a tile that some rows see in part: V may hold an infinity or NaN where a row must not see it
    // (0 x NaN is NaN); then one key at a time, kept only by the rows that see it
    auto outputs_edge = [&](int t) {
        const uint32_t at = tile_at(vlane, t);
        // keys of this lane's fragments (k index (hh, e) of step s) that hold an infinity or NaN: bit 8 s + e
        uint32_t bad = 0;
#pragma unroll 1
        for (int s = 0; s < 4; ++s) {
            u32x4 w = {0, 0, 0, 0};
#pragma unroll
            for (int d = 0; d < DB; ++d) {
                const u32x4 f = vfrag(at, s, d);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    w[i] = not_finite(w[i], f[i]);
            }
            uint32_t b8 = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                b8 |= ((w[i] >> 15) & 1u) << (2 * i) | (w[i] >> 31) << (2 * i + 1);
            bad |= b8 << (8 * s);
        }
        if (__any(bad != 0))
#pragma unroll
            for (int off = 1; off < 32; off <<= 1)
                bad |= __shfl_xor(bad, off, 64);
        const uint64_t some = ((uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)bad, 32) << 32) | (uint32_t)uniform((int)bad);
        for (uint64_t rest = some; rest; rest &= rest - 1) {
            const int bit = __ffsll((unsigned long long)rest) - 1, s = (bit & 31) >> 3, e = bit & 7;
            const int key = t * BN + 16 * s + 8 * (e >> 2) + 4 * (bit >> 5) + (e & 3);
            const bool see = key < L && (!a.causal || key <= pos) && (a.window <= 0 || key > pos - a.window);
            const uint32_t half = hh != (bit >> 5) ? 0u : (e & 1) ? 0xffff0000u : 0xffffu;
            u32x4 p;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t a0 = pf[0][i], a1 = pf[1][i], a2 = pf[2][i], a3 = pf[3][i];
                p[i] = (s & 2) ? ((s & 1) ? a3 : a2) : ((s & 1) ? a1 : a0);
            }
#pragma unroll
            for (int d = 0; d < DB; ++d) {
                u32x4 f = vfrag(at, s, d);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    f[i] &= i == (e >> 1) ? half : 0u;
                const f32x16 x = __builtin_amdgcn_mfma_f32_32x32x16_bf16(as_bf16x8(f), as_bf16x8(p), o[d], 0, 0, 0);
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    o[d][i] = see ? x[i] : o[d][i];
            }
        }
        // and the rest
        const uint32_t mine = (uint32_t)(some >> (32 * hh));
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            u32x4 keep;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                keep[i] = ((mine >> (8 * s + 2 * i)) & 1 ? 0u : 0xffffu) | ((mine >> (8 * s + 2 * i + 1)) & 1 ? 0u : 0xffff0000u);
#pragma unroll
            for (int d = 0; d < DB; ++d)
                o[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(as_bf16x8(vfrag(at, s, d) & keep), as_bf16x8(pf[s]), o[d],
                                                               0, 0, 0);
        }
    };
    // a tile on its own (K of it in place before; afterwards K of the next)
    auto single = [&](int t) {
        const bool work = t * BN < wmax && t * BN + BN > wmin;
        if (t > t0)
            issue(t);
        if (work) {
            scores(t, sa);
            all_scaled(t, sa);
            hide(t, sa);
            raise(largest(sa[1], 0, 16, largest(sa[0], 0, 16, -INFINITY)));
            all_powers(t, sa, std::true_type());
        }
        land(t);
        phase_end();
        if (work)
            outputs_edge(t);
    };

    if (t0 < t1) {
        lookup(t0);
        issue(t0 - 1);
        if (FP8)
            land(t0 - 1);
        issue(t0);
        if (!FP8)       // K of t0 has arrived when no more than the copies of V are in flight
            asm volatile("s_waitcnt vmcnt(%0)" :: "i"(IPW) : "memory");
    }
    phase_end();
    int t = t0;
    if (wrow >= rows) {             // no rows: this wave only copies
        for (; t < t1; ++t) {
            if (t > t0)
                issue(t);
            land(t);
            phase_end();
        }
    }
    const int lead = f0 < f1 ? f0 : t1;
    for (; t < lead; ++t)
        single(t);
    if (t < t1) {
        // tiles that all rows see in full
        if (t > t0)
            issue(t);
        scores(t, sa);
        all_scaled(t, sa);
        raise(largest(sa[1], 0, 16, largest(sa[0], 0, 16, -INFINITY)));
        land(t);
        phase_end();
        for (; t + 2 < f1; t += 2) {
            body(t, sa, sb);
            body(t + 1, sb, sa);
        }
        if (t + 1 < f1) {
            body(t, sa, sb);
            sa[0] = sb[0];
            sa[1] = sb[1];
            ++t;
        }
        all_powers(t, sa, std::false_type());
        outputs(t);
        for (++t; t < t1; ++t)
            single(t);
    }

    l += __shfl_xor(l, 32, 64);
    if (KG > 1) {
        // a tile took one barrier; the first half has a tile more if their number is odd
        if ((tb - ta) & 1 && kg)
            phase_end();
        phase_end();
        // the second half's sums join the first's
        f32x4 *part = (f32x4 *)(lds + GROUP) + wave * DB * 4 * 64 + lane;
        if (kg) {
#pragma unroll
            for (int d = 0; d < DB; ++d)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    part[(4 * d + i) * 64] = f32x4{o[d][4 * i], o[d][4 * i + 1], o[d][4 * i + 2], o[d][4 * i + 3]};
            joint[wave][lane][0] = m;
            joint[wave][lane][1] = l;
        }
        __syncthreads();
        if (kg)
            return it.total;
        const float m1 = joint[wave][lane][0], l1 = joint[wave][lane][1], mx = fmaxf(m, m1);
        const float s0 = __builtin_amdgcn_exp2f(m - mx), s1 = __builtin_amdgcn_exp2f(m1 - mx);
        m = mx;
        l = l * s0 + l1 * s1;
#pragma unroll
        for (int d = 0; d < DB; ++d)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const f32x4 x = part[(4 * d + i) * 64];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    o[d][4 * i + e] = o[d][4 * i + e] * s0 + x[e] * s1;
            }
    }
    if (a.n_chunks == 1) {
        // through the wave's own part of LDS (the tiles are done with), so that whole rows are stored
        const float inv = l > 0.f ? 1.f / l : l == 0.f ? 0.f : l;
        if (KG == 1)
            phase_end();
        uint16_t *part = kl + wave * 32 * D;
#pragma unroll
        for (int d = 0; d < DB; ++d)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                *(u32x2 *)(part + col * D + 8 * ((4 * d + i) ^ (col & (CPR - 1))) + 4 * hh) =
                    u32x2{cvt_bf16x2(o[d][4 * i] * inv, o[d][4 * i + 1] * inv),
                          cvt_bf16x2(o[d][4 * i + 2] * inv, o[d][4 * i + 3] * inv)};
        const int64_t to = (int64_t)(q0 + ri) * a.out_stride + (int64_t)hd * D;
#pragma unroll
        for (int j = 0; j < 32 * CPR / 64; ++j) {
            const int r = j * (64 / CPR) + lane / CPR, piece = lane & (CPR - 1);
            const u32x4 w = *(const u32x4 *)(part + r * D + 8 * (piece ^ (r & (CPR - 1))));
            const int64_t at = (int64_t)((uint64_t)(uint32_t)__shfl((int)(to >> 32), r, 64) << 32 |
                                         (uint32_t)__shfl((int)to, r, 64));
            if (wrow + r < rows)
                *(u32x4 *)(a.out + at + 8 * piece) = w;
        }
        if (row < rows && a.lse && hh == 0)
            a.lse[(int64_t)(q0 + ri) * a.hq + hd] =
                l == 0.f ? -INFINITY : (m + __builtin_amdgcn_logf(l)) * (1.f / ATTN_LOG2E);
    } else if (row < rows) {
        const int64_t slot = ((int64_t)(q0 + ri) * a.hq + hd) * a.n_chunks + by;
#pragma unroll
        for (int d = 0; d < DB; ++d)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                *(f32x4 *)(a.part_o + slot * D + 32 * d + 8 * i + 4 * hh) =
                    f32x4{o[d][4 * i], o[d][4 * i + 1], o[d][4 * i + 2], o[d][4 * i + 3]};
        if (hh == 0)
            *(f32x2 *)(a.part_ml + 2 * slot) = f32x2{m, l};
    }
    return it.total;
}

// Over pages: item and kv head bx, and every wide_x-th after it (wide_x: a multiple of the kv heads).
template <int D, int SRC>
__device__ __forceinline__ void attn_wide_pages(const AttnArgs &a, int bx, int by, int wide_x, uint8_t *smem)
{
    for (int64_t x = bx;; x += wide_x) {
        const int total = attn_wide_body<D, SRC, 1, true>(a, (int)x, by, smem);
        if (x + wide_x >= (int64_t)total * a.hkv)
            return;
        __syncthreads();
    }
}

}  // namespace mlora
