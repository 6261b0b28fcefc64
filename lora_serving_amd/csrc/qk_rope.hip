// Norm, rotation and cache write of a merged QKV layer's rows, and the cache read back.
//
// One pass: a head of D values lies in D / 8 lanes of 8 values (16 bytes), so a wave holds 8 (D =
// 64) or 4 (D = 128) heads of one token at a time and takes the token's heads group by group.
// The sum of squares and the largest value are joined over a head's lanes in registers (DPP), the
// rotation's partner half comes from the lane rot / 16 away.  Bound by HBM: each row is read
// and written once.
//
// Angles: pair i turns by frac(pos * turns[i] / 2^64) of a circle.  The product is taken modulo
// 2^64, so its top 32 bits are the exact fraction (to 2^-32) at any position; sine and cosine
// take turns as they are (v_sin_f32 / v_cos_f32).  They are computed once per wave and token and
// serve all of the wave's heads.
#include <algorithm>

#include "attention.h"
#include "common.h"

namespace mlora {

// v op'ed over the 8 or 16 lanes of a head, result in every lane
template <int LANES, class Op>
__device__ __forceinline__ float head_join(float v, Op op)
{
    v = op(v, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0xb1, 15, 15, true)));
    v = op(v, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x4e, 15, 15, true)));
    v = op(v, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x141, 15, 15, true)));
    if (LANES == 16)
        v = op(v, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x140, 15, 15, true)));
    return v;
}

// 8 values as e4m3 codes of v / scale (rounded to nearest even)
__device__ __forceinline__ u32x2 to_e4m3(const float (&v)[8], float scale)
{
    u32x2 c;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        int w = 0;
        w = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * i] / scale, v[4 * i + 1] / scale, w, false);
        w = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * i + 2] / scale, v[4 * i + 3] / scale, w, true);
        c[i] = (uint32_t)w;
    }
    return c;
}

__device__ __forceinline__ void unpack8(u32x4 r, float (&x)[8])
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = bf16_lo(r[i]);
        x[2 * i + 1] = bf16_hi(r[i]);
    }
}

__device__ __forceinline__ u32x4 pack8(const float (&x)[8])
{
    u32x4 r;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        r[i] = pack_bf16x2(x[2 * i], x[2 * i + 1]);
    return r;
}

template <int D>
__global__ __launch_bounds__(256) void qk_rope_kernel(RopeArgs a, int wpt)
{
    constexpr int LPH = D / 8;      // lanes per head
    constexpr int HPW = 64 / LPH;   // heads a wave holds at a time
    const int64_t gw = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    const int64_t t = gw / wpt;
    if (t >= a.T)
        return;
    const int part = (int)(gw - t * wpt);
    const int lane = threadIdx.x & 63, c = lane % LPH, hl = lane / LPH;
    const int heads = a.hq + 2 * a.hkv, groups = (heads + HPW - 1) / HPW;
    const uint16_t *row = a.qkv + t * a.row_stride;

    // this chunk's rotation: values 8c .. 8c+7, partner chunk pc
    const int rot = a.rot, half = rot >> 1;
    const bool turned = 8 * c < rot, inter = a.interleaved != 0;
    const bool first = 8 * c < half;
    const int pc = (inter || !turned) ? c : first ? c + (half >> 3) : c - (half >> 3);
    float cs[8], sn[8];
    if (turned) {
        const uint64_t pos = (uint64_t)(int64_t)a.pos[t];
        const int n = inter ? 4 : 8, f0 = inter ? 4 * c : (first ? 8 * c : 8 * c - half);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e < n) {
                const int32_t top = (int32_t)((pos * a.turns[f0 + e]) >> 32);
                const float turn = (float)top * 0x1p-32f;   // [-1/2, 1/2)
                cs[e] = __builtin_amdgcn_cosf(turn) * a.magnitude;
                sn[e] = __builtin_amdgcn_sinf(turn) * a.magnitude;
            }
    }
    // norm weights of this chunk and of the partner's
    float qw[8], kw[8], qp[8], kp[8];
    if (a.qw) {
        unpack8(*(const u32x4 *)(a.qw + 8 * c), qw);
        unpack8(*(const u32x4 *)(a.qw + 8 * pc), qp);
    }
    if (a.kw) {
        unpack8(*(const u32x4 *)(a.kw + 8 * c), kw);
        unpack8(*(const u32x4 *)(a.kw + 8 * pc), kp);
    }
    int64_t page = 0;
    int off = 0;
    bool stored = false;
    if (a.cache.k) {
        const int32_t s = a.slot[t];
        stored = s >= 0 && (s >> a.cache.ps) < a.cache.n_pages;
        page = s >> a.cache.ps;
        off = s & ((1 << a.cache.ps) - 1);
    }
    const int partner = (lane & ~(LPH - 1)) + pc;

    constexpr int UN = 4;           // groups loaded ahead
    for (int g0 = part; g0 < groups; g0 += UN * wpt) {
        u32x4 raw[UN];
#pragma unroll
        for (int u = 0; u < UN; ++u) {
            const int h = (g0 + u * wpt) * HPW + hl;
            raw[u] = h < heads ? *(const u32x4 *)(row + (int64_t)h * D + 8 * c) : u32x4{0, 0, 0, 0};
        }
#pragma unroll
        for (int u = 0; u < UN; ++u) {
            if (g0 + u * wpt >= groups)
                break;
            const int h = (g0 + u * wpt) * HPW + hl;
            const bool is_q = h < a.hq, is_k = !is_q && h < a.hq + a.hkv;
            float x[8];
            unpack8(raw[u], x);
            float inv = 1.f;
            const bool normed = is_q ? a.qw != nullptr : is_k && a.kw != nullptr;
            if (a.qw || a.kw) {
                float ss = 0.f;
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    ss += x[e] * x[e];
                ss = head_join<LPH>(ss, [](float p, float q) { return p + q; });
                inv = 1.f / sqrtf(ss * (1.f / D) + a.eps);
            }
            float o[8];
#pragma unroll
            for (int e = 0; e < 8; ++e)
                o[e] = normed ? x[e] * inv * (is_q ? qw[e] : kw[e]) : x[e];
            if (rot) {
                u32x4 pr;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    pr[i] = inter ? 0u : (uint32_t)__shfl((int)raw[u][i], partner, 64);
                if (turned && (is_q || is_k)) {
                    if (inter) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float p = o[2 * i], q = o[2 * i + 1];
                            o[2 * i] = p * cs[i] - q * sn[i];
                            o[2 * i + 1] = q * cs[i] + p * sn[i];
                        }
                    } else {
                        float y[8];
                        unpack8(pr, y);
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const float q = normed ? y[e] * inv * (is_q ? qp[e] : kp[e]) : y[e];
                            o[e] = o[e] * cs[e] + (first ? -q : q) * sn[e];
                        }
                    }
                }
            }
            if (is_q) {
                *(u32x4 *)(a.q_out + t * a.q_stride + (int64_t)h * D + 8 * c) = pack8(o);
                continue;
            }
            // keys and values
            const int kh = h - a.hq - (is_k ? 0 : a.hkv);
            if (is_k && a.k_out)
                *(u32x4 *)(a.k_out + t * a.k_stride + (int64_t)kh * D + 8 * c) = pack8(o);
            if (!stored || h >= heads)
                continue;
            const int64_t at = ((page * a.cache.hkv + kh) << a.cache.ps) + off;
            uint8_t *dst = is_k ? a.cache.k : a.cache.v;
            if (!a.cache.fp8) {
                *(u32x4 *)(dst + (at * D + 8 * c) * 2) = pack8(o);
            } else {
                float top = 0.f;
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    top = fmaxf(top, fabsf(o[e]));
                top = head_join<LPH>(top, [](float p, float q) { return fmaxf(p, q); });
                const float scale = fmaxf(top, 0x1p-90f) / 448.f;
                *(u32x2 *)(dst + at * D + 8 * c) = to_e4m3(o, scale);
                if (c == 0)
                    (is_k ? a.cache.k_scale : a.cache.v_scale)[at] = scale;
            }
        }
    }
}

hipError_t launch_qk_rope(const RopeArgs &a, int head_dim, hipStream_t stream)
{
    const int hpw = 64 / (head_dim / 8);
    const int groups = (a.hq + 2 * a.hkv + hpw - 1) / hpw;
    // one wave takes a whole token where there are tokens enough to fill the card (its sines serve
    // every head), more waves a token where there are few
    int wpt = 1;
    while (wpt < groups && a.T * wpt < 8192)
        wpt = std::min(groups, wpt * 2);
    const int64_t blocks = (a.T * wpt + 3) / 4;
    if (blocks > 0x7fffffff)
        return hipErrorInvalidValue;
    if (head_dim == 64)
        qk_rope_kernel<64><<<dim3((unsigned)blocks), dim3(256), 0, stream>>>(a, wpt);
    else
        qk_rope_kernel<128><<<dim3((unsigned)blocks), dim3(256), 0, stream>>>(a, wpt);
    return hipGetLastError();
}

// 8 values a thread: (token, kv head, chunk), keys (blockIdx.y = 0) and values (1)
template <int D, bool FP8>
__global__ __launch_bounds__(256) void cache_read_kernel(CacheGeom cg, const int32_t *__restrict__ slot,
                                                         int64_t n, uint16_t *k, uint16_t *v)
{
    constexpr int C = D / 8;
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    uint16_t *out = blockIdx.y == 0 ? k : v;
    if (i >= n || out == nullptr)
        return;
    const int c = (int)(i % C);
    const int64_t th = i / C, t = th / cg.hkv;
    const int h = (int)(th - t * cg.hkv);
    const int32_t s = slot[t];
    u32x4 r = {0, 0, 0, 0};
    if (s >= 0 && (s >> cg.ps) < cg.n_pages) {
        const int64_t at = (((int64_t)(s >> cg.ps) * cg.hkv + h) << cg.ps) + (s & ((1 << cg.ps) - 1));
        const uint8_t *src = blockIdx.y == 0 ? cg.k : cg.v;
        if (!FP8) {
            r = *(const u32x4 *)(src + (at * D + 8 * c) * 2);
        } else {
            const u32x2 w = *(const u32x2 *)(src + at * D + 8 * c);
            const float sc = (blockIdx.y == 0 ? cg.k_scale : cg.v_scale)[at];
            float x[8];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[j], false);
                const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[j], true);
                x[4 * j] = lo[0] * sc;
                x[4 * j + 1] = lo[1] * sc;
                x[4 * j + 2] = hi[0] * sc;
                x[4 * j + 3] = hi[1] * sc;
            }
            r = pack8(x);
        }
    }
    *(u32x4 *)(out + i * 8) = r;
}

hipError_t launch_cache_read(const CacheGeom &c, int head_dim, const int32_t *slot, int64_t T,
                             uint16_t *k, uint16_t *v, hipStream_t stream)
{
    const int64_t n = T * c.hkv * (head_dim / 8), blocks = (n + 255) / 256;
    if (blocks > 0x7fffffff)
        return hipErrorInvalidValue;
    const dim3 grid((unsigned)blocks, 2);
#define READ(D, F) cache_read_kernel<D, F><<<grid, dim3(256), 0, stream>>>(c, slot, n, k, v)
    if (head_dim == 64)
        c.fp8 ? READ(64, true) : READ(64, false);
    else
        c.fp8 ? READ(128, true) : READ(128, false);
#undef READ
    return hipGetLastError();
}

}  // namespace mlora
