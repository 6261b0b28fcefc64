// Norm, rotation and cache write of a merged QKV layer's rows, and the cache read back.
//
// One pass: a head of D values lies in D / 8 lanes of 8 values (16 bytes), so a wave holds 8 (D =
// 64) or 4 (D = 128) heads of one token at a time and takes the token's heads group by group.
// The sum of squares and the largest value are joined over a head's lanes in registers (DPP), the
// rotation's partner values come from the lane rot / 16 away.  A value becomes
// (x A + y B) / rms with its partner y; A and B (weights times cosine and sine) are made once per
// wave and token and serve all of the wave's heads.  Bound by HBM: each row is read and written
// once (D = 128, 32 + 2 x 8 heads: 16384 rows 79 us, 5.1 TB/s, the rate of a large copy; 2304 rows into
// an e4m3 cache 15 us; 64 rows 4.3 us, the latency of one launch).
//
// Angles: pair i turns by frac(pos * turns[i] / 2^64) of a circle.  The product is taken modulo
// 2^64, so its top 32 bits are the exact fraction (to 2^-32) at any position; sine and cosine
// take turns as they are (v_sin_f32 / v_cos_f32).
#include <algorithm>

#include "attention.h"
#include "attention_device.h"

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

// 8 values times `up` as e4m3 codes (rounded to nearest even)
__device__ __forceinline__ u32x2 to_e4m3(const float (&v)[8], float up)
{
    u32x2 c;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        int w = 0;
        w = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * i] * up, v[4 * i + 1] * up, w, false);
        w = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * i + 2] * up, v[4 * i + 3] * up, w, true);
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
        r[i] = cvt_bf16x2(x[2 * i], x[2 * i + 1]);
    return r;
}

template <int D>
__global__ __launch_bounds__(256) void qk_rope_kernel(RopeArgs a, int wpt_log)
{
    constexpr int LPH = D / 8;      // lanes per head
    constexpr int HPW = 64 / LPH;   // heads a wave holds at a time
    const int64_t gw = (int64_t)blockIdx.x * 4 + uniform(threadIdx.x >> 6);
    const int64_t t = gw >> wpt_log;
    const int wpt = 1 << wpt_log, part = (int)gw & (wpt - 1);
    const int lane = threadIdx.x & 63, c = lane % LPH, hl = lane / LPH;
    const int heads = a.hq + 2 * a.hkv, groups = (heads + HPW - 1) / HPW;
    if (t >= a.T || part >= groups)
        return;
    const uint16_t *row = a.qkv + t * a.row_stride;

    constexpr int UN = 4;           // groups loaded ahead
    u32x4 raw[UN];
    auto load = [&](int g0) {
#pragma unroll
        for (int u = 0; u < UN; ++u) {
            const int h = (g0 + u * wpt) * HPW + hl;
            raw[u] = h < heads ? *(const u32x4 *)(row + (int64_t)h * D + 8 * c) : u32x4{0, 0, 0, 0};
        }
    };
    load(part);

    // this chunk's rotation: values 8c .. 8c+7, partner chunk pc
    const int rot = a.rot, half = rot >> 1;
    const bool turned = 8 * c < rot, inter = a.interleaved != 0;
    const bool first = 8 * c < half;
    const int pc = (inter || !turned) ? c : first ? c + (half >> 3) : c - (half >> 3);
    float cs[8], sn[8];             // sn: with the sign of the partner's part
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        cs[e] = 1.f;
        sn[e] = 0.f;
    }
    if (turned) {
        const uint64_t pos = (uint64_t)(int64_t)a.pos[t];
        const int f0 = inter ? 4 * c : (first ? 8 * c : 8 * c - half);
        auto turn = [&](int f, float &co, float &si) {
            const int32_t top = (int32_t)((pos * a.turns[f]) >> 32);
            const float x = (float)top * 0x1p-32f;      // [-1/2, 1/2)
            co = __builtin_amdgcn_cosf(x) * a.magnitude;
            si = __builtin_amdgcn_sinf(x) * a.magnitude;
        };
        if (inter) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                turn(f0 + i, cs[2 * i], sn[2 * i + 1]);
                cs[2 * i + 1] = cs[2 * i];
                sn[2 * i] = -sn[2 * i + 1];
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                turn(f0 + e, cs[e], sn[e]);
                sn[e] = first ? -sn[e] : sn[e];
            }
        }
    }
    // A and B of queries and keys
    float qa[8], qb[8], ka[8], kb[8];
    auto coefficients = [&](const uint16_t *weight, float (&ca)[8], float (&cb)[8]) {
        float w[8], p[8];
#pragma unroll
        for (int e = 0; e < 8; ++e)
            w[e] = p[e] = 1.f;
        if (weight) {
            unpack8(*(const u32x4 *)(weight + 8 * c), w);
            u32x4 bits = {0, 0, 0, 0};      // (no partner: an infinite weight times sn = 0 would not be zero)
            if (turned)
                bits = *(const u32x4 *)(weight + 8 * pc);
            unpack8(bits, p);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            ca[e] = w[e] * cs[e];
            cb[e] = (inter ? p[e ^ 1] : p[e]) * sn[e];
        }
    };
    coefficients(a.qw, qa, qb);
    coefficients(a.kw, ka, kb);
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

    for (int g0 = part; g0 < groups;) {
        u32x4 now[UN];
#pragma unroll
        for (int u = 0; u < UN; ++u)
            now[u] = raw[u];
        const int gb = g0;
        g0 += UN * wpt;
        if (g0 < groups)
            load(g0);
#pragma unroll
        for (int u = 0; u < UN; ++u) {
            const int g = gb + u * wpt, h = g * HPW + hl;
            if (g >= groups)
                break;
            const bool is_q = h < a.hq, is_k = !is_q && h < a.hq + a.hkv;
            u32x4 bits = now[u];
            float o[8];
            unpack8(bits, o);
            if (g * HPW < a.hq + a.hkv) {       // not values alone
                float inv = 1.f;
                if (a.qw || a.kw) {
                    float ss = 0.f;
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        ss += o[e] * o[e];
                    ss = head_join<LPH>(ss, [](float p, float q) { return p + q; });
                    const bool normed = is_q ? a.qw != nullptr : a.kw != nullptr;
                    inv = normed ? __builtin_amdgcn_rsqf(ss * (1.f / D) + a.eps) : 1.f;
                }
                u32x4 pr = bits;
                if (rot) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        pr[i] = inter ? (pr[i] >> 16 | pr[i] << 16) : (uint32_t)__shfl((int)pr[i], partner, 64);
                        pr[i] = turned ? pr[i] : 0u;
                    }
                }
                float y[8], r[8];
                unpack8(pr, y);
                auto rotate = [&](const float (&ca)[8], const float (&cb)[8]) {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        r[e] = (rot ? fmaf(o[e], ca[e], y[e] * cb[e]) : o[e] * ca[e]) * inv;
                };
                if ((g + 1) * HPW <= a.hq) {
                    rotate(qa, qb);
                } else if (g * HPW >= a.hq) {
                    rotate(ka, kb);
                } else {
                    float ca[8], cb[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        ca[e] = is_q ? qa[e] : ka[e];
                        cb[e] = is_q ? qb[e] : kb[e];
                    }
                    rotate(ca, cb);
                }
                const u32x4 turned_bits = pack8(r);
                if (is_q || is_k) {
                    bits = turned_bits;
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        o[e] = r[e];
                }
            }
            if (is_q) {
                *(u32x4 *)(a.q_out + t * a.q_stride + (int64_t)h * D + 8 * c) = bits;
                continue;
            }
            // keys and values
            const int kh = h - a.hq - (is_k ? 0 : a.hkv);
            if (is_k && a.k_out)
                *(u32x4 *)(a.k_out + t * a.k_stride + (int64_t)kh * D + 8 * c) = bits;
            if (!stored || h >= heads)
                continue;
            const int64_t at = ((page * a.cache.hkv + kh) << a.cache.ps) + off;
            uint8_t *dst = is_k ? a.cache.k : a.cache.v;
            if (!a.cache.fp8) {
                *(u32x4 *)(dst + (at * D + 8 * c) * 2) = bits;
            } else {
                float top = 0.f;
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    top = fmaxf(top, fabsf(o[e]));
                top = fmaxf(head_join<LPH>(top, [](float p, float q) { return fmaxf(p, q); }), 0x1p-90f);
                *(u32x2 *)(dst + at * D + 8 * c) = to_e4m3(o, 448.f / top);
                if (c == 0)
                    (is_k ? a.cache.k_scale : a.cache.v_scale)[at] = top / 448.f;
            }
        }
    }
}

hipError_t launch_qk_rope(const RopeArgs &a, int head_dim, hipStream_t stream)
{
    const int hpw = 64 / (head_dim / 8);
    const int groups = (a.hq + 2 * a.hkv + hpw - 1) / hpw;
    // one wave takes a whole token where that makes 2048 waves (its sines and coefficients serve every head), else
    // more waves a token, a power of two (512 tokens: 6 us with 4 waves each, 10 with 16; 64 tokens: 4 us with 16)
    int wpt_log = 0;
    while ((1 << wpt_log) < groups && (a.T << wpt_log) < 2048)
        ++wpt_log;
    const int64_t blocks = ((a.T << wpt_log) + 3) / 4;
    if (blocks > 0x7fffffff)
        return hipErrorInvalidValue;
    if (head_dim == 64)
        qk_rope_kernel<64><<<dim3((unsigned)blocks), dim3(256), 0, stream>>>(a, wpt_log);
    else
        qk_rope_kernel<128><<<dim3((unsigned)blocks), dim3(256), 0, stream>>>(a, wpt_log);
    return hipGetLastError();
}

// A workgroup reads `tokens` tokens, keys (blockIdx.y = 0) or values (1), 8 values a thread at a time and 4 such
// pieces in flight.  Bound by HBM (32768 e4m3 tokens, 8 heads of 128: 43 us, 4.7 TB/s; 333 bf16 ones 2.5 us, latency).
template <int D, bool FP8>
__global__ __launch_bounds__(256) void cache_read_kernel(CacheGeom cg, const int32_t *__restrict__ slot,
                                                         int64_t T, int tokens, uint16_t *k, uint16_t *v)
{
    constexpr int C = D / 8, UN = 4;
    uint16_t *out = blockIdx.y == 0 ? k : v;
    if (out == nullptr)
        return;
    const uint8_t *src = blockIdx.y == 0 ? cg.k : cg.v;
    const float *scales = blockIdx.y == 0 ? cg.k_scale : cg.v_scale;
    const int64_t t0 = (int64_t)blockIdx.x * tokens;
    const int width = cg.hkv * C, n = (int)min((int64_t)tokens, T - t0) * width;
    const float per = 1.f / (float)width;
    out += t0 * width * 8;
    for (int i0 = threadIdx.x; i0 < n; i0 += UN * 256) {
        u32x4 w[UN];
        float sc[UN];
#pragma unroll
        for (int u = 0; u < UN; ++u) {
            const int i = i0 + 256 * u;
            if (i >= n)
                break;
            const int t = (int)(((float)i + 0.5f) * per);       // i / width (exact: i is below 2^22)
            const int c = i % C, h = (i - t * width) / C;
            const int32_t s = slot[t0 + t];
            w[u] = u32x4{0, 0, 0, 0};
            sc[u] = 0.f;
            if (s >= 0 && (s >> cg.ps) < cg.n_pages) {
                const int64_t at = (((int64_t)(s >> cg.ps) * cg.hkv + h) << cg.ps) + (s & ((1 << cg.ps) - 1));
                if (!FP8) {
                    w[u] = *(const u32x4 *)(src + (at * D + 8 * c) * 2);
                } else {
                    const u32x2 x = *(const u32x2 *)(src + at * D + 8 * c);
                    w[u][0] = x[0];
                    w[u][1] = x[1];
                    sc[u] = scales[at];
                }
            }
        }
#pragma unroll
        for (int u = 0; u < UN; ++u) {
            const int i = i0 + 256 * u;
            if (i >= n)
                break;
            if (FP8) {
                float x[8];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[u][j], false);
                    const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[u][j], true);
                    x[4 * j] = lo[0] * sc[u];
                    x[4 * j + 1] = lo[1] * sc[u];
                    x[4 * j + 2] = hi[0] * sc[u];
                    x[4 * j + 3] = hi[1] * sc[u];
                }
                w[u] = pack8(x);
            }
            *(u32x4 *)(out + (int64_t)i * 8) = w[u];
        }
    }
}

hipError_t launch_cache_read(const CacheGeom &c, int head_dim, const int32_t *slot, int64_t T,
                             uint16_t *k, uint16_t *v, hipStream_t stream)
{
    const int width = c.hkv * (head_dim / 8);           // at most 2^14
    const int tokens = std::max(1, (T * width < (1 << 19) ? 256 : 1024) / width);
    const int64_t blocks = (T + tokens - 1) / tokens;
    if (blocks > 0x7fffffff)
        return hipErrorInvalidValue;
    const dim3 grid((unsigned)blocks, 2);
#define READ(D, F) cache_read_kernel<D, F><<<grid, dim3(256), 0, stream>>>(c, slot, T, tokens, k, v)
    if (head_dim == 64)
        c.fp8 ? READ(64, true) : READ(64, false);
    else
        c.fp8 ? READ(128, true) : READ(128, false);
#undef READ
    return hipGetLastError();
}

}  // namespace mlora
