// Device-side helpers shared by the attention kernels.
//
// Both kernels compute transposed scores S^T = K Q^T and transposed outputs O^T = V^T P^T, so a
// query is a column: it stays in one lane (and the lanes that share its column), its running
// maximum is a per-lane value, and the accumulator of S^T is the B operand of the second
// product without moving a value across lanes.  The second product may take its keys in any
// order as long as both operands agree, so its k index is simply numbered the way the first
// product's accumulator holds the keys, and V^T is read from LDS in that order with transposing
// reads (ds_read_b64_tr_b16: 16 lanes read 4 keys x 16 values and get 4 keys of one value each).
#pragma once

#include "attention.h"
#include "common.h"

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));

namespace mlora {

constexpr float ATTN_LOG2E = 1.4426950408889634f;
// Start of the running maximum: finite, so that a masked score (-inf) minus it is -inf, never NaN.
constexpr float ATTN_LOWEST = -3.0e38f;
// The running maximum follows a new one only past this many powers of two: below it the
// probabilities (at most 2^6) and their fp32 sums lose nothing, and the accumulators are not
// rescaled for every small rise.
constexpr float ATTN_SLACK = 6.f;

// two floats as packed bf16, rounded to nearest even (one v_cvt_pk_bf16_f32)
__device__ __forceinline__ uint32_t cvt_bf16x2(float lo, float hi)
{
    const f32x2 v = {lo, hi};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
}

// 4 x 16 values of 16 bits, transposed over 16 lanes (see above); p: this lane's 8 bytes
__device__ __forceinline__ u32x2 lds_read_tr(const uint16_t *p)
{
    typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
    return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)p));
}

__device__ __forceinline__ bf16x8 as_bf16x8(u32x4 v) { return __builtin_bit_cast(bf16x8, v); }

// 8 e4m3 codes as bf16, exactly (e4m3's 4 significant bits fit bf16's 8)
__device__ __forceinline__ u32x4 e4m3_to_bf16x8(uint32_t a, uint32_t b)
{
    u32x4 r;
    r[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.f, false));
    r[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.f, true));
    r[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.f, false));
    r[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.f, true));
    return r;
}

// Bits of `acc` at 0x80008000 get set where a bf16 of w is infinite or NaN.
__device__ __forceinline__ uint32_t not_finite(uint32_t acc, uint32_t w)
{
    return acc | ((w & 0x7f807f80u) + 0x00800080u);
}

// a value that is the same in all lanes, as a scalar
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// Sum of the lanes up to and with this one (DPP: no trip through LDS).
__device__ __forceinline__ int wave_prefix(int v)
{
    v += __builtin_amdgcn_update_dpp(0, v, 0x111, 15, 15, false);    // row_shr 1, 2, 4, 8
    v += __builtin_amdgcn_update_dpp(0, v, 0x112, 15, 15, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x114, 15, 15, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x118, 15, 15, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x142, 10, 15, false);    // lane 15 of rows 0, 2 to rows 1, 3
    v += __builtin_amdgcn_update_dpp(0, v, 0x143, 12, 15, false);    // lane 31 to rows 2, 3
    return v;
}
// Sum over the 64 lanes of a wave, as a scalar.
__device__ __forceinline__ int wave_total(int v) { return __builtin_amdgcn_readlane(wave_prefix(v), 63); }

// Largest over the 64 lanes of a wave, as a scalar.
__device__ __forceinline__ float wave_largest(float v)
{
    const int lowest = __float_as_int(-INFINITY);
#define STEP(ctrl, rows) \
    v = fmaxf(v, __int_as_float(__builtin_amdgcn_update_dpp(lowest, __float_as_int(v), ctrl, rows, 15, false)))
    STEP(0x111, 15);
    STEP(0x112, 15);
    STEP(0x114, 15);
    STEP(0x118, 15);
    STEP(0x142, 10);
    STEP(0x143, 12);
#undef STEP
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}

// One wave: parts [ca, cb) of a row (fp32 outputs, maxima and sums at slot(c)) joined into row t of head hd.
template <int D, class Slot>
__device__ __forceinline__ void join_parts(const AttnArgs &a, int ca, int cb, Slot slot, int64_t t, int hd)
{
    constexpr int VPT = D / 64, AHEAD = 8;
    const int lane = threadIdx.x & 63;
    float mx = ATTN_LOWEST, sum = 0.f, acc[VPT];
    for (int c = ca + lane; c < cb; c += 64)
        mx = fmaxf(mx, a.part_ml[2 * slot(c)]);
    mx = wave_largest(mx);
#pragma unroll
    for (int e = 0; e < VPT; ++e)
        acc[e] = 0.f;
    for (int c0 = ca; c0 < cb; c0 += 64) {
        float f = 0.f;                          // this lane's chunk
        if (c0 + lane < cb) {
            const f32x2 ml = *(const f32x2 *)(a.part_ml + 2 * slot(c0 + lane));
            f = __builtin_amdgcn_exp2f(ml[0] - mx);
            sum += f * ml[1];
        }
        const int n = min(64, cb - c0);
        for (int i = 0; i < n; i += AHEAD) {
            float x[AHEAD][VPT];
#pragma unroll
            for (int j = 0; j < AHEAD; ++j)
#pragma unroll
                for (int e = 0; e < VPT; ++e)
                    x[j][e] = a.part_o[slot(c0 + min(i + j, n - 1)) * D + lane * VPT + e];
#pragma unroll
            for (int j = 0; j < AHEAD; ++j) {
                const float w = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(f), i + j));
#pragma unroll
                for (int e = 0; e < VPT; ++e)
                    acc[e] += i + j < n ? w * x[j][e] : 0.f;
            }
        }
    }
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1)
        sum += __shfl_xor(sum, off, 64);
    const float inv = sum > 0.f ? 1.f / sum : sum == 0.f ? 0.f : sum;
    uint16_t *dst = a.out + t * a.out_stride + (int64_t)hd * D + lane * VPT;
    if (VPT == 2)
        *(uint32_t *)dst = cvt_bf16x2(acc[0] * inv, acc[VPT - 1] * inv);
    else
        dst[0] = (uint16_t)cvt_bf16x2(acc[0] * inv, 0.f);
    if (a.lse && lane == 0)
        a.lse[t * a.hq + hd] = sum == 0.f ? -INFINITY : (mx + __builtin_amdgcn_logf(sum)) * (1.f / ATTN_LOG2E);
}

__device__ __forceinline__ int clamp_page(int page, int n_pages)
{
    return min(max(page, 0), n_pages - 1);
}

}  // namespace mlora
