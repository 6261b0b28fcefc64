// Attention of few query rows over a paged cache: kernels and launchers (attn_decode_body.h), and the join of split
// rows.
#include "attn_decode_body.h"

namespace mlora {

template <int D, int NQ, bool FP8, int KEYS, int PARTS>
__global__ __launch_bounds__(256, decode_slots(D, NQ)) void attn_decode_kernel(AttnArgs a)
{
    __shared__ __attribute__((aligned(16))) uint8_t smem[decode_lds<D, NQ>];
    attn_decode_body<D, NQ, FP8, KEYS, PARTS>(a, blockIdx.x, gridDim.x, smem);
}

// The join, a workgroup a cut between shares: the first cut within a sequence and head joins its parts, one wave a
// row.  A few MB that the shares just wrote: bound by the latency of a launch and its chain of loads (one context of
// 1003 keys 3.8 us; 511 cuts 6 to 8 us).
template <int D, int KEYS>
__global__ __launch_bounds__(256) void attn_combine_kernel(AttnArgs a, int shares)
{
    const int lane = threadIdx.x & 63, w1 = blockIdx.x + 1;
    const LaneUnits u = lane_units<KEYS>(a, lane);
    const Shares cut((uint32_t)u.total * a.hkv, (uint32_t)shares);
    if ((uint32_t)w1 >= cut.n)
        return;
    const uint32_t u1 = cut.start(w1);
    const UnitPlace at = find_unit<KEYS>(a, u, u1);
    const int w0 = w1 - 1;
    if (at.f == 0 || cut.start(w0) > u1 - at.f)     // nothing is cut here, or an earlier cut joins it
        return;
    const int end = (int)cut.of(u1 - at.f + at.sq.units - 1) + 1, rows = at.sq.n * a.group;
    for (int row = threadIdx.x >> 6; row < rows; row += 4) {
        const int i = row / a.group, hd = turned_head(a, at.b, at.h) * a.group + row - i * a.group;
        join_parts<D>(a, w0, end, [&](int w) { return part_slot(a, w, w > w0, row); }, at.sq.q0 + i, hd);
    }
}

namespace {

// (PARTS: of two column tiles)
template <int KEYS, int PARTS>
hipError_t launch_decode(const AttnArgs &a, int head_dim, int nq, int shares, hipStream_t stream)
{
    const dim3 grid((unsigned)shares);
#define DEC(D, NQ, F) \
    attn_decode_kernel<D, NQ, F, KEYS, NQ == 1 ? 2 : key_parts<KEYS, F, PARTS>><<<grid, dim3(256), 0, stream>>>(a)
#define DEC_F(D, NQ) (a.cache.fp8 ? DEC(D, NQ, true) : DEC(D, NQ, false))
#define DEC_Q(D) (nq == 1 ? DEC_F(D, 1) : DEC_F(D, 2))
    head_dim == 64 ? DEC_Q(64) : DEC_Q(128);
#undef DEC_Q
#undef DEC_F
#undef DEC
    return hipGetLastError();
}

template <int KEYS>
hipError_t launch_combine(const AttnArgs &a, int head_dim, int shares, hipStream_t stream)
{
    if (shares < 2)
        return hipSuccess;
    const dim3 grid((unsigned)(shares - 1));
    if (head_dim == 64)
        attn_combine_kernel<64, KEYS><<<grid, dim3(256), 0, stream>>>(a, shares);
    else
        attn_combine_kernel<128, KEYS><<<grid, dim3(256), 0, stream>>>(a, shares);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_attn_decode(const AttnArgs &a, int head_dim, int nq, int shares, hipStream_t stream)
{
    return few_keys(a)   ? launch_decode<KEYS_SINKS, 2>(a, head_dim, nq, shares, stream)
           : a.sinks > 0 ? launch_decode<KEYS_SINKS, 1>(a, head_dim, nq, shares, stream)
                         : launch_decode<KEYS_PLAIN, 1>(a, head_dim, nq, shares, stream);
}

hipError_t launch_attn_combine(const AttnArgs &a, int head_dim, int shares, hipStream_t stream)
{
    return a.sinks > 0 ? launch_combine<KEYS_SINKS>(a, head_dim, shares, stream)
                       : launch_combine<KEYS_PLAIN>(a, head_dim, shares, stream);
}

}  // namespace mlora
