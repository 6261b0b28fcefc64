// The mixed batch over pages: chunks of new tokens (attn_wide_body.h) and decode rows (attn_decode_body.h) in one
// launch.  The former are bound by the matrix cores, the latter by memory, and a CU holds two workgroups of either
// kind; so the launch begins with one of each on every CU and goes on with both in turn (256 tokens with contexts of
// 64 to 2048 and a chunk of 2048 tokens after 6000: 361 to 383 us, one kernel after the other 447; with contexts of 1000
// and a chunk over 8192 356 to 377 us against 432).
#include "attn_decode_body.h"
#include "attn_wide_body.h"

namespace mlora {

// MORE: there may be more wide items than workgroups for them, which then go on with further ones.  The host does not
// know the lengths, and workgroups for the most items that they allow are a cost beside a short chunk, in return for
// which long ones are spread better.  Of 210 batches (16 to 1000 single tokens over 200 or 2000 keys and a chunk of 33
// to 2048; 32 heads on 8, 16 on 16, 64 on 8) 40 are more than 3% faster than with a workgroup for each item and 9
// slower, 1% faster in the mean: 16 tokens over 2000 and a chunk of 33 over 4000 44 us (50), 250 e4m3 ones over 200 and
// 33 over 4000 66 (74), 100 over 200 and 128 over 2000 51 (54); but 200 over 1000 and 512 over 2000 228 (210), and of
// 16 heads on 16 250 e4m3 ones over 2000 and 2048 over 8192 540 (486).  Where there cannot be more items the loop is
// left out (a chunk of 2048 e4m3 tokens over 8192: 279 us, with it 286).
template <int D, bool FP8, bool MORE>
__global__ __launch_bounds__(256, 2) void attn_mixed_kernel(AttnArgs w, AttnArgs d, uint32_t wide_x, uint32_t shares)
{
    constexpr int SRC = FP8 ? AW_PAGES_E4M3 : AW_PAGES;
    constexpr int LDS = wide_lds<D, SRC, 1> > decode_lds<D, 1> ? wide_lds<D, SRC, 1> : decode_lds<D, 1>;
    __shared__ __attribute__((aligned(16))) uint8_t smem[LDS];
    // the first 256 of the wide ones, the first 256 of the others, then groups of each in turn.  Workgroups go to the 8
    // XCDs, and within one to its shader engines and their CUs, in turn: smaller groups would give each kind to some
    // of them alone (groups of 8: a chunk of 2048 with empty shares between 319 us, groups of 256 232).
    constexpr uint32_t GROUP = 256;
    const uint32_t wide = wide_x * w.n_chunks, w0 = min(wide, (uint32_t)CUS), d0 = min(shares, (uint32_t)CUS);
    uint32_t i = blockIdx.x;
    bool is_wide = i < w0;
    if (!is_wide) {
        i -= w0;
        if (i >= d0) {
            i -= d0;
            const uint32_t both = min(wide - w0, shares - d0) & ~(GROUP - 1);
            if (i < 2 * both) {
                is_wide = (i / GROUP & 1) == 0;
                i = i / (2 * GROUP) * GROUP + (i & (GROUP - 1)) + (is_wide ? w0 : d0);
            } else {
                i -= 2 * both;
                is_wide = i < wide - w0 - both;
                i = is_wide ? i + w0 + both : i - (wide - w0 - both) + d0 + both;
            }
        }
    }
    if (is_wide && MORE)
        attn_wide_pages<D, SRC>(w, (int)(i % wide_x), (int)(i / wide_x), (int)wide_x, smem);
    else if (is_wide)
        attn_wide_body<D, SRC, 1>(w, (int)(i % wide_x), (int)(i / wide_x), smem);
    else
        attn_decode_body<D, 1, FP8>(d, i, shares, smem);
}

hipError_t launch_attn_mixed(const AttnArgs &w, const AttnArgs &d, int head_dim, int shares, hipStream_t stream)
{
    const int64_t wide_x = wide_launched(w) * w.hkv, blocks = wide_x * w.n_chunks + shares;
    if (blocks > 0x7fffffff)
        return hipErrorInvalidValue;
    const bool more = wide_launched(w) < wide_items(w);
    const dim3 grid((unsigned)blocks);
#define MIX(D, F, M) attn_mixed_kernel<D, F, M><<<grid, dim3(256), 0, stream>>>(w, d, (uint32_t)wide_x, (uint32_t)shares)
#define MIX_M(D, F) (more ? MIX(D, F, true) : MIX(D, F, false))
#define MIX_F(D) (d.cache.fp8 ? MIX_M(D, true) : MIX_M(D, false))
    head_dim == 64 ? MIX_F(64) : MIX_F(128);
#undef MIX_F
#undef MIX_M
#undef MIX
    return hipGetLastError();
}

}  // namespace mlora
