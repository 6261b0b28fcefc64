// Attention of many query rows: kernels and launchers (attn_wide_body.h), and the join of rows whose keys are cut
// into chunks.
#include <algorithm>

#include "attn_wide_body.h"

namespace mlora {

template <int D, int SRC, int KG>
__global__ __launch_bounds__(KG * 256, 2) void attn_wide_kernel(AttnArgs a)
{
    __shared__ __attribute__((aligned(16))) uint8_t smem[wide_lds<D, SRC, KG>];
    attn_wide_body<D, SRC, KG>(a, blockIdx.x, blockIdx.y, smem);
}

// One wave a (token, head): the chunks that hold keys it sees, joined.
template <int D>
__global__ __launch_bounds__(256) void attn_wide_combine_kernel(AttnArgs a)
{
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
    const int ca = lo / a.chunk, cb = hi > lo ? (hi - 1) / a.chunk + 1 : ca;
    join_parts<D>(a, ca, cb, [&](int c) { return th * a.n_chunks + c; }, t, hd);
}

hipError_t launch_attn_wide(const AttnArgs &a, int head_dim, bool pages, hipStream_t stream)
{
    const int64_t items = wide_items(a);
    if (items * a.hkv > 0x7fffffff)
        return hipErrorInvalidValue;
    const dim3 grid((unsigned)(items * a.hkv), (unsigned)a.n_chunks);
    // Whole prompts that fill at most one workgroup a CU: the tiles of long rows (8 or more) go to two halves of a
    // workgroup of twice the waves, which a CU holds as well as two workgroups (10000 tokens of one head: 115 us
    // against 145; 300 tokens of 32 heads: 13.5 against 13.0).  Pages are cut into chunks instead.
    const int64_t keys = a.cu_k ? a.Tk : a.max_q, span = a.window > 0 ? std::min<int64_t>(keys, a.window) : keys;
    const bool halves = items * a.hkv <= CUS && span >= 8 * AW_BN;
#define AW(D, SRC, KG) attn_wide_kernel<D, SRC, KG><<<grid, dim3(KG * 256), 0, stream>>>(a)
#define AW_R(D) (halves ? AW(D, AW_ROWS, 2) : AW(D, AW_ROWS, 1))
#define AW_P(D) (a.cache.fp8 ? AW(D, AW_PAGES_E4M3, 1) : AW(D, AW_PAGES, 1))
#define AW_S(D) (pages ? AW_P(D) : AW_R(D))
    head_dim == 64 ? AW_S(64) : AW_S(128);
#undef AW_S
#undef AW_P
#undef AW_R
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
