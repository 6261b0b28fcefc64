// Attention of a batch whose sequences share long prefixes: a group's rows (queries x heads, of all its sequences) are
// multiplied with the prefix together, so that it is read once, and each sequence's rows with its own further keys;
// what both leave of a row, fp32 outputs o with their maximum m and sum l, is joined:
//   M = max m_c,  out = sum_c 2^(m_c - M) o_c / sum_c 2^(m_c - M) l_c
// The shared part is the wide kernel's (attn_wide_body.h: the group as one sequence of queries that see every key),
// cut into chunks of keys; the own part is the mixed batch's (attn_mixed.hip).  All of them in one launch, for the former
// is bound by the matrix cores and the latter by memory.
#include "attn_decode_body.h"
#include "attn_mixed.h"
#include "attn_wide_body.h"

namespace mlora {

template <int D, int NQ, bool FP8, bool WIDE>
__global__ __launch_bounds__(256, 2) void attn_prefix_kernel(AttnArgs s, AttnArgs w, AttnArgs d, uint32_t shared_x,
                                                             uint32_t wide_x, uint32_t shares)
{
    constexpr int SRC = FP8 ? AW_PAGES_E4M3 : AW_PAGES;
    constexpr int LDS = wide_lds<D, SRC, 1> > decode_lds<D, NQ> ? wide_lds<D, SRC, 1> : decode_lds<D, NQ>;
    __shared__ __attribute__((aligned(16))) uint8_t smem[LDS];
    uint32_t i = blockIdx.x;
    const uint32_t shared = shared_x * s.n_chunks;
    if (!mixed_place(shared + (WIDE ? wide_x * w.n_chunks : 0), shares, &i)) {
        attn_decode_body<D, NQ, FP8, KEYS_OWN>(d, i, shares, smem);
    } else if (!WIDE || i < shared) {
        attn_wide_body<D, SRC, 1, false, KEYS_SHARED>(s, (int)(i % shared_x), (int)(i / shared_x), smem);
    } else {
        i -= shared;
        attn_wide_pages<D, SRC, KEYS_OWN>(w, (int)(i % wide_x), (int)(i / wide_x), (int)wide_x, smem);
    }
}

// The join, one wave a (token, head): the chunks of the shared keys, and what its own keys left: a slot of the row, or
// (decode) the parts of the shares that it was cut between, or (wide) its chunks.
template <int D>
__global__ __launch_bounds__(256) void attn_prefix_join_kernel(AttnArgs s, AttnArgs w, AttnArgs d)
{
    const int64_t th = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    const int lane = threadIdx.x & 63;
    if (th >= d.T * d.hq)
        return;
    const int t = (int)(th / d.hq), hd = (int)(th - (int64_t)t * d.hq);
    int b = -1;
    for (int s0 = 0; s0 < d.n_seqs; s0 += 64) {
        const int i = s0 + lane;
        const uint64_t hit = ballot64(i < d.n_seqs && d.cu_q[i] <= t && t < d.cu_q[i + 1]);
        if (hit) {
            b = s0 + __ffsll((unsigned long long)hit) - 1;
            break;
        }
    }
    if (b < 0)
        return;
    const int q0 = max(d.cu_q[b], 0), n = (int)min((int64_t)d.cu_q[b + 1], d.T) - q0;
    if (n > d.max_q)
        return;
    const int L = (int)min((int64_t)max(d.kv_len[b], 0), min(d.max_kv, d.table_stride << d.cache.ps));
    const int keys = shared_keys(d, b, n, L), chunks = (keys + s.chunk - 1) / s.chunk;
    const int64_t rows = (int64_t)n * d.group;
    if (rows <= d.max_rows) {
        const int h = hd / d.group, row = (t - q0) * d.group + hd - h * d.group;
        const int32_t *const c = d.cuts + 2 * ((int64_t)b * d.hkv + h);
        const int w0 = c[0], w1 = c[1];
        if (w0 < 0 && keys == 0)        // answered whole
            return;
        join_parts<D>(d, 0, chunks + (w0 < 0 ? 1 : w1 - w0 + 1), [&](int i) {
            return i < chunks ? row_slot(s, t, hd, i)
                   : w0 < 0   ? row_slot(d, t, hd, 0)
                              : part_slot(d, w0 + i - chunks, i > chunks, row);
        }, t, hd);
    } else {
        if (w.n_chunks == 1 && keys == 0)
            return;
        const int hi = w.causal ? min(L, L - n + t - q0 + 1) : L, from = keys & ~(AW_BN - 1);
        const int own = hi > keys ? (hi - 1 - from) / w.chunk + 1 : 1;
        join_parts<D>(d, 0, chunks + own, [&](int i) { return i < chunks ? row_slot(s, t, hd, i) : row_slot(w, t, hd, i - chunks); },
                      t, hd);
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
#define PRE(D, NQ, F, W) attn_prefix_kernel<D, NQ, F, W><<<grid, dim3(256), 0, stream>>>(s, w, d, (uint32_t)shared_x, (uint32_t)wide_x, (uint32_t)shares)
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
    const unsigned blocks = (unsigned)((d.T * d.hq + 3) / 4);
    if (head_dim == 64)
        attn_prefix_join_kernel<64><<<blocks, 256, 0, stream>>>(s, w, d);
    else
        attn_prefix_join_kernel<128><<<blocks, 256, 0, stream>>>(s, w, d);
    return hipGetLastError();
}

}  // namespace mlora
