// Attention of few query rows over a paged cache (decode), and the join of split rows.
//
// The rows of one sequence and kv head (queries x heads of the group, up to 16 NQ) are the
// columns of 16x16x32 MFMA tiles, so K and V are read once for all of them.  The keys of all
// sequences and kv heads, in units of 128, are laid end to end and cut into equal shares, one a
// workgroup and as many as the card holds at a time: ragged batches end together, and few
// sequences still use every CU.  A sequence and head that crosses a cut leaves fp32 parts, which
// a second kernel joins.  A workgroup's four waves take steps of 32 keys in turn, each with its
// own running maximum, sums and accumulators, joined in LDS at the end of a piece.  K goes from
// memory straight into the fragments; V through a wave's own piece of LDS, written by rows and
// read transposed, so the loop has no barrier.  The next step's loads are issued while this
// one's softmax and second product run.  Bound by HBM (or, for a short batch, by latency).  Measured
// (D = 128, 32 heads on 8, with the join): 64 contexts of 1 to 8192 225 to 232 us (5.6 to 5.7 TB/s), 64 of
// 4096 184 to 187 us (5.8), 256 of an e4m3 cache 231 us (5.1), one of 1003 10.5 us (7 the shares, 4 the join).
// With a window and first keys (KEYS_SINKS): 64 contexts of 1 to 16384, window 2048, 105 us (5.0), 256 of an e4m3 cache, window
// 1024, 124 us (4.3: the 33 blocks of a sequence are 9 steps of four waves, the last for one of them); two steps' loads in flight
// were slower (130), three workgroups a CU too (199, 43 registers spilled).
// With two column tiles of D = 128 27 registers (e4m3: 15) are spilled, outside the loop over keys: 32 x 8 tokens
// over 4096 keys 137 us (3.9 TB/s), of an e4m3 cache 69 to 71 us (3.9).
#pragma once

#include <type_traits>

#include "attention.h"
#include "attention_device.h"

namespace mlora {

// A sequence: its queries and the units [first, first + units) of the keys [lo, L) that they see (at least one
// unit; none if this launch does not answer the sequence).  KEYS_SINKS: `sink` blocks of 32 first keys and those from lo
// on are numbered through, without the `first` blocks between them, and four in a row are a unit.
struct SeqUnits {
    int q0, n, L, lo, first, units, sink;
};

template <int KEYS> constexpr int unit_keys = KEYS == KEYS_OWN ? OWN_UNIT : DECODE_UNIT;

// (shared: KEYS_OWN, a function of b, n and L that gives the sequence's shared keys)
template <int KEYS, class Shared>
__device__ __forceinline__ SeqUnits seq_units(const AttnArgs &a, int b, Shared shared)
{
    constexpr int UNIT = unit_keys<KEYS>;
    SeqUnits s;
    s.q0 = (int)min((int64_t)max(a.cu_q[b], 0), a.T);
    s.n = (int)min((int64_t)max(a.cu_q[b + 1], 0), a.T) - s.q0;
    s.L = (int)min((int64_t)max(a.kv_len[b], 0), min(a.max_kv, a.table_stride << a.cache.ps));
    s.lo = KEYS == KEYS_OWN ? shared(b, s.n, s.L) : a.window > 0 ? max(0, s.L - s.n - a.window + 1) : 0;
    s.sink = KEYS == KEYS_SINKS ? min((a.sinks + 31) / 32, s.lo / 32) : 0;
    s.first = KEYS == KEYS_SINKS ? s.lo / 32 - s.sink : s.lo / UNIT;
    const int64_t rows = (int64_t)s.n * a.group;
    const bool mine = s.n > 0 && s.n <= a.max_q && rows >= a.min_rows && rows <= a.max_rows;
    const int units = KEYS == KEYS_SINKS ? ((s.L + 31) / 32 - s.first + UNIT / 32 - 1) / (UNIT / 32)
                                         : (s.L + UNIT - 1) / UNIT - s.first;
    s.units = mine ? max(1, units) : 0;
    return s;
}

template <int KEYS>
__device__ __forceinline__ SeqUnits seq_units(const AttnArgs &a, int b)
{
    return seq_units<KEYS>(a, b, [&](int b, int n, int L) { return shared_keys(a, b, n, L); });
}

// Units of the sequences per lane (`per` consecutive ones each): this lane's, those before it, and all (one head's);
// and the lane's last sequence.
struct LaneUnits {
    int per, mine, before, total;
    SeqUnits own;
};

template <int KEYS>
__device__ __forceinline__ LaneUnits lane_units(const AttnArgs &a, int lane)
{
    LaneUnits u{};
    u.per = (a.n_seqs + 63) / 64;
    for (int i = 0; i < u.per; ++i) {
        const int s = lane * u.per + i;
        if (s < a.n_seqs) {
            u.own = seq_units<KEYS>(a, s);
            u.mine += u.own.units;
        }
    }
    const int upto = wave_prefix(u.mine);
    u.before = upto - u.mine;
    u.total = __builtin_amdgcn_readlane(upto, 63);
    return u;
}

// `all` units (below 2^31) cut into n <= all shares, the first `more` of them one unit longer.
struct Shares {
    uint32_t n, each, more;
    __device__ __forceinline__ Shares(uint32_t all, uint32_t most) : n(min(all, most)), each(0), more(0)
    {
        if (n) {
            each = all / n;
            more = all - each * n;
        }
    }
    __device__ __forceinline__ uint32_t start(uint32_t w) const { return w * each + min(w, more); }
    __device__ __forceinline__ uint32_t of(uint32_t unit) const
    {
        const uint32_t longer = more * (each + 1);
        return unit < longer ? unit / (each + 1) : more + (unit - longer) / each;
    }
};

// The head at place h among those of sequence b.  The order of the heads turns with the sequence: shares of equal
// contexts that are whole heads long would else all read the same few heads of their pages at a time (e4m3, 256
// contexts of 2048: 256 us, turned 200; of 600: 79, turned 68; other batches: 0.5% slower at the median, 2.4% at most).
__device__ __forceinline__ int turned_head(const AttnArgs &a, int b, int h)
{
    const int t = h + (int)((unsigned)b % (unsigned)a.hkv);
    return t < a.hkv ? t : t - a.hkv;
}

// The (sequence, head's place) that holds unit `at`, and the unit's number in it.
struct UnitPlace {
    int b, h, f;
    SeqUnits sq;
};

template <int KEYS>
__device__ __forceinline__ UnitPlace find_unit(const AttnArgs &a, const LaneUnits &u, uint32_t at)
{
    UnitPlace p;
    const uint32_t first = (uint32_t)u.before * a.hkv;
    const uint64_t hit = ballot64(first <= at && at - first < (uint32_t)u.mine * a.hkv);
    const int src = __ffsll((unsigned long long)hit) - 1;
    uint32_t rest = at - (uint32_t)__builtin_amdgcn_readlane(u.before, src) * a.hkv;
    p.b = src * u.per;
    if (u.per == 1) {           // (no second trip to memory)
        p.sq.q0 = __builtin_amdgcn_readlane(u.own.q0, src);
        p.sq.n = __builtin_amdgcn_readlane(u.own.n, src);
        p.sq.L = __builtin_amdgcn_readlane(u.own.L, src);
        p.sq.lo = __builtin_amdgcn_readlane(u.own.lo, src);
        p.sq.first = __builtin_amdgcn_readlane(u.own.first, src);
        p.sq.units = __builtin_amdgcn_readlane(u.own.units, src);
        p.sq.sink = KEYS == KEYS_SINKS ? __builtin_amdgcn_readlane(u.own.sink, src) : 0;
    } else {
        p.sq = seq_units<KEYS>(a, p.b);
    }
    for (; rest >= (uint32_t)p.sq.units * a.hkv; p.sq = seq_units<KEYS>(a, ++p.b))
        rest -= (uint32_t)p.sq.units * a.hkv;
    p.h = (int)(rest / (uint32_t)p.sq.units);
    p.f = (int)rest - p.h * p.sq.units;
    return p;
}

// Slot of a part: a share leaves at most two, one of what began before it (which = true) and one of what goes on
// after it.
__device__ __forceinline__ int64_t part_slot(const AttnArgs &a, int share, bool which, int row)
{
    return (2 * (int64_t)share + (which ? 0 : 1)) * a.max_rows + row;
}

// Swizzle of the 16-byte pieces of a V row in LDS by its key: writes of one piece over 16 keys and transposing
// reads of 8 keys x 2 pieces both touch every bank once.
template <int D>
__device__ __forceinline__ int ad_swz(int key)
{
    return D == 128 ? (key & 7) << 1 | ((key >> 3) & 1) : ((key >> 1) & 3) << 1 | ((key >> 3) & 1);
}

// (KEYS_OWN: V and Q of each wave, and the first OWN_SEQS sequences; else V, the waves' parts and Q)
constexpr int OWN_SEQS = 256;
template <int D, int NQ, int KEYS = KEYS_PLAIN>
constexpr int decode_lds = KEYS == KEYS_OWN ? 4 * 2 * 32 * D + (NQ > 1 ? 4 * 16 * NQ * D * 2 : 0) + OWN_SEQS * 5 * 4
                                            : 4 * 2 * (32 * D > 32 * (D + 4) ? 32 * D : 32 * (D + 4)) + 4 * 16 * 2 * 4 +
                                                  (NQ > 1 ? 16 * NQ * D * 2 : 0);

// Share `share` of `shares` (or sequence and head `share`, see launch_attn_decode); smem: decode_lds bytes.
// KEYS_OWN: shares are not a workgroup's but a wave's (4 share + wave of 4 shares), and a wave leaves its parts to the join
// by itself: no barrier, so that the start of one wave's sequence, a chain of loads, hides behind the others' keys.  What
// comes after a shared prefix is short, and the waves of a workgroup waited for each start together (256 of an e4m3 cache
// behind four prefixes, 1 to 700 keys each: the kernel 97 us, with this and fewer chunks of the prefixes 77).
// PARTS: bf16 parts of a probability (see below).
template <int D, int NQ, bool FP8, int KEYS = KEYS_PLAIN, int PARTS = NQ == 1 || KEYS == KEYS_OWN ? 2 : 1>
__device__ __forceinline__ void attn_decode_body(const AttnArgs &a, uint32_t share, uint32_t shares, uint8_t *smem)
{
    constexpr int ESZ = FP8 ? 1 : 2;
    constexpr int KS = D / 32;          // k-steps of the first product
    constexpr int DB = D / 16;          // row blocks of the second
    constexpr int LD = FP8 ? D / 64 : D / 32;   // 16-byte loads per lane and 16-key block
    constexpr int OS = D + 4;           // row stride of the joined accumulators in LDS
    constexpr int VW = 32 * D;          // a wave's V rows in LDS
    constexpr bool OWN = KEYS == KEYS_OWN;
    constexpr int NW = 4, STEP = OWN ? 32 : 32 * NW;    // waves; keys they take at a time
    constexpr int UNIT = unit_keys<KEYS>;
    static_assert(STEP == UNIT, "units are whole steps");
    constexpr int PW = OWN || VW > 32 * OS ? VW : 32 * OS;      // a wave's V rows or, for the join, accumulators
    uint16_t *const lds = (uint16_t *)smem;
    float (*const ml)[16][2] = (float (*)[16][2])(smem + NW * PW * 2);
    const int wave = uniform(threadIdx.x >> 6), w32 = OWN ? 0 : 32 * wave;
    // two column tiles: Q
    uint16_t *const ql = (uint16_t *)(smem + NW * PW * 2 + (OWN ? wave * 16 * NQ * D * 2 : NW * 16 * 2 * 4));
    if (OWN)
        share = 4 * share + wave;

    const int lane = threadIdx.x & 63, col = lane & 15, g = lane >> 4;
    const int ps = a.cache.ps, pm = (1 << ps) - 1;
    uint16_t *vl = lds + wave * VW;

    // KEYS_OWN: up to OWN_SEQS sequences are listed in LDS, 64 a wave, from loads that do not wait for each other, instead of a
    // chain of them for each of a lane's sequences, whose group is searched for (256 of an e4m3 cache, four groups: a call 84 us,
    // listed 80)
    const bool listed = OWN && a.n_seqs <= OWN_SEQS && a.n_groups <= 64;
    u32x4 *const list = (u32x4 *)(smem + decode_lds<D, NQ, KEYS> - OWN_SEQS * 5 * 4);      // q0, n, L, lo
    int *const list_of = (int *)(list + OWN_SEQS);                                          // units
    if (listed) {
        Group mine = {0, 0, 0};
        if (lane < a.n_groups)
            mine = group_at(a, lane);
        const int s = 64 * wave + lane;
        if (64 * wave < a.n_seqs) {
            const SeqUnits q = seq_units<KEYS>(a, min(s, a.n_seqs - 1), [&](int b, int n, int L) {
                Group g = {0, 0, 0};
                for (int i = 0; i < a.n_groups; ++i) {
                    const Group x = {__builtin_amdgcn_readlane(mine.b0, i), __builtin_amdgcn_readlane(mine.b1, i),
                                     __builtin_amdgcn_readlane(mine.keys, i)};
                    if (b >= x.b0 && b < x.b1)
                        g = x;
                }
                return shared_keys(a, g, b, n, L);
            });
            list[s] = u32x4{(uint32_t)q.q0, (uint32_t)q.n, (uint32_t)q.L, (uint32_t)q.lo};
            list_of[s] = s < a.n_seqs ? q.units : 0;
        }
        __syncthreads();
    }
    auto list_at = [&](int b) {
        const u32x4 x = list[b];
        const int lo = uniform((int)x[3]);
        return SeqUnits{uniform((int)x[0]), uniform((int)x[1]), uniform((int)x[2]), lo, lo / UNIT, uniform(list_of[b]), 0};
    };
    auto list_units = [&] {         // (as lane_units)
        LaneUnits u{};
        u.per = (a.n_seqs + 63) / 64;
        for (int i = 0; i < u.per; ++i)
            u.mine += lane * u.per + i < a.n_seqs ? list_of[lane * u.per + i] : 0;
        const int upto = wave_prefix(u.mine);
        u.before = upto - u.mine;
        u.total = __builtin_amdgcn_readlane(upto, 63);
        return u;
    };
    auto list_find = [&](const LaneUnits &u, uint32_t at) {         // (as find_unit)
        UnitPlace p;
        const uint32_t first = (uint32_t)u.before * a.hkv;
        const int src = __ffsll((unsigned long long)ballot64(first <= at && at - first < (uint32_t)u.mine * a.hkv)) - 1;
        uint32_t rest = at - (uint32_t)__builtin_amdgcn_readlane(u.before, src) * a.hkv;
        p.b = src * u.per;
        p.sq = list_at(p.b);
        for (; rest >= (uint32_t)p.sq.units * a.hkv; p.sq = list_at(++p.b))
            rest -= (uint32_t)p.sq.units * a.hkv;
        p.h = (int)(rest / (uint32_t)p.sq.units);
        p.f = (int)rest - p.h * p.sq.units;
        return p;
    };

    // this workgroup's share: `left` units from unit f of (sequence b, head h) on
    UnitPlace from;
    int left;
    Shares cut(0, 0);
    uint32_t u0 = 0;            // the unit f's number among all
    if (!OWN && a.part_o == nullptr) {          // one workgroup a sequence and head
        from.b = (int)(share / a.hkv);
        from.h = (int)(share - (unsigned)from.b * a.hkv);
        from.f = 0;
        from.sq = seq_units<KEYS>(a, from.b);
        left = from.sq.units;
    } else {
        const LaneUnits u = listed ? list_units() : lane_units<KEYS>(a, lane);
        // (OWN: half of what a sequence and head has in the mean, up to four units, at the least, for each part is one more
        // for the join)
        const uint32_t all = (uint32_t)u.total * a.hkv;
        const uint32_t least = OWN ? min(max(all / (2 * (uint32_t)(a.n_seqs * a.hkv)), 1u), 4u) : 1;
        cut = Shares(all, OWN ? min(4 * shares, (all + least - 1) / least) : shares);
        if (share >= cut.n)
            return;
        u0 = cut.start(share);
        left = (int)(cut.start(share + 1) - u0);
        from = listed ? list_find(u, u0) : find_unit<KEYS>(a, u, u0);
    }
    int b = from.b, h = from.h, f = from.f;
    SeqUnits sq = from.sq;
    const float cs = a.scale * ATTN_LOG2E;
    const int last = (int)a.table_stride - 1;

    // KEYS_OWN: the pages of a sequence's first step, for its next head starts there again
    int pgf[2], seen = -1;
    while (left > 0) {
        const int end = min(sq.units, f + left);
        const int rows = sq.n * a.group, L = sq.L, head = turned_head(a, b, h);
        // keys [k0, k1) (KEYS_SINKS: of the numbered ones)
        const int skip = KEYS == KEYS_SINKS ? 32 * sq.first : 0, first = KEYS == KEYS_SINKS ? 0 : sq.first;
        const int k0 = max((first + f) * UNIT, KEYS == KEYS_SINKS ? 0 : sq.lo & ~31), k1 = min(L - skip, (first + end) * UNIT);
        // the step at k: its first key
        auto key_at = [&](int k) { return KEYS == KEYS_SINKS && k >= 32 * sq.sink ? k + skip : k; };
        const int32_t *__restrict__ table = a.table + (int64_t)b * a.table_stride;

        u32x4 kr[2][LD], vr[2][LD];
        f32x4 ks[2], vs[2];
        int pg[2];
        // pages of the two 16-key blocks of the step at kb (past the end: some page, whose keys are masked)
        auto lookup = [&](int kb) {
#pragma unroll
            for (int u = 0; u < 2; ++u)
                pg[u] = table[min((kb + 16 * u) >> ps, last)];
        };
        // (a scalar base and a constant offset a lane)
        const uint32_t off = col * D * ESZ + 16 * g;
        auto load = [&](int kb) {
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int page = clamp_page(uniform(pg[u]), a.cache.n_pages);
                const int64_t row = (((int64_t)page * a.cache.hkv + head) << ps) + ((kb + 16 * u) & pm);
                const uint8_t *kp = a.cache.k + row * D * ESZ, *vp = a.cache.v + row * D * ESZ;
#pragma unroll
                for (int s = 0; s < LD; ++s)
                    kr[u][s] = *(const u32x4 *)(kp + (off + 64 * s));
#pragma unroll
                for (int s = 0; s < LD; ++s)
                    vr[u][s] = *(const u32x4 *)(vp + (off + 64 * s));
                if (FP8) {
                    ks[u] = *(const f32x4 *)(a.cache.k_scale + row + 4 * g);
                    vs[u] = *(const f32x4 *)(a.cache.v_scale + row + 4 * g);
                }
            }
        };
        int at = k0 + w32, kb = key_at(at);     // this wave's step, and its first key
        if (OWN && b != seen && L > 0) {         // (a table may have no columns)
#pragma unroll
            for (int u = 0; u < 2; ++u)
                pgf[u] = table[min(((sq.lo & ~31) + 16 * u) >> ps, last)];
            seen = b;
        }
        if (at < k1) {
            if (OWN && f == 0) {
                pg[0] = pgf[0];
                pg[1] = pgf[1];
            } else {
                lookup(kb);
            }
            load(kb);
            if (at + STEP < k1)
                lookup(key_at(at + STEP));
        }

        // Q as B operand: column = row of the sequence, 8 values a k-step (e4m3 K comes 16 values a lane: two
        // k-steps side by side); its position.  Two column tiles leave no room for it in registers: it is read
        // from LDS each step.
        u32x4 qf[NQ == 1 ? KS : 1];
        int pos[NQ];
        auto qpiece = [&](int s) { return FP8 ? 8 * (s >> 1) + 2 * g + (s & 1) : 4 * s + g; };
#pragma unroll
        for (int j = 0; j < NQ; ++j) {
            const int r = min(16 * j + col, rows - 1), i = r / a.group, hd = head * a.group + r - i * a.group;
            pos[j] = L - sq.n + i;
            const uint16_t *qr = a.q + (sq.q0 + i) * a.q_stride + (int64_t)hd * D;
            if (NQ == 1) {
#pragma unroll
                for (int s = 0; s < KS; ++s)
                    qf[NQ == 1 ? s : 0] = *(const u32x4 *)(qr + 8 * qpiece(s));
            } else if (OWN || wave == j) {
#pragma unroll
                for (int s = 0; s < KS; ++s)
                    *(u32x4 *)(ql + (16 * j + col) * D + 8 * (qpiece(s) ^ (col & (D / 8 - 1)))) =
                        *(const u32x4 *)(qr + 8 * qpiece(s));
            }
        }
        if (NQ > 1 && !OWN)
            __syncthreads();
        const uint32_t qlane = col * D * 2 + 16 * (qpiece(0) ^ (col & (D / 8 - 1)));
        auto qfrag = [&](uint32_t at, int j, int s) {       // (piece s is piece 0 with bits of s changed)
            if (NQ == 1)
                return qf[NQ == 1 ? s : 0];
            return *(const u32x4 *)((const uint8_t *)ql + (at ^ (16 * (FP8 ? 8 * (s >> 1) + (s & 1) : 4 * s))) + 32 * j * D);
        };

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

        const uint32_t wlane = col * D * 2 + 16 * ((FP8 ? 2 * g : g) ^ ad_swz<D>(col));
        const int vk = 4 * g + (col >> 2);
        const uint32_t rlane = vk * D * 2 + 16 * (((col & 3) >> 1) ^ ad_swz<D>(vk)) + 8 * (col & 1);
        auto sees = [&](int key, int pos) {
            if (OWN)
                return key < L && (!a.causal || key <= pos) && key >= sq.lo;
            return key < L && (!a.causal || key <= pos) &&
                   (a.window <= 0 || key > pos - a.window || (KEYS == KEYS_SINKS && key < a.sinks));
        };
        auto step = [&](auto edge) {
            uint32_t qa = qlane;
            asm volatile("" : "+v"(qa));        // (keeps the compiler from holding Q and every address in registers)
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
                        st[j][u] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kf, as_bf16x8(qfrag(qa, j, s)), st[j][u], 0, 0, 0);
                }
#pragma unroll
                for (int j = 0; j < NQ; ++j)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        st[j][u][i] *= FP8 ? cs * ks[u][i] : cs;
            }
            // V rows into LDS ([key][D], pieces swizzled); rows outside [lo, L) as zeros
            uint32_t bad[2] = {0, 0}, wl = wlane;
            asm volatile("" : "+v"(wl));
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int key = 16 * u + col;
                const bool in = kb + key < L && (kb + key >= sq.lo || (KEYS == KEYS_SINKS && kb + key < a.sinks));
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
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                w[e][i] = in ? w[e][i] : 0u;
                                bad[u] = not_finite(bad[u], w[e][i]);
                            }
                        }
                        // piece 8 s + 2 g + e (e4m3) or 4 s + g
                        *(u32x4 *)((uint8_t *)vl + (wl ^ (FP8 ? 128 * s + 16 * e : 64 * s)) + 32 * u * D) = w[e];
                    }
                }
            }
            f32x4 vss[2];
            if (FP8) {
#pragma unroll
                for (int u = 0; u < 2; ++u)
                    vss[u] = vs[u];
            }
            // the next step's loads
            if (at + STEP < k1) {
                load(key_at(at + STEP));
                if (at + 2 * STEP < k1)
                    lookup(key_at(at + 2 * STEP));
            }
            u32x4 pf[PARTS][NQ];
#pragma unroll
            for (int j = 0; j < NQ; ++j) {
                if (edge)
#pragma unroll
                    for (int u = 0; u < 2; ++u)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int key = kb + 16 * u + 4 * g + i;
                            st[j][u][i] = sees(key, pos[j]) ? st[j][u][i] : -INFINITY;
                        }
                float mx = -INFINITY;
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        mx = fmaxf(mx, st[j][u][i]);
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
                // P^T for the matrix cores; the sum keeps fp32.  One column tile: as two bf16 parts, which memory leaves
                // the time for (48 batches: 0.6% slower at the median, long ones 2% at most), the first cut off below p (a step
                // of 2^-7), the rest rounded (2^-15 of p); both are positive where p is, so an infinite V stays that
                // infinity.  Two tiles: rounded to bf16 (half a step: 2^-8 relative), for two parts take registers and
                // products that are not there (32 x 8 tokens over 4096 keys 156 us, so 137; e4m3 75 and 70), but two parts
                // where a window is short (few_keys), over an e4m3 cache with sinks (key_parts), and behind a prefix, which
                // leaves a sequence few keys (own keys of up to 400, rms error of a result that is rounded alone 1: 1.25,
                // e4m3 1.4, two parts 1.0; 32 x 5 tokens, up to 600 own keys: 64 and 65 us, e4m3 72 and 74, D = 64 27 and
                // 27, up to 4000: 85 and 90, e4m3 67 and 73).
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (PARTS == 1) {
                        pf[0][j][i] = cvt_bf16x2(p[2 * i], p[2 * i + 1]);
                        continue;
                    }
                    uint32_t hi[2];
                    float lo[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        hi[e] = __builtin_elementwise_sub_sat(__float_as_uint(p[2 * i + e]), 1u) & 0xffff0000u;
                        lo[e] = p[2 * i + e] - __uint_as_float(hi[e]);
                    }
                    pf[0][j][i] = hi[0] >> 16 | hi[1];
                    pf[PARTS - 1][j][i] = cvt_bf16x2(lo[0], lo[1]);
                }
            }
            // O^T += V^T P^T; k index (g, e) is key 16 (e / 4) + 4 g + e % 4
            uint32_t rl = rlane;
            asm volatile("" : "+v"(rl));
            auto vfrag = [&](int d) {
                u32x4 f;
#pragma unroll
                for (int u = 0; u < 2; ++u) {       // keys 16 u + vk, values 16 d ..
                    const u32x2 w = lds_read_tr((const uint16_t *)((const uint8_t *)vl + (rl ^ (32 * d)) + 32 * u * D));
                    f[2 * u] = w[0];
                    f[2 * u + 1] = w[1];
                }
                return f;
            };
            if (edge && sq.n > 1) {
                // V may hold an infinity or NaN where some query must not see it (0 x NaN is NaN): such keys one at
                // a time, kept only by the queries that see them, and zeroed for the rest
                uint32_t some = 0;
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    uint64_t x = ballot64((bad[u] & 0x80008000u) != 0);
                    x |= x >> 32;
                    x |= x >> 16;
                    some |= (uint32_t)(x & 0xffff) << (16 * u);
                }
                for (; some; some &= some - 1) {
                    const int key = __ffs((int)some) - 1, e = 4 * (key >> 4) + (key & 3), ka = kb + key;
                    const uint32_t half = g != ((key & 15) >> 2) ? 0u : (e & 1) ? 0xffff0000u : 0xffffu;
#pragma unroll
                    for (int d = 0; d < DB; ++d) {
                        u32x4 f = vfrag(d);
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            f[i] &= i == (e >> 1) ? half : 0u;
#pragma unroll
                        for (int j = 0; j < NQ; ++j) {
                            f32x4 t = o[j][d];
#pragma unroll
                            for (int w = 0; w < PARTS; ++w)
                                t = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(f), as_bf16x8(pf[w][j]), t, 0, 0, 0);
                            const bool see = sees(ka, pos[j]);
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                o[j][d][i] = see ? t[i] : o[j][d][i];
                        }
                    }
                    if (lane < D / 8)
                        *(u32x4 *)(vl + key * D + 8 * lane) = u32x4{0, 0, 0, 0};
                }
            }
#pragma unroll
            for (int d = 0; d < DB; ++d) {
                const bf16x8 vf = as_bf16x8(vfrag(d));
#pragma unroll
                for (int w = 0; w < PARTS; ++w)
#pragma unroll
                    for (int j = 0; j < NQ; ++j)
                        o[j][d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vf, as_bf16x8(pf[w][j]), o[j][d], 0, 0, 0);
                if (d & 1)
                    __builtin_amdgcn_sched_barrier(0);      // (not all fragments at once: registers)
            }
        };
        // steps that hold a key which some query of the sequence does not see: below `free` and from `full` on
        const int full = L - sq.n + 1 - 32, free = OWN ? sq.lo : a.window > 0 ? L - a.window : 0;
        for (; at < k1 && kb < free; at += STEP, kb = key_at(at))
            step(std::true_type());
        for (; at < k1 && kb <= full; at += STEP, kb = key_at(at))
            step(std::false_type());
        for (; at < k1; at += STEP, kb = key_at(at))
            step(std::true_type());

        const bool whole = f == 0 && end == sq.units;
        if (OWN) {
#pragma unroll
            for (int j = 0; j < NQ; ++j) {
                float sum = l[j] + __shfl_xor(l[j], 16, 64);
                sum += __shfl_xor(sum, 32, 64);
                const int row = 16 * j + col;
                if (row >= rows)
                    continue;
                const int i = row / a.group, hd = head * a.group + row - i * a.group;
                if (whole && sq.lo == 0) {
                    const float inv = sum > 0.f ? 1.f / sum : sum == 0.f ? 0.f : sum;
                    uint16_t *dst = a.out + (sq.q0 + i) * a.out_stride + (int64_t)hd * D + 4 * g;
#pragma unroll
                    for (int d = 0; d < DB; ++d)
                        *(u32x2 *)(dst + 16 * d) = u32x2{cvt_bf16x2(o[j][d][0] * inv, o[j][d][1] * inv),
                                                         cvt_bf16x2(o[j][d][2] * inv, o[j][d][3] * inv)};
                    if (a.lse && g == 0)
                        a.lse[(int64_t)(sq.q0 + i) * a.hq + hd] =
                            sum == 0.f ? -INFINITY : (m[j] + __builtin_amdgcn_logf(sum)) * (1.f / ATTN_LOG2E);
                } else {
                    const int64_t slot = whole ? row_slot(a, sq.q0 + i, hd, 0) : part_slot(a, share, f > 0, row);
                    float *dst = a.part_o + slot * D + 4 * g;
#pragma unroll
                    for (int d = 0; d < DB; ++d)
                        *(f32x4 *)(dst + 16 * d) = o[j][d];
                    if (g == 0)
                        *(f32x2 *)(a.part_ml + 2 * slot) = f32x2{m[j], sum};
                }
            }
            if (f == 0 && lane == 0)
                *(u32x4 *)(a.cuts + 4 * ((int64_t)b * a.hkv + head)) =
                    u32x4{whole ? ~0u : share, (uint32_t)cut.of(u0 + sq.units - 1), (uint32_t)sq.lo, 0};
        }
        // join the waves, 16 rows at a time
        float *of = (float *)lds;
#pragma unroll
        for (int j = 0; j < (OWN ? 0 : NQ); ++j) {
            if (j > 0 && 16 * j >= rows)
                break;
            float lj = l[j] + __shfl_xor(l[j], 16, 64);
            lj += __shfl_xor(lj, 32, 64);
            __syncthreads();
            if (16 * j + col < rows) {
#pragma unroll
                for (int d = 0; d < DB; ++d)
                    *(f32x4 *)(of + (wave * 16 + col) * OS + 16 * d + 4 * g) = o[j][d];
                if (g == 0) {
                    ml[wave][col][0] = m[j];
                    ml[wave][col][1] = lj;
                }
            }
            __syncthreads();
            const int r = threadIdx.x >> 4, part = threadIdx.x & 15;
            const int row = 16 * j + r;
            if (r < 16 && row < rows) {
                float mx = ml[0][r][0];
#pragma unroll
                for (int w = 1; w < NW; ++w)
                    mx = fmaxf(mx, ml[w][r][0]);
                constexpr int VPT = D / 16;   // values a thread
                float sum = 0.f, acc[VPT];
#pragma unroll
                for (int e = 0; e < VPT; ++e)
                    acc[e] = 0.f;
#pragma unroll
                for (int w = 0; w < NW; ++w) {
                    const float f = __builtin_amdgcn_exp2f(ml[w][r][0] - mx);
                    sum += f * ml[w][r][1];
#pragma unroll
                    for (int e = 0; e < VPT; e += 4) {
                        const f32x4 x = *(const f32x4 *)(of + (w * 16 + r) * OS + part * VPT + e);
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            acc[e + i] += f * x[i];
                    }
                }
                const int i = row / a.group, hd = head * a.group + row - i * a.group;
                if (whole) {
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
                    const int64_t slot = part_slot(a, share, f > 0, row);
                    float *dst = a.part_o + slot * D + part * VPT;
#pragma unroll
                    for (int e = 0; e < VPT; e += 4)
                        *(f32x4 *)(dst + e) = f32x4{acc[e], acc[e + 1], acc[e + 2], acc[e + 3]};
                    if (part == 0)
                        *(f32x2 *)(a.part_ml + 2 * slot) = f32x2{mx, sum};
                }
            }
        }
        // the next head or sequence
        u0 += end - f;
        left -= end - f;
        if (left <= 0)
            break;
        f = 0;
        if (++h == a.hkv) {
            h = 0;
            do
                sq = listed ? list_at(++b) : seq_units<KEYS>(a, ++b);
            while (sq.units == 0);
        }
        if (!OWN)
            __syncthreads();
    }
}

}  // namespace mlora
