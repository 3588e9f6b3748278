// K6s: one decode step of attention for a batch that shares a prefix: the
// kernel (its instantiations: attn_shared_f16.cu, attn_shared_bf16.cu; plan and
// merge: attn_shared.cu).
//
// Sequence b's newest query q[b, h] attends to the prefix's P keys, stored
// once for the batch (k/v_prefix [Hk, P, d]), and to its own cache. Softmax
// parts over disjoint key sets merge by their (max, sum), so each part can run
// in the form that suits it. (The attention of nnterp "stablelm" 03 Notes;
// ALiBi as in "Bloom in a sovereign engine", Contribution, with the query at
// position P + lens[b] - 1.)
//
// The prefix is one product for the whole batch: for a kv head, the queries of
// all sequences and of the head's group are the rows of Q, and S = Q K^T,
// O = P V run on the tensor cores with each prefix byte read once instead of
// once per sequence. A unit is (kv head, 128 query rows = 128 / G sequences)
// of ceil(P / 128) key tiles.
//
// The own caches: a sequence's query heads of one kv head are few (G = 1 ..
// 8), its keys many, so the pass is bound by the bytes of K and V. On the CUDA
// cores each key costs 4 d G flops and as many shared-memory reads and
// shuffles, which a G of 4 or 8 does not hide behind the bytes (measured: 2.0
// TB/s at 32/8 heads x 128, 2.9 TB/s at 32 x 64). So the products run on the
// tensor cores with the roles turned: keys are the rows, heads the (padded) 16
// columns,
//     S^T [128 keys, 16] = K Q^T,    O^T [d, 16] = V^T P^T,
// with K and V straight from the TMA tiles, one softmax thread per key, and
// the per-head maximum a warp reduction. An MMA's unused columns are whatever
// shared memory holds: columns do not mix, and none of them is read. A unit is
// (sequence, kv head) of ceil(len / 128) key tiles. The lengths are device
// data: each CTA sums them itself to find its range, and one leaves the
// running tile counts for the merge. A last, part-filled tile is loaded in
// boxes of 16 keys, multiplied over ceil(keys / 16) steps, and the values
// behind its end are cleared: 0 times what an unused cache entry holds need
// not be 0.
//
// Work: the tiles of all units of a part, in one line, are cut into equal
// ranges, one per CTA; a CTA's stay in a unit is a segment with a partial
// result (max, sum, O) of its own. There are two CTAs per SM, so that one's
// chain of scores, softmax and product fills the other's gaps; each does its
// prefix range and then its own caches' range, whose loads begin as the
// prefix's last tiles are consumed (32 sequences of 32 x 64 heads, 8192 shared
// and 279 own keys: in launches of their own 37.9 us, in one 34.9, 32.4 with the
// ranges found beside the first loads; with one CTA of an SM on the prefix and
// the other on the own caches the softmax of the prefix took three times as
// long, and the whole half as long again).
// Tiles go from the newest key down (with ALiBi the bias is largest there, so
// the rescale of O stays rare).
// Measured and bound: the bytes where rows are few (16 sequences of 16 x 128 heads,
// 32771 shared keys: 67.2 us, 6.3 TB/s, 0.93 of the copy rate); else the tensor cores'
// chain of scores, softmax and product per tile, and both parts' fixed ends: 64
// sequences of 32/8 x 128 heads, 16384 shared keys, 44.8 us for 27.6 of bytes and
// 9.4 of products. Tiles of 64 keys with two S buffers at head_dim 128, so that the
// next scores come beside the softmax: 45.9; the SM's other CTA fills that gap.
// 6 warps: TMA; MMA issue; four of softmax.
#pragma once

#include "internal.h"

namespace blk {

namespace {

constexpr int kThreads = 192;
constexpr int kTQ = 128, kTK = 128;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kRescaleThreshold = 8.0f;  // log2 of the largest unnormalised p

template <int D>
struct Cfg {
    static constexpr int kSub = D / 64;
    static constexpr int kTile = kSub * 128 * 128;      // Q, K or V tile
    static constexpr int kPool = D == 64 ? 6 : 3;       // tiles of shared memory: 96 KB
    static constexpr int kSlotsP = kPool - 1;           // prefix: Q, then a ring
    static constexpr int kSlots = kPool;                // own caches: a ring
    // own caches' queries and weights: 8 rows of 128 bytes per 64 columns; the
    // operands' rows 8 .. 15 are what follows (any bytes will do)
    static constexpr int kQBytes = kSub * 1024, kPBytes = 2 * 1024;
    static constexpr int kOffQ = kPool * kTile;
    static constexpr int kOffP = kOffQ + 2 * kQBytes;
    static constexpr int kOffMax = kOffP + 2 * kPBytes + 1024;  // [2][8][4] floats
    static constexpr int kOffSum = kOffMax + 2 * 8 * 4 * 4;     // [2][8][4] floats
    static constexpr int kOffBar = kOffSum + 2 * 8 * 4 * 4;     // prefix, then own caches
    static constexpr int kSmem = kOffBar + 512 + 1024;          // + alignment slack
    static_assert(kSmem <= 112 * 1024, "two CTAs per SM");
    // TMEM, prefix: S [0, 128); head_dim 64: P [128, 192), O [192, 256);
    // head_dim 128: P over S (so the next S waits for the PV that reads P), O
    // [128, 256). Own caches: S^T [0, 32), O^T [32, 64), each twice (by tile, by
    // segment).
    static constexpr bool kPOverS = D != 64;
    static constexpr uint32_t kColP = kPOverS ? 0 : 128, kColO = 256 - D;
};

// tcgen05.ld of N consecutive columns of this thread's lane, waited.
template <int N>
__device__ __forceinline__ void tmem_ldn(uint32_t taddr, uint32_t (&r)[N]) {
    if constexpr (N == 1)
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];\n\t"
                     "tcgen05.wait::ld.sync.aligned;" : "=r"(r[0]) : "r"(taddr) : "memory");
    else if constexpr (N == 2)
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x2.b32 {%0, %1}, [%2];\n\t"
                     "tcgen05.wait::ld.sync.aligned;"
                     : "=r"(r[0]), "=r"(r[1]) : "r"(taddr) : "memory");
    else if constexpr (N == 4)
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];\n\t"
                     "tcgen05.wait::ld.sync.aligned;"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(taddr) : "memory");
    else
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n\t"
                     "tcgen05.wait::ld.sync.aligned;"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
                       "=r"(r[6]), "=r"(r[7]) : "r"(taddr) : "memory");
}
template <int N>
__device__ __forceinline__ void tmem_stn(uint32_t taddr, const uint32_t (&r)[N]) {
    if constexpr (N == 1)
        asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" ::"r"(taddr), "r"(r[0])
                     : "memory");
    else if constexpr (N == 2)
        asm volatile("tcgen05.st.sync.aligned.32x32b.x2.b32 [%0], {%1, %2};" ::"r"(taddr), "r"(r[0]),
                     "r"(r[1]) : "memory");
    else if constexpr (N == 4)
        asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};" ::"r"(taddr),
                     "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]) : "memory");
    else
        asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
                     ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]),
                     "r"(r[6]), "r"(r[7]) : "memory");
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// max over the warp's lanes: floats as integers of the same order
__device__ __forceinline__ float warp_max(float v) {
    int i = __float_as_int(v);
    i = i < 0 ? i ^ 0x7fffffff : i;
    i = __reduce_max_sync(0xffffffffu, i);
    return __int_as_float(i < 0 ? i ^ 0x7fffffff : i);
}

// 32 bytes to global memory in one store (32-byte aligned).
__device__ __forceinline__ void store_sector(float* p, const float (&f)[8]) {
    asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(f[0]),
                 "f"(f[1]), "f"(f[2]), "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7])
                 : "memory");
}

__device__ __forceinline__ float alibi_slope(const SharedKernelArgs& a, int h) {
    return a.slopes ? a.slopes[h]
                    : exp2f(-8.0f * static_cast<float>(h + 1) / static_cast<float>(a.H));
}

// Descriptor of `off` (in 16 bytes) behind the one of d: the address is the
// low word's field and does not carry out of it, so that 32 bits are enough. A
// form of this kernel that added 64-bit offsets in unrolled loops gave wrong O =
// P V at head_dim 64 (as if of keys 0, 16, 32, ... only) and right ones with the
// loop not unrolled, or with this function. The cause is not known: the two
// additions are equal for these addresses, and attn_pair.cu does the other one.
__device__ __forceinline__ uint64_t desc_at(uint64_t d, uint32_t off) {
    uint32_t lo, hi;
    asm("mov.b64 {%0, %1}, %2;" : "=r"(lo), "=r"(hi) : "l"(d));
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(lo + off), "r"(hi));
    return r;
}

// mbarriers of the prefix part ...
template <int SLOTS>
struct PrefixBars {
    uint32_t at;
    static constexpr int kBytes = 64 + 16 * SLOTS;
    __device__ __forceinline__ uint32_t q_full() const { return at; }
    __device__ __forceinline__ uint32_t q_empty() const { return at + 8u; }
    __device__ __forceinline__ uint32_t s_full() const { return at + 16u; }
    __device__ __forceinline__ uint32_t s_free() const { return at + 24u; }
    __device__ __forceinline__ uint32_t p_full() const { return at + 32u; }
    __device__ __forceinline__ uint32_t pv_done() const { return at + 40u; }
    __device__ __forceinline__ uint32_t o_free() const { return at + 48u; }
    __device__ __forceinline__ uint32_t drain() const { return at + 56u; }
    __device__ __forceinline__ uint32_t full(int i) const { return at + 64u + 8u * i; }
    __device__ __forceinline__ uint32_t empty(int i) const { return at + 64u + 8u * (SLOTS + i); }
    __device__ __forceinline__ void init() const {
        mbar_init(q_full(), 1);
        mbar_init(q_empty(), 1);
        mbar_init(s_full(), 1);
        mbar_init(s_free(), 4);
        mbar_init(p_full(), 4);
        mbar_init(pv_done(), 1);
        mbar_init(o_free(), 4);
        mbar_init(drain(), 1);
        for (int i = 0; i < SLOTS; ++i) {
            mbar_init(full(i), 1);
            mbar_init(empty(i), 1);
        }
    }
};
// ... and of the own caches' part (pairs: by tile or by segment)
template <int SLOTS>
struct OwnBars {
    uint32_t at;
    static constexpr int kBytes = 144 + 16 * SLOTS;
    __device__ __forceinline__ uint32_t q_full(int i) const { return at + 8u * i; }
    __device__ __forceinline__ uint32_t q_empty(int i) const { return at + 16u + 8u * i; }
    __device__ __forceinline__ uint32_t s_full(int i) const { return at + 32u + 8u * i; }
    __device__ __forceinline__ uint32_t s_free(int i) const { return at + 48u + 8u * i; }
    __device__ __forceinline__ uint32_t p_full(int i) const { return at + 64u + 8u * i; }
    __device__ __forceinline__ uint32_t pv_done(int i) const { return at + 80u + 8u * i; }
    __device__ __forceinline__ uint32_t o_free(int i) const { return at + 96u + 8u * i; }
    __device__ __forceinline__ uint32_t max_full() const { return at + 112u; }
    __device__ __forceinline__ uint32_t sum_full() const { return at + 120u; }
    __device__ __forceinline__ uint32_t drain() const { return at + 128u; }
    __device__ __forceinline__ uint32_t range_full() const { return at + 136u; }
    __device__ __forceinline__ uint32_t full(int i) const { return at + 144u + 8u * i; }
    __device__ __forceinline__ uint32_t empty(int i) const { return at + 144u + 8u * (SLOTS + i); }
    __device__ __forceinline__ void init() const {
        for (int i = 0; i < 2; ++i) {
            mbar_init(q_full(i), 1);
            mbar_init(q_empty(i), 1);
            mbar_init(s_full(i), 1);
            mbar_init(s_free(i), 4);
            mbar_init(p_full(i), 4);
            mbar_init(pv_done(i), 1);
            mbar_init(o_free(i), 4);
        }
        mbar_init(max_full(), 4);
        mbar_init(sum_full(), 4);
        mbar_init(drain(), 1);
        mbar_init(range_full(), 4);
        for (int i = 0; i < SLOTS; ++i) {
            mbar_init(full(i), 1);
            mbar_init(empty(i), 1);
        }
    }
};

// -------------------------------------------------------------- prefix ----
// A CTA's segments: tiles [t, t + n) of unit u, key tiles from klo.
struct PrefixSegments {
    int t, end, u, n, klo, it;
    bool valid;
    __device__ __forceinline__ void set(const SharedKernelArgs& a) {
        valid = t < end;
        if (!valid) return;
        u = t / a.nkt;
        klo = t - u * a.nkt;
        n = min(end - t, a.nkt - klo);
    }
    __device__ __forceinline__ void start(const SharedKernelArgs& a) {
        const int64_t c = blockIdx.x;
        t = c < a.prefix_ctas ? static_cast<int>(c * a.W / a.prefix_ctas) : 0;
        end = c < a.prefix_ctas ? static_cast<int>((c + 1) * a.W / a.prefix_ctas) : 0;
        it = 0;
        set(a);
    }
    __device__ __forceinline__ void next(const SharedKernelArgs& a) {
        t += n;
        ++it;
        set(a);
    }
};

// Returns false if a wait gave up.
template <typename T, int D>
__device__ __forceinline__ bool prefix_phase(const SharedKernelArgs& a, const CUtensorMap& tmQ,
                                             const CUtensorMap& tmK, const CUtensorMap& tmV,
                                             uint32_t pool, uint32_t bar0, uint32_t tmem, int warp,
                                             int lane) {
    using C = Cfg<D>;
    constexpr int kSlots = C::kSlotsP;
    const uint32_t sQ = pool, sRing = pool + C::kTile;
    const PrefixBars<kSlots> bar{bar0};
    PrefixSegments c;
    c.start(a);
    bool ok = true;
    if (warp == 0) {
        if (lane == 0) {
            // read again by the kv head's other row tiles, if it has any
            const uint64_t pol = a.nrt > 1 ? l2_evict_last_policy() : l2_evict_first_policy();
            int r = 0, nq = 0;  // tiles and query tiles on their way so far
            while (ok && c.valid) {
                const int g = c.u / a.nrt, rt = c.u - g * a.nrt;
                if (!(ok = mbar_wait(bar.q_empty(), (c.it & 1) ^ 1u, a.err))) break;
                mbar_expect_tx(bar.q_full(), C::kTile);
                ++nq;
#pragma unroll
                for (int sub = 0; sub < C::kSub; ++sub)
                    tma_load_4d(sQ + sub * kTQ * 128, &tmQ, bar.q_full(), sub * 64, 0, g,
                                rt * (kTQ / a.G));
                for (int i = 0; i < 2 * c.n; ++i, ++r) {  // K, V, K, V, ...
                    const int sl = r % kSlots;
                    if (!(ok = mbar_wait(bar.empty(sl), ((r / kSlots) & 1) ^ 1u, a.err))) break;
                    mbar_expect_tx(bar.full(sl), C::kTile);
                    const int row = (c.klo + c.n - 1 - i / 2) * kTK;
#pragma unroll
                    for (int sub = 0; sub < C::kSub; ++sub)
                        tma_load_3d_hint(sRing + sl * C::kTile + sub * kTK * 128,
                                         i & 1 ? &tmV : &tmK, bar.full(sl), sub * 64, row, g, pol);
                }
                c.next(a);
            }
            // the tiles are the own caches' next: all of them consumed
            for (int i = r > kSlots ? r - kSlots : 0; i < r && ok; ++i)
                ok = mbar_wait(bar.empty(i % kSlots), (i / kSlots) & 1, a.err);
            if (ok && c.it > 0) ok = mbar_wait(bar.q_empty(), (c.it - 1) & 1, a.err);
            if (!ok) {  // gave up: no copy may land behind this block's end
                for (int i = r > kSlots ? r - kSlots : 0; i < r; ++i)
                    mbar_wait(bar.full(i % kSlots), (i / kSlots) & 1, a.err);
                if (nq > 0) mbar_wait(bar.q_full(), (nq - 1) & 1, a.err);
            }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            constexpr uint32_t fmt = dt_traits<T>::mma_fmt;
            constexpr uint32_t idesc_s = make_idesc_f16(fmt, kTQ, kTK, false);
            constexpr uint32_t idesc_o = make_idesc_f16(fmt, kTQ, D, true);
            constexpr uint64_t kAtom = (kTQ * 128) >> 4;
            constexpr uint64_t kSlotStep = C::kTile >> 4;
            const uint64_t dq = make_sdesc_sw128(sQ, 16, 1024);
            const uint64_t dk0 = make_sdesc_sw128(sRing, 16, 1024);
            const uint64_t dv0 = make_sdesc_sw128(sRing, kTK * 128, 1024);
            const uint32_t tS = tmem, tP = tmem + C::kColP, tO = tmem + C::kColO;
            // S = Q K^T of tile t, once the softmax has read the previous S (P
            // over S: the previous PV has read P)
            auto issue_s = [&](int t) -> bool {
                const int r = 2 * t, sl = r % kSlots;
                if (!mbar_wait(bar.full(sl), (r / kSlots) & 1, a.err)) return false;
                if (t > 0 && !mbar_wait(C::kPOverS ? bar.pv_done() : bar.s_free(), (t - 1) & 1, a.err))
                    return false;
                tc_fence_after();
                const uint64_t dk = dk0 + sl * kSlotStep;
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks) {
                    const uint32_t off = static_cast<uint32_t>((ks / 4) * kAtom) + (ks % 4) * 2;
                    tc_mma_ss(tS, desc_at(dq, off), desc_at(dk, off), idesc_s, ks > 0 ? 1u : 0u);
                }
                tc_commit(bar.s_full());
                tc_commit(bar.empty(sl));
                return true;
            };
            auto issue_pv = [&](int t, bool first, int it) -> bool {
                const int r = 2 * t + 1, sl = r % kSlots;
                if (!mbar_wait(bar.full(sl), (r / kSlots) & 1, a.err) ||
                    !mbar_wait(bar.p_full(), t & 1, a.err) ||
                    (first && it > 0 && !mbar_wait(bar.o_free(), (it - 1) & 1, a.err)))
                    return false;
                tc_fence_after();
                const uint64_t dv = dv0 + sl * kSlotStep;
#pragma unroll
                for (int ks = 0; ks < kTK / 16; ++ks)
                    tc_mma_ts(tO, tP + ks * 8, desc_at(dv, ks * ((16 * 128) >> 4)), idesc_o,
                              (!first || ks > 0) ? 1u : 0u);
                tc_commit(bar.pv_done());
                tc_commit(bar.empty(sl));
                return true;
            };
            int t = 0;  // tiles so far
            while (ok && c.valid) {
                if (!(ok = mbar_wait(bar.q_full(), c.it & 1, a.err))) break;
                if (!C::kPOverS) ok = issue_s(t);
                for (int i = 0; i < c.n && ok; ++i, ++t) {
                    // head_dim 64: S of the next tile ahead of PV of this one
                    if (C::kPOverS) ok = issue_s(t);
                    else if (i + 1 < c.n) ok = issue_s(t + 1);
                    if (ok && i + (C::kPOverS ? 1 : 2) == c.n) tc_commit(bar.q_empty());
                    if (ok && !C::kPOverS && c.n == 1) tc_commit(bar.q_empty());
                    ok = ok && issue_pv(t, i == 0, c.it);
                }
                c.next(a);
            }
            // ... and the columns of S and P
            if (ok && t > 0) ok = mbar_wait(bar.pv_done(), (t - 1) & 1, a.err);
            tc_fence_after();
            if (!ok) {  // gave up: nor any product
                tc_commit(bar.drain());
                mbar_wait(bar.drain(), 0, a.err);
            }
        }
    } else {
        const int quarter = warp & 3;
        const int row = quarter * 32 + lane;
        const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
        const uint32_t tS = tmem + lane_off, tP = tmem + C::kColP + lane_off;
        const uint32_t tO = tmem + C::kColO + lane_off;
        const float scale_l2 = a.scale * kLog2e;
        const float mul = a.alibi ? 1.f : scale_l2;  // what is left to multiply a score by
        int t = 0;
        while (ok && c.valid) {
            const int kvh = c.u / a.nrt, rt = c.u - kvh * a.nrt;
            // a warp all of whose rows lie behind the batch only keeps the
            // barriers going: its P and O are whatever they are, and unread
            const bool live = rt * (kTQ / a.G) + quarter * 32 / a.G < a.B;
            float m_used = -INFINITY;  // running max, log2 domain
            float l = 0.f;
            const float slope_l2 = a.alibi ? kLog2e * alibi_slope(a, kvh * a.G + row % a.G) : 0.f;
            for (int i = 0; i < c.n; ++i, ++t) {
                if (!(ok = mbar_wait(bar.s_full(), t & 1, a.err))) break;
                tc_fence_after();
                if (!live) {
                    if (i > 0 && !(ok = mbar_wait(bar.pv_done(), (t - 1) & 1, a.err))) break;
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        if (!C::kPOverS) mbar_arrive(bar.s_free());
                        mbar_arrive(bar.p_full());
                    }
                    continue;
                }
                uint32_t r[kTK];
                tmem_ld128(tS, r);
                if (!C::kPOverS) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar.s_free());
                }
                const int kbase = (c.klo + c.n - 1 - i) * kTK;
                if (a.alibi) {
                    // + slope * (key - P), the distance to the query's own part
                    // of the row's bias being left to the merge
                    const float sk = slope_l2 * static_cast<float>(kbase - a.P);
                    const uint64_t sc2 = f2_pack(scale_l2, scale_l2);
                    const uint64_t sl2 = f2_pack(slope_l2, slope_l2), sk2 = f2_pack(sk, sk);
#pragma unroll
                    for (int k = 0; k < kTK; k += 2) {
                        float b0, b1, u0, u1;
                        ffma2(static_cast<float>(k), static_cast<float>(k + 1), sl2, sk2, b0, b1);
                        ffma2(__uint_as_float(r[k]), __uint_as_float(r[k + 1]), sc2,
                              f2_pack(b0, b1), u0, u1);
                        r[k] = __float_as_uint(u0);
                        r[k + 1] = __float_as_uint(u1);
                    }
                }
                if (kbase + kTK > a.P) {
                    const int lim = a.P - 1 - kbase;  // keys <= lim exist
#pragma unroll
                    for (int k = 0; k < kTK; ++k)
                        if (k > lim) r[k] = __float_as_uint(-INFINITY);
                }
                float m0 = -INFINITY, m1 = -INFINITY, m2 = -INFINITY, m3 = -INFINITY;
#pragma unroll
                for (int k = 0; k < kTK; k += 8) {
                    m0 = fmax3f(m0, __uint_as_float(r[k]), __uint_as_float(r[k + 1]));
                    m1 = fmax3f(m1, __uint_as_float(r[k + 2]), __uint_as_float(r[k + 3]));
                    m2 = fmax3f(m2, __uint_as_float(r[k + 4]), __uint_as_float(r[k + 5]));
                    m3 = fmax3f(m3, __uint_as_float(r[k + 6]), __uint_as_float(r[k + 7]));
                }
                const float mx = fmaxf(fmaxf(m0, m1), fmaxf(m2, m3)) * mul;  // mul > 0
                float corr = 1.f;
                if (mx > m_used + kRescaleThreshold) {
                    corr = ex2_approx(m_used - mx);
                    m_used = mx;
                }
                // weights in the storage type for the product (half a step each,
                // see attn_pair.cu), in 32 bits for the sum
                const uint64_t mul2 = f2_pack(mul, mul), neg2 = f2_pack(-m_used, -m_used);
                uint64_t acc0 = f2_pack(0.f, 0.f), acc1 = acc0;
                // P over S: nothing but this row's own scores is there, and they
                // are in registers; else the previous PV has to have read P
                if (i > 0 && !(ok = mbar_wait(bar.pv_done(), (t - 1) & 1, a.err))) break;
                tc_fence_after();
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    uint32_t pk[16];
#pragma unroll
                    for (int e = 0; e < 16; e += 2) {
                        const int k = q * 32 + 2 * e;
                        float e0, e1, e2, e3;
                        ffma2(__uint_as_float(r[k]), __uint_as_float(r[k + 1]), mul2, neg2, e0, e1);
                        ffma2(__uint_as_float(r[k + 2]), __uint_as_float(r[k + 3]), mul2, neg2, e2, e3);
                        const float p0 = ex2_approx(e0), p1 = ex2_approx(e1);
                        const float p2 = ex2_approx(e2), p3 = ex2_approx(e3);
                        fadd2_acc(acc0, p0, p1);
                        fadd2_acc(acc1, p2, p3);
                        pk[e] = dt_traits<T>::pack2(p0, p1);
                        pk[e + 1] = dt_traits<T>::pack2(p2, p3);
                    }
                    tmem_st16_nowait(tP + q * 16, pk);
                }
                if (i > 0 && __any_sync(0xffffffffu, corr != 1.f)) {
#pragma unroll 1
                    for (int cc = 0; cc < D / 16; ++cc) {
                        uint32_t o[16];
                        tmem_ld16(tO + cc * 16, o);
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            o[e] = __float_as_uint(__uint_as_float(o[e]) * corr);
                        tmem_st16_nowait(tO + cc * 16, o);
                    }
                }
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar.p_full());
                float s0, s1, s2, s3;
                f2_unpack(acc0, s0, s1);
                f2_unpack(acc1, s2, s3);
                l = l * corr + ((s0 + s1) + (s2 + s3));
            }
            if (!ok || !(ok = mbar_wait(bar.pv_done(), (t - 1) & 1, a.err))) break;
            tc_fence_after();
            // the segment's result
            const bool mine = rt * (kTQ / a.G) + row / a.G < a.B;
            const int64_t rec = (static_cast<int64_t>(blockIdx.x) + c.u) * kTQ;
            if (mine) a.pm[rec + row] = make_float2(m_used, l);
            float* dst = a.po + rec * D + row * 8;
#pragma unroll 1
            for (int cc = 0; cc < D / 32 && live; ++cc) {
                uint32_t o[32];
                tmem_ld32(tO + cc * 32, o);
                if (mine) {
#pragma unroll
                    for (int v = 0; v < 4; ++v) {
                        float f[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e) f[e] = __uint_as_float(o[v * 8 + e]);
                        store_sector(dst + (cc * 4 + v) * kTQ * 8, f);
                    }
                }
                __syncwarp();  // TMEM loads are whole-warp instructions
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar.o_free());
            c.next(a);
        }
    }
    return ok;
}

// ---------------------------------------------------------- own caches ----
// Ranges are dealt from the last CTA down: where there are fewer tiles than
// CTAs, others than the prefix's get them.
__device__ __forceinline__ int own_index() {
    return static_cast<int>(gridDim.x - 1 - blockIdx.x);
}
__device__ __forceinline__ int own_len(const SharedKernelArgs& a, int b) {
    return min(max(a.lens[b], 0), a.S_max);
}

// A CTA's segments: tiles [t, t + n) of unit (b, g), key tiles first ..
// first + n - 1 of the unit; t counts all units' tiles.
struct OwnSegments {
    int64_t t, end;
    int b, g, first, n, len, it;
    bool valid;
    __device__ __forceinline__ void set(const SharedKernelArgs& a) {
        valid = t < end;
        if (!valid) return;
        const int left = (len + kTK - 1) / kTK - first;
        n = static_cast<int>(min(static_cast<int64_t>(left), end - t));
    }
    // base: tiles ahead of sequence b0's first unit; the range starts in b0
    __device__ __forceinline__ void start(const SharedKernelArgs& a, int64_t lo, int64_t hi, int b0,
                                          int64_t base) {
        t = lo;
        end = hi;
        it = 0;
        b = b0;
        valid = t < end;
        if (!valid) return;
        len = own_len(a, b);
        const int nt = (len + kTK - 1) / kTK;
        g = static_cast<int>((t - base) / nt);
        first = static_cast<int>((t - base) % nt);
        set(a);
    }
    __device__ __forceinline__ void next(const SharedKernelArgs& a) {
        t += n;
        ++it;
        first = 0;
        if (t < end && ++g == a.Hk) {
            g = 0;
            do {
                len = own_len(a, ++b);
            } while (len == 0);
        }
        set(a);
    }
};


// This CTA's range of the own caches' tiles, by the four softmax warps: tiles
// [lo, hi), the first in sequence b0, `base` tiles ahead of that sequence.
struct OwnRange {
    int64_t lo, hi, base;
    int b0;
    int sum[4];
};
__device__ __forceinline__ void find_own_range(const SharedKernelArgs& a, OwnRange& out,
                                               uint32_t range_full) {
    const int t = static_cast<int>(threadIdx.x) - 64, lane = t & 31, w = t / 32;
    // thread t sums the tiles of a run of sequences
    const int per = (a.B + 127) / 128;
    const int b_lo = min(t * per, a.B), b_hi = min(b_lo + per, a.B);
    int mine = 0;
    for (int b = b_lo; b < b_hi; ++b) mine += (own_len(a, b) + kTK - 1) / kTK;
    int upto = mine;  // inclusive sum over the warp's threads, then over all
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += v;
    }
    if (lane == 31) out.sum[w] = upto;
    // (all four warps come here before any wait that can give up)
    asm volatile("bar.sync 1, 128;" ::: "memory");
    int before = upto - mine, total = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (i < w) before += out.sum[i];
        total += out.sum[i];
    }
    // with fewer tiles than CTAs, one for each of the first W (the merge counts
    // on every CTA of a unit's span having some of it)
    const int64_t W = static_cast<int64_t>(total) * a.Hk;
    const int64_t ctas = min(static_cast<int64_t>(gridDim.x), W), me = own_index();
    const int64_t lo = me < ctas ? me * W / ctas : 0, hi = me < ctas ? (me + 1) * W / ctas : 0;
    if (t == 0) {
        out.lo = lo;
        out.hi = hi;
    }
    // the thread whose run holds the first tile finds its sequence
    if (lo < hi && static_cast<int64_t>(before) * a.Hk <= lo &&
        lo < static_cast<int64_t>(before + mine) * a.Hk) {
        int64_t base = static_cast<int64_t>(before) * a.Hk;
        int b = b_lo;
        for (;; ++b) {
            const int nt = (own_len(a, b) + kTK - 1) / kTK;
            if (lo < base + static_cast<int64_t>(nt) * a.Hk) break;
            base += static_cast<int64_t>(nt) * a.Hk;
        }
        out.b0 = b;
        out.base = base;
    }
    if (me == 0) {
        int c = before;
        for (int b = b_lo; b < b_hi; ++b) {
            a.cum[b] = c;
            c += (own_len(a, b) + kTK - 1) / kTK;
        }
        if (t == 0) a.cum[a.B] = total;
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(range_full);
}

template <typename T, int D, int G>
__device__ __forceinline__ void own_phase(const SharedKernelArgs& a, const CUtensorMap& tmQ,
                                          const CUtensorMap& tmK, const CUtensorMap& tmV,
                                          const CUtensorMap& tmK16, const CUtensorMap& tmV16,
                                          OwnSegments c, uint8_t* smem, uint32_t bar0, uint32_t tmem,
                                          int warp, int lane) {
    using C = Cfg<D>;
    constexpr int kSlots = C::kSlots;
    const uint32_t sKV = smem_u32(smem);
    const uint32_t sQ = sKV + C::kOffQ, sP = sKV + C::kOffP;
    const OwnBars<kSlots> bar{bar0};
    bool ok = true;
    if (warp == 0) {
        if (lane == 0) {
            const uint64_t pol = l2_evict_first_policy();
            int r = 0, nq = 0;  // tiles and query boxes on their way so far
            while (ok && c.valid) {
                const int qb = c.it & 1;
                if (!(ok = mbar_wait(bar.q_empty(qb), ((c.it >> 1) & 1) ^ 1u, a.err))) break;
                mbar_expect_tx(bar.q_full(qb), G * 128 * C::kSub);
                ++nq;
#pragma unroll
                for (int sub = 0; sub < C::kSub; ++sub)
                    tma_load_2d(sQ + qb * C::kQBytes + sub * 1024, &tmQ, bar.q_full(qb), sub * 64,
                                c.b * a.H + c.g * G);
                for (int i = 0; i < c.n && ok; ++i) {
                    const int row = (c.first + c.n - 1 - i) * kTK;
                    const int keys = c.len - row;  // of this tile, if less than kTK
                    for (int kv = 0; kv < 2; ++kv, ++r) {
                        const int sl = r % kSlots;
                        if (!mbar_wait(bar.empty(sl), ((r / kSlots) & 1) ^ 1u, a.err)) {
                            ok = false;
                            break;
                        }
                        const uint32_t dst = sKV + sl * C::kTile;
                        if (keys >= kTK) {
                            mbar_expect_tx(bar.full(sl), C::kTile);
#pragma unroll
                            for (int sub = 0; sub < C::kSub; ++sub)
                                tma_load_3d_hint(dst + sub * kTK * 128, kv ? &tmV : &tmK, bar.full(sl),
                                                 sub * 64, row, c.b * a.Hk + c.g, pol);
                        } else {
                            const int boxes = (keys + 15) / 16;
                            mbar_expect_tx(bar.full(sl), boxes * 16 * 128 * C::kSub);
                            for (int x = 0; x < boxes; ++x)
#pragma unroll
                                for (int sub = 0; sub < C::kSub; ++sub)
                                    tma_load_3d_hint(dst + sub * kTK * 128 + x * 2048,
                                                     kv ? &tmV16 : &tmK16, bar.full(sl), sub * 64,
                                                     row + x * 16, c.b * a.Hk + c.g, pol);
                        }
                    }
                }
                c.next(a);
            }
            // whatever the others met, no copy lands behind this block's end
            for (int i = r > kSlots ? r - kSlots : 0; i < r; ++i)
                mbar_wait(bar.full(i % kSlots), (i / kSlots) & 1, a.err);
            for (int i = nq > 2 ? nq - 2 : 0; i < nq; ++i)
                mbar_wait(bar.q_full(i & 1), (i >> 1) & 1, a.err);
        }
    } else if (warp == 1) {
        if (lane == 0) {
            constexpr uint32_t fmt = dt_traits<T>::mma_fmt;
            constexpr uint32_t idesc_s = make_idesc_f16(fmt, kTK, 16, false);
            constexpr uint32_t idesc_o = make_idesc_f16(fmt, D, 16, false) | (1u << 15);  // A MN-major
            constexpr uint64_t kAtom = (kTK * 128) >> 4;
            constexpr uint64_t kSlotStep = C::kTile >> 4;
            const uint64_t dk0 = make_sdesc_sw128(sKV, 16, 1024);
            const uint64_t dv0 = make_sdesc_sw128(sKV, kTK * 128, 1024);
            const uint64_t dq0 = make_sdesc_sw128(sQ, 16, 1024);
            const uint64_t dp0 = make_sdesc_sw128(sP, 16, 1024);
            struct Tile {
                int t, it, keys;  // running number, segment, keys of it (may exceed kTK)
                bool first, last; // of its segment
            };
            int i = 0;
            auto next_tile = [&](Tile& x, int t) -> bool {
                if (!c.valid) return false;
                x.t = t;
                x.it = c.it;
                x.keys = c.len - (c.first + c.n - 1 - i) * kTK;
                x.first = i == 0;
                x.last = ++i == c.n;
                if (x.last) {
                    c.next(a);
                    i = 0;
                }
                return true;
            };
            // S^T = K Q^T: the keys and (first tile) queries are there, and the
            // softmax has read the S buffer's last tile
            auto s_ready = [&](const Tile& x) {
                const int r = 2 * x.t;
                return mbar_test(bar.full(r % kSlots), (r / kSlots) & 1) &&
                       (!x.first || mbar_test(bar.q_full(x.it & 1), (x.it >> 1) & 1)) &&
                       (x.t < 2 || mbar_test(bar.s_free(x.t & 1), ((x.t >> 1) - 1) & 1));
            };
            auto issue_s = [&](const Tile& x) {
                tc_fence_after();
                const int sl = 2 * x.t % kSlots;
                const uint64_t dk = dk0 + sl * kSlotStep;
                const uint64_t dq = dq0 + (x.it & 1) * (C::kQBytes >> 4);
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks)
                    tc_mma_ss(tmem + 16u * (x.t & 1),
                              desc_at(dk, static_cast<uint32_t>((ks / 4) * kAtom) + (ks % 4) * 2),
                              desc_at(dq, (ks / 4) * (1024 >> 4) + (ks % 4) * 2), idesc_s,
                              ks > 0 ? 1u : 0u);
                tc_commit(bar.s_full(x.t & 1));
                tc_commit(bar.empty(sl));
                if (x.last) tc_commit(bar.q_empty(x.it & 1));
            };
            // O^T += V^T P^T: the values and P are there, and (first tile) the O
            // buffer's last segment has been read out
            auto pv_ready = [&](const Tile& x) {
                const int r = 2 * x.t + 1;
                return mbar_test(bar.full(r % kSlots), (r / kSlots) & 1) &&
                       mbar_test(bar.p_full(x.t & 1), (x.t >> 1) & 1) &&
                       (!x.first || x.it < 2 || mbar_test(bar.o_free(x.it & 1), ((x.it >> 1) - 1) & 1));
            };
            auto issue_pv = [&](const Tile& x) {
                tc_fence_after();
                const int sl = (2 * x.t + 1) % kSlots;
                const uint64_t dv = dv0 + sl * kSlotStep;
                const uint64_t dp = dp0 + (x.t & 1) * (C::kPBytes >> 4);
                const int steps = (min(x.keys, kTK) + 15) / 16;
#pragma unroll
                for (int ks = 0; ks < kTK / 16; ++ks)
                    if (ks < steps)
                        tc_mma_ss(tmem + 32u + 16u * (x.it & 1), desc_at(dv, ks * ((16 * 128) >> 4)),
                                  desc_at(dp, (ks / 4) * (1024 >> 4) + (ks % 4) * 2), idesc_o,
                                  (!x.first || ks > 0) ? 1u : 0u);
                tc_commit(bar.pv_done(x.t & 1));
                tc_commit(bar.empty(sl));
            };
            Tile now, nxt;
            bool have = next_tile(now, 0), more = true, s_out = false, pv_out = false;
            bool ahead = false;  // S of nxt is out
            if (have) more = next_tile(nxt, 1);
            uint64_t t0 = globaltimer_ns();
            for (uint32_t spin = 1; have; ++spin) {
                bool did = false;
                if (!s_out) {
                    if (s_ready(now)) {
                        issue_s(now);
                        s_out = did = true;
                    }
                } else if (more && !ahead && s_ready(nxt)) {
                    issue_s(nxt);
                    ahead = did = true;
                }
                if (s_out && !pv_out && pv_ready(now)) {
                    issue_pv(now);
                    pv_out = did = true;
                }
                if (pv_out) {  // on to the next tile
                    have = more;
                    now = nxt;
                    s_out = ahead;
                    pv_out = ahead = false;
                    if (more) more = next_tile(nxt, now.t + 1);
                }
                if (did) {
                    spin = 0;
                } else if (spin == 1) {
                    t0 = globaltimer_ns();
                } else if ((spin & 63u) == 0u && globaltimer_ns() - t0 > kWaitLimitNs) {
                    report_error(a.err, DEV_ERR_TIMEOUT);
                    break;
                }
            }
            // ... and no product
            tc_commit(bar.drain());
            mbar_wait(bar.drain(), 0, a.err);
        }
    } else {
        const int quarter = warp & 3;
        const int key = quarter * 32 + lane;  // TMEM lane: key of a tile
        // ... and row of O^T: head_dim 64 takes 16 lanes of each quarter
        const int dim = D == 64 ? quarter * 16 + lane : key;
        const bool has_dim = D != 64 || lane < 16;
        const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
        const uint32_t tS = tmem + lane_off, tO = tmem + lane_off + 32u;
        const float scale_l2 = a.scale * kLog2e;
        float* red_max = reinterpret_cast<float*>(smem + C::kOffMax);
        float* red_sum = reinterpret_cast<float*>(smem + C::kOffSum);
        int t = 0;
        // a segment's O is in TMEM until its last PV has completed: read out
        // behind the next segment's first tile
        bool pend = false;
        int pend_t = 0, pend_buf = 0;
        int64_t pend_rec = 0;
        auto read_out = [&]() -> bool {
            if (!mbar_wait(bar.pv_done(pend_t & 1), (pend_t >> 1) & 1, a.err)) return false;
            tc_fence_after();
            uint32_t o[G];
            tmem_ldn<G>(tO + 16u * pend_buf, o);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar.o_free(pend_buf));
            if (has_dim) {
#pragma unroll
                for (int h = 0; h < G; ++h)
                    a.own_po[(pend_rec * G + h) * D + dim] = __uint_as_float(o[h]);
            }
            __syncwarp();
            return true;
        };
        while (ok && c.valid) {
            float m[G], l[G], slope[G];
#pragma unroll
            for (int h = 0; h < G; ++h) {
                m[h] = -INFINITY;
                l[h] = 0.f;
                slope[h] = 0.f;
                if (a.alibi) {
                    const int hq = c.g * G + h;
                    slope[h] = kLog2e * (a.slopes ? a.slopes[hq]
                                                  : exp2f(-8.0f * static_cast<float>(hq + 1) /
                                                          static_cast<float>(a.H)));
                }
            }
            for (int i = 0; i < c.n; ++i, ++t) {
                const int j = (c.first + c.n - 1 - i) * kTK + key;
                const int keys = c.len - (c.first + c.n - 1 - i) * kTK;
                if (!mbar_wait(bar.s_full(t & 1), (t >> 1) & 1, a.err)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                uint32_t r[G];
                tmem_ldn<G>(tS + 16u * (t & 1), r);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar.s_free(t & 1));
                const float back = static_cast<float>(j - (c.len - 1));
                float s[G];
#pragma unroll
                for (int h = 0; h < G; ++h) {
                    s[h] = fmaf(__uint_as_float(r[h]), scale_l2, slope[h] * back);
                    if (key >= keys) s[h] = -INFINITY;
                }
                float* rm = red_max + (t & 1) * 32;
#pragma unroll
                for (int h = 0; h < G; ++h) {
                    const float w = warp_max(s[h]);
                    if (lane == h) rm[h * 4 + quarter] = w;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(bar.max_full());
                if (!mbar_wait(bar.max_full(), t & 1, a.err)) {
                    ok = false;
                    break;
                }
                // the same decision in every thread
                float corr[G];
                bool moved = false;
#pragma unroll
                for (int h = 0; h < G; ++h) {
                    const float4 w = *reinterpret_cast<const float4*>(rm + h * 4);
                    const float mx = fmaxf(fmaxf(w.x, w.y), fmaxf(w.z, w.w));
                    corr[h] = 1.f;
                    if (mx > m[h] + kRescaleThreshold) {
                        corr[h] = ex2_approx(m[h] - mx);
                        m[h] = mx;
                        moved = true;
                    }
                }
                // P^T buffer t & 1 was read by the PV of tile t - 2
                if (t > 1 && !mbar_wait(bar.pv_done(t & 1), ((t >> 1) - 1) & 1, a.err)) {
                    ok = false;
                    break;
                }
                const uint32_t p_row = sP + (t & 1) * C::kPBytes + (key / 64) * 1024;
#pragma unroll
                for (int h = 0; h < G; ++h) {
                    // in the storage type for the product, as the prefix's (on
                    // the CUDA cores, in 32 bits, the pass was bound by them)
                    const float p = ex2_approx(s[h] - m[h]);
                    l[h] = fmaf(l[h], corr[h], p);
                    const uint32_t at =
                        p_row + h * 128 + (((key & 63) * 2) ^ (static_cast<uint32_t>(h) << 4));
                    const uint16_t bits = static_cast<uint16_t>(dt_traits<T>::pack2(p, 0.f));
                    asm volatile("st.shared.b16 [%0], %1;" ::"r"(at), "h"(bits) : "memory");
                }
                if (keys < kTK && (keys & 15) && quarter == 0) {
                    // values behind the tile's end, up to the product's steps of 16
                    const int rv = 2 * t + 1, sl = rv % kSlots;
                    if (!mbar_wait(bar.full(sl), (rv / kSlots) & 1, a.err)) {
                        ok = false;
                        break;
                    }
                    const int pieces = (16 - (keys & 15)) * 8;
#pragma unroll
                    for (int sub = 0; sub < C::kSub; ++sub)
                        for (int x = lane; x < pieces; x += 32)
                            st_shared_v4(sKV + sl * C::kTile + sub * kTK * 128 + keys * 128 + x * 16,
                                         0u, 0u, 0u, 0u);
                }
                fence_proxy_async_smem();
                if (i > 0 && moved) {
                    if (!mbar_wait(bar.pv_done((t - 1) & 1), ((t - 1) >> 1) & 1, a.err)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    uint32_t o[G];
                    const uint32_t col = tO + 16u * (c.it & 1);
                    tmem_ldn<G>(col, o);
#pragma unroll
                    for (int h = 0; h < G; ++h)
                        o[h] = __float_as_uint(__uint_as_float(o[h]) * corr[h]);
                    tmem_stn<G>(col, o);
                    tc_fence_before();
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(bar.p_full(t & 1));
                if (pend) {
                    ok = read_out();
                    pend = false;
                    if (!ok) break;
                }
            }
            if (!ok) break;
            // the segment's result
#pragma unroll
            for (int h = 0; h < G; ++h) {
                float v = l[h];
#pragma unroll
                for (int x = 16; x > 0; x >>= 1) v += __shfl_xor_sync(0xffffffffu, v, x);
                if (lane == h) red_sum[(c.it & 1) * 32 + h * 4 + quarter] = v;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(bar.sum_full());
            if (!mbar_wait(bar.sum_full(), c.it & 1, a.err)) {
                ok = false;
                break;
            }
            const int64_t rec = static_cast<int64_t>(own_index()) +
                                (static_cast<int64_t>(c.b) * a.Hk + c.g);
            pend = true;
            pend_t = t - 1;
            pend_buf = c.it & 1;
            pend_rec = rec;
            if (quarter == 0 && lane < G) {
                const float4 w = *reinterpret_cast<const float4*>(red_sum + (c.it & 1) * 32 + lane * 4);
                float mh = m[0];
#pragma unroll
                for (int h = 1; h < G; ++h)
                    if (lane == h) mh = m[h];
                a.own_pm[rec * G + lane] = make_float2(mh, (w.x + w.y) + (w.z + w.w));
            }
            c.next(a);
        }
        if (ok && pend) ok = read_out();
    }
}

template <typename T, int D, int G>
__global__ void __launch_bounds__(kThreads, 2)
    shared_kernel(const __grid_constant__ SharedMaps tm, const SharedKernelArgs a) {
    using C = Cfg<D>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ OwnRange range;
    uint8_t* smem = align_1024(smem_raw);
    const uint32_t bar_p = smem_u32(smem) + C::kOffBar;
    const uint32_t bar_o = bar_p + PrefixBars<C::kSlotsP>::kBytes;
    constexpr int kOffSlot = C::kOffBar + PrefixBars<C::kSlotsP>::kBytes + OwnBars<C::kSlots>::kBytes;
    static_assert(kOffSlot + 4 <= C::kOffBar + 512, "barrier space");
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kOffSlot);
    const int warp = threadIdx.x / 32;
    const int lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        PrefixBars<C::kSlotsP>{bar_p}.init();
        OwnBars<C::kSlots>{bar_o}.init();
        fence_barrier_init();
        tma_prefetch_desc(&tm.pq);
        tma_prefetch_desc(&tm.pk);
        tma_prefetch_desc(&tm.pv);
        tma_prefetch_desc(&tm.oq);
        tma_prefetch_desc(&tm.ok);
        tma_prefetch_desc(&tm.ov);
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(tmem_slot), 256);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    if (a.pdl) pdl_wait();
    // the softmax warps find the range while the first tiles are on their way
    if (warp >= 2) find_own_range(a, range, OwnBars<C::kSlots>{bar_o}.range_full());

    // each warp goes on to the own caches as it is done with the prefix
    bool ok = prefix_phase<T, D>(a, tm.pq, tm.pk, tm.pv, smem_u32(smem), bar_p, tmem, warp, lane);
    if (ok) ok = mbar_wait(OwnBars<C::kSlots>{bar_o}.range_full(), 0, a.err);
    if (ok) {
        OwnSegments own;
        own.start(a, range.lo, range.hi, range.b0, range.base);
        own_phase<T, D, G>(a, tm.oq, tm.ok, tm.ov, tm.ok16, tm.ov16, own, smem, bar_o, tmem, warp, lane);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, 256);
    // The merge may come in now. Earlier its blocks only took the SM's room as
    // CTAs ended (at the start of this kernel: 36.9 us against 33.6 for 32 x 32 x
    // 64 heads, 8192 shared keys).
    if (a.pdl) pdl_launch_dependents();
}

template <typename T, int D, int G>
cudaError_t launch_shared_g(const SharedMaps& tm, const SharedKernelArgs& a, cudaStream_t s) {
    using C = Cfg<D>;
    auto kern = shared_kernel<T, D, G>;
    const cudaError_t e = set_smem_attr_once(reinterpret_cast<const void*>(kern), C::kSmem);
    if (e != cudaSuccess) return e;
    return launch_pdl(a.pdl != 0, kern, dim3(a.grid), dim3(kThreads), C::kSmem, s, tm, a);
}

template <typename T>
cudaError_t launch_shared_t(int d, const SharedMaps& tm, const SharedKernelArgs& a, cudaStream_t s) {
    switch (d * 16 + a.G) {
        case 64 * 16 + 1: return launch_shared_g<T, 64, 1>(tm, a, s);
        case 64 * 16 + 2: return launch_shared_g<T, 64, 2>(tm, a, s);
        case 64 * 16 + 4: return launch_shared_g<T, 64, 4>(tm, a, s);
        case 64 * 16 + 8: return launch_shared_g<T, 64, 8>(tm, a, s);
        case 128 * 16 + 1: return launch_shared_g<T, 128, 1>(tm, a, s);
        case 128 * 16 + 2: return launch_shared_g<T, 128, 2>(tm, a, s);
        case 128 * 16 + 4: return launch_shared_g<T, 128, 4>(tm, a, s);
        case 128 * 16 + 8: return launch_shared_g<T, 128, 8>(tm, a, s);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace

}  // namespace blk
