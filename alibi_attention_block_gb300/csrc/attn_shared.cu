// K6s: one decode step of attention for a batch that shares a prefix.
//
// Sequence b's newest query q[b, h] attends to the prefix's P keys, stored
// once for the batch (k/v_prefix [Hk, P, d]), and to its own cache. Softmax
// parts over disjoint key sets merge by their (max, sum), so the prefix is one
// product for the whole batch: for a kv head, the queries of all sequences and
// of the head's group are the rows of Q, and S = Q K^T, O = P V run on the
// tensor cores with each prefix byte read once instead of once per sequence.
// (the attention of nnterp "stablelm" 03 Notes; ALiBi as in "Bloom in a
// sovereign engine", Contribution, with the query at position
// P + lens[b] - 1.)
//
// Pass 1 (prefix_kernel): persistent, one CTA per SM. A unit is (kv head, 128
// or 256 query rows; 128 rows are 128 / G sequences); its P keys are nkt tiles
// of 128. The units' tiles in one line are cut into equal ranges, one per CTA
// (no CTA has more than one tile above another), and a CTA's stay in a unit is
// a segment with a partial result of its own. A chain of one query tile
// (scores, softmax, PV, one after the other) leaves tensor core and memory
// idle most of the time, so two streams A and B run side by side:
//   one row tile per kv head: A and B have the same queries and take the
//     segment's key tiles in turn, each with its own running maximum, sum and
//     O, merged at the end;
//   more (PAIR): A and B are two row tiles on the same key tiles, which halves
//     the bytes each row tile brings into shared memory (16384 keys, 8 kv
//     heads x 128, 256 rows each: 25.0 us apart, where the L2-to-SM traffic
//     bounds it, @PAIR@ us paired).
// 12 warps as in attn_pair.cu:
//   warp 0      TMA: the segment's queries (4D boxes: d, group, kv head,
//               batch), then K and V tiles into a ring; one ring per stream
//               unless they share the tiles. (In a ring that both read, each
//               slot needs both to release it: a stream that skips the other's
//               tiles cannot tell a slot's phases apart by their parity.)
//   warps 1, 2  MMA-issuing thread of stream A, of stream B
//   warps 4..7, 8..11  softmax of A, of B, one thread per query row. At the
//               end of a segment the result goes to the workspace in fp32:
//               paired, each stream's own O; else both streams' statistics
//               meet in shared memory, and each warpgroup merges half of the
//               columns of the two O from TMEM.
// TMEM columns: S_A [0, 128), S_B [128, 256); head_dim 64: P_A, P_B
// [256, 384), O_A, O_B [384, 512); head_dim 128: P over its own S, O_A, O_B
// [256, 512) (so the next S waits for the PV that reads P).
// Pass 2 (own_kernel, attn_own.cu): the sequences' own caches.
// Pass 3 (shared_combine_kernel): one warp per (b, query head) merges the
// segments of both passes.
#include "internal.h"

namespace blk {

namespace {

constexpr int kThreads = 384;
constexpr int kTQ = 128, kTK = 128;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kRescaleThreshold = 8.0f;  // log2 of the largest unnormalised p
constexpr uint32_t kLaunchRegs = 168;

struct PrefixArgs {
    int pdl;
    // partial outputs [segments][row tiles of a unit][D / 8][128 rows][8]: a
    // thread holds a row and writes whole 32-byte sectors that join its
    // neighbours' (row-major, the epilogue of a full tile took 5 us)
    float* po;
    float2* pm;    // [segments][rows of a unit] (max, sum), log2 domain
    const float* slopes;
    unsigned* err;
    int B, H, Hk, G, P;
    int nkt;       // key tiles
    int nrt;       // row tiles per kv head
    int nu;        // units per kv head
    int W;         // tiles in all: Hk * nu * nkt
    float scale;
    int alibi;
};

template <int D, bool PAIR>
struct Cfg {
    static constexpr int kSub = D / 64;
    static constexpr int kTile = kSub * 128 * 128;     // Q, K or V tile
    // slots of a ring of K and V tiles, and rings
    static constexpr int kSlots = PAIR ? (D == 64 ? 10 : 4) : (D == 64 ? 6 : 3);
    static constexpr int kRings = PAIR ? 1 : 2;
    static constexpr int kRows = PAIR ? 2 * kTQ : kTQ;  // of a unit
    static constexpr int kOffRing = (PAIR ? 2 : 1) * kTile;
    static constexpr int kOffStats = kOffRing + kRings * kSlots * kTile;  // [2][128] float2
    static constexpr int kOffBar = kOffStats + 2 * 128 * 8;
    // no alignment slack (three slots would not fit): the kernel has no other
    // shared memory, so the tiles start where dynamic shared memory does
    static constexpr int kSmem = kOffBar + 512;
    static constexpr bool kPOverS = D != 64;
    // per-thread registers of the control warps and of the softmax warps
    static constexpr uint32_t kRegsControl = 88;
    static constexpr uint32_t kRegsSoftmax = 208;
    static constexpr uint32_t kColP = kPOverS ? 0 : 256, kPStep = kPOverS ? 128 : 64;
    static constexpr uint32_t kColO = kPOverS ? 256 : 384;
    static_assert(kColO + 2 * D <= 512 && kSmem <= 232448, "TMEM or shared memory");
};

// A CTA's segments: tiles [t, hi) of unit u, key tiles from klo; processed
// from the last key tile down (with ALiBi the bias is largest there).
struct Segments {
    int t, end, u, n, klo, it;
    bool valid;
    __device__ __forceinline__ void set(const PrefixArgs& a) {
        valid = t < end;
        if (!valid) return;
        u = t / a.nkt;
        klo = t - u * a.nkt;
        n = min(end - t, a.nkt - klo);
    }
    __device__ __forceinline__ void start(const PrefixArgs& a) {
        t = static_cast<int>(static_cast<int64_t>(blockIdx.x) * a.W / gridDim.x);
        end = static_cast<int>(static_cast<int64_t>(blockIdx.x + 1) * a.W / gridDim.x);
        it = 0;
        set(a);
    }
    __device__ __forceinline__ void next(const PrefixArgs& a) {
        t += n;
        ++it;
        set(a);
    }
};

// 32 bytes to global memory in one store (32-byte aligned).
__device__ __forceinline__ void store_sector(float* p, const float (&f)[8]) {
    asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(f[0]),
                 "f"(f[1]), "f"(f[2]), "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7])
                 : "memory");
}

template <typename T, int D, bool ALIBI, bool PAIR>
__global__ void __launch_bounds__(kThreads, 1)
    prefix_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                  const __grid_constant__ CUtensorMap tmV, const PrefixArgs a) {
    using C = Cfg<D, PAIR>;
    constexpr int kSlots = C::kSlots;
    extern __shared__ __align__(1024) uint8_t smem[];
    if (smem_u32(smem) & 1023u) {  // the swizzled tiles need it
        if (threadIdx.x == 0) report_error(a.err, DEV_ERR_TIMEOUT);
        return;
    }
    const uint32_t sQ = smem_u32(smem);
    const uint32_t sRing = sQ + C::kOffRing;
    const uint32_t bar0 = sQ + C::kOffBar;
    auto s_full = [&](int x) { return bar0 + 8u * x; };
    auto s_free = [&](int x) { return bar0 + 16u + 8u * x; };
    auto p_full = [&](int x) { return bar0 + 32u + 8u * x; };
    auto pv_done = [&](int x) { return bar0 + 48u + 8u * x; };
    const uint32_t q_full = bar0 + 64u, q_empty = bar0 + 72u;
    const uint32_t stats_full = bar0 + 80u;
    // stream x's O has been read (paired), or both (else one barrier for both)
    auto o_free = [&](int x) { return bar0 + 88u + 8u * (PAIR ? x : 0); };
    // slot i of stream x's ring (paired: of the one ring)
    auto ring_of = [&](int x) { return PAIR ? 0 : kSlots * x; };
    auto full = [&](int x, int i) { return bar0 + 104u + 8u * (ring_of(x) + i); };
    auto empty = [&](int x, int i) { return bar0 + 104u + 8u * (kSlots * C::kRings + ring_of(x) + i); };
    static_assert(104 + 16 * C::kRings * kSlots + 4 <= 512, "barrier space");
    uint32_t* tmem_slot =
        reinterpret_cast<uint32_t*>(smem + C::kOffBar + 104 + 16 * C::kRings * kSlots);
    // key tiles of stream x in a segment, and the key tile of its i-th
    auto has_rows = [&](const Segments& c, int x) {
        return !PAIR || x == 0 || 2 * (c.u % a.nu) + 1 < a.nrt;
    };
    auto tiles = [&](const Segments& c, int x) {
        return PAIR ? (has_rows(c, x) ? c.n : 0) : (c.n + 1 - x) / 2;
    };

    const int warp = threadIdx.x / 32;
    const int lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int x = 0; x < 2; ++x) {
            mbar_init(s_full(x), 1);
            mbar_init(s_free(x), 4);
            mbar_init(p_full(x), 4);
            mbar_init(pv_done(x), 1);
            mbar_init(o_free(x), PAIR ? 4 : 8);
            for (int i = 0; i < kSlots; ++i) {
                mbar_init(full(x, i), 1);
                mbar_init(empty(x, i), PAIR ? 2 : 1);
            }
        }
        mbar_init(q_full, 1);
        mbar_init(q_empty, 2);
        mbar_init(stats_full, 8);
        fence_barrier_init();
        tma_prefetch_desc(&tmQ);
        tma_prefetch_desc(&tmK);
        tma_prefetch_desc(&tmV);
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(tmem_slot), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    if (a.pdl) {
        pdl_wait();
        pdl_launch_dependents();
    }
    static_assert(4 * C::kRegsControl + 8 * C::kRegsSoftmax <= 12 * kLaunchRegs,
                  "register split exceeds the launch's registers");
    if (warp < 4) {
        setmaxnreg_dec<C::kRegsControl>();
        if (warp == 0 && lane == 0) {
            // read again by the kv head's other units, if it has any
            const uint64_t pol = a.nu > 1 ? l2_evict_last_policy() : l2_evict_first_policy();
            Segments c;
            c.start(a);
            int rx[2] = {0, 0};  // tiles put into each ring
            bool ok = true;
            while (ok && c.valid) {
                const int g = c.u / a.nu, rt = (c.u - g * a.nu) * (PAIR ? 2 : 1);
                const int nq = PAIR && has_rows(c, 1) ? 2 : 1;  // query tiles
                if (!mbar_wait_inl(q_empty, (c.it & 1) ^ 1u, a.err)) break;
                mbar_expect_tx(q_full, nq * C::kTile);
                for (int x = 0; x < nq; ++x)
#pragma unroll
                    for (int sub = 0; sub < C::kSub; ++sub)
                        tma_load_4d(sQ + x * C::kTile + sub * kTQ * 128, &tmQ, q_full, sub * 64, 0,
                                    g, (rt + x) * (kTQ / a.G));
                // step i's tile, for stream x (paired: for both)
                auto load = [&](const CUtensorMap* m, int i, int x) -> bool {
                    const int r = rx[x], sl = r % kSlots;
                    if (!mbar_wait_inl(empty(x, sl), ((r / kSlots) & 1) ^ 1u, a.err)) return false;
                    mbar_expect_tx(full(x, sl), C::kTile);
                    const int row = (c.klo + c.n - 1 - i) * kTK;
#pragma unroll
                    for (int sub = 0; sub < C::kSub; ++sub)
                        tma_load_3d_hint(sRing + (ring_of(x) + sl) * C::kTile + sub * kTK * 128, m,
                                         full(x, sl), sub * 64, row, g, pol);
                    ++rx[x];
                    return true;
                };
                if (PAIR)
                    for (int i = 0; i < c.n && ok; ++i) ok = load(&tmK, i, 0) && load(&tmV, i, 0);
                for (int i = 0; !PAIR && i < c.n && ok; i += 2) {
                    const bool two = i + 1 < c.n;
                    ok = load(&tmK, i, 0) && (!two || load(&tmK, i + 1, 1)) &&
                         load(&tmV, i, 0) && (!two || load(&tmV, i + 1, 1));
                }
                c.next(a);
            }
        } else if ((warp == 1 || warp == 2) && lane == 0) {
            const int x = warp - 1;
            constexpr uint32_t fmt = dt_traits<T>::mma_fmt;
            constexpr uint32_t idesc_s = make_idesc_f16(fmt, kTQ, kTK, false);
            constexpr uint32_t idesc_o = make_idesc_f16(fmt, kTQ, D, true);
            constexpr uint64_t kAtom = (kTQ * 128) >> 4;
            constexpr uint64_t kSlotStep = C::kTile >> 4;
            const uint64_t dq = make_sdesc_sw128(sQ + (PAIR ? x * C::kTile : 0), 16, 1024);
            const uint32_t ring = sRing + ring_of(x) * C::kTile;
            const uint64_t dk0 = make_sdesc_sw128(ring, 16, 1024);
            const uint64_t dv0 = make_sdesc_sw128(ring, kTK * 128, 1024);
            const uint32_t tS = tmem_base + 128u * x;
            const uint32_t tP = tmem_base + C::kColP + C::kPStep * x;
            const uint32_t tO = tmem_base + C::kColO + D * x;
            int gs = 0, gp = 0;  // S and PV products issued
            auto issue_s = [&](int r) -> bool {
                const int sl = r % kSlots;
                if (!mbar_wait_inl(full(x, sl), (r / kSlots) & 1, a.err)) return false;
                if (gs > 0) {
                    // the softmax has read the previous S; P over S: the
                    // previous PV has read P
                    if (C::kPOverS ? !mbar_wait_inl(pv_done(x), (gs - 1) & 1, a.err)
                                   : !mbar_wait_inl(s_free(x), (gs - 1) & 1, a.err))
                        return false;
                }
                tc_fence_after();
                const uint64_t dk = dk0 + sl * kSlotStep;
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks) {
                    const uint64_t off = (ks / 4) * kAtom + (ks % 4) * 2;
                    tc_mma_ss(tS, dq + off, dk + off, idesc_s, ks > 0 ? 1u : 0u);
                }
                tc_commit(s_full(x));
                tc_commit(empty(x, sl));
                ++gs;
                return true;
            };
            auto issue_pv = [&](int r, bool first, int it) -> bool {
                const int sl = r % kSlots;
                if (!mbar_wait_inl(full(x, sl), (r / kSlots) & 1, a.err)) return false;
                if (!mbar_wait_inl(p_full(x), gp & 1, a.err)) return false;
                if (first && it > 0 && !mbar_wait_inl(o_free(x), (it - 1) & 1, a.err)) return false;
                tc_fence_after();
                const uint64_t dv = dv0 + sl * kSlotStep;
#pragma unroll
                for (int ks = 0; ks < kTK / 16; ++ks)
                    tc_mma_ts(tO, tP + ks * 8, dv + ks * ((16 * 128) >> 4), idesc_o,
                              (!first || ks > 0) ? 1u : 0u);
                tc_commit(pv_done(x));
                tc_commit(empty(x, sl));
                ++gp;
                return true;
            };
            Segments c;
            c.start(a);
            int r0 = 0;  // ring position of the segment's first tile (K, V, K, V, ...)
            bool ok = true;
            while (ok && c.valid) {
                const int nx = tiles(c, x);
                auto pos_k = [&](int i) { return r0 + 2 * i; };
                auto pos_v = [&](int i) { return r0 + 2 * i + 1; };
                if (!mbar_wait_inl(q_full, c.it & 1, a.err)) break;
                if (C::kPOverS) {
                    for (int i = 0; i < nx && ok; ++i) {
                        ok = issue_s(pos_k(i));
                        if (ok && i + 1 == nx) tc_commit(q_empty);
                        ok = ok && issue_pv(pos_v(i), i == 0, c.it);
                    }
                } else {
                    // S of the next tile ahead of PV of this one
                    if (nx > 0) ok = issue_s(pos_k(0));
                    if (ok && nx == 1) tc_commit(q_empty);
                    for (int i = 0; i < nx && ok; ++i) {
                        if (i + 1 < nx) {
                            ok = issue_s(pos_k(i + 1));
                            if (ok && i + 2 == nx) tc_commit(q_empty);
                        }
                        ok = ok && issue_pv(pos_v(i), i == 0, c.it);
                    }
                }
                if (ok && nx == 0) {
                    tc_commit(q_empty);
                    // paired, without a second row tile: release the slots
                    for (int r = r0; PAIR && ok && r < r0 + 2 * c.n; ++r) {
                        ok = mbar_wait_inl(full(x, r % kSlots), (r / kSlots) & 1, a.err);
                        if (ok) mbar_arrive(empty(x, r % kSlots));
                    }
                }
                r0 += 2 * (PAIR ? c.n : nx);
                c.next(a);
            }
        }
    } else {
        setmaxnreg_inc<C::kRegsSoftmax>();
        const int x = (warp - 4) >> 2;
        const int quarter = warp & 3;
        const int row = quarter * 32 + lane;
        const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
        const uint32_t tS = tmem_base + 128u * x + lane_off;
        const uint32_t tP = tmem_base + C::kColP + C::kPStep * x + lane_off;
        const uint32_t tO = tmem_base + C::kColO + D * x + lane_off;
        const float scale_l2 = a.scale * kLog2e;
        float2* stats = reinterpret_cast<float2*>(smem + C::kOffStats);
        Segments c;
        c.start(a);
        int g = 0;             // tiles of this stream so far
        int gy = 0;            // of the other stream
        bool ok = true;
        while (ok && c.valid) {
            const int kvh = c.u / a.nu;
            const int rt = PAIR ? 2 * (c.u - kvh * a.nu) + x : c.u - kvh * a.nu;
            const int nx = tiles(c, x), ny = tiles(c, 1 - x);
            // a warp all of whose rows lie behind the batch only keeps the
            // barriers going: its P and O are whatever they are, and unread
            const bool live = rt * (kTQ / a.G) + quarter * 32 / a.G < a.B;
            if (PAIR && nx == 0) {
                // no rows: still one phase of o_free per segment
                __syncwarp();
                if (lane == 0) mbar_arrive(o_free(x));
                c.next(a);
                continue;
            }
            float m_used = -INFINITY;  // running max, log2 domain
            float l = 0.f;
            float slope_l2 = 0.f;
            if constexpr (ALIBI) {
                const int h = kvh * a.G + row % a.G;
                slope_l2 = kLog2e * (a.slopes ? a.slopes[h]
                                              : exp2f(-8.0f * static_cast<float>(h + 1) /
                                                      static_cast<float>(a.H)));
            }
            for (int i = 0; i < nx; ++i, ++g) {
                if (!mbar_wait_inl(s_full(x), g & 1, a.err)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                if (!live) {
                    if (i > 0 && !mbar_wait_inl(pv_done(x), (g - 1) & 1, a.err)) {
                        ok = false;
                        break;
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        if (!C::kPOverS) mbar_arrive(s_free(x));
                        mbar_arrive(p_full(x));
                    }
                    continue;
                }
                uint32_t r[kTK];
                tmem_ld128(tS, r);
                if (!C::kPOverS) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(s_free(x));
                }
                const int kbase = (c.klo + c.n - 1 - (PAIR ? i : 2 * i + x)) * kTK;
                if constexpr (ALIBI) {
                    // + slope * (key - P), the distance to the query's own
                    // part of the row's bias being left to the merge
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
                float mx = fmaxf(fmaxf(m0, m1), fmaxf(m2, m3));
                if constexpr (!ALIBI) mx *= scale_l2;  // scale > 0: max commutes with it
                float corr = 1.f;
                if (mx > m_used + kRescaleThreshold) {
                    corr = ex2_approx(m_used - mx);
                    m_used = mx;
                }
                const uint64_t mul2 = f2_pack(ALIBI ? 1.f : scale_l2, ALIBI ? 1.f : scale_l2);
                const uint64_t neg2 = f2_pack(-m_used, -m_used);
                uint64_t acc0 = f2_pack(0.f, 0.f), acc1 = acc0;
                uint32_t pk[kTK / 2];
#pragma unroll
                for (int k = 0; k < kTK; k += 4) {
                    float e0, e1, e2, e3;
                    ffma2(__uint_as_float(r[k]), __uint_as_float(r[k + 1]), mul2, neg2, e0, e1);
                    ffma2(__uint_as_float(r[k + 2]), __uint_as_float(r[k + 3]), mul2, neg2, e2,
                          e3);
                    const float p0 = ex2_approx(e0), p1 = ex2_approx(e1);
                    const float p2 = ex2_approx(e2), p3 = ex2_approx(e3);
                    fadd2_acc(acc0, p0, p1);
                    fadd2_acc(acc1, p2, p3);
                    pk[k / 2] = dt_traits<T>::pack2(p0, p1);
                    pk[k / 2 + 1] = dt_traits<T>::pack2(p2, p3);
                }
                if (i > 0) {  // the previous PV has read P, and O is settled
                    if (!mbar_wait_inl(pv_done(x), (g - 1) & 1, a.err)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                }
                tmem_st64_nowait(tP, pk);
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
                if (lane == 0) mbar_arrive(p_full(x));
                float s0, s1, s2, s3;
                f2_unpack(acc0, s0, s1);
                f2_unpack(acc1, s2, s3);
                l = l * corr + ((s0 + s1) + (s2 + s3));
            }
            if (!ok) break;
            const bool mine = rt * (kTQ / a.G) + row / a.G < a.B;
            const int64_t rec = (static_cast<int64_t>(blockIdx.x) + c.u) * C::kRows +
                                (PAIR ? x * kTQ : 0) + row;
            if constexpr (PAIR) {
                if (!mbar_wait_inl(pv_done(x), (g - 1) & 1, a.err)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                if (mine) a.pm[rec] = make_float2(m_used, l);
                float* dst = a.po + (rec - row) * D + row * 8;
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
            } else {
                gy += ny;
                // both streams' statistics through shared memory (once all
                // have read the previous segment's), then this warpgroup's
                // half of the columns of both O
                if (c.it > 0 && !mbar_wait_inl(o_free(0), (c.it - 1) & 1, a.err)) {
                    ok = false;
                    break;
                }
                float2* st = stats;
                st[x * kTQ + row] = make_float2(m_used, l);
                __syncwarp();
                if (lane == 0) mbar_arrive(stats_full);
                if (!mbar_wait_inl(stats_full, c.it & 1, a.err) ||
                    (nx > 0 && !mbar_wait_inl(pv_done(x), (g - 1) & 1, a.err)) ||
                    (ny > 0 && !mbar_wait_inl(pv_done(1 - x), (gy - 1) & 1, a.err))) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const float2 sa = st[row], sb = st[kTQ + row];
                const float m = fmaxf(sa.x, sb.x);
                const float wa = sa.x == -INFINITY ? 0.f : ex2_approx(sa.x - m);
                const float wb = sb.x == -INFINITY ? 0.f : ex2_approx(sb.x - m);
                const bool has_b = c.n > 1;
                if (mine && x == 0) a.pm[rec] = make_float2(m, wa * sa.y + wb * sb.y);
                float* dst = a.po + (rec - row) * D + x * (D / 2) * kTQ + row * 8;
                const uint32_t tA = tmem_base + C::kColO + lane_off + x * (D / 2);
#pragma unroll 1
                for (int cc = 0; cc < D / 32 && live; ++cc) {
                    uint32_t oa[16], ob[16];
                    tmem_ld16(tA + cc * 16, oa);
                    if (has_b) tmem_ld16(tA + D + cc * 16, ob);
                    if (mine) {
#pragma unroll
                        for (int v = 0; v < 2; ++v) {
                            float f[8];
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                f[e] = wa * __uint_as_float(oa[v * 8 + e]);
                                if (has_b) f[e] = fmaf(wb, __uint_as_float(ob[v * 8 + e]), f[e]);
                            }
                            store_sector(dst + (cc * 2 + v) * kTQ * 8, f);
                        }
                    }
                    __syncwarp();
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(o_free(x));
            c.next(a);
        }
    }
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem_base, 512);
    }
}

// o = sum_i w_i O_i / sum_i w_i l_i over the prefix's segments and the own
// cache's, w_i = 2^(m_i - max m): one warp per (b, query head). With
// ALiBi the prefix's maxima still lack the row's -slope * (lens[b] - 1).
struct CombineArgs {
    int pdl;
    const float* po;
    const float2* pm;
    const float* own_po;
    const float2* own_pm;
    const int32_t* cum;
    const int32_t* lens;
    const float* slopes;
    void* o;
    int B, H, G, max_seq, alibi, own_grid;
    int nkt, nu, W, grid, rows;  // of the prefix pass (rows: of a unit); W 0: no prefix
};

template <typename T, int D>
__global__ void __launch_bounds__(128, 6) shared_combine_kernel(const CombineArgs a) {
    // a record's D floats are read 16 bytes per lane: head_dim 64 takes half a
    // warp, so two records at a time
    constexpr int kLanes = D / 4, kAtOnce = 32 / kLanes;
    if (a.pdl) {
        pdl_wait();
        pdl_launch_dependents();
    }
    const int lane = threadIdx.x & 31;
    const int64_t w = static_cast<int64_t>(blockIdx.x) * 4 + threadIdx.x / 32;
    if (w >= static_cast<int64_t>(a.B) * a.H) return;
    const int b = static_cast<int>(w / a.H), h = static_cast<int>(w - static_cast<int64_t>(b) * a.H);
    const int Hk = a.H / a.G, g = h / a.G;
    const int c4 = lane % kLanes, half = lane / kLanes;
    // The prefix's segments of this row: CTAs c0 .. c1, record c + unit. Where
    // they are is known at once, so the first of them are on their way while
    // the lengths, which say where the own cache's are, still come.
    int64_t seg0 = 0;  // the first one's first row
    int nseg = 0, row = 0;
    if (a.W) {
        const int per = a.rows / a.G;  // sequences per unit
        const int u = g * a.nu + b / per;
        row = b % per * a.G + h % a.G;  // of the unit
        const int64_t p0 = static_cast<int64_t>(u) * a.nkt;
        const int c0 = static_cast<int>(((p0 + 1) * a.grid - 1) / a.W);
        const int c1 = static_cast<int>(((p0 + a.nkt) * a.grid - 1) / a.W);
        seg0 = static_cast<int64_t>(c0 + u) * a.rows;
        nseg = c1 - c0 + 1;
    }
    auto prefix_part = [&](int k) -> const float4& {
        return *reinterpret_cast<const float4*>(
            a.po + (seg0 + static_cast<int64_t>(k) * a.rows + row / kTQ * kTQ) * D +
            (c4 / 2 * kTQ + row % kTQ) * 8 + c4 % 2 * 4);
    };
    auto prefix_stat = [&](int k) { return a.pm[seg0 + static_cast<int64_t>(k) * a.rows + row]; };
    constexpr int kLoads = 8 / kAtOnce;  // of 8 records, in flight together
    float4 f[kLoads];
#pragma unroll
    for (int x = 0; x < kLoads; ++x)
        if (x * kAtOnce + half < nseg) f[x] = prefix_part(x * kAtOnce + half);
    float2 stat = make_float2(-INFINITY, 0.f);  // lane i: record i's (max, sum)
    if (lane < nseg) stat = prefix_stat(lane);
    const int tiles = a.cum[a.B], before = a.cum[b];
    const int n = min(max(a.lens[b], 0), a.max_seq);
    float o[4] = {0.f, 0.f, 0.f, 0.f};
    float mx = -INFINITY, lsum = 0.f;
    if (n > 0) {
        // the own cache's segments, of unit (b, kv head)
        const int64_t own_w = static_cast<int64_t>(tiles) * Hk;
        const int nt = (n + kTK - 1) / kTK;
        const int64_t t0 = static_cast<int64_t>(before) * Hk + static_cast<int64_t>(g) * nt;
        const int64_t ctas = min(static_cast<int64_t>(a.own_grid), own_w);
        const int c0 = static_cast<int>(((t0 + 1) * ctas - 1) / own_w);
        const int c1 = static_cast<int>(((t0 + nt) * ctas - 1) / own_w);
        const int64_t own0 = (static_cast<int64_t>(c0) + static_cast<int64_t>(b) * Hk + g) * a.G + h % a.G;
        const int total = nseg + c1 - c0 + 1;
        float shift = 0.f;
        if (a.alibi) {
            const float sl = a.slopes ? a.slopes[h]
                                      : exp2f(-8.0f * static_cast<float>(h + 1) /
                                              static_cast<float>(a.H));
            shift = sl * kLog2e * static_cast<float>(n - 1);
        }
        for (int base = 0; base < total; base += 32) {
            const int i = base + lane;
            if (i >= nseg || base > 0) {
                stat = make_float2(-INFINITY, 0.f);
                if (i < nseg) stat = prefix_stat(i);
                else if (i < total) stat = a.own_pm[own0 + static_cast<int64_t>(i - nseg) * a.G];
            }
            const float m = i < nseg ? stat.x - shift : stat.x;
            float mb = m;
#pragma unroll
            for (int s = 16; s > 0; s >>= 1) mb = fmaxf(mb, __shfl_xor_sync(0xffffffffu, mb, s));
            const float mn = fmaxf(mx, mb);
            const float keep = mx == -INFINITY ? 0.f : exp2f(mx - mn);
            const float wgt = m == -INFINITY ? 0.f : exp2f(m - mn);
            float ls = wgt * stat.y;
#pragma unroll
            for (int s = 16; s > 0; s >>= 1) ls += __shfl_xor_sync(0xffffffffu, ls, s);
            lsum = fmaf(lsum, keep, ls);
            mx = mn;
#pragma unroll
            for (int e = 0; e < 4; ++e) o[e] *= keep;
            // (each half of a warp, or the whole, in record order)
            const int cnt = min(32, total - base);
#pragma unroll 1
            for (int j0 = 0; j0 < cnt; j0 += 8) {
#pragma unroll
                for (int x = 0; x < kLoads; ++x) {
                    const int j = j0 + x * kAtOnce + half, k = base + j;
                    if (k < nseg) {
                        if (base + j0 > 0) f[x] = prefix_part(k);
                    } else if (j < cnt) {
                        f[x] = reinterpret_cast<const float4*>(
                            a.own_po + (own0 + static_cast<int64_t>(k - nseg) * a.G) * D)[c4];
                    }
                }
#pragma unroll
                for (int x = 0; x < kLoads; ++x) {
                    const int j = j0 + x * kAtOnce + half;
                    const float wj = __shfl_sync(0xffffffffu, wgt, j & 31);
                    if (j < cnt) {
                        o[0] = fmaf(wj, f[x].x, o[0]);
                        o[1] = fmaf(wj, f[x].y, o[1]);
                        o[2] = fmaf(wj, f[x].z, o[2]);
                        o[3] = fmaf(wj, f[x].w, o[3]);
                    }
                }
            }
        }
    }
    if constexpr (kAtOnce == 2) {
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] += __shfl_xor_sync(0xffffffffu, o[e], 16);
    }
    const float inv = lsum > 0.f ? 1.0f / lsum : 0.f;
    if (lane < kLanes) {
        const uint2 v = make_uint2(dt_traits<T>::pack2(o[0] * inv, o[1] * inv),
                                   dt_traits<T>::pack2(o[2] * inv, o[3] * inv));
        *reinterpret_cast<uint2*>(static_cast<T*>(a.o) + w * D + lane * 4) = v;
    }
}

template <typename T, int D, bool ALIBI, bool PAIR>
cudaError_t launch_prefix(DType dt, const SharedArgs& s, const PrefixArgs& p, int grid,
                          cudaStream_t st) {
    using C = Cfg<D, PAIR>;
    CUtensorMap tq, tk, tv;
    if (!make_tmap_queries(&tq, dt, s.own.q, p.B, p.Hk, p.G, D, kTQ / p.G) ||
        !make_tmap_3d(&tk, dt, s.k_prefix, p.Hk, p.P, D, kTK) ||
        !make_tmap_3d(&tv, dt, s.v_prefix, p.Hk, p.P, D, kTK))
        return cudaErrorInvalidValue;
    auto kern = prefix_kernel<T, D, ALIBI, PAIR>;
    const cudaError_t e = set_smem_attr_once(reinterpret_cast<const void*>(kern), C::kSmem);
    if (e != cudaSuccess) return e;
    PrefixArgs a = p;
    a.pdl = pdl_allowed(st);
    return launch_pdl(a.pdl != 0, kern, dim3(grid), dim3(kThreads), C::kSmem, st, tq, tk, tv, a);
}

template <typename T, int D>
cudaError_t launch_t(DType dt, const SharedArgs& s, cudaStream_t st) {
    const DecodeArgs& d = s.own;
    const int G = d.H / d.Hk;
    PrefixArgs p{};
    p.nkt = (s.P + kTK - 1) / kTK;
    p.nrt = (d.B + kTQ / G - 1) / (kTQ / G);
    const bool pair = p.nrt > 1;
    p.nu = pair ? (p.nrt + 1) / 2 : 1;
    p.W = d.Hk * p.nu * p.nkt;
    int grid = s.num_sms < kSharedMaxGrid ? s.num_sms : kSharedMaxGrid;
    if (grid > p.W) grid = p.W;
    const SharedLayout L = shared_layout(d.B, d.H, d.Hk, D, s.P);
    p.po = reinterpret_cast<float*>(s.ws + L.po);
    p.pm = reinterpret_cast<float2*>(s.ws + L.pm);
    p.slopes = d.slopes;
    p.err = s.err;
    p.B = d.B;
    p.H = d.H;
    p.Hk = d.Hk;
    p.G = G;
    p.P = s.P;
    p.scale = d.scale;
    p.alibi = d.alibi;
    cudaError_t e;
    if (p.W) {
        if (pair)
            e = d.alibi ? launch_prefix<T, D, true, true>(dt, s, p, grid, st)
                        : launch_prefix<T, D, false, true>(dt, s, p, grid, st);
        else
            e = d.alibi ? launch_prefix<T, D, true, false>(dt, s, p, grid, st)
                        : launch_prefix<T, D, false, false>(dt, s, p, grid, st);
        if (e != cudaSuccess) return e;
    }
    OwnArgs own{};
    own.po = reinterpret_cast<float*>(s.ws + L.own_po);
    own.pm = reinterpret_cast<float2*>(s.ws + L.own_pm);
    own.cum = reinterpret_cast<int32_t*>(s.ws + L.cum);
    own.lens = d.lens;
    own.slopes = d.slopes;
    own.err = s.err;
    own.B = d.B;
    own.H = d.H;
    own.Hk = d.Hk;
    own.S_max = d.S_max;
    own.after_prefix = p.W != 0;
    own.grid = 2 * s.num_sms < kOwnMaxGrid ? 2 * s.num_sms : kOwnMaxGrid;
    own.scale = d.scale;
    own.alibi = d.alibi;
    e = launch_attention_own(dt, own, D, d.q, d.k, d.v, st);
    if (e != cudaSuccess) return e;
    CombineArgs c{};
    c.po = p.po;
    c.pm = p.pm;
    c.own_po = own.po;
    c.own_pm = own.pm;
    c.cum = own.cum;
    c.own_grid = own.grid;
    c.lens = d.lens;
    c.slopes = d.slopes;
    c.o = d.o;
    c.B = d.B;
    c.H = d.H;
    c.G = G;
    c.max_seq = d.S_max;
    c.alibi = d.alibi;
    c.nkt = p.nkt;
    c.nu = p.nu;
    c.rows = pair ? 2 * kTQ : kTQ;
    c.W = p.W;
    c.grid = grid;
    c.pdl = pdl_allowed(st);
    const int64_t warps = static_cast<int64_t>(d.B) * d.H;
    return launch_pdl(c.pdl != 0, shared_combine_kernel<T, D>,
                      dim3(static_cast<unsigned>((warps + 3) / 4)), dim3(128), 0, st, c);
}

}  // namespace

SharedLayout shared_layout(int64_t B, int64_t H, int64_t Hk, int64_t d, int64_t P) {
    const int64_t G = H / Hk, nrt = (B + kTQ / G - 1) / (kTQ / G);
    const int64_t nu = nrt > 1 ? (nrt + 1) / 2 : 1, rows = nrt > 1 ? 2 * kTQ : kTQ;
    const int64_t recs = P ? (kSharedMaxGrid + Hk * nu) * rows : 0;
    auto up = [](int64_t n) { return (n + 255) / 256 * 256; };
    SharedLayout L;
    L.po = 0;
    L.pm = up(recs * d * 4);
    L.own_po = L.pm + up(recs * 8);
    const int64_t own = (kOwnMaxGrid + B * Hk) * G;
    L.own_pm = L.own_po + up(own * d * 4);
    L.cum = L.own_pm + up(own * 8);
    L.total = L.cum + up((B + 1) * 4);
    return L;
}

int64_t shared_tiles(int64_t B, int64_t H, int64_t Hk, int64_t P) {
    const int64_t G = H / Hk;
    return Hk * ((B + kTQ / G - 1) / (kTQ / G)) * ((P + kTK - 1) / kTK);
}

cudaError_t launch_attention_decode_shared(DType dt, const SharedArgs& s, cudaStream_t st) {
    if (dt == DType::F16)
        return s.own.d == 64 ? launch_t<__half, 64>(dt, s, st) : launch_t<__half, 128>(dt, s, st);
    return s.own.d == 64 ? launch_t<__nv_bfloat16, 64>(dt, s, st)
                         : launch_t<__nv_bfloat16, 128>(dt, s, st);
}

}  // namespace blk
