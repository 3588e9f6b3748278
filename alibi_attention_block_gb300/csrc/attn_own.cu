// K6o: one decode step of attention over the sequences' own caches, as partial
// results (pass 2 of attn_shared.cu).
//
// A sequence's query heads of one kv head are few (G = 1 .. 8), its keys many:
// the pass is bound by the bytes of K and V. On the CUDA cores each key costs
// 4 d G flops and as many shared-memory reads and shuffles, which a G of 4 or
// 8 does not hide behind the bytes (measured: 2.0 TB/s at 32/8 heads x 128,
// 2.9 TB/s at 32 x 64). So the products run on the tensor cores with the roles
// turned: keys are the rows, heads the (padded) 16 columns,
//     S^T [128 keys, 16] = K Q^T,    O^T [d, 16] = V^T P^T,
// with K and V straight from the TMA tiles, one softmax thread per key, and
// the per-head maximum a warp reduction. An MMA's unused columns are whatever
// shared memory holds: columns do not mix, and none of them is read.
//
// Work: (sequence, kv head) units of ceil(len / 128) key tiles in one line,
// cut into equal ranges, one per CTA (two CTAs per SM); a CTA's stay in a unit
// is a segment with a partial result (max, sum, O) of its own. The lengths are
// device data: each CTA sums them itself to find its range, and CTA 0 leaves
// the running tile counts for the merge. Tiles go from the newest key down
// (with ALiBi the bias is largest there). A last, part-filled tile is loaded
// in boxes of 16 keys, multiplied over ceil(keys / 16) steps, and the values
// behind its end are cleared: 0 times what an unused cache entry holds need
// not be 0.
// 6 warps: TMA; MMA issue; four of softmax. The MMA thread issues what is ready
// first, S of the next tile or PV of this one: with S always ahead, a tile's PV
// waited for the next tile's keys to arrive (a memory latency per tile, 3000
// to 4000 clocks). A segment's O is read out during the next one's first tile.
// TMEM columns: S [0, 32) and O^T [32, 64), both double-buffered (by tile, by
// segment).
#include "internal.h"

namespace blk {

namespace {

constexpr int kThreads = 192;
constexpr int kTK = 128;  // keys per tile
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kRescaleThreshold = 8.0f;  // log2 of the largest unnormalised p

template <int D>
struct Cfg {
    static constexpr int kSub = D / 64;
    static constexpr int kTile = kSub * kTK * 128;
    static constexpr int kSlots = D == 64 ? 6 : 3;  // K and V tiles in flight: 96 KB
    // queries and weights: 8 rows of 128 bytes per 64 columns; the operands'
    // rows 8 .. 15 are what follows (any bytes will do)
    static constexpr int kQBytes = kSub * 1024, kPBytes = 2 * 1024;
    static constexpr int kOffQ = kSlots * kTile;
    static constexpr int kOffP = kOffQ + 2 * kQBytes;
    static constexpr int kOffMax = kOffP + 2 * kPBytes + 1024;  // [2][8][4] floats
    static constexpr int kOffSum = kOffMax + 2 * 8 * 4 * 4;     // [2][8][4] floats
    static constexpr int kOffBar = kOffSum + 2 * 8 * 4 * 4;
    static constexpr int kSmem = kOffBar + 512 + 1024;  // + alignment slack
    static_assert(kSmem <= 113 * 1024, "two CTAs per SM");
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

__device__ __forceinline__ int own_len(const OwnArgs& a, int b) {
    return min(max(a.lens[b], 0), a.S_max);
}

// A CTA's segments: tiles [t, t + n) of unit (b, g), key tiles first ..
// first + n - 1 of the unit; t counts all units' tiles.
struct Segments {
    int64_t t, end;
    int b, g, first, n, len, it;
    bool valid;
    __device__ __forceinline__ void set(const OwnArgs& a) {
        valid = t < end;
        if (!valid) return;
        const int left = (len + kTK - 1) / kTK - first;
        n = static_cast<int>(min(static_cast<int64_t>(left), end - t));
    }
    // base: tiles ahead of sequence b0's first unit; the range starts in b0
    __device__ __forceinline__ void start(const OwnArgs& a, int64_t lo, int64_t hi, int b0,
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
    __device__ __forceinline__ void next(const OwnArgs& a) {
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

template <typename T, int D, int G>
__global__ void __launch_bounds__(kThreads, 2)
    own_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
               const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmK16,
               const __grid_constant__ CUtensorMap tmV16, const OwnArgs a) {
    using C = Cfg<D>;
    constexpr int kSlots = C::kSlots;
    extern __shared__ uint8_t smem_raw[];
    __shared__ int64_t sh_lo, sh_hi, sh_base;
    __shared__ int sh_b0;
    __shared__ int sh_sum[kThreads / 32];
    uint8_t* smem = align_1024(smem_raw);
    const uint32_t sKV = smem_u32(smem);
    const uint32_t sQ = sKV + C::kOffQ, sP = sKV + C::kOffP;
    const uint32_t bar0 = sKV + C::kOffBar;
    auto full = [&](int i) { return bar0 + 8u * i; };
    auto empty = [&](int i) { return bar0 + 8u * (kSlots + i); };
    const uint32_t bar1 = bar0 + 16u * kSlots;
    auto q_full = [&](int i) { return bar1 + 8u * i; };
    auto q_empty = [&](int i) { return bar1 + 16u + 8u * i; };
    auto s_full = [&](int i) { return bar1 + 32u + 8u * i; };
    auto s_free = [&](int i) { return bar1 + 48u + 8u * i; };
    auto p_full = [&](int i) { return bar1 + 64u + 8u * i; };
    auto pv_done = [&](int i) { return bar1 + 80u + 8u * i; };
    auto o_free = [&](int i) { return bar1 + 96u + 8u * i; };
    const uint32_t max_full = bar1 + 112u, sum_full = bar1 + 120u;
    static_assert(16 * kSlots + 132 <= 512, "barrier space");
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffBar + 16 * kSlots + 128);

    const int warp = threadIdx.x / 32;
    const int lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kSlots; ++i) {
            mbar_init(full(i), 1);
            mbar_init(empty(i), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(q_full(i), 1);
            mbar_init(q_empty(i), 1);
            mbar_init(s_full(i), 1);
            mbar_init(s_free(i), 4);
            mbar_init(p_full(i), 4);
            mbar_init(pv_done(i), 1);
            mbar_init(o_free(i), 4);
        }
        mbar_init(max_full, 4);
        mbar_init(sum_full, 4);
        fence_barrier_init();
        tma_prefetch_desc(&tmQ);
        tma_prefetch_desc(&tmK);
        tma_prefetch_desc(&tmV);
        tma_prefetch_desc(&tmK16);
        tma_prefetch_desc(&tmV16);
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(tmem_slot), 64);
        tmem_relinquish();
    }
    // Behind the prefix pass there is nothing to wait for: that kernel lets
    // this one start only after its own wait, when everything enqueued before
    // it (the caches' writers, the previous merge, which reads this workspace)
    // has completed. The wait is made up for at the end, so that this grid's
    // completion stands for both.
    if (a.pdl) {
        if (!a.after_prefix) pdl_wait();
        pdl_launch_dependents();
    }
    // this CTA's range of tiles: thread i sums the tiles of a run of sequences
    const int per = (a.B + kThreads - 1) / kThreads;
    const int b_lo = min(static_cast<int>(threadIdx.x) * per, a.B), b_hi = min(b_lo + per, a.B);
    int mine = 0;
    for (int b = b_lo; b < b_hi; ++b) mine += (own_len(a, b) + kTK - 1) / kTK;
    int upto = mine;  // inclusive sum over the warp's threads, then over all
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += v;
    }
    if (lane == 31) sh_sum[warp] = upto;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    int before = upto - mine, total = 0;
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) {
        if (i < warp) before += sh_sum[i];
        total += sh_sum[i];
    }
    const int64_t W = static_cast<int64_t>(total) * a.Hk;
    // with fewer tiles than CTAs, one for each of the first W (the merge
    // counts on every CTA of a unit's span having some of it)
    const int64_t ctas = min(static_cast<int64_t>(gridDim.x), W), me = blockIdx.x;
    const int64_t lo = me < ctas ? me * W / ctas : 0, hi = me < ctas ? (me + 1) * W / ctas : 0;
    if (threadIdx.x == 0) {
        sh_lo = lo;
        sh_hi = hi;
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
        sh_b0 = b;
        sh_base = base;
    }
    if (blockIdx.x == 0) {
        int c = before;
        for (int b = b_lo; b < b_hi; ++b) {
            a.cum[b] = c;
            c += (own_len(a, b) + kTK - 1) / kTK;
        }
        if (threadIdx.x == 0) a.cum[a.B] = total;
    }
    __syncthreads();

    Segments c;
    c.start(a, sh_lo, sh_hi, sh_b0, sh_base);
    if (warp == 0) {
        if (lane == 0) {
            const uint64_t pol = l2_evict_first_policy();
            int r = 0;
            bool ok = true;
            while (ok && c.valid) {
                const int qb = c.it & 1;
                if (!mbar_wait(q_empty(qb), ((c.it >> 1) & 1) ^ 1u, a.err)) break;
                mbar_expect_tx(q_full(qb), G * 128 * C::kSub);
#pragma unroll
                for (int sub = 0; sub < C::kSub; ++sub)
                    tma_load_2d(sQ + qb * C::kQBytes + sub * 1024, &tmQ, q_full(qb), sub * 64,
                                c.b * a.H + c.g * G);
                for (int i = 0; i < c.n && ok; ++i) {
                    const int row = (c.first + c.n - 1 - i) * kTK;
                    const int keys = c.len - row;  // of this tile, if less than kTK
                    for (int kv = 0; kv < 2; ++kv, ++r) {
                        const int sl = r % kSlots;
                        if (!mbar_wait(empty(sl), ((r / kSlots) & 1) ^ 1u, a.err)) {
                            ok = false;
                            break;
                        }
                        const uint32_t dst = sKV + sl * C::kTile;
                        if (keys >= kTK) {
                            mbar_expect_tx(full(sl), C::kTile);
#pragma unroll
                            for (int sub = 0; sub < C::kSub; ++sub)
                                tma_load_3d_hint(dst + sub * kTK * 128, kv ? &tmV : &tmK, full(sl),
                                                 sub * 64, row, c.b * a.Hk + c.g, pol);
                        } else {
                            const int boxes = (keys + 15) / 16;
                            mbar_expect_tx(full(sl), boxes * 16 * 128 * C::kSub);
                            for (int x = 0; x < boxes; ++x)
#pragma unroll
                                for (int sub = 0; sub < C::kSub; ++sub)
                                    tma_load_3d_hint(dst + sub * kTK * 128 + x * 2048,
                                                     kv ? &tmV16 : &tmK16, full(sl), sub * 64,
                                                     row + x * 16, c.b * a.Hk + c.g, pol);
                        }
                    }
                }
                c.next(a);
            }
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
                return mbar_test(full(r % kSlots), (r / kSlots) & 1) &&
                       (!x.first || mbar_test(q_full(x.it & 1), (x.it >> 1) & 1)) &&
                       (x.t < 2 || mbar_test(s_free(x.t & 1), ((x.t >> 1) - 1) & 1));
            };
            auto issue_s = [&](const Tile& x) {
                tc_fence_after();
                const int sl = 2 * x.t % kSlots;
                const uint64_t dk = dk0 + sl * kSlotStep;
                const uint64_t dq = dq0 + (x.it & 1) * (C::kQBytes >> 4);
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks)
                    tc_mma_ss(tmem_base + 16u * (x.t & 1), dk + (ks / 4) * kAtom + (ks % 4) * 2,
                              dq + (ks / 4) * (1024 >> 4) + (ks % 4) * 2, idesc_s, ks > 0 ? 1u : 0u);
                tc_commit(s_full(x.t & 1));
                tc_commit(empty(sl));
                if (x.last) tc_commit(q_empty(x.it & 1));
            };
            // O^T += V^T P^T: the values and P are there, and (first tile) the O
            // buffer's last segment has been read out
            auto pv_ready = [&](const Tile& x) {
                const int r = 2 * x.t + 1;
                return mbar_test(full(r % kSlots), (r / kSlots) & 1) &&
                       mbar_test(p_full(x.t & 1), (x.t >> 1) & 1) &&
                       (!x.first || x.it < 2 || mbar_test(o_free(x.it & 1), ((x.it >> 1) - 1) & 1));
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
                        tc_mma_ss(tmem_base + 32u + 16u * (x.it & 1), dv + ks * ((16 * 128) >> 4),
                                  dp + (ks / 4) * (1024 >> 4) + (ks % 4) * 2, idesc_o,
                                  (!x.first || ks > 0) ? 1u : 0u);
                tc_commit(pv_done(x.t & 1));
                tc_commit(empty(sl));
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
        }
    } else {
        const int quarter = warp & 3;
        const int key = quarter * 32 + lane;  // TMEM lane: key of a tile
        // ... and row of O^T: head_dim 64 takes 16 lanes of each quarter
        const int dim = D == 64 ? quarter * 16 + lane : key;
        const bool has_dim = D != 64 || lane < 16;
        const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
        const uint32_t tS = tmem_base + lane_off, tO = tmem_base + lane_off + 32u;
        const float scale_l2 = a.scale * kLog2e;
        float* red_max = reinterpret_cast<float*>(smem + C::kOffMax);
        float* red_sum = reinterpret_cast<float*>(smem + C::kOffSum);
        int t = 0;
        bool ok = true;
        // a segment's O is in TMEM until its last PV has completed: read out
        // behind the next segment's first tile
        bool pend = false;
        int pend_t = 0, pend_buf = 0;
        int64_t pend_rec = 0;
        auto read_out = [&]() -> bool {
            if (!mbar_wait(pv_done(pend_t & 1), (pend_t >> 1) & 1, a.err)) return false;
            tc_fence_after();
            uint32_t o[G];
            tmem_ldn<G>(tO + 16u * pend_buf, o);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(o_free(pend_buf));
            if (has_dim) {
#pragma unroll
                for (int h = 0; h < G; ++h)
                    a.po[(pend_rec * G + h) * D + dim] = __uint_as_float(o[h]);
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
                if (!mbar_wait(s_full(t & 1), (t >> 1) & 1, a.err)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                uint32_t r[G];
                tmem_ldn<G>(tS + 16u * (t & 1), r);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(s_free(t & 1));
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
                if (lane == 0) mbar_arrive(max_full);
                if (!mbar_wait(max_full, t & 1, a.err)) {
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
                if (t > 1 && !mbar_wait(pv_done(t & 1), ((t >> 1) - 1) & 1, a.err)) {
                    ok = false;
                    break;
                }
                const uint32_t p_row = sP + (t & 1) * C::kPBytes + (key / 64) * 1024;
#pragma unroll
                for (int h = 0; h < G; ++h) {
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
                    if (!mbar_wait(full(sl), (rv / kSlots) & 1, a.err)) {
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
                    if (!mbar_wait(pv_done((t - 1) & 1), ((t - 1) >> 1) & 1, a.err)) {
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
                if (lane == 0) mbar_arrive(p_full(t & 1));
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
            if (lane == 0) mbar_arrive(sum_full);
            if (!mbar_wait(sum_full, c.it & 1, a.err)) {
                ok = false;
                break;
            }
            const int64_t rec = static_cast<int64_t>(blockIdx.x) +
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
                a.pm[rec * G + lane] = make_float2(mh, (w.x + w.y) + (w.z + w.w));
            }
            c.next(a);
        }
        if (ok && pend) read_out();
    }
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem_base, 64);
    }
    if (a.pdl && a.after_prefix) pdl_wait();
}

template <typename T, int D, int G>
cudaError_t launch_g(DType dt, const OwnArgs& a, const void* q, const void* k, const void* v,
                     cudaStream_t s) {
    using C = Cfg<D>;
    CUtensorMap tq, tk, tv, tk16, tv16;
    const uint64_t planes = static_cast<uint64_t>(a.B) * a.Hk;
    if (!make_tmap_2d(&tq, dt, q, static_cast<uint64_t>(a.B) * a.H, D, G) ||
        !make_tmap_3d(&tk, dt, k, planes, a.S_max, D, kTK) ||
        !make_tmap_3d(&tv, dt, v, planes, a.S_max, D, kTK) ||
        !make_tmap_3d(&tk16, dt, k, planes, a.S_max, D, 16) ||
        !make_tmap_3d(&tv16, dt, v, planes, a.S_max, D, 16))
        return cudaErrorInvalidValue;
    auto kern = own_kernel<T, D, G>;
    const cudaError_t e = set_smem_attr_once(reinterpret_cast<const void*>(kern), C::kSmem);
    if (e != cudaSuccess) return e;
    OwnArgs ap = a;
    ap.pdl = pdl_allowed(s);
    return launch_pdl(ap.pdl != 0, kern, dim3(a.grid), dim3(kThreads), C::kSmem, s, tq, tk, tv, tk16,
                      tv16, ap);
}

template <typename T, int D>
cudaError_t launch_d(DType dt, const OwnArgs& a, const void* q, const void* k, const void* v,
                     cudaStream_t s) {
    switch (a.H / a.Hk) {
        case 1: return launch_g<T, D, 1>(dt, a, q, k, v, s);
        case 2: return launch_g<T, D, 2>(dt, a, q, k, v, s);
        case 4: return launch_g<T, D, 4>(dt, a, q, k, v, s);
        case 8: return launch_g<T, D, 8>(dt, a, q, k, v, s);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace

cudaError_t launch_attention_own(DType dt, const OwnArgs& a, int d, const void* q, const void* k,
                                 const void* v, cudaStream_t s) {
    if (dt == DType::F16)
        return d == 64 ? launch_d<__half, 64>(dt, a, q, k, v, s)
                       : launch_d<__half, 128>(dt, a, q, k, v, s);
    return d == 64 ? launch_d<__nv_bfloat16, 64>(dt, a, q, k, v, s)
                   : launch_d<__nv_bfloat16, 128>(dt, a, q, k, v, s);
}

}  // namespace blk
