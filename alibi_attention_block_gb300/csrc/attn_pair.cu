// K3 at head_dim 64: causal softmax attention on tcgen05 tensor cores, two
// 128-query tiles per work item.
//
// At head_dim 64 a 128x128 score tile costs 64 FLOP of MMA per exponential,
// so the softmax (one ex2 per score, 32 per clock per SM) and the tensor core
// take about as long as each other on a tile: the kernel has to keep both busy
// at once. Each CTA owns one SM and works on a pair of query tiles A = 2i and
// B = 2i + 1 of one (batch, head); they share every K/V tile, and while one
// tile's exponentials are computed the tensor core runs the other tile's
// products. The MMA thread issues, per key tile j,
//     S_A(j+1) = Q_A K_{j+1}^T,  O_A += P_A(j) V_j,  S_B(j+1),  O_B += P_B(j) V_j
// so the scores of the next tile are ready when a softmax warpgroup finishes
// the current one (each query tile's products come from its own issuing
// thread, in that order). 12 warps:
//   warp 0      TMA: both Q tiles of an item (double-buffered across items),
//               then K and V tiles of 128 keys into a four-stage ring
//               (128-byte swizzle, 64-column boxes, zero fill past S). K
//               and V load with an evict-last L2 policy (the head's other
//               query-tile pairs read the same key prefix), Q evict-first.
//   warps 1, 2  one MMA-issuing thread per query tile (M=128, K=16 per
//               instruction): S (N=128) from Q and K in shared memory, PV
//               (N=64) from P in TMEM and V in shared memory (V MN-major).
//               An MMA issue returns only about when the tensor core takes
//               it, and a barrier test costs on the order of a hundred
//               clocks, so one issuing thread that waits between groups
//               leaves the tensor core idle; with one thread per query tile
//               the other tile's products fill those gaps. Warp 1 also
//               allocates TMEM.
//               Keeping P out of shared memory matters: the tensor core's
//               operand reads, the TMA writes and any P traffic share the
//               SM's shared-memory bandwidth, and an all-shared-memory PV
//               would make that the bound.
//   warp 3      idle.
//   warps 4..7  softmax of tile A, one thread per query row (TMEM lane);
//   warps 8..11 softmax of tile B. Per key tile: one tcgen05.ld of the row's
//               128 scores (the S buffer is released at once), the causal
//               mask on the diagonal (and ragged last) tile only, the row max
//               (3-input max), one paired (f32x2) FMA per two scores into ex2
//               (scale log2(e)/sqrt(d) folded in; for ALiBi the bias
//               -slope*(i-j), "Bloom in a sovereign engine", Contribution,
//               enters as +slope*j, the -slope*i part being constant along
//               the row), P rounded to the storage type and held in
//               registers until the previous PV has read this tile's P
//               columns in TMEM, so the exponentials overlap that PV.
//               O is rescaled in TMEM only when the running max
//               grows by more than 2^8. An item's O / l is read out of TMEM
//               and written as [B, S, H, d] during the first tile of the
//               warpgroup's next item, so no softmax waits on a last PV.
// TMEM columns: S_A [0, 128), S_B [128, 256), P_A [256, 320), P_B [320, 384)
// (two 16-bit values per column), O_A [384, 448), O_B [448, 512).
// Items are (query-tile pair, batch, head), heaviest pairs first, dealt to
// the persistent CTAs in alternating directions.
// Query scale head_dim^-0.5 and GQA (kv head = h / (H/Hk)) follow nnterp
// "stablelm" 03 Notes.
#include "attn_plan.cuh"
#include "internal.h"

namespace blk {

namespace {

constexpr int kPairThreads = 384;
constexpr int kTQ = 128;  // query rows per tile
constexpr int kTK = 128;  // keys per tile
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kRescaleThreshold = 8.0f;  // log2 of the largest unnormalised p
// per-thread registers: at launch (65536 / 384, rounded down to a multiple of
// 8), and after the split for warpgroup 0 and for the softmax warpgroups
constexpr uint32_t kLaunchRegs = 168, kRegsControl = 64, kRegsSoftmax = 208;

template <int D>
struct PairCfg {
    static_assert(D == 64, "the pair kernel is built for head_dim 64");
    static constexpr int kSub = D / 64;                 // 64-column boxes per row
    static constexpr int kQBytes = kSub * kTQ * 128;    // one Q tile
    static constexpr int kKVBytes = kSub * kTK * 128;   // one K or V tile
    static constexpr int kQBufs = 2;
    static constexpr int kStages = 4;
    static constexpr int kOffKV = kQBufs * 2 * kQBytes;
    static constexpr int kOffBar = kOffKV + kStages * 2 * kKVBytes;
    // ALiBi: per softmax warpgroup an mbarrier (its four warps' arrivals)
    // and two 128-float tables slope*log2(e)*i (i = key column within a
    // tile), one per item parity
    static constexpr int kOffTabBar = kOffBar + 256;
    static constexpr int kOffBias = kOffTabBar + 16;
    // packed prompts: one more barrier per V stage; and one for the end
    static constexpr int kOffVReady = kOffBias + 2 * 2 * kTK * 4;
    static constexpr int kOffDrain = kOffVReady + 8 * kStages;
    static constexpr int kSmem = kOffDrain + 8 + 1024;  // + alignment slack
    static constexpr uint32_t kColP = 256;              // P_x at kColP + 64 x
    static constexpr uint32_t kColO = 384;              // O_x at kColO + D x
    static constexpr uint32_t kTmemCols = 512;
};

// This CTA's items: (pair i, batch b, head h), pair i = query tiles 2i and
// 2i+1 (the second absent when the tile count is odd and i is the last pair).
// Round r gives item r*G + blockIdx on even rounds and r*G + G-1-blockIdx on
// odd ones; items are numbered heaviest pair first.
//
// Packed prompts (PACKED): items are (unit, head); a unit is a query-tile
// pair of one prompt, from the plan's list (heaviest first), and the prompt's
// nP prefix tiles come ahead of its own key tiles. A prompt's tiles are paired
// from its end, so that where their number is odd the single one is the first,
// which has one key tile, and not the last, which has all (17 tiles: 81 steps for
// 89). 32 x 64 heads: two prompts of 8192 and 5330 tokens 389 us, 1.01 PFLOP/s (the
// dense kernel 1.04 at S = 8192); eight of 1273 on average 98.8 us, 0.66. As there, each
// query tile's chain of scores, softmax and product is the bound. Shortening it did
// not pay: a row's softmax in two halves on 16 warps, with an exchange of the maxima,
// 487 us; P handed over in two halves of the tile, 397.
template <bool PACKED>
struct PairCursor {
    using Plan = typename PlanStorage<PACKED>::type;
    int item, it, i, b, h, g, nA, nB;
    bool valid;
    // packed: the prompt's first row and length, the prefix's key tiles; t0:
    // query tile A (B is t0 + 1)
    int start_row, len, nP, prefix, t0;
    __device__ __forceinline__ int item_of(int round) const {
        const int G = static_cast<int>(gridDim.x), c = static_cast<int>(blockIdx.x);
        return round * G + ((round & 1) ? G - 1 - c : c);
    }
    __device__ __forceinline__ void decode(const AttnArgs& a, const AttnPack<PACKED>& pack,
                                           const Plan& plan, int nq, int np) {
        if constexpr (PACKED) {
            const PlanUnit u = plan_unit(pack, plan, item / a.H);
            h = item % a.H;
            b = 0;
            g = h / (a.H / a.Hk);
            start_row = u.first;
            len = u.len;
            i = u.l;
            prefix = pack.prefix;
            nP = (prefix + kTK - 1) / kTK;
            const bool odd = ((len + kTQ - 1) / kTQ) & 1;
            t0 = odd ? max(2 * i - 1, 0) : 2 * i;
            nA = nP + t0 + 1;
            nB = odd && i == 0 ? 0 : nP + t0 + 2;
            return;
        }
        const int bh_count = a.B * a.H;
        i = np - 1 - item / bh_count;
        const int bh = item % bh_count;
        b = bh / a.H;
        h = bh - b * a.H;
        g = h / (a.H / a.Hk);
        nA = 2 * i + 1;                          // key tiles of query tile 2i
        nB = (2 * i + 1 < nq) ? 2 * i + 2 : 0;   // of query tile 2i+1, if present
    }
    __device__ __forceinline__ void start(const AttnArgs& a, const AttnPack<PACKED>& pack,
                                         const Plan& plan, int nq, int np, int n_items) {
        it = 0;
        item = item_of(0);
        valid = item < n_items;
        if (valid) decode(a, pack, plan, nq, np);
    }
    __device__ __forceinline__ void next(const AttnArgs& a, const AttnPack<PACKED>& pack,
                                         const Plan& plan, int nq, int np, int n_items) {
        ++it;
        item = item_of(it);
        valid = item < n_items;
        if (valid) decode(a, pack, plan, nq, np);
    }
    __device__ __forceinline__ int n_kv() const { return nB ? nB : nA; }
};

template <typename T, int D, bool ALIBI, bool PACKED>
__global__ void __launch_bounds__(kPairThreads, 1)
    attn_pair_kernel(const __grid_constant__ CUtensorMap tmQ,
                     const __grid_constant__ CUtensorMap tmK,
                     const __grid_constant__ CUtensorMap tmV, const AttnArgs a,
                     const __grid_constant__ AttnPack<PACKED> pack) {
    using Cfg = PairCfg<D>;
    constexpr int kStages = Cfg::kStages;
    // With ALiBi the key tiles are walked from the diagonal down: the bias
    // +slope*j is largest there, so the row max is set by the first tile and
    // the O rescale (max grown past 2^8) stays rare; walked upwards, the max
    // rises by slope*128*log2(e) per tile, past 2^8 on most tiles for
    // slopes above 1/23.
    constexpr bool kRev = ALIBI;
    extern __shared__ uint8_t smem_raw[];
    __shared__ typename PlanStorage<PACKED>::type plan;
    uint8_t* smem = align_1024(smem_raw);
    const uint32_t sQ = smem_u32(smem);      // Q[buf][x] at (2 buf + x) tiles
    const uint32_t sKV = sQ + Cfg::kOffKV;   // stage s: K at 2s, V at 2s + 1 tiles
    const uint32_t bar0 = sQ + Cfg::kOffBar;
    // barriers (8 bytes each); x = 0 for query tile A, 1 for B
    auto s_full = [&](int x) { return bar0 + 8u * x; };
    auto s_free = [&](int x) { return bar0 + 16u + 8u * x; };
    auto p_full = [&](int x) { return bar0 + 32u + 8u * x; };
    auto pv_done = [&](int x) { return bar0 + 48u + 8u * x; };
    auto o_free = [&](int x) { return bar0 + 64u + 8u * x; };
    auto q_full = [&](int i) { return bar0 + 80u + 8u * i; };
    auto q_empty = [&](int i) { return bar0 + 96u + 8u * i; };
    auto k_full = [&](int i) { return bar0 + 112u + 8u * i; };
    auto v_full = [&](int i) { return bar0 + 112u + 8u * (kStages + i); };
    auto k_empty = [&](int i) { return bar0 + 112u + 8u * (2 * kStages + i); };
    auto v_empty = [&](int i) { return bar0 + 112u + 8u * (3 * kStages + i); };
    // packed: V tile i is ready once warp 3 has seen it land and cleared the
    // rows behind the prompt's end
    auto v_ready = [&](int i) { return PACKED ? sQ + Cfg::kOffVReady + 8u * i : v_full(i); };
    const uint32_t drain = sQ + Cfg::kOffDrain;
    uint32_t* tmem_slot =
        reinterpret_cast<uint32_t*>(smem + Cfg::kOffBar + 112 + 32 * kStages);

    const int warp = threadIdx.x / 32;
    const int lane = threadIdx.x & 31;
    const int nq = (a.S + kTQ - 1) / kTQ;
    const int np = (nq + 1) / 2;
    int n_items = np * a.B * a.H;

    if (threadIdx.x == 0) {
        for (int x = 0; x < 2; ++x) {
            mbar_init(s_full(x), 1);
            mbar_init(s_free(x), 4);
            mbar_init(p_full(x), 4);
            mbar_init(pv_done(x), 1);
            mbar_init(o_free(x), 4);
            mbar_init(q_full(x), 1);
            mbar_init(q_empty(x), 2);
        }
        mbar_init(drain, 2);
        if (ALIBI)
            for (int x = 0; x < 2; ++x) mbar_init(sQ + Cfg::kOffTabBar + 8u * x, 4);
        for (int i = 0; i < kStages; ++i) {
            mbar_init(k_full(i), 1);
            mbar_init(v_full(i), 1);
            mbar_init(k_empty(i), 2);
            mbar_init(v_empty(i), 2);
            if (PACKED) mbar_init(v_ready(i), 1);
        }
        fence_barrier_init();
        tma_prefetch_desc(&tmQ);
        tma_prefetch_desc(&tmK);
        tma_prefetch_desc(&tmV);
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(tmem_slot), Cfg::kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    if (a.pdl) {  // launched for programmatic dependent launch
        pdl_wait();  // inputs written by the previous kernel are visible from here on
        pdl_launch_dependents();
    }
    if constexpr (PACKED) {
        if (!pack.plan) build_plan(plan, pack.cu_seqlens, pack.prompts, a.S, 2 * kTQ, kTQ);
        n_items = plan_units(pack, plan) * a.H;
    }
    // registers: the launch gives every thread kLaunchRegs; warpgroup 0 (TMA,
    // MMA issue) gives most of its share to the two softmax warpgroups, which
    // hold a row's 128 scores and 64 packed probabilities at once
    static_assert(4 * kRegsControl + 8 * kRegsSoftmax <= 12 * kLaunchRegs,
                  "register split exceeds the launch's registers");
    if (warp < 4) {
        setmaxnreg_dec<kRegsControl>();
    if (warp == 0) {
        if (lane == 0) {
            const uint64_t pol_kv = l2_evict_last_policy(), pol_q = l2_evict_first_policy();
            PairCursor<PACKED> c;
            c.start(a, pack, plan, nq, np, n_items);
            int gkv = 0;   // K/V tiles loaded so far (ring position)
            int half = 0;  // 1: and a K tile without its V
            bool ok = true;
            while (ok && c.valid) {
                const int qb = c.it & 1;
                if (!mbar_wait_inl(q_empty(qb), ((c.it >> 1) & 1) ^ 1u, a.err)) break;
                mbar_expect_tx(q_full(qb), (c.nB ? 2 : 1) * Cfg::kQBytes);
                for (int x = 0; x < (c.nB ? 2 : 1); ++x) {
#pragma unroll
                    for (int sub = 0; sub < Cfg::kSub; ++sub)
                        tma_load_3d_hint(sQ + (2 * qb + x) * Cfg::kQBytes + sub * kTQ * 128, &tmQ,
                                    q_full(qb), sub * 64, PACKED ? c.start_row + (c.t0 + x) * kTQ : (2 * c.i + x) * kTQ,
                                    c.b * a.H + c.h, pol_q);
                }
                const int nkv = c.n_kv();
                for (int j = 0; j < nkv; ++j, ++gkv) {
                    const int kt = kRev ? nkv - 1 - j : j;  // key tile of shared step j
                    const int st = gkv % kStages;
                    const uint32_t ph = (gkv / kStages) & 1;
                    const uint32_t sK = sKV + (2 * st) * Cfg::kKVBytes;
                    const CUtensorMap *mK = &tmK, *mV = &tmV;
                    int krow = kt * kTK;
                    if constexpr (PACKED) {
                        if (kt < c.nP) {
                            mK = &pack.tmPK;
                            mV = &pack.tmPV;
                        } else {
                            krow = c.start_row + (kt - c.nP) * kTK;
                        }
                    }
                    if (!mbar_wait_inl(k_empty(st), ph ^ 1u, a.err)) {
                        ok = false;
                        break;
                    }
                    mbar_expect_tx(k_full(st), Cfg::kKVBytes);
#pragma unroll
                    for (int sub = 0; sub < Cfg::kSub; ++sub)
                        tma_load_3d_hint(sK + sub * kTK * 128, mK, k_full(st), sub * 64, krow,
                                    c.b * a.Hk + c.g, pol_kv);
                    if (!mbar_wait_inl(v_empty(st), ph ^ 1u, a.err)) {
                        half = 1;
                        ok = false;
                        break;
                    }
                    mbar_expect_tx(v_full(st), Cfg::kKVBytes);
#pragma unroll
                    for (int sub = 0; sub < Cfg::kSub; ++sub)
                        tma_load_3d_hint(sK + Cfg::kKVBytes + sub * kTK * 128, mV, v_full(st),
                                    sub * 64, krow, c.b * a.Hk + c.g, pol_kv);
                }
                c.next(a, pack, plan, nq, np, n_items);
            }
            // whatever the others met, no copy lands behind this block's end:
            // the last fill of each K, V and Q buffer. One wait in the code: with
            // a loop for each kind, and the products' wait in their threads'
            // branch, the whole kernel ran 0.5 to 2% longer
#pragma unroll 1
            for (int i = 0; i < 2 * kStages + 2; ++i) {
                const bool q = i >= 2 * kStages;  // v_full(0) is k_full(kStages)
                const int buf = i % kStages;
                const int fills = q ? (c.it + 1 - (i & 1)) / 2
                                    : (gkv + (i < kStages ? half : 0) + kStages - 1 - buf) / kStages;
                if (fills > 0)
                    mbar_wait_inl(q ? q_full(i & 1) : k_full(0) + 8u * i, (fills - 1) & 1, a.err);
            }
        }
    } else if (warp == 1 || warp == 2) {
        if (lane == 0) {
            // MMA issuer of query tile x (warp 1: A, warp 2: B). Two issuing
            // threads keep the tensor core fed while either one waits on a
            // barrier; each commits to the shared K/V and Q release barriers
            // (count 2), also for key tiles its query tile does not use.
            const int x = warp - 1;
            constexpr uint32_t fmt = dt_traits<T>::mma_fmt;
            constexpr uint32_t idesc_s = make_idesc_f16(fmt, kTQ, kTK, false);
            constexpr uint32_t idesc_o = make_idesc_f16(fmt, kTQ, D, true);
            constexpr uint64_t kQStep = Cfg::kQBytes >> 4;
            constexpr uint64_t kStageStep = (2 * Cfg::kKVBytes) >> 4;
            constexpr uint64_t kAtom = (kTQ * 128) >> 4;  // next 64-column atom
            const uint64_t dq0 = make_sdesc_sw128(sQ, 16, 1024) + x * kQStep;
            const uint64_t dk0 = make_sdesc_sw128(sKV, 16, 1024);
            const uint64_t dv0 = make_sdesc_sw128(sKV + Cfg::kKVBytes, kTK * 128, 1024);
            const uint32_t tS = tmem_base + 128u * x;
            const uint32_t tP = tmem_base + Cfg::kColP + 64u * x;
            const uint32_t tO = tmem_base + Cfg::kColO + D * x;
            int gs = 0, gp = 0, itx = 0;  // S and PV tiles issued, items with this tile
            // S_x = Q_x K^T, once the softmax has read the previous S_x
            auto issue_s = [&](uint64_t dq, uint64_t dk) -> bool {
                if (gs > 0 && !mbar_wait_inl(s_free(x), (gs - 1) & 1, a.err)) return false;
                tc_fence_after();
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks) {
                    const uint64_t off = (ks / 4) * kAtom + (ks % 4) * 2;
                    tc_mma_ss(tS, dq + off, dk + off, idesc_s, ks > 0 ? 1u : 0u);
                }
                tc_commit(s_full(x));
                ++gs;
                return true;
            };
            // O_x += P_x V once the softmax has written P_x (the first PV of an
            // item overwrites O_x, so it also waits for the previous read-out)
            auto issue_pv = [&](uint64_t dv, bool first) -> bool {
                if (!mbar_wait_inl(p_full(x), gp & 1, a.err)) return false;
                if (first && itx > 0 && !mbar_wait_inl(o_free(x), (itx - 1) & 1, a.err)) return false;
                tc_fence_after();
#pragma unroll
                for (int ks = 0; ks < kTK / 16; ++ks)
                    tc_mma_ts(tO, tP + ks * 8, dv + ks * ((16 * 128) >> 4), idesc_o,
                              (!first || ks > 0) ? 1u : 0u);
                tc_commit(pv_done(x));
                ++gp;
                return true;
            };
            PairCursor<PACKED> c;
            c.start(a, pack, plan, nq, np, n_items);
            int gkv = 0;
            bool ok = true;
            while (ok && c.valid) {
                const int qb = c.it & 1;
                const int nx = x ? c.nB : c.nA, nkv = c.n_kv();
                // this tile's shared steps [lo, hi): the first nx in key order,
                // the last nx when the walk runs down from the diagonal
                const int lo = kRev ? nkv - nx : 0, hi = kRev ? nkv : nx;
                const int qlast = nx > 0 ? hi - 1 : 0;  // Q_x is released after this step's S
                if (!mbar_wait_inl(q_full(qb), (c.it >> 1) & 1, a.err)) break;
                const uint64_t dq = dq0 + (2 * qb) * kQStep;
                // S of step 0
                {
                    const int st = gkv % kStages;
                    if (!mbar_wait_inl(k_full(st), (gkv / kStages) & 1, a.err)) break;
                    if (lo == 0 && nx > 0 && !issue_s(dq, dk0 + st * kStageStep)) break;
                    tc_commit(k_empty(st));
                    if (qlast == 0) tc_commit(q_empty(qb));
                }
                for (int j = 0; j < nkv; ++j) {
                    const int gj = gkv + j;
                    const int stj = gj % kStages;
                    if (j + 1 < nkv) {
                        // S of step j+1 ahead of PV of step j
                        const int stn = (gj + 1) % kStages;
                        if (!mbar_wait_inl(k_full(stn), ((gj + 1) / kStages) & 1, a.err)) {
                            ok = false;
                            break;
                        }
                        if (j + 1 >= lo && j + 1 < hi && !issue_s(dq, dk0 + stn * kStageStep)) {
                            ok = false;
                            break;
                        }
                        tc_commit(k_empty(stn));
                        if (j + 1 == qlast) tc_commit(q_empty(qb));
                    }
                    if (!mbar_wait_inl(v_ready(stj), (gj / kStages) & 1, a.err)) {
                        ok = false;
                        break;
                    }
                    if (j >= lo && j < hi && !issue_pv(dv0 + stj * kStageStep, j == lo)) {
                        ok = false;
                        break;
                    }
                    tc_commit(v_empty(stj));
                }
                gkv += nkv;
                if (nx > 0) ++itx;
                c.next(a, pack, plan, nq, np, n_items);
            }
            tc_commit(drain);
        }
    } else if constexpr (PACKED) {
        // warp 3: passes each V tile on once it has landed, the rows behind
        // the prompt's end (the next prompt's) cleared: their P is 0, but 0
        // times a non-finite value of another prompt is not
        PairCursor<PACKED> c;
        c.start(a, pack, plan, nq, np, n_items);
        int gkv = 0;
        bool ok = true;
        while (ok && c.valid) {
            const int nkv = c.n_kv();
            for (int j = 0; j < nkv; ++j, ++gkv) {
                const int kt = kRev ? nkv - 1 - j : j;
                const int st = gkv % kStages;
                if (!mbar_wait_inl(v_full(st), (gkv / kStages) & 1, a.err)) {
                    ok = false;
                    break;
                }
                const int rows = kt < c.nP ? kTK : c.len - (kt - c.nP) * kTK;
                if (rows < kTK)
                    clear_tile_rows<Cfg::kSub>(sKV + (2 * st + 1) * Cfg::kKVBytes, kTK, rows, lane);
                __syncwarp();
                if (lane == 0) mbar_arrive(v_ready(st));
            }
            c.next(a, pack, plan, nq, np, n_items);
        }
    }
    } else {
        setmaxnreg_inc<kRegsSoftmax>();
        // softmax: warpgroup x = 0 (warps 4..7) for tile A, 1 (8..11) for B;
        // warp w reads TMEM lanes 32 (w % 4) .. +31, one query row per thread
        const int x = (warp - 4) >> 2;
        const int quarter = warp & 3;
        const int row = quarter * 32 + lane;
        const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
        const uint32_t tS = tmem_base + 128u * x;
        const uint32_t tO = tmem_base + Cfg::kColO + D * x;
        const uint32_t tP = tmem_base + Cfg::kColP + 64u * x;
        const float scale_l2 = a.scale * kLog2e;
        PairCursor<PACKED> c;
        c.start(a, pack, plan, nq, np, n_items);
        int g = 0;  // key tiles processed (across items)
        bool ok = true;
        // The read-out of an item's O waits for its last PV; it is deferred to
        // the first tile of this warpgroup's next item (after that tile's
        // exponentials), so the next item's softmax overlaps the last PV.
        bool pend = false;  // an item's O is still in TMEM
        float pend_l = 0.f;
        int64_t pend_row = -1;  // output row (b * S + qpos) * H + h, or -1 past S
        int n_done = 0;         // items this warpgroup has started (ALiBi table parity)
        while (ok && c.valid) {
            const int nx = x ? c.nB : c.nA;
            if (nx == 0) {
                c.next(a, pack, plan, nq, np, n_items);
                continue;
            }
            const int qt = (PACKED ? c.t0 : 2 * c.i) + x;
            const int qpos = qt * kTQ + row;
            float m_used = -INFINITY;  // running max, log2 domain
            float l = 0.f;
            float slope_l2 = 0.f;
            uint32_t bias_tab = 0;
            if constexpr (ALIBI) {
                const float slope = a.slopes ? a.slopes[c.h]
                                             : exp2f(-8.0f * static_cast<float>(c.h + 1) /
                                                     static_cast<float>(a.H));
                slope_l2 = slope * kLog2e;
                // the item's column bias table, in the buffer the warpgroup's
                // previous item did not use (its last readers may still be on
                // that item); each warp's arrival publishes its 32 entries,
                // and no warp reads before all four have arrived
                const int off = Cfg::kOffBias + (2 * x + (n_done & 1)) * kTK * 4;
                reinterpret_cast<float*>(smem + off)[row] = slope_l2 * static_cast<float>(row);
                bias_tab = sQ + off;
                const uint32_t tab_bar = sQ + Cfg::kOffTabBar + 8u * x;
                __syncwarp();
                if (lane == 0) mbar_arrive(tab_bar);
                if (!mbar_wait_inl(tab_bar, n_done & 1, a.err)) {
                    ok = false;
                    break;
                }
            }
            ++n_done;
            for (int j = 0; j < nx; ++j, ++g) {
                if (!mbar_wait_inl(s_full(x), g & 1, a.err,
                                   PACKED ? idle_limit_ns(c.it, c.nP) : kWaitLimitNs)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                uint32_t r[kTK];
                tmem_ld128(tS + lane_off, r);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(s_free(x));
                const int kt = kRev ? nx - 1 - j : j;  // key tile of this step
                // packed ALiBi: key positions count from the query tile's first
                // (a row's constant), so that slope * position stays small,
                // hence exact, where its weight is not
                const int kbase = !PACKED        ? kt * kTK
                                  : kt >= c.nP ? (kt - c.nP - qt) * kTK
                                               : kt * kTK - c.prefix - qt * kTK;
                // ALiBi: u = s*scale*log2(e) + slope*log2(e)*i, one paired FMA
                // per two scores from the column table; the tile's uniform
                // part slope*log2(e)*kbase joins the max and the exponent
                const float sk = ALIBI ? slope_l2 * static_cast<float>(kbase) : 0.f;
                if constexpr (ALIBI) {
                    const uint64_t sc2 = f2_pack(scale_l2, scale_l2);
#pragma unroll
                    for (int i = 0; i < kTK; i += 4) {
                        uint64_t c01, c23;
                        ld_shared_v2_u64(bias_tab + i * 4, c01, c23);
                        float u0, u1, u2, u3;
                        ffma2(__uint_as_float(r[i]), __uint_as_float(r[i + 1]), sc2, c01, u0, u1);
                        ffma2(__uint_as_float(r[i + 2]), __uint_as_float(r[i + 3]), sc2, c23, u2,
                              u3);
                        r[i] = __float_as_uint(u0);
                        r[i + 1] = __float_as_uint(u1);
                        r[i + 2] = __float_as_uint(u2);
                        r[i + 3] = __float_as_uint(u3);
                    }
                }
                bool masked;
                int lim;  // keys <= lim are visible
                if constexpr (PACKED) {
                    const int kown = (kt - c.nP) * kTK;  // own key position, < 0 in the prefix
                    masked = kt >= c.nP ? kt - c.nP == qt || kown + kTK > c.len
                                        : (kt + 1) * kTK > c.prefix;
                    lim = kt >= c.nP ? min(qpos, c.len - 1) - kown : c.prefix - 1 - kt * kTK;
                } else {
                    masked = kt == qt || kbase + kTK > a.S;
                    lim = min(qpos, a.S - 1) - kbase;
                }
                if (masked) {
#pragma unroll
                    for (int i = 0; i < kTK; ++i)
                        if (i > lim) r[i] = __float_as_uint(-INFINITY);
                }
                float m0 = -INFINITY, m1 = -INFINITY, m2 = -INFINITY, m3 = -INFINITY;
#pragma unroll
                for (int i = 0; i < kTK; i += 8) {
                    m0 = fmax3f(m0, __uint_as_float(r[i]), __uint_as_float(r[i + 1]));
                    m1 = fmax3f(m1, __uint_as_float(r[i + 2]), __uint_as_float(r[i + 3]));
                    m2 = fmax3f(m2, __uint_as_float(r[i + 4]), __uint_as_float(r[i + 5]));
                    m3 = fmax3f(m3, __uint_as_float(r[i + 6]), __uint_as_float(r[i + 7]));
                }
                float mx = fmaxf(fmaxf(m0, m1), fmaxf(m2, m3));
                if constexpr (!ALIBI) mx *= scale_l2;  // scale > 0: max commutes with it
                if constexpr (ALIBI) mx += sk;
                float corr = 1.f;
                if (mx > m_used + kRescaleThreshold) {
                    corr = ex2_approx(m_used - mx);
                    m_used = mx;
                }
                // p = 2^(logit - m) in the storage type, and the row sum; P is
                // held in registers until the previous PV has read P_x. The
                // product takes P from TMEM in 16 bits, with V's type: each
                // weight is off by half a step at most, relative (2^-8 in bf16,
                // 2^-11 in fp16), about what the output's own rounding costs. The
                // sum takes the 32-bit weights
                const uint64_t mul2 = f2_pack(ALIBI ? 1.f : scale_l2, ALIBI ? 1.f : scale_l2);
                const float off = ALIBI ? sk - m_used : -m_used;
                const uint64_t neg2 = f2_pack(off, off);
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
                // the previous PV has read P_x and O_x is settled: read out the
                // previous item's O if pending, publish P_x, then rescale O if
                // the max moved (before this tile's PV)
                if (j > 0 || pend) {
                    if (!mbar_wait_inl(pv_done(x), (g - 1) & 1, a.err)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                }
                if (j == 0 && pend) {
                    uint32_t o[D];
                    tmem_ld64(tO + lane_off, o);
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(o_free(x));
                    if (pend_row >= 0) {
                        const float inv_l = 1.0f / pend_l;
                        T* dst = static_cast<T*>(a.o) + pend_row * static_cast<int64_t>(D);
#pragma unroll
                        for (int v = 0; v < D / 8; ++v) {
                            float f[8];
#pragma unroll
                            for (int e = 0; e < 8; ++e) f[e] = __uint_as_float(o[v * 8 + e]) * inv_l;
                            store8(dst + v * 8, f);
                        }
                    }
                    pend = false;
                }
                tmem_st64_nowait(tP + lane_off, pk);
                if (j > 0 && __any_sync(0xffffffffu, corr != 1.f)) {
#pragma unroll 1
                    for (int cc = 0; cc < D / 16; ++cc) {
                        uint32_t o[16];
                        const uint32_t col = tO + lane_off + cc * 16;
                        tmem_ld16(col, o);
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            o[i] = __float_as_uint(__uint_as_float(o[i]) * corr);
                        tmem_st16_nowait(col, o);
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
            pend = true;
            pend_l = l;
            if constexpr (PACKED)
                pend_row = qpos < c.len ? (static_cast<int64_t>(c.start_row) + qpos) * a.H + c.h : -1;
            else
                pend_row = qpos < a.S ? (static_cast<int64_t>(c.b) * a.S + qpos) * a.H + c.h : -1;
            c.next(a, pack, plan, nq, np, n_items);
        }
        // the last item's O
        if (ok && pend && mbar_wait_inl(pv_done(x), (g - 1) & 1, a.err)) {
            tc_fence_after();
            uint32_t o[D];
            tmem_ld64(tO + lane_off, o);
            tc_fence_before();
            if (pend_row >= 0) {
                const float inv_l = 1.0f / pend_l;
                T* dst = static_cast<T*>(a.o) + pend_row * static_cast<int64_t>(D);
#pragma unroll
                for (int v = 0; v < D / 8; ++v) {
                    float f[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) f[e] = __uint_as_float(o[v * 8 + e]) * inv_l;
                    store8(dst + v * 8, f);
                }
            }
        }
    }
    __syncthreads();
    if (warp == 1) {
        mbar_wait_inl(drain, 0, a.err);  // ... nor is a product still under way
        tc_fence_after();
        tmem_dealloc(tmem_base, Cfg::kTmemCols);
    }
}

template <typename T, bool ALIBI, bool PACKED>
cudaError_t launch_pair(DType dt, const AttnArgs& a, const AttnPack<PACKED>& pack, int64_t items,
                        cudaStream_t s) {
    constexpr int D = 64;
    using Cfg = PairCfg<D>;
    CUtensorMap tq, tk, tv;
    if (!make_tmap_3d(&tq, dt, a.q, static_cast<uint64_t>(a.B) * a.H, a.S, D, kTQ) ||
        !make_tmap_3d(&tk, dt, a.k, static_cast<uint64_t>(a.B) * a.Hk, a.S, D, kTK) ||
        !make_tmap_3d(&tv, dt, a.v, static_cast<uint64_t>(a.B) * a.Hk, a.S, D, kTK))
        return cudaErrorInvalidValue;
    auto kern = attn_pair_kernel<T, D, ALIBI, PACKED>;
    {
        const cudaError_t e = set_smem_attr_once(reinterpret_cast<const void*>(kern), Cfg::kSmem);
        if (e != cudaSuccess) return e;
    }
    if (items > 0x7fffffff) return cudaErrorInvalidValue;
    const int64_t grid = items < a.num_sms ? items : a.num_sms;
    AttnArgs ap = a;
    ap.pdl = pdl_allowed(s);
    (void)launch_pdl(ap.pdl != 0, kern, dim3(static_cast<unsigned>(grid)), dim3(kPairThreads), Cfg::kSmem, s,
                     tq, tk, tv, ap, pack);
    return cudaGetLastError();
}

template <bool PACKED>
cudaError_t launch_pair_t(DType dt, const AttnArgs& a, const AttnPack<PACKED>& pack, int64_t items,
                          cudaStream_t s) {
    if (dt == DType::F16)
        return a.alibi ? launch_pair<__half, true>(dt, a, pack, items, s)
                       : launch_pair<__half, false>(dt, a, pack, items, s);
    return a.alibi ? launch_pair<__nv_bfloat16, true>(dt, a, pack, items, s)
                   : launch_pair<__nv_bfloat16, false>(dt, a, pack, items, s);
}

}  // namespace

cudaError_t launch_attention_pair64(DType dt, const AttnArgs& a, cudaStream_t s) {
    if (a.d != 64) return cudaErrorInvalidValue;
    const int64_t nq = (a.S + kTQ - 1) / kTQ;
    return launch_pair_t(dt, a, AttnPack<false>{}, (nq + 1) / 2 * a.B * a.H, s);
}

cudaError_t launch_attention_pair64_packed(DType dt, const AttnArgs& a, const AttnPack<true>& pack,
                                           int64_t max_units, cudaStream_t s) {
    if (a.d != 64) return cudaErrorInvalidValue;
    return launch_pair_t(dt, a, pack, max_units * a.H, s);
}

}  // namespace blk
