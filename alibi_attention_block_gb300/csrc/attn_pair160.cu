// K3 over packed prompts at head_dim 160: causal softmax attention on tcgen05
// tensor cores, two 128-row query tiles per work item.
//
// Two tiles' S, P and O fit TMEM's 512 columns at head_dim 160 with key tiles of
// 64: S_A [0, 64), S_B [64, 128), P_A [128, 160), P_B [160, 192) (16-bit pairs),
// O_A [192, 352), O_B [352, 512). So one tile's products run beside the other's
// softmax, and each tile's next scores beside its own, as in attn_pair.cu; with
// one tile of 128-key steps in flight (attn_gqa.cu) the chain of scores, softmax
// and product is the bound. Grouped heads are packed into a tile's rows as there.
// A 64-key score product reads its query tile from shared memory twice as often
// (N = 64: 52 clocks a K step of 16 for 66 at N = 128): 1,700 clocks of products per
// 128 keys for 1,320, but the chain left the tensor core idle for longer. Six
// prompts of 654 tokens on average, 32/8 x 160 heads: 74.9 us with one tile, 64.4
// with two; the narrower key tiles also waste less at the diagonal. (At head_dim
// 128, where a step of 128 keys fits, attn_pair128.cu is as fast or faster: 91.7 us
// for 91.8, 174 for 178.)
//
// The issuing threads are close to a bound: an iteration of S, PV, two barrier
// tests each and four commits took 2,235 clocks, of which the products 1,050. A
// test of a barrier that has completed costs some 110, a commit more. Two tests go
// out together, and the softmax passes the K tiles back: 67.6 -> 64.4 us.
// 12 warps:
//   warp 0      TMA: each query tile's Q (its own buffer, reloaded once the tile's
//               last S of the item has completed), K and V tiles into a ring of
//               three stages. The last 32 columns of Q and K are a slice of
//               64-byte rows with the 64-byte swizzle; V is padded to 192 columns.
//   warps 1, 2  one MMA-issuing thread per query tile: S (M=128, N=64), PV
//               (N=160: P from TMEM, V MN-major). Warp 1 also allocates TMEM.
//   warp 3      passes V tiles on, the rows behind the prompt's end cleared.
//   warps 4..7  softmax of tile A, 8..11 of tile B, one thread per row (see
//               attn_pair.cu).
// Query scale head_dim^-0.5 and GQA (kv head = h / (H/Hk)) follow nnterp
// "stablelm" 03 Notes; ALiBi "Bloom in a sovereign engine", Contribution.
#include "attn_plan.cuh"
#include "internal.h"

namespace blk {

namespace {

constexpr int kPair160Threads = 384;
constexpr int kTQ = 128;  // query rows per tile
constexpr int kTK = 64;   // keys per tile
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kRescaleThreshold = 8.0f;  // log2 of the largest unnormalised p
// per-thread registers, as in attn_pair128.cu
constexpr uint32_t kLaunchRegs = 168, kRegsControl = 96, kRegsSoftmax = 192;

constexpr int D = 160;

struct C {
    // whole 64-column slices of a row and a half one: 64-byte rows for Q and K,
    // padded to a whole slice for V
    static constexpr int kFull = D / 64, kSub = kFull + 1;
    static constexpr int kQBytes = kFull * kTQ * 128 + kTQ * 64;
    static constexpr int kKBytes = kFull * kTK * 128 + kTK * 64;
    static constexpr int kVBytes = kSub * kTK * 128;
    static constexpr int kStageBytes = kKBytes + kVBytes;
    static constexpr int kStages = 3;
    static constexpr int kOffKV = 2 * kQBytes;  // Q_A, Q_B
    static constexpr int kOffBar = kOffKV + kStages * kStageBytes;
    // ALiBi (one head a tile): per softmax warpgroup an mbarrier (its four
    // warps' arrivals) and two tables slope*log2(e)*i (i = key column within a
    // tile), one per item parity
    static constexpr int kOffTabBar = kOffBar + 512;
    static constexpr int kOffBias = kOffTabBar + 16;
    static constexpr int kSmem = kOffBias + 2 * 2 * kTK * 4 + 1024;  // + alignment slack
    static constexpr uint32_t kColP = 128;              // P_x at kColP + 32 x
    static constexpr uint32_t kColO = 192;              // O_x at kColO + D x
    static constexpr uint32_t kTmemCols = 512;
};

// This CTA's items: (unit of the plan's list, kv head, head chunk). A unit is a
// query-tile pair of one prompt, 2 R positions; row r of tile x is head g * G +
// hc * Gt + r / R at position (t0 + x) R + r % R (see attn_gqa.cu; R = 128 for
// MHA). Tiles are paired from the prompt's end (see attn_pair.cu). The prefix's
// nP key tiles come ahead of the prompt's own.
struct Cursor {
    int item, it, g, h, hc, start_row, len, nP, prefix, t0, nA, nB;
    bool valid;
    __device__ __forceinline__ void decode(const AttnArgs& a, const AttnPack<true>& pack,
                                           const PlanSmem& plan) {
        const int per_unit = a.Hk * pack.nhc;
        const PlanUnit u = plan_unit(pack, plan, item / per_unit);
        const int rest = item % per_unit;
        hc = rest % pack.nhc;
        g = rest / pack.nhc;
        h = g * pack.G + hc * pack.Gt;  // the tile's first head
        start_row = u.first;
        len = u.len;
        prefix = pack.prefix;
        nP = (prefix + kTK - 1) / kTK;
        const bool odd = ((len + pack.R - 1) / pack.R) & 1;
        t0 = odd ? max(2 * u.l - 1, 0) : 2 * u.l;
        const int endA = (t0 + 1) * pack.R;  // one past tile A's last position
        nA = nP + (min(endA, len) + kTK - 1) / kTK;
        nB = odd && u.l == 0 ? 0 : nP + (min(endA + pack.R, len) + kTK - 1) / kTK;
    }
    __device__ __forceinline__ void at(const AttnArgs& a, const AttnPack<true>& pack,
                                       const PlanSmem& plan, int round, int n_items) {
        const int G = static_cast<int>(gridDim.x), c = static_cast<int>(blockIdx.x);
        it = round;
        item = round * G + ((round & 1) ? G - 1 - c : c);
        valid = item < n_items;
        if (valid) decode(a, pack, plan);
    }
    __device__ __forceinline__ void start(const AttnArgs& a, const AttnPack<true>& pack,
                                          const PlanSmem& plan, int n_items) {
        at(a, pack, plan, 0, n_items);
    }
    __device__ __forceinline__ void next(const AttnArgs& a, const AttnPack<true>& pack,
                                         const PlanSmem& plan, int n_items) {
        at(a, pack, plan, it + 1, n_items);
    }
    __device__ __forceinline__ int n_kv() const { return nB ? nB : nA; }
};

template <typename T, bool ALIBI>
__global__ void __launch_bounds__(kPair160Threads, 1)
    attn_pair160_kernel(const __grid_constant__ CUtensorMap tmQ,
                        const __grid_constant__ CUtensorMap tmK,
                        const __grid_constant__ CUtensorMap tmV,
                        const __grid_constant__ CUtensorMap tmQ2,
                        const __grid_constant__ CUtensorMap tmK2, const AttnArgs a,
                        const __grid_constant__ AttnPack<true> pack) {
    constexpr int kStages = C::kStages;
    // ALiBi: key tiles from the diagonal down (see attn_pair.cu)
    constexpr bool kRev = ALIBI;
    extern __shared__ uint8_t smem_raw[];
    __shared__ PlanSmem plan;
    uint8_t* smem = align_1024(smem_raw);
    const uint32_t sQ = smem_u32(smem);     // Q_x at x tiles
    const uint32_t sKV = sQ + C::kOffKV;    // stage s: K, then V
    const uint32_t bar0 = sQ + C::kOffBar;
    // barriers (8 bytes each); x = 0 for query tile A, 1 for B
    auto s_full = [&](int x) { return bar0 + 8u * x; };
    auto s_free = [&](int x) { return bar0 + 16u + 8u * x; };
    auto p_full = [&](int x) { return bar0 + 32u + 8u * x; };
    auto pv_done = [&](int x) { return bar0 + 48u + 8u * x; };
    auto o_free = [&](int x) { return bar0 + 64u + 8u * x; };
    auto q_full = [&](int x) { return bar0 + 80u + 8u * x; };
    auto q_empty = [&](int x) { return bar0 + 96u + 8u * x; };
    auto k_full = [&](int i) { return bar0 + 112u + 8u * i; };
    auto v_full = [&](int i) { return bar0 + 112u + 8u * (kStages + i); };
    auto k_empty = [&](int i) { return bar0 + 112u + 8u * (2 * kStages + i); };
    auto v_empty = [&](int i) { return bar0 + 112u + 8u * (3 * kStages + i); };
    // V tile i is ready once warp 3 has seen it land and cleared the rows
    // behind the prompt's end
    auto v_ready = [&](int i) { return bar0 + 112u + 8u * (4 * kStages + i); };
    auto drain = [&](int x) { return bar0 + 112u + 8u * (5 * kStages + x); };
    static_assert(128 + 40 * kStages + 4 <= 512, "barrier space");
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffBar + 128 + 40 * kStages);

    const int warp = threadIdx.x / 32;
    const int lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int x = 0; x < 2; ++x) {
            mbar_init(s_full(x), 1);
            mbar_init(s_free(x), 4);
            mbar_init(p_full(x), 4);
            mbar_init(pv_done(x), 1);
            mbar_init(o_free(x), 4);
            mbar_init(q_full(x), 1);
            mbar_init(q_empty(x), 1);
            mbar_init(drain(x), 1);
        }
        if (ALIBI)
            for (int x = 0; x < 2; ++x) mbar_init(sQ + C::kOffTabBar + 8u * x, 4);
        for (int i = 0; i < kStages; ++i) {
            mbar_init(k_full(i), 1);
            mbar_init(v_full(i), 1);
            mbar_init(k_empty(i), 2);
            mbar_init(v_empty(i), 2);
            mbar_init(v_ready(i), 1);
        }
        fence_barrier_init();
        tma_prefetch_desc(&tmQ);
        tma_prefetch_desc(&tmK);
        tma_prefetch_desc(&tmV);
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(tmem_slot), C::kTmemCols);
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
    if (!pack.plan) build_plan(plan, pack.cu_seqlens, pack.prompts, a.S, 2 * pack.R, pack.R);
    const int n_items = plan_units(pack, plan) * a.Hk * pack.nhc;
    static_assert(4 * kRegsControl + 8 * kRegsSoftmax <= 12 * kLaunchRegs,
                  "register split exceeds the launch's registers");
    if (warp < 4) {
        setmaxnreg_dec<kRegsControl>();
    if (warp == 0) {
        if (lane == 0) {
            const uint64_t pol_kv = l2_evict_last_policy(), pol_q = l2_evict_first_policy();
            Cursor c;
            c.start(a, pack, plan, n_items);
            int gkv = 0;           // K/V tiles loaded so far (ring position)
            int nk = 0, nv = 0;    // K and V fills
            int itq[2] = {0, 0};   // Q fills per query tile
            bool ok = true;
            while (ok && c.valid) {
                const int nh = min(pack.Gt, pack.G - c.hc * pack.Gt), R = pack.R;
                for (int x = 0; x < (c.nB ? 2 : 1) && ok; ++x) {
                    if (!(ok = mbar_wait_inl(q_empty(x), (itq[x] & 1) ^ 1u, a.err))) break;
                    ++itq[x];
                    // boxes of R rows per head and slice; rows behind the
                    // chunk's heads keep stale values and are never written out
                    mbar_expect_tx(q_full(x), static_cast<uint32_t>(nh * R * D * 2));
                    const int qrow = c.start_row + (c.t0 + x) * R;
                    const uint32_t dst = sQ + x * C::kQBytes;
                    for (int k = 0; k < nh; ++k) {
#pragma unroll
                        for (int sub = 0; sub < C::kFull; ++sub)
                            tma_load_3d_hint(dst + sub * kTQ * 128 + k * R * 128, &tmQ, q_full(x),
                                             sub * 64, qrow, c.h + k, pol_q);
                        tma_load_3d_hint(dst + C::kFull * kTQ * 128 + k * R * 64, &tmQ2, q_full(x),
                                         C::kFull * 64, qrow, c.h + k, pol_q);
                    }
                }
                const int nkv = c.n_kv();
                for (int j = 0; j < nkv && ok; ++j, ++gkv) {
                    const int kt = kRev ? nkv - 1 - j : j;  // key tile of shared step j
                    const int st = gkv % kStages;
                    const uint32_t ph = (gkv / kStages) & 1;
                    const uint32_t sK = sKV + st * C::kStageBytes;
                    const bool own = kt >= c.nP;
                    const CUtensorMap* mK = own ? &tmK : &pack.tmPK;
                    const CUtensorMap* mK2 = own ? &tmK2 : &pack.tmPK2;
                    const CUtensorMap* mV = own ? &tmV : &pack.tmPV;
                    const int krow = own ? c.start_row + (kt - c.nP) * kTK : kt * kTK;
                    if (!(ok = mbar_wait_inl(k_empty(st), ph ^ 1u, a.err))) break;
                    mbar_expect_tx(k_full(st), C::kKBytes);
                    ++nk;
#pragma unroll
                    for (int sub = 0; sub < C::kFull; ++sub)
                        tma_load_3d_hint(sK + sub * kTK * 128, mK, k_full(st), sub * 64, krow, c.g, pol_kv);
                    tma_load_3d_hint(sK + C::kFull * kTK * 128, mK2, k_full(st), C::kFull * 64, krow, c.g,
                                     pol_kv);
                    if (!(ok = mbar_wait_inl(v_empty(st), ph ^ 1u, a.err))) break;
                    mbar_expect_tx(v_full(st), C::kVBytes);
                    ++nv;
#pragma unroll
                    for (int sub = 0; sub < C::kSub; ++sub)
                        tma_load_3d_hint(sK + C::kKBytes + sub * kTK * 128, mV, v_full(st), sub * 64, krow,
                                         c.g, pol_kv);
                }
                c.next(a, pack, plan, n_items);
            }
            // whatever the others met, no copy lands behind this block's end
            for (int i = max(nk - kStages, 0); i < nk; ++i)
                mbar_wait_inl(k_full(i % kStages), (i / kStages) & 1, a.err);
            for (int i = max(nv - kStages, 0); i < nv; ++i)
                mbar_wait_inl(v_full(i % kStages), (i / kStages) & 1, a.err);
            for (int x = 0; x < 2; ++x)
                if (itq[x] > 0) mbar_wait_inl(q_full(x), (itq[x] - 1) & 1, a.err);
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
            constexpr uint64_t kStageStep = C::kStageBytes >> 4;
            constexpr uint64_t kAtomQ = (kTQ * 128) >> 4, kAtomK = (kTK * 128) >> 4;
            const uint32_t sQx = sQ + x * C::kQBytes;
            const uint64_t dq = make_sdesc_sw128(sQx, 16, 1024);
            const uint64_t dk0 = make_sdesc_sw128(sKV, 16, 1024);
            const uint64_t dv0 = make_sdesc_sw128(sKV + C::kKBytes, kTK * 128, 1024);
            // the half slice of Q and K
            const uint64_t dqh = make_sdesc_sw64(sQx + C::kFull * kTQ * 128, 16, 512);
            const uint64_t dkh0 = make_sdesc_sw64(sKV + C::kFull * kTK * 128, 16, 512);
            const uint32_t tS = tmem_base + 64u * x;
            const uint32_t tP = tmem_base + C::kColP + 32u * x;
            const uint32_t tO = tmem_base + C::kColO + D * x;
            int gs = 0, gp = 0, itx = 0;  // S and PV tiles issued, items with this tile
            // S_x = Q_x K^T, once the K tile is there and the softmax has read
            // the previous S_x. The softmax passes the K tile back: a commit
            // costs this thread more than a hundred clocks, and a barrier test
            // as much, so two tests go out together
            auto issue_s = [&](int gj) -> bool {
                const int st = gj % kStages;
                const uint32_t ph = (gj / kStages) & 1;
                if (gs > 0 ? !mbar_wait2_inl(k_full(st), ph, s_free(x), (gs - 1) & 1, a.err)
                           : !mbar_wait_inl(k_full(st), ph, a.err))
                    return false;
                tc_fence_after();
                const uint64_t dk = dk0 + st * kStageStep;
#pragma unroll
                for (int ks = 0; ks < C::kFull * 4; ++ks)
                    tc_mma_ss(tS, dq + (ks / 4) * kAtomQ + (ks % 4) * 2,
                              dk + (ks / 4) * kAtomK + (ks % 4) * 2, idesc_s, ks > 0 ? 1u : 0u);
                const uint64_t dkh = dkh0 + st * kStageStep;
#pragma unroll
                for (int ks = 0; ks < 2; ++ks)
                    tc_mma_ss(tS, dqh + ks * 2, dkh + ks * 2, idesc_s, 1u);
                tc_commit(s_full(x));
                ++gs;
                return true;
            };
            // O_x += P_x V once the V tile is there and the softmax has written
            // P_x (the first PV of an item overwrites O_x, so it also waits for
            // the previous read-out)
            auto issue_pv = [&](int gj, bool first) -> bool {
                const int st = gj % kStages;
                if (!mbar_wait2_inl(v_ready(st), (gj / kStages) & 1, p_full(x), gp & 1, a.err))
                    return false;
                if (first && itx > 0 && !mbar_wait_inl(o_free(x), (itx - 1) & 1, a.err)) return false;
                tc_fence_after();
                const uint64_t dv = dv0 + st * kStageStep;
#pragma unroll
                for (int ks = 0; ks < kTK / 16; ++ks)
                    tc_mma_ts(tO, tP + ks * 8, dv + ks * ((16 * 128) >> 4), idesc_o,
                              (!first || ks > 0) ? 1u : 0u);
                tc_commit(pv_done(x));
                tc_commit(v_empty(st));
                ++gp;
                return true;
            };
            // a tile that this query tile does not use goes straight back
            auto skip = [&](uint32_t full, uint32_t empty, int gj) -> bool {
                if (!mbar_wait_inl(full, (gj / kStages) & 1, a.err)) return false;
                mbar_arrive(empty);
                return true;
            };
            Cursor c;
            c.start(a, pack, plan, n_items);
            int gkv = 0;
            bool ok = true;
            while (ok && c.valid) {
                const int nx = x ? c.nB : c.nA, nkv = c.n_kv();
                // this tile's shared steps [lo, hi): the first nx in key order,
                // the last nx when the walk runs down from the diagonal; Q_x is
                // released after the last one's S
                const int lo = kRev ? nkv - nx : 0, hi = kRev ? nkv : nx;
                if (nx > 0 && !mbar_wait_inl(q_full(x), itx & 1, a.err)) break;
                auto s_step = [&](int j) -> bool {
                    const int gj = gkv + j, st = gj % kStages;
                    if (!(j >= lo && j < hi ? issue_s(gj) : skip(k_full(st), k_empty(st), gj)))
                        return false;
                    if (nx > 0 && j + 1 == hi) tc_commit(q_empty(x));
                    return true;
                };
                if (!s_step(0)) break;
                for (int j = 0; j < nkv && ok; ++j) {
                    // S of step j+1 ahead of PV of step j
                    const int gj = gkv + j, st = gj % kStages;
                    ok = (j + 1 == nkv || s_step(j + 1)) &&
                         (j >= lo && j < hi ? issue_pv(gj, j == lo) : skip(v_ready(st), v_empty(st), gj));
                }
                gkv += nkv;
                if (nx > 0) ++itx;
                c.next(a, pack, plan, n_items);
            }
            // ... nor a product
            tc_commit(drain(x));
            mbar_wait_inl(drain(x), 0, a.err);
        }
    } else {
        // warp 3: passes each V tile on once it has landed, the rows behind
        // the prompt's end (the next prompt's) cleared: their P is 0, but 0
        // times a non-finite value of another prompt is not
        Cursor c;
        c.start(a, pack, plan, n_items);
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
                    clear_tile_rows<C::kSub>(sKV + st * C::kStageBytes + C::kKBytes, kTK, rows, lane);
                __syncwarp();
                if (lane == 0) mbar_arrive(v_ready(st));
            }
            c.next(a, pack, plan, n_items);
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
        const uint32_t tS = tmem_base + 64u * x;
        const uint32_t tO = tmem_base + C::kColO + D * x;
        const uint32_t tP = tmem_base + C::kColP + 32u * x;
        const float scale_l2 = a.scale * kLog2e;
        Cursor c;
        c.start(a, pack, plan, n_items);
        int g = 0;    // key tiles processed (across items)
        int gkv = 0;  // shared steps of the items so far
        bool ok = true;
        // The read-out of an item's O waits for its last PV; it is deferred to
        // the first tile of this warpgroup's next item (after that tile's
        // exponentials), so the next item's softmax overlaps the last PV.
        bool pend = false;  // an item's O is still in TMEM
        float pend_l = 0.f;
        int64_t pend_row = -1;  // output row, or -1: none
        int n_done = 0;         // items this warpgroup has started (ALiBi table parity)
        // O / l of the previous item, 32 columns at a time, once its last PV
        // has completed
        auto flush = [&]() {
            const float inv_l = 1.0f / pend_l;
#pragma unroll 1
            for (int cc = 0; cc < D / 32; ++cc) {
                uint32_t o[32];
                tmem_ld32(tO + lane_off + cc * 32, o);
                if (pend_row >= 0) {
                    T* dst = static_cast<T*>(a.o) + pend_row * static_cast<int64_t>(D) + cc * 32;
#pragma unroll
                    for (int v = 0; v < 4; ++v) {
                        float f[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e) f[e] = __uint_as_float(o[v * 8 + e]) * inv_l;
                        store8(dst + v * 8, f);
                    }
                }
                __syncwarp();
            }
        };
        while (ok && c.valid) {
            const int nx = x ? c.nB : c.nA, nkv = c.n_kv();
            const int gk = gkv + (kRev ? nkv - nx : 0);  // ring position of this tile's first step
            gkv += nkv;
            if (nx == 0) {
                c.next(a, pack, plan, n_items);
                continue;
            }
            // this row's head of the tile, and its position
            const int hl = row / pack.R;
            const int qfirst = (c.t0 + x) * pack.R;
            const int qpos = qfirst + row - hl * pack.R;
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
                const int off = C::kOffBias + (2 * x + (n_done & 1)) * kTK * 4;
                if (row < kTK)
                    reinterpret_cast<float*>(smem + off)[row] = slope_l2 * static_cast<float>(row);
                bias_tab = sQ + off;
                const uint32_t tab_bar = sQ + C::kOffTabBar + 8u * x;
                __syncwarp();
                if (lane == 0) mbar_arrive(tab_bar);
                if (!mbar_wait_inl(tab_bar, n_done & 1, a.err)) {
                    ok = false;
                    break;
                }
            }
            ++n_done;
            for (int j = 0; j < nx; ++j, ++g) {
                if (!mbar_wait_inl(s_full(x), g & 1, a.err, idle_limit_ns(c.it, c.nP))) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                if (quarter == 0 && lane == 0) mbar_arrive(k_empty((gk + j) % kStages));
                uint32_t r[kTK];
                tmem_ld64(tS + lane_off, r);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(s_free(x));
                const int kt = kRev ? nx - 1 - j : j;  // key tile of this step
                // packed ALiBi: key positions count from the query tile's first
                // (a row's constant), so that slope * position stays small,
                // hence exact, where its weight is not
                const int kown = (kt - c.nP) * kTK;  // own key position, < 0 in the prefix
                const int kbase = kt >= c.nP ? kown - qfirst : kt * kTK - c.prefix - qfirst;
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
                const bool masked = kt >= c.nP ? kown + kTK - 1 > qfirst || kown + kTK > c.len
                                               : (kt + 1) * kTK > c.prefix;
                const int lim = kt >= c.nP ? min(qpos, c.len - 1) - kown  // keys <= lim are visible
                                           : c.prefix - 1 - kt * kTK;
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
                // held in registers until the previous PV has read P_x
                const uint64_t mul2 = f2_pack(ALIBI ? 1.f : scale_l2, ALIBI ? 1.f : scale_l2);
                // (walking down from the diagonal, a row's first tiles may hold
                // no key that it sees: every weight 0, not inf - inf)
                const float m_off = ALIBI && m_used == -INFINITY ? 0.f : m_used;
                const float off = ALIBI ? sk - m_off : -m_off;
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
                    flush();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(o_free(x));
                    pend = false;
                }
                tmem_st32_nowait(tP + lane_off, pk);
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
            pend_row = qpos < c.len && hl < pack.Gt && c.hc * pack.Gt + hl < pack.G
                           ? (static_cast<int64_t>(c.start_row) + qpos) * a.H + c.h + hl
                           : -1;
            c.next(a, pack, plan, n_items);
        }
        // the last item's O
        if (ok && pend && mbar_wait_inl(pv_done(x), (g - 1) & 1, a.err)) {
            tc_fence_after();
            flush();
            tc_fence_before();
        }
    }
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem_base, C::kTmemCols);
    }
}

template <typename T, bool ALIBI>
cudaError_t launch_pair160(DType dt, const AttnArgs& a, const AttnPack<true>& pack, int64_t items,
                           cudaStream_t s) {
    CUtensorMap tq, tk, tv, tq2, tk2;  // *2: the half slice
    const uint64_t H = a.H, Hk = a.Hk;
    const uint32_t R = pack.R;
    if (!make_tmap_3d(&tq, dt, a.q, H, a.S, D, R) || !make_tmap_3d(&tk, dt, a.k, Hk, a.S, D, kTK) ||
        !make_tmap_3d(&tv, dt, a.v, Hk, a.S, D, kTK) || !make_tmap_3d(&tq2, dt, a.q, H, a.S, D, R, 32) ||
        !make_tmap_3d(&tk2, dt, a.k, Hk, a.S, D, kTK, 32))
        return cudaErrorInvalidValue;
    auto kern = attn_pair160_kernel<T, ALIBI>;
    const cudaError_t e = set_smem_attr_once(reinterpret_cast<const void*>(kern), C::kSmem);
    if (e != cudaSuccess) return e;
    if (items > 0x7fffffff) return cudaErrorInvalidValue;
    const int64_t grid = items < a.num_sms ? items : a.num_sms;
    AttnArgs ap = a;
    ap.pdl = pdl_allowed(s);
    (void)launch_pdl(ap.pdl != 0, kern, dim3(static_cast<unsigned>(grid)), dim3(kPair160Threads), C::kSmem,
                     s, tq, tk, tv, tq2, tk2, ap, pack);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attention_pair160_packed(DType dt, const AttnArgs& a, const AttnPack<true>& pack,
                                            int64_t max_units, cudaStream_t s) {
    // ALiBi takes one slope per tile: grouped heads go to attn_gqa.cu
    if (a.d != D || (a.alibi && a.H != a.Hk)) return cudaErrorInvalidValue;
    AttnPack<true> p = pack;
    gqa_tile(a.H, a.Hk, &p.G, &p.Gt, &p.R, &p.nhc);
    const int64_t items = max_units * a.Hk * p.nhc;
    if (dt == DType::F16)
        return a.alibi ? launch_pair160<__half, true>(dt, a, p, items, s)
                       : launch_pair160<__half, false>(dt, a, p, items, s);
    return a.alibi ? launch_pair160<__nv_bfloat16, true>(dt, a, p, items, s)
                   : launch_pair160<__nv_bfloat16, false>(dt, a, p, items, s);
}

}  // namespace blk
