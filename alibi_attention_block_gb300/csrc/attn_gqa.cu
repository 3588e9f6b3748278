// K3 for grouped-query attention at head_dim 128 and 160: the query heads
// that share one key/value head are packed into the rows of one 128-row
// query tile, so every K/V tile a CTA loads serves the whole group.
//
// GQA (nnterp "stablelm", 03 Notes: on the 12B model kv head j serves query
// heads 4j .. 4j+3; kv head = h / (H/Hk)). With G = H/Hk query heads per kv
// head, a tile holds Gt = min(G, 16) of them (all G unless G > 16; a larger
// group is split into chunks of Gt heads) and R = 128/Gt consecutive
// positions (rounded down to a multiple of 8) of each: row r is head
// g*G + chunk*Gt + r/R at position p0 + r%R. MHA (G = 1) is the plain
// 128-position tile. The scores S = Q K^T of one 128-key tile are then one
// M=128, N=128 product for all G heads at once, and one PV product
// (M=128, N=d) follows it; both run at the tensor core's full-size shapes
// (K=d for S, N=d for PV), with each K/V tile read from L2 once per group
// and position block instead of once per head. Work items are
// (position block, batch, kv head, head chunk), latest (heaviest) blocks
// first, dealt to the persistent CTAs in alternating directions.
//
// 6 warps, one CTA per SM:
//   warp 0      TMA: the item's Q tile (G boxes of R rows per 64-column
//               slice), then K tiles one ahead of V tiles (each 128 keys,
//               128-byte swizzle, zero fill past S), K and V in rings of
//               their own; K and V load with an evict-last L2 policy (other
//               position blocks of the group read the same key prefix), Q
//               evict-first
//   warp 1      TMEM allocator and single-thread MMA issuer, in the order
//               S(0), S(1), PV(0), S(2), PV(1), ...: S is double-buffered in
//               TMEM, so the next tile's scores are computed while the
//               softmax works on this one
//   warps 2..5  softmax, one thread per query row (TMEM lane; a warp reaches
//               the lane quarter of its index mod 4): one tcgen05.ld of the
//               row's 128 scores (the S buffer is released at once), the
//               causal mask on the key tiles past the block's first
//               position, the row max (3-input max), one paired (f32x2) FMA
//               per two scores into ex2 (scale log2(e)/sqrt(d) folded in;
//               ALiBi, "Bloom in a sovereign engine", Contribution, enters as
//               +slope*key with the row's own head slope), P packed to the
//               storage type in registers and stored to TMEM once the
//               previous PV has read the old P. O is rescaled in TMEM only
//               when the running max grows by more than 2^8. An item's O / l
//               is read out and written as [B, S, H, d] during the first
//               tile of the next item, so no softmax waits on a last PV.
// TMEM columns: S0 [0, 128), S1 [128, 256), P [256, 320) (two 16-bit values
// per column), O [320, 320 + d).
// Query scale head_dim^-0.5 follows nnterp "stablelm" 03 Notes.
#include "attn_plan.cuh"
#include "internal.h"

namespace blk {

namespace {

constexpr int gqa_threads(bool packed) { return packed ? 224 : 192; }  // packed: one more warp
constexpr int kTQ = 128;  // query rows per tile (G heads x R positions)
constexpr int kTK = 128;  // keys per tile
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kRescaleThreshold = 8.0f;  // log2 of the largest unnormalised p
constexpr uint32_t kColP = 256, kColO = 320;

template <int D>
struct GqaCfg {
    static_assert(D == 128 || D == 160, "GQA-packed attention is built for head_dim 128 and 160");
    static constexpr int kSub = (D + 63) / 64;          // 64-column slices per row
    // V tile: 128 rows x kSub x 128 B (head_dim 160 padded to 192 columns, one
    // descriptor for the whole row). Q and K tiles keep only the 32 columns of
    // head_dim 160's last slice, as a slice of 64-byte rows with the 64-byte
    // swizzle: what that saves makes room for a second V stage (with one, the
    // next V was loaded only after the PV product; B2 S4096, 32/8 heads: 333 -> 308
    // us).
    static constexpr bool kHalf = D % 64 != 0;
    static constexpr int kFull = D / 64;                 // whole slices
    static constexpr int kTileBytes = kSub * 128 * 128;
    static constexpr int kQKBytes = kFull * 128 * 128 + (kHalf ? 128 * 64 : 0);
    static constexpr int kQBufs = D > 128 ? 1 : 2;
    static constexpr int kKStages = 2;
    static constexpr int kVStages = 2;
    static constexpr int kOffK = kQBufs * kQKBytes;
    static constexpr int kOffV = kOffK + kKStages * kQKBytes;
    static constexpr int kOffBar = kOffV + kVStages * kTileBytes;
    static constexpr int kSmem = kOffBar + 256 + 1024;   // + barriers + alignment slack
    static constexpr uint32_t kTmemCols = 512;
};

// Packing of a group's query heads into 128-row tiles.
struct GqaPack {
    int G;     // query heads per kv head
    int Gt;    // query heads per tile
    int R;     // positions per head in a tile (multiple of 8)
    int nhc;   // head chunks per group
};

// This CTA's items: (position block pb, batch b, kv head g, head chunk hc).
// Round r gives item r*Gd + blockIdx on even rounds and r*Gd + Gd-1-blockIdx
// on odd ones (Gd = grid size); items are numbered latest block first.
// Packed prompts (PACKED; with ALiBi over grouped heads, a slope per row, as
// attn_pair128.cu and attn_pair160.cu take the others): a unit is a block of R
// positions of one prompt; the prefix's nP key tiles come ahead of the
// prompt's own.
template <bool PACKED>
struct GqaCursor {
    using Plan = typename PlanStorage<PACKED>::type;
    int item, it, pb, b, g, hc, p0, nkv;
    bool valid;
    int start_row, len, nP, prefix;
    __device__ __forceinline__ int item_of(int round) const {
        const int Gd = static_cast<int>(gridDim.x), c = static_cast<int>(blockIdx.x);
        return round * Gd + ((round & 1) ? Gd - 1 - c : c);
    }
    __device__ __forceinline__ void decode(const AttnArgs& a, const GqaPack& pk,
                                           const AttnPack<PACKED>& pack, const Plan& plan, int nblk) {
        if constexpr (PACKED) {
            const int per_unit = a.Hk * pk.nhc;
            const PlanUnit u = plan_unit(pack, plan, item / per_unit);
            const int rest = item % per_unit;
            hc = rest % pk.nhc;
            g = rest / pk.nhc;
            b = 0;
            start_row = u.first;
            len = u.len;
            p0 = u.l * pk.R;
            prefix = pack.prefix;
            nP = (prefix + kTK - 1) / kTK;
            nkv = nP + (min(p0 + pk.R, len) + kTK - 1) / kTK;
            return;
        }
        const int per_block = a.B * a.Hk * pk.nhc;
        pb = nblk - 1 - item / per_block;
        int rest = item % per_block;
        hc = rest % pk.nhc;
        rest /= pk.nhc;
        b = rest / a.Hk;
        g = rest - b * a.Hk;
        p0 = pb * pk.R;
        const int last = min(p0 + pk.R, a.S);  // one past the block's last position
        nkv = (last + kTK - 1) / kTK;
    }
    __device__ __forceinline__ void start(const AttnArgs& a, const GqaPack& pk,
                                         const AttnPack<PACKED>& pack, const Plan& plan, int nblk,
                                         int n_items) {
        it = 0;
        item = item_of(0);
        valid = item < n_items;
        if (valid) decode(a, pk, pack, plan, nblk);
    }
    __device__ __forceinline__ void next(const AttnArgs& a, const GqaPack& pk,
                                         const AttnPack<PACKED>& pack, const Plan& plan, int nblk,
                                         int n_items) {
        ++it;
        item = item_of(it);
        valid = item < n_items;
        if (valid) decode(a, pk, pack, plan, nblk);
    }
};

template <typename T, int D, bool ALIBI, bool PACKED>
__global__ void __launch_bounds__(gqa_threads(PACKED), 1)
    attn_gqa_kernel(const __grid_constant__ CUtensorMap tmQ,
                    const __grid_constant__ CUtensorMap tmK,
                    const __grid_constant__ CUtensorMap tmV,
                    const __grid_constant__ CUtensorMap tmQ2,
                    const __grid_constant__ CUtensorMap tmK2, const AttnArgs a,
                    const GqaPack pk, const __grid_constant__ AttnPack<PACKED> pack) {
    using Cfg = GqaCfg<D>;
    constexpr int kQB = Cfg::kQBufs, kKS = Cfg::kKStages, kVS = Cfg::kVStages;
    // packed ALiBi: key tiles from the diagonal down, as in attn_pair.cu (the
    // bias is largest there, so the rescale of O stays rare)
    constexpr bool kRev = ALIBI && PACKED;
    extern __shared__ uint8_t smem_raw[];
    __shared__ typename PlanStorage<PACKED>::type plan;
    uint8_t* smem = align_1024(smem_raw);
    const uint32_t sQ = smem_u32(smem);
    const uint32_t sK = sQ + Cfg::kOffK;
    const uint32_t sV = sQ + Cfg::kOffV;
    const uint32_t bar0 = sQ + Cfg::kOffBar;
    // barriers (8 bytes each)
    auto s_full = [&](int i) { return bar0 + 8u * i; };
    auto s_free = [&](int i) { return bar0 + 16u + 8u * i; };
    const uint32_t p_full = bar0 + 32u;
    const uint32_t pv_done = bar0 + 40u;
    const uint32_t o_free = bar0 + 48u;
    auto q_full = [&](int i) { return bar0 + 56u + 8u * i; };
    auto q_empty = [&](int i) { return bar0 + 72u + 8u * i; };
    auto k_full = [&](int i) { return bar0 + 88u + 8u * i; };
    auto k_empty = [&](int i) { return bar0 + 104u + 8u * i; };
    auto v_full = [&](int i) { return bar0 + 120u + 8u * i; };
    auto v_empty = [&](int i) { return bar0 + 136u + 8u * i; };
    // packed: V tile i is ready once the last warp has seen it land and
    // cleared the rows behind the prompt's end
    auto v_ready = [&](int i) { return PACKED ? bar0 + 160u + 8u * i : v_full(i); };
    const uint32_t drain = bar0 + 176u;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + Cfg::kOffBar + 152);

    const int warp = threadIdx.x / 32;
    const int lane = threadIdx.x & 31;
    const int G = pk.G, R = pk.R;
    const int nblk = (a.S + R - 1) / R;
    int n_items = nblk * a.B * a.Hk * pk.nhc;

    if (threadIdx.x == 0) {
        for (int x = 0; x < 2; ++x) {
            mbar_init(s_full(x), 1);
            mbar_init(s_free(x), 4);
            mbar_init(q_full(x), 1);
            mbar_init(q_empty(x), 1);
            mbar_init(k_full(x), 1);
            mbar_init(k_empty(x), 1);
            mbar_init(v_full(x), 1);
            mbar_init(v_empty(x), 1);
            if (PACKED) mbar_init(v_ready(x), 1);
        }
        mbar_init(p_full, 4);
        mbar_init(pv_done, 1);
        mbar_init(o_free, 4);
        mbar_init(drain, 1);
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
        if (!pack.plan) build_plan(plan, pack.cu_seqlens, pack.prompts, a.S, pk.R, 0);
        n_items = plan_units(pack, plan) * a.Hk * pk.nhc;
    }

    if (warp == 0) {
        if (lane == 0) {
            const uint64_t pol_kv = l2_evict_last_policy(), pol_q = l2_evict_first_policy();
            GqaCursor<PACKED> c;
            c.start(a, pk, pack, plan, nblk, n_items);
            int gk = 0, gv = 0;  // K and V tiles loaded so far (ring positions)
            bool ok = true;
            // the first row of step j's key tile, and whether it is the prefix's
            auto tile_source = [&](int j, int& krow) -> bool {
                if constexpr (PACKED) {
                    const int kt = kRev ? c.nkv - 1 - j : j;
                    krow = kt < c.nP ? kt * kTK : c.start_row + (kt - c.nP) * kTK;
                    return kt < c.nP;
                } else {
                    krow = j * kTK;
                    return false;
                }
            };
            auto load_k = [&](int j) -> bool {
                const int st = gk % kKS;
                if (!mbar_wait(k_empty(st), ((gk / kKS) & 1) ^ 1u, a.err)) return false;
                mbar_expect_tx(k_full(st), Cfg::kQKBytes);
                int krow;
                const CUtensorMap *m = &tmK, *m2 = &tmK2;
                if (tile_source(j, krow)) {
                    if constexpr (PACKED) {
                        m = &pack.tmPK;
                        m2 = &pack.tmPK2;
                    }
                }
                const uint32_t dst = sK + st * Cfg::kQKBytes;
#pragma unroll
                for (int sub = 0; sub < Cfg::kFull; ++sub)
                    tma_load_3d_hint(dst + sub * kTK * 128, m, k_full(st), sub * 64, krow,
                                     c.b * a.Hk + c.g, pol_kv);
                if constexpr (Cfg::kHalf)
                    tma_load_3d_hint(dst + Cfg::kFull * kTK * 128, m2, k_full(st), Cfg::kFull * 64, krow,
                                     c.b * a.Hk + c.g, pol_kv);
                ++gk;
                return true;
            };
            auto load_v = [&](int j) -> bool {
                const int st = gv % kVS;
                if (!mbar_wait(v_empty(st), ((gv / kVS) & 1) ^ 1u, a.err)) return false;
                mbar_expect_tx(v_full(st), Cfg::kTileBytes);
                int krow;
                const CUtensorMap* m = &tmV;
                if (tile_source(j, krow)) {
                    if constexpr (PACKED) m = &pack.tmPV;
                }
#pragma unroll
                for (int sub = 0; sub < Cfg::kSub; ++sub)
                    tma_load_3d_hint(sV + st * Cfg::kTileBytes + sub * kTK * 128, m, v_full(st),
                                sub * 64, krow, c.b * a.Hk + c.g, pol_kv);
                ++gv;
                return true;
            };
            while (ok && c.valid) {
                const int qb = c.it % kQB;
                if (!mbar_wait(q_empty(qb), ((c.it / kQB) & 1) ^ 1u, a.err)) break;
                // one box of R rows per head of the chunk and 64-column
                // slice; rows past the chunk's heads keep stale values and are
                // never written out
                const int nh = min(pk.Gt, G - c.hc * pk.Gt);
                mbar_expect_tx(q_full(qb), static_cast<uint32_t>(nh * R * D * 2));
                for (int i = 0; i < nh; ++i) {
                    const int qrow = (PACKED ? c.start_row : 0) + c.p0;
                    const int plane = c.b * a.H + c.g * G + c.hc * pk.Gt + i;
                    const uint32_t dst = sQ + qb * Cfg::kQKBytes;
#pragma unroll
                    for (int sub = 0; sub < Cfg::kFull; ++sub)
                        tma_load_3d_hint(dst + sub * kTQ * 128 + i * R * 128, &tmQ, q_full(qb), sub * 64,
                                         qrow, plane, pol_q);
                    if constexpr (Cfg::kHalf)
                        tma_load_3d_hint(dst + Cfg::kFull * kTQ * 128 + i * R * 64, &tmQ2, q_full(qb),
                                         Cfg::kFull * 64, qrow, plane, pol_q);
                }
                // consumption order: K(0), then K(j+1) ahead of V(j)
                ok = load_k(0);
                for (int j = 0; ok && j < c.nkv; ++j) {
                    if (j + 1 < c.nkv) ok = load_k(j + 1);
                    if (ok) ok = load_v(j);
                }
                c.next(a, pk, pack, plan, nblk, n_items);
            }
            // whatever the others met, no copy lands behind this block's end
            for (int i = max(gk - kKS, 0); i < gk; ++i)
                mbar_wait(k_full(i % kKS), (i / kKS) & 1, a.err);
            for (int i = max(gv - kVS, 0); i < gv; ++i)
                mbar_wait(v_full(i % kVS), (i / kVS) & 1, a.err);
            for (int i = max(c.it - kQB, 0); i < c.it; ++i)
                mbar_wait(q_full(i % kQB), (i / kQB) & 1, a.err);
        }
    } else if (warp == 1) {
        if (lane == 0) {
            constexpr uint32_t fmt = dt_traits<T>::mma_fmt;
            constexpr uint32_t idesc_s = make_idesc_f16(fmt, kTQ, kTK, false);
            constexpr uint32_t idesc_o = make_idesc_f16(fmt, kTQ, D, true);
            constexpr uint64_t kVStep = Cfg::kTileBytes >> 4, kQKStep = Cfg::kQKBytes >> 4;
            constexpr uint64_t kSubStep = (kTQ * 128) >> 4;  // next 64-column slice
            const uint64_t dq0 = make_sdesc_sw128(sQ, 16, 1024);
            const uint64_t dk0 = make_sdesc_sw128(sK, 16, 1024);
            const uint64_t dv0 = make_sdesc_sw128(sV, kTK * 128, 1024);
            // the half slice of Q and K (64-byte rows)
            const uint64_t dqh0 = make_sdesc_sw64(sQ + Cfg::kFull * kTQ * 128, 16, 512);
            const uint64_t dkh0 = make_sdesc_sw64(sK + Cfg::kFull * kTK * 128, 16, 512);
            const uint32_t tP = tmem_base + kColP;
            const uint32_t tO = tmem_base + kColO;
            int gk = 0, gv = 0, gs = 0, gp = 0, itx = 0;
            // S(buffer gs % 2) = Q K^T, once the softmax has read that buffer's
            // previous scores
            auto issue_s = [&](int qb) -> bool {
                const int st = gk % kKS;
                const int sb = gs & 1;
                if (!mbar_wait(k_full(st), (gk / kKS) & 1, a.err)) return false;
                if (gs >= 2 && !mbar_wait(s_free(sb), ((gs >> 1) - 1) & 1, a.err)) return false;
                tc_fence_after();
                const uint64_t dq = dq0 + qb * kQKStep, dk = dk0 + st * kQKStep;
#pragma unroll
                for (int ks = 0; ks < Cfg::kFull * 4; ++ks) {
                    const uint64_t off = (ks / 4) * kSubStep + (ks % 4) * 2;
                    tc_mma_ss(tmem_base + 128u * sb, dq + off, dk + off, idesc_s, ks > 0 ? 1u : 0u);
                }
                if constexpr (Cfg::kHalf) {
                    const uint64_t dqh = dqh0 + qb * kQKStep, dkh = dkh0 + st * kQKStep;
#pragma unroll
                    for (int ks = 0; ks < 2; ++ks)
                        tc_mma_ss(tmem_base + 128u * sb, dqh + ks * 2, dkh + ks * 2, idesc_s, 1u);
                }
                tc_commit(s_full(sb));
                tc_commit(k_empty(st));
                ++gk;
                ++gs;
                return true;
            };
            // O += P V once the softmax has written P (the first PV of an item
            // overwrites O, so it also waits for the previous item's read-out)
            auto issue_pv = [&](bool first) -> bool {
                const int st = gv % kVS;
                if (!mbar_wait(v_ready(st), (gv / kVS) & 1, a.err)) return false;
                if (!mbar_wait(p_full, gp & 1, a.err)) return false;
                if (first && itx > 0 && !mbar_wait(o_free, (itx - 1) & 1, a.err)) return false;
                tc_fence_after();
                const uint64_t dv = dv0 + st * kVStep;
#pragma unroll
                for (int ks = 0; ks < kTK / 16; ++ks)
                    tc_mma_ts(tO, tP + ks * 8, dv + ks * ((16 * 128) >> 4), idesc_o,
                              (!first || ks > 0) ? 1u : 0u);
                tc_commit(pv_done);
                tc_commit(v_empty(st));
                ++gv;
                ++gp;
                return true;
            };
            GqaCursor<PACKED> c;
            c.start(a, pk, pack, plan, nblk, n_items);
            bool ok = true;
            while (ok && c.valid) {
                const int qb = c.it % kQB;
                if (!mbar_wait(q_full(qb), (c.it / kQB) & 1, a.err)) break;
                ok = issue_s(qb);
                if (ok && c.nkv == 1) tc_commit(q_empty(qb));
                for (int j = 0; ok && j < c.nkv; ++j) {
                    if (j + 1 < c.nkv) {
                        ok = issue_s(qb);
                        if (ok && j + 2 == c.nkv) tc_commit(q_empty(qb));
                    }
                    if (ok) ok = issue_pv(j == 0);
                }
                ++itx;
                c.next(a, pk, pack, plan, nblk, n_items);
            }
            // ... nor a product
            tc_commit(drain);
            mbar_wait(drain, 0, a.err);
        }
    } else if (PACKED && warp == 6) {
        if constexpr (PACKED) {
            // passes each V tile on, the rows behind the prompt's end cleared
            // (see attn_pair.cu)
            GqaCursor<PACKED> c;
            c.start(a, pk, pack, plan, nblk, n_items);
            int gv = 0;
            bool ok = true;
            while (ok && c.valid) {
                for (int j = 0; j < c.nkv; ++j, ++gv) {
                    const int kt = kRev ? c.nkv - 1 - j : j;
                    const int st = gv % kVS;
                    if (!mbar_wait(v_full(st), (gv / kVS) & 1, a.err)) {
                        ok = false;
                        break;
                    }
                    const int rows = kt < c.nP ? kTK : c.len - (kt - c.nP) * kTK;
                    if (rows < kTK)
                        clear_tile_rows<Cfg::kSub>(sV + st * Cfg::kTileBytes, kTK, rows, lane);
                    __syncwarp();
                    if (lane == 0) mbar_arrive(v_ready(st));
                }
                c.next(a, pk, pack, plan, nblk, n_items);
            }
        }
    } else {
        // softmax: warp w reads TMEM lanes 32 (w % 4) .. +31, one query row
        // per thread
        const int quarter = warp & 3;
        const int row = quarter * 32 + lane;
        const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
        const uint32_t tO = tmem_base + kColO;
        const uint32_t tP = tmem_base + kColP;
        const float scale_l2 = a.scale * kLog2e;
        const int hl = row / R;          // head of this row within the tile
        const int rpos = row - hl * R;   // position offset within the block
        float slope_l2 = 0.f;
        GqaCursor<PACKED> c;
        c.start(a, pk, pack, plan, nblk, n_items);
        int g = 0;  // key tiles processed (across items)
        bool ok = true;
        bool pend = false;      // an item's O is still in TMEM
        float pend_l = 0.f;
        int64_t pend_row = -1;  // output row (b * S + pos) * H + h, or -1
        while (ok && c.valid) {
            const int pos = c.p0 + rpos;
            // rows past the chunk's heads are padding
            const bool in_group = hl < pk.Gt && c.hc * pk.Gt + hl < G;
            const int h = c.g * G + (in_group ? c.hc * pk.Gt + hl : 0);
            if constexpr (ALIBI) {
                const float slope = a.slopes ? a.slopes[h]
                                             : exp2f(-8.0f * static_cast<float>(h + 1) /
                                                     static_cast<float>(a.H));
                slope_l2 = slope * kLog2e;
            }
            const int S_own = PACKED ? c.len : a.S;
            const int lim_abs = min(pos, S_own - 1);  // (own) keys <= lim_abs are visible
            float m_used = -INFINITY;  // running max, log2 domain
            float l = 0.f;
            for (int j = 0; j < c.nkv; ++j, ++g) {
                const int sb = g & 1;
                if (!mbar_wait(s_full(sb), (g >> 1) & 1, a.err)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                uint32_t r[kTK];
                tmem_ld128(tmem_base + 128u * sb + lane_off, r);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(s_free(sb));
                const int kt = kRev ? c.nkv - 1 - j : j;  // key tile of this step
                const int kbase = (PACKED ? kt - c.nP : j) * kTK;  // packed: < 0 in the prefix
                if constexpr (ALIBI) {
                    // packed: key positions from the block's first (a row's
                    // constant), small where the weight is not
                    const int kpos = !PACKED      ? kbase
                                     : kbase >= 0 ? kbase - c.p0
                                                  : kt * kTK - c.prefix - c.p0;
                    const float sk = slope_l2 * static_cast<float>(kpos);
#pragma unroll
                    for (int i = 0; i < kTK; ++i)
                        r[i] = __float_as_uint(fmaf(__uint_as_float(r[i]), scale_l2,
                                                    fmaf(slope_l2, static_cast<float>(i), sk)));
                }
                bool masked;
                int lim;
                if constexpr (PACKED) {
                    masked = kbase >= 0 ? kbase + kTK - 1 > c.p0 || kbase + kTK > c.len
                                        : (kt + 1) * kTK > c.prefix;
                    lim = kbase >= 0 ? lim_abs - kbase : c.prefix - 1 - kt * kTK;
                } else {
                    masked = kbase + kTK - 1 > c.p0 || kbase + kTK > a.S;
                    lim = lim_abs - kbase;
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
                float corr = 1.f;
                if (mx > m_used + kRescaleThreshold) {
                    corr = ex2_approx(m_used - mx);
                    m_used = mx;
                }
                // a row with no visible key in this tile and none before it
                // keeps m = -inf: use 0. Padding rows, and, with packed ALiBi's
                // walk down from the diagonal, the first rows of a block of
                // positions that crosses a key tile's edge
                const float m_eff = m_used == -INFINITY ? 0.f : m_used;
                const uint64_t mul2 = f2_pack(ALIBI ? 1.f : scale_l2, ALIBI ? 1.f : scale_l2);
                const uint64_t neg2 = f2_pack(-m_eff, -m_eff);
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
                // the previous PV has read P and O is settled: read out the
                // previous item's O if pending, publish P, rescale O if the
                // max moved (before this tile's PV)
                if (j > 0 || pend) {
                    if (!mbar_wait(pv_done, (g - 1) & 1, a.err)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                }
                if (j == 0 && pend) {
                    float inv_l = pend_l > 0.f ? 1.0f / pend_l : 0.f;
                    T* dst = pend_row >= 0 ? static_cast<T*>(a.o) + pend_row * static_cast<int64_t>(D)
                                           : nullptr;
#pragma unroll 1
                    for (int cc = 0; cc < D / 32; ++cc) {
                        uint32_t o[32];
                        tmem_ld32(tO + lane_off + cc * 32, o);
                        if (dst) {
                            float f[32];
#pragma unroll
                            for (int e = 0; e < 32; ++e) f[e] = __uint_as_float(o[e]) * inv_l;
#pragma unroll
                            for (int v = 0; v < 4; ++v)
                                store8(dst + cc * 32 + v * 8,
                                       *reinterpret_cast<const float(*)[8]>(&f[v * 8]));
                        }
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(o_free);
                    pend = false;
                }
                tmem_st64_nowait(tP + lane_off, *reinterpret_cast<const uint32_t(*)[64]>(pk));
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
                if (lane == 0) mbar_arrive(p_full);
                float s0, s1, s2, s3;
                f2_unpack(acc0, s0, s1);
                f2_unpack(acc1, s2, s3);
                l = l * corr + ((s0 + s1) + (s2 + s3));
            }
            if (!ok) break;
            pend = true;
            pend_l = l;
            const int64_t row0 = PACKED ? c.start_row : static_cast<int64_t>(c.b) * a.S;
            pend_row = (in_group && pos < S_own) ? (row0 + pos) * a.H + h : -1;
            c.next(a, pk, pack, plan, nblk, n_items);
        }
        // the last item's O
        if (ok && pend && mbar_wait(pv_done, (g - 1) & 1, a.err)) {
            tc_fence_after();
            const float inv_l = pend_l > 0.f ? 1.0f / pend_l : 0.f;
            T* dst = pend_row >= 0 ? static_cast<T*>(a.o) + pend_row * static_cast<int64_t>(D)
                                   : nullptr;
#pragma unroll 1
            for (int cc = 0; cc < D / 32; ++cc) {
                uint32_t o[32];
                tmem_ld32(tO + lane_off + cc * 32, o);
                if (dst) {
                    float f[32];
#pragma unroll
                    for (int e = 0; e < 32; ++e) f[e] = __uint_as_float(o[e]) * inv_l;
#pragma unroll
                    for (int v = 0; v < 4; ++v)
                        store8(dst + cc * 32 + v * 8, *reinterpret_cast<const float(*)[8]>(&f[v * 8]));
                }
            }
            tc_fence_before();
        }
    }
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem_base, Cfg::kTmemCols);
    }
}

template <typename T, int D, bool ALIBI, bool PACKED>
cudaError_t launch_gqa_d(DType dt, const AttnArgs& a, const GqaPack& pk,
                         const AttnPack<PACKED>& pack, int64_t items, cudaStream_t s) {
    const int R = pk.R;
    using Cfg = GqaCfg<D>;
    // (the half-slice maps are used at head_dim 160 only)
    CUtensorMap tq, tk, tv, tq2, tk2;
    if (!make_tmap_3d(&tq, dt, a.q, static_cast<uint64_t>(a.B) * a.H, a.S, D, R) ||
        !make_tmap_3d(&tq2, dt, a.q, static_cast<uint64_t>(a.B) * a.H, a.S, D, R, 32) ||
        !make_tmap_3d(&tk2, dt, a.k, static_cast<uint64_t>(a.B) * a.Hk, a.S, D, kTK, 32) ||
        !make_tmap_3d(&tk, dt, a.k, static_cast<uint64_t>(a.B) * a.Hk, a.S, D, kTK) ||
        !make_tmap_3d(&tv, dt, a.v, static_cast<uint64_t>(a.B) * a.Hk, a.S, D, kTK))
        return cudaErrorInvalidValue;
    auto kern = attn_gqa_kernel<T, D, ALIBI, PACKED>;
    {
        const cudaError_t e = set_smem_attr_once(reinterpret_cast<const void*>(kern), Cfg::kSmem);
        if (e != cudaSuccess) return e;
    }
    if (items > 0x7fffffff) return cudaErrorInvalidValue;
    const int64_t grid = items < a.num_sms ? items : a.num_sms;
    AttnArgs ap = a;
    ap.pdl = pdl_allowed(s);
    (void)launch_pdl(ap.pdl != 0, kern, dim3(static_cast<unsigned>(grid)), dim3(gqa_threads(PACKED)),
                     Cfg::kSmem, s, tq, tk, tv, tq2, tk2, ap, pk, pack);
    return cudaGetLastError();
}

template <typename T, int D, bool PACKED>
cudaError_t launch_gqa_a(DType dt, const AttnArgs& a, const GqaPack& pk,
                         const AttnPack<PACKED>& pack, int64_t items, cudaStream_t s) {
    if constexpr (!PACKED)  // packed prompts come here with ALiBi only
        if (!a.alibi) return launch_gqa_d<T, D, false>(dt, a, pk, pack, items, s);
    return launch_gqa_d<T, D, true>(dt, a, pk, pack, items, s);
}

template <bool PACKED>
cudaError_t launch_gqa(DType dt, const AttnArgs& a, const GqaPack& pk, const AttnPack<PACKED>& pack,
                       int64_t items, cudaStream_t s) {
    if (dt == DType::F16)
        return a.d == 128 ? launch_gqa_a<__half, 128>(dt, a, pk, pack, items, s)
                          : launch_gqa_a<__half, 160>(dt, a, pk, pack, items, s);
    return a.d == 128 ? launch_gqa_a<__nv_bfloat16, 128>(dt, a, pk, pack, items, s)
                      : launch_gqa_a<__nv_bfloat16, 160>(dt, a, pk, pack, items, s);
}

GqaPack gqa_pack(int H, int Hk) {
    GqaPack pk;
    pk.G = H / Hk;
    pk.Gt = pk.G < 16 ? pk.G : 16;
    pk.R = (kTQ / pk.Gt) / 8 * 8;
    pk.nhc = (pk.G + pk.Gt - 1) / pk.Gt;
    return pk;
}

}  // namespace

void gqa_tile(int H, int Hk, int* G, int* Gt, int* R, int* nhc) {
    const GqaPack pk = gqa_pack(H, Hk);
    *G = pk.G;
    *Gt = pk.Gt;
    *R = pk.R;
    *nhc = pk.nhc;
}

cudaError_t launch_attention_gqa(DType dt, const AttnArgs& a, cudaStream_t s) {
    if (a.Hk <= 0 || a.H % a.Hk || (a.d != 128 && a.d != 160)) return cudaErrorInvalidValue;
    if (a.B == 0 || a.S == 0) return cudaSuccess;
    const GqaPack pk = gqa_pack(a.H, a.Hk);
    const int64_t items = static_cast<int64_t>((a.S + pk.R - 1) / pk.R) * a.B * a.Hk * pk.nhc;
    return launch_gqa(dt, a, pk, AttnPack<false>{}, items, s);
}

cudaError_t launch_attention_gqa_packed(DType dt, const AttnArgs& a, const AttnPack<true>& pack,
                                        int64_t max_units, cudaStream_t s) {
    if (a.Hk <= 0 || a.H % a.Hk || (a.d != 128 && a.d != 160) || !a.alibi) return cudaErrorInvalidValue;
    const GqaPack pk = gqa_pack(a.H, a.Hk);
    return launch_gqa(dt, a, pk, pack, max_units * a.Hk * pk.nhc, s);
}

}  // namespace blk
