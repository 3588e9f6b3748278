// K3 dispatch: causal softmax attention by head_dim and group size.
//   head_dim 64            attn_pair.cu     (two query tiles per item; any GQA)
//   head_dim 128, MHA      attn_pair128.cu  (two query tiles, shared S buffer)
//   head_dim 128, GQA      attn_gqa.cu      (the group's query heads packed
//   head_dim 160, any      attn_gqa.cu       into one 128-row tile)
// Packed prompts: head_dim 64 as above; 128 and 160 two query tiles of packed
// heads (attn_pair128.cu, attn_pair160.cu), or one where ALiBi meets grouped heads
// (attn_gqa.cu).
#include "internal.h"

namespace blk {

namespace {

// ---- packed prompts: the work list -----------------------------------
// The prompts' lengths are device data, so the list of work units is built on
// the device: a short one by every CTA of the attention kernel for itself
// (attn_plan.cuh), a long one by one block ahead of it. Unit l of a prompt
// attends to about l key tiles more than unit 0, so a counting sort by l (in
// kPlanBins bins of 2^shift units), largest first, orders the units heaviest
// first, as the dense kernels order theirs. The order within a bin is whatever
// the shared atomics give; every unit is computed alike wherever it stands, so
// results do not depend on it. The table cannot be checked on the host: its
// entries are clamped to [0, tokens] and each raised to the greatest before it,
// so that the prompts' lengths add up to at most tokens whatever it holds, and
// the units to at most max_units.
constexpr int kPlanThreads = 1024, kPlanBins = 2048;

__global__ void __launch_bounds__(kPlanThreads)
    plan_kernel(const int32_t* cu, int prompts, int tokens, int unit, int shift, int max_units,
                int4* plan, int pdl) {
    __shared__ int at[kPlanBins];
    __shared__ int warp_sum[kPlanThreads / 32];
    __shared__ int first_of[kPlanThreads + 1];
    if (pdl) {
        pdl_wait();
        pdl_launch_dependents();
    }
    const int t = threadIdx.x, lane = t & 31, warp = t / 32;
    at[t] = 0;
    at[t + kPlanThreads] = 0;
    __syncthreads();
    // the table in pieces of kPlanThreads prompts; of a piece one warp per
    // prompt, one lane per unit
    auto each_unit = [&](auto&& f) {
        int before = 0;  // the greatest entry ahead of the piece
        for (int base = 0; base < prompts; base += kPlanThreads) {
            const int e = base + t;
            int v = e <= prompts ? min(max(cu[e], 0), tokens) : 0;
            const int behind = base + kPlanThreads <= prompts && t == kPlanThreads - 1
                                   ? min(max(cu[base + kPlanThreads], 0), tokens)
                                   : 0;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int u = __shfl_up_sync(0xffffffffu, v, o);
                if (lane >= o) v = max(v, u);
            }
            if (lane == 31) warp_sum[warp] = v;
            __syncthreads();
            v = max(max(v, before), __reduce_max_sync(0xffffffffu, lane < warp ? warp_sum[lane] : 0));
            first_of[t] = v;
            if (t == kPlanThreads - 1) first_of[kPlanThreads] = max(v, behind);
            __syncthreads();
            const int n_here = min(prompts - base, kPlanThreads);
            for (int i = warp; i < n_here; i += kPlanThreads / 32) {
                const int first = first_of[i], len = first_of[i + 1] - first;
                const int n = len / unit + (len % unit != 0);
                for (int l = lane; l < n; l += 32) f(first, len, l);
            }
            before = first_of[kPlanThreads - 1];
            __syncthreads();
        }
    };
    each_unit([&](int, int, int l) { atomicAdd(&at[l >> shift], 1); });
    __syncthreads();
    // exclusive sums from the last bin down: thread t owns bins hi and hi - 1
    const int hi = kPlanBins - 1 - 2 * t;
    const int c0 = at[hi], c1 = at[hi - 1];
    int sum = c0 + c1;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += v;
    }
    if (lane == 31) warp_sum[warp] = sum;
    __syncthreads();
    if (warp == 0) {
        int w = warp_sum[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, w, o);
            if (lane >= o) w += v;
        }
        warp_sum[lane] = w;
    }
    __syncthreads();
    const int end = sum + (warp ? warp_sum[warp - 1] : 0);
    at[hi] = end - c0 - c1;
    at[hi - 1] = end - c1;
    if (t == 0) plan[0] = make_int4(min(warp_sum[kPlanThreads / 32 - 1], max_units), 0, 0, 0);
    __syncthreads();
    each_unit([&](int first, int len, int l) {
        const int i = atomicAdd(&at[l >> shift], 1);
        if (i < max_units) plan[1 + i] = make_int4(first, len, l, 0);
    });
}

// a query-tile pair per item, or one tile (attn_gqa.cu)
bool packed_pairs(int H, int Hk, int d, bool alibi) {
    return d == 64 || H == Hk || !alibi;
}
// positions per unit
int packed_unit(int H, int Hk, int d, bool alibi) {
    if (d == 64) return 256;
    int G, Gt, R, nhc;
    gqa_tile(H, Hk, &G, &Gt, &R, &nhc);
    return packed_pairs(H, Hk, d, alibi) ? 2 * R : R;
}

}  // namespace

int64_t packed_max_units(int64_t tokens, int64_t prompts, int H, int Hk, int d, bool alibi) {
    return tokens / packed_unit(H, Hk, d, alibi) + prompts;
}

int64_t packed_plan_entries(int64_t tokens, int64_t prompts, int H, int Hk, int d, bool alibi) {
    const int64_t units = packed_max_units(tokens, prompts, H, Hk, d, alibi);
    return prompts <= kPlanCtaPrompts && units <= kPlanCtaUnits ? 0 : 1 + units;
}

cudaError_t launch_attention_packed(DType dt, const AttnArgs& a, const PackedArgs& p,
                                    cudaStream_t s) {
    const int unit = packed_unit(a.H, a.Hk, a.d, a.alibi != 0);
    const int64_t max_units = packed_max_units(a.S, p.prompts, a.H, a.Hk, a.d, a.alibi != 0);
    int shift = 0;
    while ((static_cast<int64_t>(a.S / unit) >> shift) >= kPlanBins) ++shift;
    AttnPack<true> pack;
    const bool listed = packed_plan_entries(a.S, p.prompts, a.H, a.Hk, a.d, a.alibi != 0) != 0;
    pack.plan = listed ? p.plan : nullptr;
    pack.cu_seqlens = p.cu_seqlens;
    pack.prompts = p.prompts;
    pack.prefix = p.prefix;
    // without a prefix the maps are never used: any valid one will do
    const void* kp = p.prefix ? p.k_prefix : a.k;
    const void* vp = p.prefix ? p.v_prefix : a.v;
    const uint64_t rows = p.prefix ? p.prefix : a.S;
    const bool pair160 = a.d == 160 && packed_pairs(a.H, a.Hk, a.d, a.alibi != 0);
    const uint32_t tile = pair160 ? 64 : 128;  // keys per tile
    if (!make_tmap_3d(&pack.tmPK, dt, kp, a.Hk, rows, a.d, tile) ||
        !make_tmap_3d(&pack.tmPK2, dt, kp, a.Hk, rows, a.d, tile, 32) ||
        !make_tmap_3d(&pack.tmPV, dt, vp, a.Hk, rows, a.d, tile))
        return cudaErrorInvalidValue;
    if (listed) {
        const bool pdl = pdl_allowed(s);
        const cudaError_t e = launch_pdl(pdl, plan_kernel, dim3(1), dim3(kPlanThreads), 0, s,
                                         p.cu_seqlens, p.prompts, a.S, unit, shift,
                                         static_cast<int>(max_units), p.plan, pdl ? 1 : 0);
        if (e != cudaSuccess) return e;
    }
    if (a.d == 64) return launch_attention_pair64_packed(dt, a, pack, max_units, s);
    if (pair160) return launch_attention_pair160_packed(dt, a, pack, max_units, s);
    if (packed_pairs(a.H, a.Hk, a.d, a.alibi != 0))
        return launch_attention_pair128_packed(dt, a, pack, max_units, s);
    return launch_attention_gqa_packed(dt, a, pack, max_units, s);
}

cudaError_t launch_attention(DType dt, const AttnArgs& a, cudaStream_t s) {
    if (a.B == 0 || a.S == 0) return cudaSuccess;
    switch (a.d) {
        case 64: return launch_attention_pair64(dt, a, s);
        case 128:
            return a.H == a.Hk ? launch_attention_pair128(dt, a, s) : launch_attention_gqa(dt, a, s);
        case 160: return launch_attention_gqa(dt, a, s);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace blk
