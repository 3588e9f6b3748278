// The work list of packed prompts (see attn.cu), as the attention kernels read
// it: from the workspace, or built by every CTA for itself in shared memory.
#pragma once

#include "internal.h"

namespace blk {

// One unit of work: unit l (256 or R positions from l * unit on) of the prompt
// at rows first .. first + len - 1.
struct PlanUnit {
    int first, len, l;
};

// A small list is built by each CTA: the table's entries are in L2, and a kernel
// that only builds the list costs 2.6 us, its launch and a workspace. In a graph, in
// us, built by each CTA and in the workspace (16 x 64 heads, ALiBi, turns of 25
// tokens):
//    16 turns  11.7  15.7     64   30.7  31.2    128   57.2  51.9    255  106.3  90.3
// (32 x 64 heads: 4 prompts of 2000 90.9 and 96.2, 8 of 1273 83.8 and 89.4). Where
// all prompts are one unit there is one level, which one thread lists: above some
// 64 such prompts that costs more than the launch. Every CTA has to come to the same
// order, so no atomics: prompts are ranked by their number of units (ties by
// index), and unit l of the prompt of rank r comes behind all units above l, in
// the order of the ranks among those of level l. Where a unit is a pair of query
// tiles, those of prompts with an odd number of tiles are the last of their
// level: paired from the end, they attend to a key tile less (five prompts of
// 1788 tokens on average, 16 x 128 heads: 96.4 us without, 91.8 with; eight of 1273,
// 32 x 64 heads: 100.6 and 97.8).
//
// Items go round the CTAs in this order, every other round reversed. A model says
// that giving each round's items by the CTAs' loads so far saves 4 to 7 % more;
// done by a warp of its own, beside the products, it saved 2 % at 16 x 128 heads
// and cost 4 to 16 % elsewhere.
struct PlanSmem {
    int first[kPlanCtaPrompts], len[kPlanCtaPrompts];
    int n[kPlanCtaPrompts], sorted_n[kPlanCtaPrompts];  // 2 * units + odd
    uint16_t sorted_b[kPlanCtaPrompts];
    uint32_t list[kPlanCtaUnits];  // prompt << 16 | l
    int total;
};
struct PlanNone {};
template <bool PACKED>
struct PlanStorage { using type = PlanNone; };
template <>
struct PlanStorage<true> { using type = PlanSmem; };

// All threads of the block; ends with a block barrier. The table's entries are
// clamped to a nondecreasing pair within [0, tokens], and units past the
// list's room dropped. tile: positions of a query tile where a unit is a pair of
// them, else 0.
__device__ __forceinline__ void build_plan(PlanSmem& p, const int32_t* cu, int prompts, int tokens,
                                           int unit, int tile) {
    const int nt = static_cast<int>(blockDim.x), t = static_cast<int>(threadIdx.x);
    for (int b = t; b < prompts; b += nt) {
        const int first = min(max(cu[b], 0), tokens);
        const int len = min(max(cu[b + 1], first), tokens) - first;
        p.first[b] = first;
        p.len[b] = len;
        p.n[b] = (len + unit - 1) / unit * 2 + (tile ? (len + tile - 1) / tile & 1 : 0);
    }
    __syncthreads();
    for (int b = t; b < prompts; b += nt) {
        const int n = p.n[b];
        int rank = 0;
        for (int o = 0; o < prompts; ++o) {
            const int v = p.n[o];
            rank += v > n || (v == n && o < b);
        }
        p.sorted_n[rank] = n;
        p.sorted_b[rank] = static_cast<uint16_t>(b);
    }
    __syncthreads();
    const int levels = p.sorted_n[0] >> 1;
    if (t == 0 && levels == 0) p.total = 0;
    for (int l = t; l < levels; l += nt) {
        // units above level l; prompts that have level l, and the even ones
        int at = 0, r = 0, evens = 0;
        for (; r < prompts && (p.sorted_n[r] >> 1) > l; ++r) {
            at += (p.sorted_n[r] >> 1) - 1 - l;
            evens += !(p.sorted_n[r] & 1);
        }
        if (l == 0) p.total = min(at + r, kPlanCtaUnits);
        int odd_at = at + evens;
        for (int i = 0; i < r; ++i) {
            const int to = p.sorted_n[i] & 1 ? odd_at++ : at++;
            if (to < kPlanCtaUnits)
                p.list[to] = static_cast<uint32_t>(p.sorted_b[i]) << 16 | static_cast<uint32_t>(l);
        }
    }
    __syncthreads();
}

// Limit of a softmax warpgroup's wait for scores. A work item without a second
// query tile leaves the second tile's warpgroup waiting through it, and a long
// prefix behind many short prompts makes such items last seconds together (13200
// prompts of one token, 4 heads of 64, behind 2^20 shared keys: 2.7 s). Such an
// item has the prefix's key tiles and two of its own at most, and a tile takes 1 to
// 2 us; this allows 10 for each item that the CTA has been through.
__device__ __forceinline__ unsigned long long idle_limit_ns(int items, int prefix_tiles) {
    return kWaitLimitNs + static_cast<unsigned long long>(items + 1) * (prefix_tiles + 2) * 10000ull;
}

template <typename Plan>
__device__ __forceinline__ int plan_units(const AttnPack<true>& pack, const Plan& p) {
    return pack.plan ? pack.plan[0].x : p.total;
}
template <typename Plan>
__device__ __forceinline__ PlanUnit plan_unit(const AttnPack<true>& pack, const Plan& p, int i) {
    if (pack.plan) {
        const int4 u = pack.plan[1 + i];
        return PlanUnit{u.x, u.y, u.z};
    }
    const uint32_t e = p.list[i];
    return PlanUnit{p.first[e >> 16], p.len[e >> 16], static_cast<int>(e & 0xffffu)};
}

}  // namespace blk
