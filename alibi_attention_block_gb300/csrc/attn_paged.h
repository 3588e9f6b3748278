// Host side of the paged decode step and its kernels (attn_paged.cu, attn_paged_*.cu).
#pragma once

#include "paged.h"

namespace blk {

constexpr int kPagedMaxGrid = 640;  // CTAs at most

// [K, V][boxes of a page's rows, of 16][128-byte slices, the 64-byte slice]
struct PagedMapSet {
    CUtensorMap m[2][2][2];
};
struct PagedMaps {
    const CUtensorMap* m[2][2];
};

struct PagedArgs {
    PagedCache c;
    const void* q;
    int64_t qs[2];  // strides of sequences and heads, in elements
    // partial results: [records][GP][d], [records][GP] (reference, sum; log2 domain); record
    // cta + b * units + u for a CTA's stay in unit (b, u)
    float* po;
    float2* pm;
    int64_t* cum;  // [B + 1] 128-key tiles ahead of each sequence (per unit)
    const float* slopes;
    unsigned* err;
    int H, G, GP;   // query heads; of a kv head; of a unit, at most
    int groups;     // units of a kv head: ceil(G / GP)
    int units;      // of a sequence
    int grid;
    float scale;
    int alibi, pdl;
    int direct;  // a unit per CTA, rows to o
    void* o;
};

cudaError_t launch_paged_f16(bool e8, const PagedMapSet& tm, PagedArgs& a, int sms, cudaStream_t s);
cudaError_t launch_paged_bf16(bool e8, const PagedMapSet& tm, PagedArgs& a, int sms, cudaStream_t s);

}  // namespace blk
