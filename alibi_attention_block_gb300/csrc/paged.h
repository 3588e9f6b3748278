// The paged cache as its kernels see it (kv_append.cu, attn_paged.cu).
#pragma once

#include "internal.h"

namespace blk {

struct PagedCache {
    void* k;  // [pages][Hk][page tokens][d] from page_stride to page_stride, 16-bit values or e4m3 codes
    void* v;
    float* k_scale;  // [pages][Hk] (e4m3), else nullptr
    float* v_scale;
    const int32_t* table;  // [B][max_pages]
    const int32_t* lens;   // [B]
    int64_t page_stride;   // elements
    int pages, page_log2, max_pages, B, Hk, d;
};

// Checks a cache's descriptor, or a cache with its pointers (written: by the append).
blk_status check_paged_desc(const blk_paged_desc* d);
blk_status make_paged_cache(const blk_paged_desc* d, const void* k, const void* v,
                            const float* k_scale, const float* v_scale, const int32_t* table,
                            const int32_t* lens, PagedCache* out);

}  // namespace blk
