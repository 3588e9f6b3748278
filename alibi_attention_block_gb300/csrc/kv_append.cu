// K7: new tokens into a paged key/value cache, the rotary applied on the way
// (blk_kv_append_paged).
//
// Sequence b has lens[b] tokens with its new ones, which are rows cu[b] ..
// cu[b+1] - 1 of k and v (without cu: row b) at the positions ending at lens[b] - 1.
// Position p lies in page table[b][p / page], row p % page. The keys are turned at
// their positions (nnterp "stablelm" 03 Notes; angles: turn.cuh), the values
// are not; the queries, if given, are turned in the same launch.
//
// 8 bits: value = e4m3 code * scale, one scale for each page and kv head, K and V
// apart: the smallest power of two of at least 2^-60 with which no finite value of
// the page needs a code above 448. A power of two costs e4m3 nothing (its steps are
// relative), and makes a page's contents independent of how its tokens came: where
// a later token needs a larger scale, the codes held are divided by a power of two,
// which is exact down to e4m3's subnormals (only codes of below 2^-6 after the division
// are rounded a second time). A page's scale never falls while the page fills.
//
// Work: a block takes one page's new rows of one head of K or V, so that the page's
// largest value is found and used in one place, without atomics: each thread holds
// its turned values in registers between the two. Blocks of queries take a
// group of heads and reuse the angles. The number of pages that a sequence
// touches is device data: sequence b's blocks are numbers floor(cu[b] / page) + 2 b and
// up, which leaves room for floor(n / page) + 2 pages, enough for n tokens from any
// offset; surplus blocks end at once. Bound by bytes: the new rows read once, their
// codes and scales written once.
#include <cuda_fp8.h>

#include <cmath>

#include "paged.h"
#include "turn.cuh"

namespace blk {

namespace {

struct AppendArgs {
    TurnArgs turn;
    PagedCache c;
    const void* x[3];  // k, v, q
    void* q_out;
    int64_t xs[3][2], qs[2];  // strides of heads and tokens, in elements
    const int32_t* cu;         // or nullptr: one token per sequence
    const int32_t* positions;  // of the rotary, or nullptr: the cache's
    int tokens, H, per;        // query heads, and of them per block
    int pdl;
};

// The new rows of one page of one sequence.
struct PageRows {
    int b, first, n;   // sequence; first row in the page, rows
    int page;          // column of the table
    int64_t row, pos;  // of the first: row of k, v and q, position
};

__device__ __forceinline__ int start_of(const AppendArgs& a, int b) {
    return min(max(a.cu[b], 0), a.tokens);
}

// Rows of item i, in every thread of a warp alike; false: none.
__device__ __forceinline__ bool rows_of(const AppendArgs& a, int64_t i, int lane, PageRows& r) {
    const int lg = a.c.page_log2;
    int64_t c0, n, at;
    if (a.cu) {
        // the last sequence whose numbers begin at or ahead of i
        int lo = 0, hi = a.c.B;
        while (hi - lo > 1) {
            const int step = (hi - lo + 31) / 32;
            const int64_t b = lo + static_cast<int64_t>(lane + 1) * step;
            const bool ahead =
                b < hi && (start_of(a, static_cast<int>(b)) >> lg) + 2 * b <= i;
            lo += __popc(__ballot_sync(0xffffffffu, ahead)) * step;
            hi = min(hi, lo + step);
        }
        r.b = lo;
        c0 = start_of(a, lo);
        n = start_of(a, lo + 1) - c0;
        at = i - ((c0 >> lg) + 2 * static_cast<int64_t>(lo));
    } else {
        r.b = static_cast<int>(i);
        c0 = i;
        n = 1;
        at = 0;
    }
    const int64_t end = a.c.lens[r.b];
    int64_t p0 = end - n;  // of the sequence's first new row
    c0 -= p0;              // row of position 0
    p0 = p0 < 0 ? 0 : p0;
    const int64_t page = (p0 >> lg) + at;
    const int64_t lo = max(p0, page << lg), hi = min(end, (page + 1) << lg);
    if (at < 0 || lo >= hi) return false;
    r.first = static_cast<int>(lo - (page << lg));
    r.n = static_cast<int>(hi - lo);
    r.page = static_cast<int>(page);
    r.row = c0 + lo;
    r.pos = lo;
    return true;
}

__device__ __forceinline__ uint32_t finite_bits(float x) {
    const uint32_t u = __float_as_uint(x) & 0x7fffffffu;
    return u < 0x7f800000u ? u : 0u;
}

// The smallest power of two of at least 2^-60 with which |x| (its bits) takes at most 448 = 1.75 * 2^8.
__device__ __forceinline__ float scale_for(uint32_t bits) {
    const int e = static_cast<int>((bits + 0x1fffffu) >> 23) - 127 - 8;
    return __uint_as_float(static_cast<uint32_t>(max(e, -60) + 127) << 23);
}

__device__ __forceinline__ uint32_t e4m3_pair(float x, float y) {
    return __nv_cvt_float2_to_fp8x2(make_float2(x, y), __NV_SATFINITE, __NV_E4M3);
}
template <int VP>
__device__ __forceinline__ void store_codes(uint8_t* p, const float* f, float inv) {
    if constexpr (VP == 8) {
        const uint32_t lo = e4m3_pair(f[0] * inv, f[1] * inv) | e4m3_pair(f[2] * inv, f[3] * inv) << 16;
        const uint32_t hi = e4m3_pair(f[4] * inv, f[5] * inv) | e4m3_pair(f[6] * inv, f[7] * inv) << 16;
        *reinterpret_cast<uint2*>(p) = make_uint2(lo, hi);
    } else if constexpr (VP == 4) {
        *reinterpret_cast<uint32_t*>(p) =
            e4m3_pair(f[0] * inv, f[1] * inv) | e4m3_pair(f[2] * inv, f[3] * inv) << 16;
    } else {
        *p = static_cast<uint8_t>(e4m3_pair(f[0] * inv, 0.f));
    }
}

// Four codes times a factor, rounded to codes again.
__device__ __forceinline__ uint32_t rescaled(uint32_t codes, float by) {
    uint32_t out = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(
            static_cast<__nv_fp8x2_storage_t>(codes >> (16 * i)), __NV_E4M3);
        const float2 f = __half22float2(__half2(h));
        out |= e4m3_pair(f.x * by, f.y * by) << (16 * i);
    }
    return out;
}

// Threads: so many that IT rounds of them take a whole page (threads_for).
template <typename T, bool E8, int VP, int IT>
__global__ void __launch_bounds__(512) kv_append_kernel(const __grid_constant__ AppendArgs a) {
    __shared__ uint32_t most[16];
    const int d = a.c.d, units = d / (2 * VP);
    const int rows = blockDim.x / units;  // of a round
    const int u = threadIdx.x % units, r0 = threadIdx.x / units;
    const int lane = threadIdx.x & 31;
    const bool mine = r0 < rows;
    // heads of K, then of V, then groups of query heads
    const int what = blockIdx.y < a.c.Hk ? 0 : blockIdx.y < 2 * a.c.Hk ? 1 : 2;
    const int head = blockIdx.y - what * a.c.Hk;
    const Unit<VP> at(u, what == 1 ? 0 : a.turn.plan.pairs, a.turn.plan.interleaved);
    uint64_t turns[VP];
#pragma unroll
    for (int i = 0; i < VP; ++i) turns[i] = at.turned ? a.turn.plan.turns[u * VP + i] : 0;
    const float m = a.turn.plan.amplitude;
    if (a.pdl) pdl_wait();
    PageRows r;
    if (!rows_of(a, blockIdx.x, lane, r)) return;
    const T* x = static_cast<const T*>(a.x[what]) + r.row * a.xs[what][1];

    if (what == 2) {
        const int h1 = min((head + 1) * a.per, a.H);
        for (int k = mine ? r0 : r.n; k < r.n; k += rows) {
            Angles<VP> ang;
            if (at.turned)
                ang.set(turns, a.positions ? a.positions[r.row + k] : static_cast<int>(r.pos + k), m, m);
#pragma unroll 4
            for (int h = head * a.per; h < h1; ++h) {
                const T* src = x + h * a.xs[2][0] + k * a.xs[2][1];
                T* dst = static_cast<T*>(a.q_out) + h * a.qs[0] + (r.row + k) * a.qs[1];
                float p[VP], q[VP];
                load_piece(src + at.a, p);
                load_piece(src + at.b, q);
                if (at.turned) ang.turn(p, q, a.turn.plan.interleaved);
                store_piece(dst + at.a, p);
                store_piece(dst + at.b, q);
            }
        }
        return;
    }

    // a page of the sequence's that is not there takes nothing
    if (r.page >= a.c.max_pages) return;
    const int page = a.c.table[static_cast<int64_t>(r.b) * a.c.max_pages + r.page];
    if (page < 0 || page >= a.c.pages) return;
    const int64_t base = page * a.c.page_stride + (static_cast<int64_t>(head) << a.c.page_log2) * d;
    x += head * a.xs[what][0];
    float v[IT][2][VP];
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < IT; ++i) {
        const int k = r0 + i * rows;
        if (mine && k < r.n) {
            load_piece(x + k * a.xs[what][1] + at.a, v[i][0]);
            load_piece(x + k * a.xs[what][1] + at.b, v[i][1]);
        }
    }
#pragma unroll
    for (int i = 0; i < IT; ++i) {
        const int k = r0 + i * rows;
        if (mine && k < r.n) {
            if (at.turned) {
                Angles<VP> ang;
                ang.set(turns, a.positions ? a.positions[r.row + k] : static_cast<int>(r.pos + k), m, m);
                ang.turn(v[i][0], v[i][1], a.turn.plan.interleaved);
            }
            if constexpr (E8) {
#pragma unroll
                for (int e = 0; e < VP; ++e)
                    top = max(top, max(finite_bits(v[i][0][e]), finite_bits(v[i][1][e])));
            }
        }
    }
    if constexpr (E8) {
        float* scales = what ? a.c.v_scale : a.c.k_scale;
        float* scale = scales + static_cast<int64_t>(page) * a.c.Hk + head;
        uint8_t* codes = static_cast<uint8_t*>(what ? a.c.v : a.c.k) + base;
        // a page's first row begins its scale anew
        const float held = r.first > 0 ? *scale : 0.f;
        top = __reduce_max_sync(0xffffffffu, top);
        if (lane == 0) most[threadIdx.x / 32] = top;
        __syncthreads();
        for (int w = 0; w < static_cast<int>(blockDim.x) / 32; ++w) top = max(top, most[w]);
        const float now = fmaxf(scale_for(top), held);
        if (threadIdx.x == 0) *scale = now;
        if (r.first > 0 && held < now) {
            const float by = held / now;
            uint4* old = reinterpret_cast<uint4*>(codes);
            for (int i = threadIdx.x; i < r.first * (d / 16); i += blockDim.x) {
                uint4 o = old[i];
                o.x = rescaled(o.x, by);
                o.y = rescaled(o.y, by);
                o.z = rescaled(o.z, by);
                o.w = rescaled(o.w, by);
                old[i] = o;
            }
        }
        const float inv = 1.0f / now;
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            const int k = r0 + i * rows;
            if (mine && k < r.n) {
                uint8_t* dst = codes + (r.first + k) * d;
                store_codes<VP>(dst + at.a, v[i][0], inv);
                store_codes<VP>(dst + at.b, v[i][1], inv);
            }
        }
    } else {
        T* cache = static_cast<T*>(what ? a.c.v : a.c.k) + base;
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            const int k = r0 + i * rows;
            if (mine && k < r.n) {
                T* dst = cache + (r.first + k) * d;
                store_piece(dst + at.a, v[i][0]);
                store_piece(dst + at.b, v[i][1]);
            }
        }
    }
}

template <typename T, bool E8, int VP, int IT>
cudaError_t launch_append(const AppendArgs& a, int64_t items, int slots, cudaStream_t s) {
    const int units = a.c.d / (2 * VP), page = 1 << a.c.page_log2;
    const int threads = (units * ((page + IT - 1) / IT) + 31) / 32 * 32;
    return launch_pdl(a.pdl != 0, kv_append_kernel<T, E8, VP, IT>,
                      dim3(static_cast<unsigned>(items), static_cast<unsigned>(slots)), dim3(threads), 0,
                      s, a);
}
template <typename T, bool E8>
cudaError_t launch_append_w(const AppendArgs& a, int64_t items, int slots, cudaStream_t s) {
    switch (turn_width(a.turn.plan.pairs)) {  // 64 values held per thread
        case 8: return launch_append<T, E8, 8, 4>(a, items, slots, s);
        case 4: return launch_append<T, E8, 4, 8>(a, items, slots, s);
        default: return launch_append<T, E8, 1, 32>(a, items, slots, s);
    }
}

#define REQUIRE(cond, ...)                                                \
    do {                                                                  \
        if (!(cond)) return report_error_status(BLK_EINVAL, __VA_ARGS__); \
    } while (0)

}  // namespace

blk_status check_paged_desc(const blk_paged_desc* d) {
    REQUIRE(d, "cache desc is NULL");
    REQUIRE(d->kind == BLK_CACHE_16BIT || d->kind == BLK_CACHE_E4M3, "unknown kind of cache");
    REQUIRE(d->pages >= 1 && d->pages <= (int64_t(1) << 30), "pages out of range");
    REQUIRE(d->max_pages >= 1 && d->batch >= 1 && d->batch <= (int64_t(1) << 24) &&
                d->max_pages <= (int64_t(1) << 24),
            "batch or max_pages out of range");
    if (d->page_tokens != 16 && d->page_tokens != 32 && d->page_tokens != 64 && d->page_tokens != 128)
        return report_error_status(BLK_EUNSUPPORTED, "page_tokens must be 16, 32, 64 or 128");
    REQUIRE(d->max_pages * d->page_tokens <= 0x7fffff80, "max_pages * page_tokens out of range");
    REQUIRE(d->n_kv_heads >= 1 && d->n_kv_heads <= 4096, "n_kv_heads out of range");
    if (d->head_dim < 16 || d->head_dim % 16 != 0 || d->head_dim > 256)
        return report_error_status(BLK_EUNSUPPORTED, "head_dim must be a multiple of 16 in [16, 256]");
    const int64_t least = d->n_kv_heads * d->page_tokens * d->head_dim;
    REQUIRE(d->page_stride >= least && d->page_stride % 16 == 0 && d->page_stride <= (int64_t(1) << 36),
            "page_stride must be a multiple of 16 elements and hold a page");
    REQUIRE(d->pages <= (int64_t(1) << 48) / d->page_stride, "cache too large");
    return BLK_OK;
}

blk_status make_paged_cache(const blk_paged_desc* d, const void* k, const void* v,
                            const float* k_scale, const float* v_scale, const int32_t* table,
                            const int32_t* lens, PagedCache* out) {
    const blk_status st = check_paged_desc(d);
    if (st != BLK_OK) return st;
    REQUIRE(k && (reinterpret_cast<uintptr_t>(k) & 15u) == 0 && v &&
                (reinterpret_cast<uintptr_t>(v) & 15u) == 0,
            "k_cache and v_cache must be 16-byte aligned device pointers");
    if (d->kind == BLK_CACHE_E4M3)
        REQUIRE(k_scale && (reinterpret_cast<uintptr_t>(k_scale) & 3u) == 0 && v_scale &&
                    (reinterpret_cast<uintptr_t>(v_scale) & 3u) == 0,
                "an e4m3 cache has k_scale and v_scale, 4-byte aligned");
    else
        REQUIRE(!k_scale && !v_scale, "a 16-bit cache has no scales");
    REQUIRE(table && (reinterpret_cast<uintptr_t>(table) & 3u) == 0 && lens &&
                (reinterpret_cast<uintptr_t>(lens) & 3u) == 0,
            "block_table and lens must be 4-byte aligned device pointers");
    out->k = const_cast<void*>(k);
    out->v = const_cast<void*>(v);
    out->k_scale = const_cast<float*>(k_scale);
    out->v_scale = const_cast<float*>(v_scale);
    out->table = table;
    out->lens = lens;
    out->page_stride = d->page_stride;
    out->pages = static_cast<int>(d->pages);
    out->page_log2 = d->page_tokens == 16 ? 4 : d->page_tokens == 32 ? 5 : d->page_tokens == 64 ? 6 : 7;
    out->max_pages = static_cast<int>(d->max_pages);
    out->B = static_cast<int>(d->batch);
    out->Hk = static_cast<int>(d->n_kv_heads);
    out->d = static_cast<int>(d->head_dim);
    return BLK_OK;
}

}  // namespace blk

using namespace blk;

extern "C" blk_status blk_kv_append_paged(const blk_append_desc* d, const blk_rope_plan* rope,
                                          const void* k, const void* v, const void* q,
                                          const int32_t* cu_seqlens, const int32_t* positions,
                                          const int32_t* block_table, const int32_t* lens,
                                          void* k_cache, void* v_cache, float* k_scale,
                                          float* v_scale, void* q_out, blk_dtype dt, blk_stream_t s) {
    REQUIRE(dt == BLK_F16 || dt == BLK_BF16, "dtype must be BLK_F16 or BLK_BF16");
    REQUIRE(d, "desc is NULL");
    AppendArgs a{};
    blk_status st = make_paged_cache(&d->cache, k_cache, v_cache, k_scale, v_scale, block_table, lens, &a.c);
    if (st != BLK_OK) return st;
    REQUIRE(d->tokens >= 1 && d->tokens <= (int64_t(1) << 30), "tokens out of range");
    REQUIRE(cu_seqlens || d->tokens == d->cache.batch, "without cu_seqlens there is one token per sequence");
    REQUIRE((reinterpret_cast<uintptr_t>(cu_seqlens) & 3u) == 0 &&
                (reinterpret_cast<uintptr_t>(positions) & 3u) == 0,
            "cu_seqlens and positions must be 4-byte aligned");
    REQUIRE(rope || !positions, "positions given without a rotary");
    REQUIRE(!rope || plan_made(rope, d->cache.head_dim),
            "rope was not made by blk_rope_plan_init, or its span is above head_dim");
    REQUIRE(d->n_heads >= 0 && d->n_heads <= 16384 && (d->n_heads > 0) == (q != nullptr) &&
                (q != nullptr) == (q_out != nullptr),
            "q, q_out and n_heads go together");
    const void* ptrs[4] = {k, v, q, q_out};
    const int64_t strides[4][2] = {{d->k_head_stride, d->k_token_stride},
                                   {d->v_head_stride, d->v_token_stride},
                                   {d->q_head_stride, d->q_token_stride},
                                   {d->q_out_head_stride, d->q_out_token_stride}};
    REQUIRE(k && v, "k or v is NULL");
    for (int i = 0; i < (q ? 4 : 2); ++i) {
        REQUIRE((reinterpret_cast<uintptr_t>(ptrs[i]) & 15u) == 0, "tensors must be 16-byte aligned");
        for (int j = 0; j < 2; ++j)
            REQUIRE(strides[i][j] >= 0 && strides[i][j] % 8 == 0 && strides[i][j] <= (int64_t(1) << 40),
                    "strides must be multiples of 8 elements");
    }
    REQUIRE(!q || q != q_out || (strides[2][0] == strides[3][0] && strides[2][1] == strides[3][1]),
            "an output in place has the input's strides");
    for (int i = 0; i < 3; ++i) {
        a.x[i] = ptrs[i];
        for (int j = 0; j < 2; ++j) a.xs[i][j] = strides[i][j];
    }
    a.q_out = q_out;
    a.qs[0] = strides[3][0];
    a.qs[1] = strides[3][1];
    if (rope) a.turn.plan = *rope;
    a.cu = cu_seqlens;
    a.positions = positions;
    a.tokens = static_cast<int>(d->tokens);
    a.H = static_cast<int>(d->n_heads);
    int sms = 0;
    unsigned* err = nullptr;
    if ((st = current_device_info(&sms, &err)) != BLK_OK) return st;
    const cudaStream_t cs = reinterpret_cast<cudaStream_t>(s);
    a.pdl = pdl_allowed(cs);
    const int64_t items = cu_seqlens ? (d->tokens >> a.c.page_log2) + 2 * d->cache.batch : d->tokens;
    REQUIRE(items <= 0x7fffffff, "tokens and batch too large");
    // query heads per block: fewer where there are few tokens
    const int64_t rows = d->tokens * d->n_heads / (1 << a.c.page_log2);
    int64_t per = rows / (8 * sms);
    per = per < 1 ? 1 : per > 8 ? 8 : per;
    a.per = static_cast<int>(per);
    const int slots = static_cast<int>(2 * d->cache.n_kv_heads + (d->n_heads + per - 1) / per);
    const bool e8 = d->cache.kind == BLK_CACHE_E4M3;
    const cudaError_t e =
        dt == BLK_F16 ? (e8 ? launch_append_w<__half, true>(a, items, slots, cs)
                            : launch_append_w<__half, false>(a, items, slots, cs))
                      : (e8 ? launch_append_w<__nv_bfloat16, true>(a, items, slots, cs)
                            : launch_append_w<__nv_bfloat16, false>(a, items, slots, cs));
    return e == cudaSuccess ? BLK_OK
                            : report_error_status(BLK_ECUDA, "append launch: %s", cudaGetErrorString(e));
}
