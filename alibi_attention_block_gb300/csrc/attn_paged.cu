// K8 host side and merge: one decode step of attention over a paged cache. The kernel
// (attn_paged.cuh) leaves a partial result for each CTA's stay in a unit; the merge
// joins them: o = sum_i w_i O_i / sum_i w_i l_i, w_i = 2^(m_i - max m) (as the square of 2^((m_i - max m) / 2): with
// 8 bits w_i alone may be too small a number, where l_i is large). m_i = -inf: no key seen (l_i = 0), or each with a score of
// -inf (l_i their number), which leaves no softmax, NaN, where no other record has a finite one.
#include <cmath>

#include "attn_paged.h"

namespace blk {

namespace {

constexpr int kTK = 128;
constexpr int kMergeThreads = 128;

struct MergeArgs {
    const float* po;
    const float2* pm;
    const int64_t* cum;
    const int32_t* lens;
    void* o;
    int64_t rows;  // batch * H
    int batch, H, G, GP, groups, units, capacity, grid, pdl;
};

// The CTA whose range [c * W / n, (c + 1) * W / n) holds tile t, n CTAs in all (W >= n):
// c * W < (t + 1) * n <= (c + 1) * W, from an estimate in floating point that is off by
// one at most (n is at most kPagedMaxGrid).
__device__ __forceinline__ int cta_of(int64_t t, int64_t W, int n) {
    const int64_t x = (t + 1) * n;
    int c = static_cast<int>(static_cast<float>(t) * (static_cast<float>(n) / static_cast<float>(W)));
    while (c * W >= x) --c;
    while ((c + 1) * W < x) ++c;
    return c;
}

// The records of a row: the first one's number and how many they are (0: no key).
struct Records {
    int64_t first;
    int n;
};
__device__ __forceinline__ Records records_of(const MergeArgs& a, int64_t row) {
    const int b = static_cast<int>(row / a.H), h = static_cast<int>(row - static_cast<int64_t>(b) * a.H);
    const int g = h / a.G, in = h - g * a.G;  // kv head, and head of its group
    const int u = g * a.groups + in / a.GP;
    const int n = min(max(a.lens[b], 0), a.capacity);
    if (n == 0) return {0, 0};
    const int64_t W = a.cum[a.batch] * a.units, nt = (n + kTK - 1) / kTK;
    const int64_t t0 = a.cum[b] * a.units + u * nt;
    const int ctas = static_cast<int>(min(static_cast<int64_t>(a.grid), W));
    const int c0 = cta_of(t0, W, ctas), c1 = cta_of(t0 + nt - 1, W, ctas);
    return {(c0 + static_cast<int64_t>(b) * a.units + u) * a.GP + in % a.GP, c1 - c0 + 1};
}

// Eight columns of records [from, n) in steps, joined: f of sum l and reference m.
template <int D>
__device__ __forceinline__ void join(const MergeArgs& a, const Records& r, int col, int from, int step, float& m,
                                     float& l, float (&f)[8]) {
    const float* p = a.po + r.first * D + col;
    const float2* s = a.pm + r.first;
    m = -INFINITY;
    l = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = 0.f;
    // Four records' loads at a time, the ones behind the last without effect: a row of two or three has
    // them all on their way at once (64 sequences of up to 1000 keys, 32/8 x 128: 18.0 -> 17.3 us).
    for (int k = from; k < r.n; k += 4 * step) {
        float4 x[4], y[4];
        float2 ml[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[i] = y[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            ml[i] = make_float2(-INFINITY, 0.f);
            if (k + i * step < r.n) {
                const int64_t at = static_cast<int64_t>(k + i * step) * a.GP;
                const float4* q = reinterpret_cast<const float4*>(p + at * D);
                x[i] = q[0];
                y[i] = q[1];
                ml[i] = s[at];
            }
        }
        float mn = m;
#pragma unroll
        for (int i = 0; i < 4; ++i) mn = fmaxf(mn, ml[i].x);
        const float keep = m == mn ? 1.f : ex2_approx(0.5f * (m - mn));
        m = mn;
        l = l * keep * keep;
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] *= keep * keep;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float half = ml[i].x == mn ? 1.f : ex2_approx(0.5f * (ml[i].x - mn));
            const float w = half * half;
            l = fmaf(half, half * ml[i].y, l);
            const float v[8] = {x[i].x, x[i].y, x[i].z, x[i].w, y[i].x, y[i].y, y[i].z, y[i].w};
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = fmaf(w, v[e], f[e]);
        }
    }
}

// What a row's sums are multiplied by: zeros where no key was seen.
__device__ __forceinline__ float share(float m, float l) {
    return l == 0.f ? 0.f : m == -INFINITY ? NAN : 1.0f / l;
}

// D / 8 threads per row of 8 columns each.
template <typename T, int D>
__global__ void __launch_bounds__(kMergeThreads) paged_merge_kernel(const MergeArgs a) {
    constexpr int kPer = D / 8, kRows = kMergeThreads / kPer;
    if (a.pdl) pdl_wait();
    const int64_t row = static_cast<int64_t>(blockIdx.x) * kRows + threadIdx.x / kPer;
    const int col = threadIdx.x % kPer * 8;
    if (threadIdx.x >= kRows * kPer || row >= a.rows) return;
    float m, l, f[8];
    join<D>(a, records_of(a, row), col, 0, 1, m, l, f);
    const float inv = share(m, l);
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] *= inv;
    store8(static_cast<T*>(a.o) + row * D + col, f);
}

// The same by a block per row, whose teams of D / 8 threads take records in turn and join theirs
// through shared memory, for few rows: then a row's records are many (one of nearly each CTA where a
// long sequence has few heads) and one load behind the other is what takes the time. One sequence, e4m3,
// 32/8 x 128, 4096, 16384 and 65536 keys: 16.3 -> 8.2 us, 23.8 -> 13.9 and 36.1 -> 27.0; 16 of up to
// 2000: 14.6 -> 13.7. With more rows than in launch_merge_d the blocks are many more than the GPU
// holds at a time, and most rows have two records: 200 of up to 600 keys 28.1 -> 36.3. Blocks of 256 and
// 512 threads: level for one sequence, 14.3 and 16.5 for the sixteen.
constexpr int kRowThreads = 128;
template <typename T, int D>
__global__ void __launch_bounds__(kRowThreads) paged_merge_row_kernel(const MergeArgs a) {
    constexpr int kPer = D / 8, kTeams = kRowThreads / kPer;
    __shared__ __align__(16) float parts[kTeams][D];
    __shared__ float2 ml[kTeams];
    if (a.pdl) pdl_wait();
    const int64_t row = blockIdx.x;
    const int team = threadIdx.x / kPer, col = threadIdx.x % kPer * 8;
    const Records r = records_of(a, row);
    if (team < kTeams && team < r.n) {
        float m, l, f[8];
        join<D>(a, r, col, team, kTeams, m, l, f);
        float4* to = reinterpret_cast<float4*>(parts[team] + col);
        to[0] = make_float4(f[0], f[1], f[2], f[3]);
        to[1] = make_float4(f[4], f[5], f[6], f[7]);
        if (col == 0) ml[team] = make_float2(m, l);
    }
    __syncthreads();
    const int n = min(r.n, kTeams);
    float top = -INFINITY;
    for (int k = 0; k < n; ++k) top = fmaxf(top, ml[k].x);
    for (int c = threadIdx.x; c < D; c += kRowThreads) {
        float l = 0.f, f = 0.f;
#pragma unroll 4
        for (int k = 0; k < n; ++k) {
            const float2 x = ml[k];
            const float half = x.x == top ? 1.f : ex2_approx(0.5f * (x.x - top));
            l = fmaf(half, half * x.y, l);
            f = fmaf(half * half, parts[k][c], f);
        }
        f *= share(top, l);
        static_cast<uint16_t*>(a.o)[row * D + c] = static_cast<uint16_t>(dt_traits<T>::pack2(f, 0.f));
    }
}

template <typename T, int D>
cudaError_t launch_merge_d(const MergeArgs& a, int sms, cudaStream_t s) {
    if (a.rows <= 8 * sms)  // one round of such blocks
        return launch_pdl(a.pdl != 0, paged_merge_row_kernel<T, D>, dim3(static_cast<unsigned>(a.rows)),
                          dim3(kRowThreads), 0, s, a);
    constexpr int per = kMergeThreads / (D / 8);
    return launch_pdl(a.pdl != 0, paged_merge_kernel<T, D>, dim3(static_cast<unsigned>((a.rows + per - 1) / per)),
                      dim3(kMergeThreads), 0, s, a);
}
template <typename T>
cudaError_t launch_merge(const MergeArgs& a, int d, int sms, cudaStream_t s) {
    switch (d) {
        case 64: return launch_merge_d<T, 64>(a, sms, s);
        case 128: return launch_merge_d<T, 128>(a, sms, s);
        default: return launch_merge_d<T, 160>(a, sms, s);
    }
}

#define REQUIRE(cond, ...)                                                \
    do {                                                                  \
        if (!(cond)) return report_error_status(BLK_EINVAL, __VA_ARGS__); \
    } while (0)

blk_status check_desc(const blk_decode_paged_desc* d) {
    REQUIRE(d, "desc is NULL");
    const blk_status st = check_paged_desc(&d->cache);
    if (st != BLK_OK) return st;
    if (d->cache.head_dim != 64 && d->cache.head_dim != 128 && d->cache.head_dim != 160)
        return report_error_status(BLK_EUNSUPPORTED, "head_dim must be 64, 128 or 160");
    REQUIRE(d->n_heads >= 1 && d->n_heads <= 16384 && d->n_heads % d->cache.n_kv_heads == 0,
            "n_heads must be a positive multiple of n_kv_heads");
    REQUIRE(d->q_batch_stride >= 0 && d->q_head_stride >= 0 && d->q_batch_stride % 2 == 0 &&
                d->q_head_stride % 2 == 0 && d->q_batch_stride <= (int64_t(1) << 40) &&
                d->q_head_stride <= (int64_t(1) << 40),
            "q's strides must be even");
    REQUIRE(d->cache.batch * d->n_heads <= (int64_t(1) << 28), "batch and n_heads too large");
    REQUIRE(std::isfinite(d->softmax_scale), "softmax_scale must be finite");
    REQUIRE(d->alibi == 0 || d->alibi == 1, "alibi must be 0 or 1");
    return BLK_OK;
}

// Whether a sequence's tiles, and the units (of eight heads), are so few that a CTA takes each unit whole: 512 keys, and
// 256 units for each CTA that an SM holds (Cfg::kCtas), not much over one round of CTAs. Above that a CTA's start for every unit, and
// units of unequal length, cost more than the second launch. One launch and two, in us, bf16 (units: of up to 100 keys, of up to 500):
//   16/16 x 64, e4m3 (4):     512: 5.7, 9.1 and 8.1, 11.4     1024: 9.7, 11.8 and 15.2, 15.4   1536: 13.6, 13.1 and 20.1, 16.9
//   32/8 x 128, e4m3 (2):     256: 5.3, 9.1 and 7.9, 11.0     512: 10.1, 10.3 and 14.4, 13.9   1024: 18.8, 14.2 and 24.9, 19.2
//   16/16 x 128, 16 bits (2): 256: 4.9, 8.1 and 9.0, 10.7     512: 8.8, 10.4 and 13.4, 13.8    1024: 17.4, 14.5 and 24.8, 22.1
//   32/8 x 160, 16 bits (1):  256: 10.1, 12.3 and 15.5, 14.8  512: 19.8, 16.0 and 28.6, 22.3
// and four sequences of up to 1000 keys (in a graph): 10.3-13.8 and 8.9-10.3.
constexpr int64_t kDirectTiles = 4, kDirectUnits = 256;
bool is_direct(const blk_decode_paged_desc* d) {
    const blk_paged_desc& c = d->cache;
    const int64_t G = d->n_heads / c.n_kv_heads;
    const bool e8 = c.kind == BLK_CACHE_E4M3;
    const int ctas = e8 && c.head_dim == 64 && G <= 4 ? 4 : !e8 && c.head_dim == 160 ? 1 : 2;
    return c.max_pages * c.page_tokens <= kDirectTiles * kTK &&
           c.batch * c.n_kv_heads * ((G + 7) / 8) <= kDirectUnits * ctas;
}

// Query heads of a unit. Sixteen, each reading of the cache for twice the heads, where the bytes bound
// (256 sequences of up to 8192 keys, 16 heads on one, 16 bits: 93 -> 67 us at head_dim 128, 144 -> 94 at 160;
// 32 on one: 178 -> 123, 280 -> 177); not at 64 (59 -> 57, but a call of 32 sequences 16.7 -> 17.6), not over e4m3,
// where the softmax of each head costs more than its bytes (64 -> 77), and not where a CTA takes a unit
// whole, which halves the CTAs (4 sequences of 500 keys, 32/2: 9.0 -> 9.8).
int unit_heads(const blk_decode_paged_desc* d) {
    const int64_t G = d->n_heads / d->cache.n_kv_heads;
    if (G <= 8) return G == 1 ? 1 : G <= 4 ? 4 : 8;
    return d->cache.kind == BLK_CACHE_16BIT && d->cache.head_dim >= 128 && !is_direct(d) ? 16 : 8;
}
// ... and units of a kv head
int64_t unit_groups(const blk_decode_paged_desc* d) {
    const int n = unit_heads(d);
    return (d->n_heads / d->cache.n_kv_heads + n - 1) / n;
}

struct Layout {
    size_t po, pm, cum, total;
};
Layout layout(const blk_decode_paged_desc* d) {
    const size_t recs = static_cast<size_t>(kPagedMaxGrid + d->cache.batch * d->cache.n_kv_heads * unit_groups(d)) *
                        unit_heads(d);
    auto up = [](size_t n) { return (n + 255) / 256 * 256; };
    Layout L{};
    if (is_direct(d)) return L;
    L.po = 0;
    L.pm = up(recs * d->cache.head_dim * 4);
    L.cum = L.pm + up(recs * 8);
    L.total = L.cum + up((d->cache.batch + 1) * 8);
    return L;
}

}  // namespace

}  // namespace blk

using namespace blk;

extern "C" {

blk_status blk_attn_decode_paged_workspace_size(const blk_decode_paged_desc* d, size_t* bytes) {
    const blk_status st = check_desc(d);
    if (st != BLK_OK) return st;
    REQUIRE(bytes, "bytes is NULL");
    *bytes = layout(d).total;
    return BLK_OK;
}

blk_status blk_attn_decode_paged(const blk_decode_paged_desc* d, const void* q, const void* k_cache,
                                 const void* v_cache, const float* k_scale, const float* v_scale,
                                 const int32_t* block_table, const int32_t* lens,
                                 const float* alibi_slopes, void* o, void* workspace,
                                 size_t ws_bytes, blk_dtype dt, blk_stream_t s) {
    REQUIRE(dt == BLK_F16 || dt == BLK_BF16, "dtype must be BLK_F16 or BLK_BF16");
    blk_status st = check_desc(d);
    if (st != BLK_OK) return st;
    PagedArgs a{};
    st = make_paged_cache(&d->cache, k_cache, v_cache, k_scale, v_scale, block_table, lens, &a.c);
    if (st != BLK_OK) return st;
    REQUIRE(q && (reinterpret_cast<uintptr_t>(q) & 15u) == 0 && o &&
                (reinterpret_cast<uintptr_t>(o) & 15u) == 0,
            "q and o must be 16-byte aligned device pointers");
    REQUIRE(d->alibi || !alibi_slopes, "alibi_slopes given with alibi = 0");
    REQUIRE((reinterpret_cast<uintptr_t>(alibi_slopes) & 3u) == 0, "alibi_slopes must be 4-byte aligned");
    if (d->alibi && !alibi_slopes && (d->n_heads & (d->n_heads - 1)) != 0)
        return report_error_status(BLK_EUNSUPPORTED,
                                   "standard ALiBi slopes need a power-of-two head count");
    const Layout L = layout(d);
    if (L.total && (!workspace || ws_bytes < L.total || (reinterpret_cast<uintptr_t>(workspace) & 15u) != 0))
        return report_error_status(BLK_EWORKSPACE, "workspace needs %zu bytes, 16-byte aligned", L.total);
    int sms = 0;
    if ((st = current_device_info(&sms, &a.err)) != BLK_OK) return st;
    const cudaStream_t cs = reinterpret_cast<cudaStream_t>(s);
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    a.q = q;
    a.qs[0] = d->q_batch_stride;
    a.qs[1] = d->q_head_stride;
    a.po = reinterpret_cast<float*>(ws + L.po);
    a.pm = reinterpret_cast<float2*>(ws + L.pm);
    a.cum = reinterpret_cast<int64_t*>(ws + L.cum);
    a.direct = L.total == 0;
    a.o = o;
    a.slopes = alibi_slopes;
    a.H = static_cast<int>(d->n_heads);
    a.G = a.H / a.c.Hk;
    a.GP = unit_heads(d);
    a.groups = static_cast<int>(unit_groups(d));
    a.units = a.c.Hk * a.groups;
    a.scale = d->softmax_scale > 0.f ? d->softmax_scale : 1.0f / std::sqrt(static_cast<float>(a.c.d));
    a.alibi = d->alibi;
    a.pdl = pdl_allowed(cs);
    const bool e8 = d->cache.kind == BLK_CACHE_E4M3;
    const uint32_t elem = e8 ? 1 : 2;
    const bool wide = !e8 || a.c.d >= 128, narrow = e8 && a.c.d % 128 != 0;
    PagedMapSet tm;  // (a slice of a width that a head does not have: never used)
    for (int kv = 0; kv < 2; ++kv)
        for (int i = wide ? 0 : 1; i <= (narrow ? 1 : 0); ++i) {
            const void* base = kv ? v_cache : k_cache;
            const uint32_t page = static_cast<uint32_t>(d->cache.page_tokens);
            bool ok = make_tmap_pages(&tm.m[kv][0][i], elem, base, a.c.pages, a.c.Hk, page, a.c.d,
                                      d->cache.page_stride, page, i ? 64 : 128);
            if (page == 16) tm.m[kv][1][i] = tm.m[kv][0][i];
            else ok = ok && make_tmap_pages(&tm.m[kv][1][i], elem, base, a.c.pages, a.c.Hk, page, a.c.d,
                                            d->cache.page_stride, 16, i ? 64 : 128);
            if (!ok) return report_error_status(BLK_EINVAL, "no tensor map for this cache");
        }
    cudaError_t e = dt == BLK_F16 ? launch_paged_f16(e8, tm, a, sms, cs) : launch_paged_bf16(e8, tm, a, sms, cs);
    if (e == cudaSuccess && !a.direct) {
        MergeArgs m{};
        m.po = a.po;
        m.pm = a.pm;
        m.cum = a.cum;
        m.lens = lens;
        m.o = o;
        m.rows = d->cache.batch * d->n_heads;
        m.batch = a.c.B;
        m.H = a.H;
        m.G = a.G;
        m.GP = a.GP;
        m.groups = a.groups;
        m.units = a.units;
        m.capacity = a.c.max_pages << a.c.page_log2;
        m.grid = a.grid;
        m.pdl = a.pdl;
        e = dt == BLK_F16 ? launch_merge<__half>(m, a.c.d, sms, cs) : launch_merge<__nv_bfloat16>(m, a.c.d, sms, cs);
    }
    return e == cudaSuccess ? BLK_OK
                            : report_error_status(BLK_ECUDA, "paged decode launch: %s", cudaGetErrorString(e));
}

}  // extern "C"
