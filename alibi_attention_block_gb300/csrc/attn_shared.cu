// K6s host side and merge: one decode step of attention for a batch that
// shares a prefix. The kernel (attn_shared.cuh) leaves partial results of the
// prefix and of the sequences' own caches; the merge has a lane per
// query row.
#include "internal.h"

namespace blk {

namespace {

constexpr int kTQ = 128, kTK = 128;
constexpr float kLog2e = 1.4426950408889634f;

// o = sum_i w_i O_i / sum_i w_i l_i over the prefix's segments and the own
// cache's, w_i = 2^(m_i - max m), in one pass with a running maximum. With
// ALiBi the prefix's maxima still lack the row's -slope * (lens[b] - 1).
// A lane holds one query row (of 32 rows of a kv head that lie together in the
// prefix's records), a warp eight output columns: a record's 32 bytes per lane
// are 1 KB in one piece, and no value crosses lanes. (One warp per row, 16 bytes
// per lane: 806 instructions per row, 10.9 us for 8192 rows, latency-bound in
// 2.25 waves; this: 6.6.) Where a row has eight segments or more (SPLIT) the
// four warps of a block take them in turn and join their sums in shared memory:
// a warp alone waits for four loads at a time (16 rows of 16 heads x 128 with 20
// segments: 8.4 us, split 4.5).
struct CombineArgs {
    int pdl;
    const float* po;
    const float2* pm;
    const float* own_po;
    const float2* own_pm;
    const int32_t* cum;
    const int32_t* lens;
    const float* slopes;
    void* o;
    int B, H, G, max_seq, alibi, grid;
    int nkt, nrt, W, prefix_ctas;  // of the prefix; W 0: none
    int row_blocks;                // blocks of 32 rows per kv head
};

// The CTA whose range [c * W / n, (c + 1) * W / n) holds tile t, n CTAs in all
// (at most kSharedMaxGrid, W >= n): c * W < (t + 1) * n <= (c + 1) * W, from an estimate
// in floating point that is off by one at most.
__device__ __forceinline__ int cta_of(int64_t t, int64_t W, int n) {
    const int64_t x = (t + 1) * n;
    int c = static_cast<int>(static_cast<float>(t) * (static_cast<float>(n) / static_cast<float>(W)));
    while (c * W >= x) --c;
    while ((c + 1) * W < x) ++c;
    return c;
}

struct Merge {
    float m = -INFINITY, l = 0.f, o[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    __device__ __forceinline__ void add(float pm, float pl, const float4 x, const float4 y) {
        const float mn = fmaxf(m, pm);
        const float keep = m == -INFINITY ? 0.f : exp2f(m - mn);
        const float w = pm == -INFINITY ? 0.f : exp2f(pm - mn);
        m = mn;
        l = fmaf(l, keep, w * pl);
        const float f[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = fmaf(o[e], keep, w * f[e]);
    }
};

template <typename T, int D, bool SPLIT>
__global__ void __launch_bounds__(128) shared_combine_kernel(const CombineArgs a) {
    constexpr int kCols = SPLIT ? D / 8 : D / 32;  // blocks over the columns
    constexpr int kStep = SPLIT ? 4 : 1;           // a warp's step over segments
    __shared__ float part[SPLIT ? 4 : 1][10][32];
    if (a.pdl) {
        pdl_wait();
        pdl_launch_dependents();
    }
    const int lane = threadIdx.x & 31;
    const int warp = threadIdx.x / 32;
    const int blk = blockIdx.x / kCols;  // (kv head, 32 rows)
    const int col8 = SPLIT ? blockIdx.x % kCols : blockIdx.x % kCols * 4 + warp;
    const int first = SPLIT ? warp : 0;  // this warp's first segment
    const int g = blk / a.row_blocks;
    const int R = (blk - g * a.row_blocks) * 32 + lane;  // row of the kv head
    const bool mine = R / a.G < a.B;
    const int b = mine ? R / a.G : a.B - 1, h = g * a.G + R % a.G;
    const int Hk = a.H / a.G;
    const int n = min(max(a.lens[b], 0), a.max_seq);
    const int tiles = a.cum[a.B], before = a.cum[b];
    Merge r;
    float shift = 0.f;
    if (a.alibi) {
        const float sl = a.slopes ? a.slopes[h]
                                  : exp2f(-8.0f * static_cast<float>(h + 1) / static_cast<float>(a.H));
        shift = sl * kLog2e * static_cast<float>(n - 1);
    }
    if (a.W) {
        // the prefix's segments of this row tile: CTAs c0 .. c1, record c + unit
        const int u = g * a.nrt + R / kTQ, row = R % kTQ;
        const int64_t t0 = static_cast<int64_t>(u) * a.nkt;
        const int c0 = cta_of(t0, a.W, a.prefix_ctas), c1 = cta_of(t0 + a.nkt - 1, a.W, a.prefix_ctas);
        const int64_t rec = static_cast<int64_t>(c0 + u) * kTQ;
        const float* p = a.po + rec * D + (col8 * kTQ + row) * 8;
        const float2* s = a.pm + rec + row;
#pragma unroll 4
        for (int k = first; k <= c1 - c0; k += kStep) {
            const float4* q = reinterpret_cast<const float4*>(p + static_cast<int64_t>(k) * kTQ * D);
            const float4 x = q[0], y = q[1];
            const float2 ml = s[static_cast<int64_t>(k) * kTQ];
            r.add(ml.x - shift, ml.y, x, y);
        }
    }
    if (n > 0) {
        // the own cache's segments, of unit (b, kv head)
        const int64_t W = static_cast<int64_t>(tiles) * Hk;
        const int nt = (n + kTK - 1) / kTK;
        const int64_t t0 = static_cast<int64_t>(before) * Hk + static_cast<int64_t>(g) * nt;
        const int ctas = static_cast<int>(min(static_cast<int64_t>(a.grid), W));
        const int c0 = cta_of(t0, W, ctas), c1 = cta_of(t0 + nt - 1, W, ctas);
        const int64_t rec = (static_cast<int64_t>(c0) + static_cast<int64_t>(b) * Hk + g) * a.G + R % a.G;
        const float* p = a.own_po + rec * D + col8 * 8;
        const float2* s = a.own_pm + rec;
#pragma unroll 2
        for (int k = first; k <= c1 - c0; k += kStep) {
            const float4* q = reinterpret_cast<const float4*>(p + static_cast<int64_t>(k) * a.G * D);
            const float4 x = q[0], y = q[1];
            const float2 ml = s[static_cast<int64_t>(k) * a.G];
            r.add(ml.x, ml.y, x, y);
        }
    }
    if constexpr (SPLIT) {
        part[warp][0][lane] = r.m;
        part[warp][1][lane] = r.l;
#pragma unroll
        for (int e = 0; e < 8; ++e) part[warp][2 + e][lane] = r.o[e];
        __syncthreads();
        if (warp > 0) return;
        for (int i = 1; i < 4; ++i)
            r.add(part[i][0][lane], part[i][1][lane],
                  make_float4(part[i][2][lane], part[i][3][lane], part[i][4][lane], part[i][5][lane]),
                  make_float4(part[i][6][lane], part[i][7][lane], part[i][8][lane], part[i][9][lane]));
    }
    if (!mine) return;
    // a sequence of length 0 takes no part
    const float inv = n > 0 && r.l > 0.f ? 1.0f / r.l : 0.f;
    float f[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = n > 0 ? r.o[e] * inv : 0.f;
    store8(static_cast<T*>(a.o) + (static_cast<int64_t>(b) * a.H + h) * D + col8 * 8, f);
}

template <typename T, int D>
cudaError_t launch_combine(const CombineArgs& c, cudaStream_t st) {
    const int Hk = c.H / c.G;
    const bool split = c.W && c.prefix_ctas >= 7 * Hk * c.nrt;  // segments of a unit, less one
    const int64_t blocks = static_cast<int64_t>(Hk) * c.row_blocks * (split ? D / 8 : D / 32);
    return launch_pdl(c.pdl != 0,
                      split ? shared_combine_kernel<T, D, true> : shared_combine_kernel<T, D, false>,
                      dim3(static_cast<unsigned>(blocks)), dim3(128), 0, st, c);
}

}  // namespace

SharedLayout shared_layout(int64_t B, int64_t H, int64_t Hk, int64_t d, int64_t P) {
    const int64_t G = H / Hk, nrt = (B + kTQ / G - 1) / (kTQ / G);
    const int64_t recs = P ? (kSharedMaxGrid + Hk * nrt) * kTQ : 0;
    auto up = [](int64_t n) { return (n + 255) / 256 * 256; };
    SharedLayout L;
    L.po = 0;
    L.pm = up(recs * d * 4);
    L.own_po = L.pm + up(recs * 8);
    const int64_t own = (kSharedMaxGrid + B * Hk) * G;
    L.own_pm = L.own_po + up(own * d * 4);
    L.cum = L.own_pm + up(own * 8);
    L.total = L.cum + up((B + 1) * 4);
    return L;
}

int64_t shared_tiles(int64_t B, int64_t H, int64_t Hk, int64_t P) {
    const int64_t G = H / Hk;
    return Hk * ((B + kTQ / G - 1) / (kTQ / G)) * ((P + kTK - 1) / kTK);
}

cudaError_t launch_attention_decode_shared(DType dt, const SharedArgs& s, cudaStream_t st) {
    const DecodeArgs& d = s.own;
    const SharedLayout L = shared_layout(d.B, d.H, d.Hk, d.d, s.P);
    SharedKernelArgs a{};
    a.pdl = pdl_allowed(st);
    a.G = d.H / d.Hk;
    a.nkt = (s.P + kTK - 1) / kTK;
    a.nrt = (d.B + kTQ / a.G - 1) / (kTQ / a.G);
    a.W = d.Hk * a.nrt * a.nkt;
    a.grid = 2 * s.num_sms < kSharedMaxGrid ? 2 * s.num_sms : kSharedMaxGrid;
    a.prefix_ctas = a.grid < a.W ? a.grid : a.W;
    a.po = reinterpret_cast<float*>(s.ws + L.po);
    a.pm = reinterpret_cast<float2*>(s.ws + L.pm);
    a.own_po = reinterpret_cast<float*>(s.ws + L.own_po);
    a.own_pm = reinterpret_cast<float2*>(s.ws + L.own_pm);
    a.cum = reinterpret_cast<int32_t*>(s.ws + L.cum);
    a.lens = d.lens;
    a.slopes = d.slopes;
    a.err = s.err;
    a.B = d.B;
    a.H = d.H;
    a.Hk = d.Hk;
    a.P = s.P;
    a.S_max = d.S_max;
    a.scale = d.scale;
    a.alibi = d.alibi;
    SharedMaps m;
    const uint64_t planes = static_cast<uint64_t>(d.B) * d.Hk;
    // without a prefix its maps are never used: any valid ones will do
    const void* kp = s.P ? s.k_prefix : d.k;
    const void* vp = s.P ? s.v_prefix : d.v;
    const uint64_t prows = s.P ? s.P : d.S_max;
    if (!make_tmap_queries(&m.pq, dt, d.q, d.B, d.Hk, a.G, d.d, kTQ / a.G) ||
        !make_tmap_3d(&m.pk, dt, kp, d.Hk, prows, d.d, kTK) ||
        !make_tmap_3d(&m.pv, dt, vp, d.Hk, prows, d.d, kTK) ||
        !make_tmap_2d(&m.oq, dt, d.q, static_cast<uint64_t>(d.B) * d.H, d.d, a.G) ||
        !make_tmap_3d(&m.ok, dt, d.k, planes, d.S_max, d.d, kTK) ||
        !make_tmap_3d(&m.ov, dt, d.v, planes, d.S_max, d.d, kTK) ||
        !make_tmap_3d(&m.ok16, dt, d.k, planes, d.S_max, d.d, 16) ||
        !make_tmap_3d(&m.ov16, dt, d.v, planes, d.S_max, d.d, 16))
        return cudaErrorInvalidValue;
    const cudaError_t e = dt == DType::F16 ? launch_shared_f16(d.d, m, a, st)
                                           : launch_shared_bf16(d.d, m, a, st);
    if (e != cudaSuccess) return e;
    CombineArgs c{};
    c.pdl = a.pdl;
    c.po = a.po;
    c.pm = a.pm;
    c.own_po = a.own_po;
    c.own_pm = a.own_pm;
    c.cum = a.cum;
    c.lens = a.lens;
    c.slopes = a.slopes;
    c.o = d.o;
    c.B = a.B;
    c.H = a.H;
    c.G = a.G;
    c.max_seq = a.S_max;
    c.alibi = a.alibi;
    c.grid = a.grid;
    c.nkt = a.nkt;
    c.nrt = a.nrt;
    c.W = a.W;
    c.prefix_ctas = a.prefix_ctas;
    c.row_blocks = static_cast<int>((static_cast<int64_t>(a.B) * a.G + 31) / 32);
    if (dt == DType::F16)
        return d.d == 64 ? launch_combine<__half, 64>(c, st) : launch_combine<__half, 128>(c, st);
    return d.d == 64 ? launch_combine<__nv_bfloat16, 64>(c, st)
                     : launch_combine<__nv_bfloat16, 128>(c, st);
}

}  // namespace blk
