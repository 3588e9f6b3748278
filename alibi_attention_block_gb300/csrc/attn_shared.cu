// K6s host side and merge: one decode step of attention for a batch that
// shares a prefix. The kernel (attn_shared.cuh) leaves partial results of the
// prefix and of the sequences' own caches; the merge has one warp per
// (sequence, query head).
#include "internal.h"

namespace blk {

namespace {

constexpr int kTQ = 128, kTK = 128;
constexpr float kLog2e = 1.4426950408889634f;

// o = sum_i w_i O_i / sum_i w_i l_i over the prefix's segments and the own
// cache's, w_i = 2^(m_i - max m): one warp per (b, query head). With
// ALiBi the prefix's maxima still lack the row's -slope * (lens[b] - 1).
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
};

// The CTA whose range [c * W / n, (c + 1) * W / n) holds tile t, n CTAs in all
// (at most 512, W >= n): c * W < (t + 1) * n <= (c + 1) * W, from an estimate
// in floating point that is off by one at most. (Four 64-bit divisions per row
// were most of the merge's instructions: 11.3 us for 8192 rows, @COMB@ without.)
__device__ __forceinline__ int cta_of(int64_t t, int64_t W, int n) {
    const int64_t x = (t + 1) * n;
    int c = static_cast<int>(static_cast<float>(t) * (static_cast<float>(n) / static_cast<float>(W)));
    while (c * W >= x) --c;
    while ((c + 1) * W < x) ++c;
    return c;
}

template <typename T, int D>
__global__ void __launch_bounds__(128, 6) shared_combine_kernel(const CombineArgs a) {
    // a record's D floats are read 16 bytes per lane: head_dim 64 takes half a
    // warp, so two records at a time
    constexpr int kLanes = D / 4, kAtOnce = 32 / kLanes;
    if (a.pdl) {
        pdl_wait();
        pdl_launch_dependents();
    }
    const int lane = threadIdx.x & 31;
    const unsigned w = blockIdx.x * 4 + threadIdx.x / 32;  // B * H < 2^31
    if (w >= static_cast<unsigned>(a.B) * static_cast<unsigned>(a.H)) return;
    const int b = static_cast<int>(w / static_cast<unsigned>(a.H)), h = static_cast<int>(w) - b * a.H;
    const int Hk = a.H / a.G, g = h / a.G;
    const int c4 = lane % kLanes, half = lane / kLanes;
    // The prefix's segments of this row: CTAs c0 .. c1, record c + unit. Where
    // they are is known at once, so the first of them are on their way while
    // the lengths, which say where the own cache's are, still come.
    int64_t seg0 = 0;  // the first one's first row
    int nseg = 0, row = 0;
    if (a.W) {
        const int per = kTQ / a.G;  // sequences per unit
        const int u = g * a.nrt + b / per;
        row = b % per * a.G + h % a.G;  // of the unit
        const int64_t p0 = static_cast<int64_t>(u) * a.nkt;
        const int c0 = cta_of(p0, a.W, a.prefix_ctas), c1 = cta_of(p0 + a.nkt - 1, a.W, a.prefix_ctas);
        seg0 = static_cast<int64_t>(c0 + u) * kTQ;
        nseg = c1 - c0 + 1;
    }
    auto prefix_part = [&](int k) -> const float4& {
        return *reinterpret_cast<const float4*>(
            a.po + (seg0 + static_cast<int64_t>(k) * kTQ) * D + (c4 / 2 * kTQ + row) * 8 + c4 % 2 * 4);
    };
    auto prefix_stat = [&](int k) { return a.pm[seg0 + static_cast<int64_t>(k) * kTQ + row]; };
    constexpr int kLoads = 8 / kAtOnce;  // of 8 records, in flight together
    float4 f[kLoads];
#pragma unroll
    for (int x = 0; x < kLoads; ++x)
        if (x * kAtOnce + half < nseg) f[x] = prefix_part(x * kAtOnce + half);
    float2 stat = make_float2(-INFINITY, 0.f);  // lane i: record i's (max, sum)
    if (lane < nseg) stat = prefix_stat(lane);
    const int tiles = a.cum[a.B], before = a.cum[b];
    const int n = min(max(a.lens[b], 0), a.max_seq);
    float o[4] = {0.f, 0.f, 0.f, 0.f};
    float mx = -INFINITY, lsum = 0.f;
    if (n > 0) {
        // the own cache's segments, of unit (b, kv head)
        const int64_t own_w = static_cast<int64_t>(tiles) * Hk;
        const int nt = (n + kTK - 1) / kTK;
        const int64_t t0 = static_cast<int64_t>(before) * Hk + static_cast<int64_t>(g) * nt;
        const int ctas = static_cast<int>(min(static_cast<int64_t>(a.grid), own_w));
        const int c0 = cta_of(t0, own_w, ctas), c1 = cta_of(t0 + nt - 1, own_w, ctas);
        const int64_t own0 = (static_cast<int64_t>(c0) + static_cast<int64_t>(b) * Hk + g) * a.G + h % a.G;
        const int total = nseg + c1 - c0 + 1;
        float shift = 0.f;
        if (a.alibi) {
            const float sl = a.slopes ? a.slopes[h]
                                      : exp2f(-8.0f * static_cast<float>(h + 1) /
                                              static_cast<float>(a.H));
            shift = sl * kLog2e * static_cast<float>(n - 1);
        }
        for (int base = 0; base < total; base += 32) {
            const int i = base + lane;
            if (i >= nseg || base > 0) {
                stat = make_float2(-INFINITY, 0.f);
                if (i < nseg) stat = prefix_stat(i);
                else if (i < total) stat = a.own_pm[own0 + static_cast<int64_t>(i - nseg) * a.G];
            }
            const float m = i < nseg ? stat.x - shift : stat.x;
            float mb = m;
#pragma unroll
            for (int s = 16; s > 0; s >>= 1) mb = fmaxf(mb, __shfl_xor_sync(0xffffffffu, mb, s));
            const float mn = fmaxf(mx, mb);
            const float keep = mx == -INFINITY ? 0.f : exp2f(mx - mn);
            const float wgt = m == -INFINITY ? 0.f : exp2f(m - mn);
            float ls = wgt * stat.y;
#pragma unroll
            for (int s = 16; s > 0; s >>= 1) ls += __shfl_xor_sync(0xffffffffu, ls, s);
            lsum = fmaf(lsum, keep, ls);
            mx = mn;
#pragma unroll
            for (int e = 0; e < 4; ++e) o[e] *= keep;
            // (each half of a warp, or the whole, in record order)
            const int cnt = min(32, total - base);
#pragma unroll 1
            for (int j0 = 0; j0 < cnt; j0 += 8) {
#pragma unroll
                for (int x = 0; x < kLoads; ++x) {
                    const int j = j0 + x * kAtOnce + half, k = base + j;
                    if (k < nseg) {
                        if (base + j0 > 0) f[x] = prefix_part(k);
                    } else if (j < cnt) {
                        f[x] = reinterpret_cast<const float4*>(
                            a.own_po + (own0 + static_cast<int64_t>(k - nseg) * a.G) * D)[c4];
                    }
                }
#pragma unroll
                for (int x = 0; x < kLoads; ++x) {
                    const int j = j0 + x * kAtOnce + half;
                    const float wj = __shfl_sync(0xffffffffu, wgt, j & 31);
                    if (j < cnt) {
                        o[0] = fmaf(wj, f[x].x, o[0]);
                        o[1] = fmaf(wj, f[x].y, o[1]);
                        o[2] = fmaf(wj, f[x].z, o[2]);
                        o[3] = fmaf(wj, f[x].w, o[3]);
                    }
                }
            }
        }
    }
    if constexpr (kAtOnce == 2) {
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] += __shfl_xor_sync(0xffffffffu, o[e], 16);
    }
    const float inv = lsum > 0.f ? 1.0f / lsum : 0.f;
    if (lane < kLanes) {
        const uint2 v = make_uint2(dt_traits<T>::pack2(o[0] * inv, o[1] * inv),
                                   dt_traits<T>::pack2(o[2] * inv, o[3] * inv));
        *reinterpret_cast<uint2*>(static_cast<T*>(a.o) + static_cast<int64_t>(w) * D + lane * 4) = v;
    }
}

template <typename T, int D>
cudaError_t launch_combine(const CombineArgs& c, cudaStream_t st) {
    const int64_t warps = static_cast<int64_t>(c.B) * c.H;
    return launch_pdl(c.pdl != 0, shared_combine_kernel<T, D>,
                      dim3(static_cast<unsigned>((warps + 3) / 4)), dim3(128), 0, st, c);
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
    if (dt == DType::F16)
        return d.d == 64 ? launch_combine<__half, 64>(c, st) : launch_combine<__half, 128>(c, st);
    return d.d == 64 ? launch_combine<__nv_bfloat16, 64>(c, st)
                     : launch_combine<__nv_bfloat16, 128>(c, st);
}

}  // namespace blk
