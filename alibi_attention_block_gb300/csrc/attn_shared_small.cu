// K6s for few keys: the decode step of a batch that shares a prefix, in one
// launch and without a workspace.
//
// One block per (sequence, query head) over the prefix's keys and the sequence's
// own, the softmax in two passes: the scores go to shared memory, then their
// maximum, the weights 2^(s - max) and their sum, then the weighted values. (The
// attention of nnterp "stablelm" 03 Notes; ALiBi as in "Bloom in a sovereign
// engine", Contribution.) Nothing is split over blocks, so there are no partial
// results and no merge; the prefix comes from L2 for each sequence, a group's keys
// for each of its heads. D / 8 lanes hold a key, 16 bytes each, on the CUDA cores,
// with the weights in 32 bits throughout (the kernel for many keys rounds them for
// its products).
//
// What bounds it is latency: the launch, and in a warp's two passes a load, products
// and shuffles per 16 keys (head_dim 64). In a graph, in us, here and with the kernel
// for many keys (attn_shared.cuh; whose launch, ranges and merge take 8 to 10):
//   16 heads x 64    4 sequences,  64 keys  3.4  9.4    310 keys  5.0 10.3
//                                 564 keys  6.7 10.9   1020 keys  8.9  9.2 (2 kv heads)
//   32 heads x 64    8 sequences, 310 keys  7.2 13.2    564 keys  9.7 13.7
//   16 heads x 128   4 sequences, 310 keys  7.0 10.6    564 keys 10.3 11.2
//                   16 sequences, 310 keys 10.0 11.0
//   16 heads x 64, 2 kv heads     32 sequences (512 blocks), 310 keys 12.9 9.5
// Hence its limits: 768 keys at head_dim 64 or 384 at 128, two blocks of 512 threads
// per SM, and less of one with more of the other. The keys counted are the caches'
// capacity, as the host does not know the lengths.
#include "internal.h"

namespace blk {

namespace {

constexpr int kWarps = 16, kThreads = 32 * kWarps;
constexpr float kLog2e = 1.4426950408889634f;

struct SmallArgs {
    const void *q, *kp, *vp, *k, *v;
    void* o;
    const int32_t* lens;
    const float* slopes;
    int H, Hk, P, S_max, alibi, pdl;
    float scale;
};

// over the lanes whose indexes differ in the bits first, 2 first, ... below end
__device__ __forceinline__ float group_sum(float v, int first, int end) {
#pragma unroll
    for (int x = first; x < end; x <<= 1) v += __shfl_xor_sync(0xffffffffu, v, x);
    return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, x));
    return v;
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) shared_small_kernel(const SmallArgs a) {
    constexpr int L = D / 8;                  // lanes per key
    constexpr int kStep = kWarps * (32 / L);  // keys per step of the block
    constexpr int U = 4;                      // steps in flight
    __shared__ float sc[kSharedSmallDims / D];
    __shared__ __align__(16) float part[kWarps][D];  // written as float4, read as float2
    __shared__ float red_max[kWarps], red_sum[kWarps];
    if (a.pdl) {
        pdl_wait();
        pdl_launch_dependents();
    }
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
    const int b = blockIdx.x / a.H, h = blockIdx.x % a.H, g = h / (a.H / a.Hk);
    const int n = min(max(a.lens[b], 0), a.S_max);
    T* o = static_cast<T*>(a.o) + (static_cast<int64_t>(b) * a.H + h) * D;
    if (n == 0) {  // takes no part
        if (threadIdx.x < D / 2) reinterpret_cast<uint32_t*>(o)[threadIdx.x] = 0u;
        return;
    }
    const int keys = a.P + n;
    const int at = lane % L * 8;  // this lane's dimensions
    const int64_t own_row = (static_cast<int64_t>(b) * a.Hk + g) * a.S_max;
    auto row = [&](const void* prefix, const void* cache, int key) {
        return key < a.P ? static_cast<const T*>(prefix) + (static_cast<int64_t>(g) * a.P + key) * D + at
                         : static_cast<const T*>(cache) + (own_row + key - a.P) * D + at;
    };
    auto unpack = [](const uint4& u, float (&f)[8]) {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 t = dt_traits<T>::unpack2(w[i]);
            f[2 * i] = t.x;
            f[2 * i + 1] = t.y;
        }
    };
    float q[8];
    load8(static_cast<const T*>(a.q) + (static_cast<int64_t>(b) * a.H + h) * D + at, q);
#pragma unroll
    for (int e = 0; e < 8; ++e) q[e] *= a.scale * kLog2e;
    float slope = 0.f;
    if (a.alibi)
        slope = kLog2e * (a.slopes ? a.slopes[h]
                                   : exp2f(-8.0f * static_cast<float>(h + 1) / static_cast<float>(a.H)));
    const int key0 = warp * (32 / L) + lane / L;
    // scores (every lane of a warp makes the same trips); the values' lines come
    // into L1 meanwhile
    float mx = -INFINITY;
    for (int k0 = key0; k0 - key0 < keys; k0 += U * kStep) {
        uint4 kv[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int key = k0 + u * kStep;
            kv[u] = make_uint4(0, 0, 0, 0);
            if (key < keys) {
                kv[u] = *reinterpret_cast<const uint4*>(row(a.kp, a.k, key));
                asm volatile("prefetch.global.L1 [%0];" ::"l"(row(a.vp, a.v, key)));
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int key = k0 + u * kStep;
            float f[8], s = 0.f;
            unpack(kv[u], f);
#pragma unroll
            for (int e = 0; e < 8; ++e) s = fmaf(q[e], f[e], s);
            s = fmaf(slope, static_cast<float>(key - (keys - 1)), group_sum(s, 1, L));
            if (key < keys) {
                mx = fmaxf(mx, s);
                if (lane % L == 0) sc[key] = s;
            }
        }
    }
    mx = warp_max(mx);
    if (lane == 0) red_max[warp] = mx;
    __syncthreads();
    // weights and their sum
    mx = warp_max(red_max[lane % kWarps]);
    float l = 0.f;
    for (int key = threadIdx.x; key < keys; key += kThreads) {
        const float p = ex2_approx(sc[key] - mx);
        sc[key] = p;
        l += p;
    }
    l = group_sum(l, 1, 32);
    if (lane == 0) red_sum[warp] = l;
    __syncthreads();
    // weighted values
    float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int k0 = key0; k0 < keys; k0 += U * kStep) {
        uint4 kv[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int key = k0 + u * kStep;
            kv[u] = make_uint4(0, 0, 0, 0);
            if (key < keys) kv[u] = *reinterpret_cast<const uint4*>(row(a.vp, a.v, key));
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int key = k0 + u * kStep;
            const float p = key < keys ? sc[key] : 0.f;
            float f[8];
            unpack(kv[u], f);
#pragma unroll
            for (int e = 0; e < 8; ++e) acc[e] = fmaf(p, f[e], acc[e]);
        }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] = group_sum(acc[e], L, 32);
    if (lane < L) {
        float4* to = reinterpret_cast<float4*>(&part[warp][at]);
        to[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
        to[1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
    }
    __syncthreads();
    if (threadIdx.x < D / 2) {
        float x = 0.f, y = 0.f;
        l = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float2 t = *reinterpret_cast<const float2*>(&part[w][2 * threadIdx.x]);
            x += t.x;
            y += t.y;
            l += red_sum[w];
        }
        const float inv = 1.0f / l;
        reinterpret_cast<uint32_t*>(o)[threadIdx.x] = dt_traits<T>::pack2(x * inv, y * inv);
    }
}

template <typename T>
cudaError_t launch_small(int d, const SmallArgs& a, int blocks, cudaStream_t st) {
    return launch_pdl(a.pdl != 0, d == 64 ? shared_small_kernel<T, 64> : shared_small_kernel<T, 128>,
                      dim3(blocks), dim3(kThreads), 0, st, a);
}

}  // namespace

bool shared_small(int64_t B, int64_t H, int64_t d, int64_t P, int64_t S_max) {
    const int64_t dims = (P + S_max) * d, blocks = B * H;
    return dims <= kSharedSmallDims && blocks <= kSharedSmallBlocks && dims * blocks <= kSharedSmallWork;
}

cudaError_t launch_attention_decode_shared_small(DType dt, const SharedArgs& s, cudaStream_t st) {
    const DecodeArgs& d = s.own;
    SmallArgs a{};
    a.q = d.q;
    a.kp = s.k_prefix;
    a.vp = s.v_prefix;
    a.k = d.k;
    a.v = d.v;
    a.o = d.o;
    a.lens = d.lens;
    a.slopes = d.slopes;
    a.H = d.H;
    a.Hk = d.Hk;
    a.P = s.P;
    a.S_max = d.S_max;
    a.alibi = d.alibi;
    a.scale = d.scale;
    a.pdl = pdl_allowed(st);
    return dt == DType::F16 ? launch_small<__half>(d.d, a, d.B * d.H, st)
                            : launch_small<__nv_bfloat16>(d.d, a, d.B * d.H, st);
}

}  // namespace blk
