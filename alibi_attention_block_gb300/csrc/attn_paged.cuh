// K8: one decode step of attention over a paged cache of 16-bit values or e4m3 codes: the
// kernel (its instantiations: attn_paged_*.cu; plan and merge: attn_paged.cu).
//
//   o[b, h] = sum_j p_j v_j,  p = softmax_j(scale q[b, h] . k_j - slope_h (lens[b] - 1 - j))
//
// over the keys j < lens[b] that page table[b][j / page] holds (the attention of
// nnterp "stablelm" 03 Notes; ALiBi as in "Bloom in a sovereign engine", Contribution). A step
// reads each key and value once for the 4 d flops of each of the group's few heads, so
// it is bound by the cache's bytes, if the products cost little enough. On the CUDA cores
// an 8-bit cache leaves 23 elements per clock and SM to be unpacked and multiplied G times
// each, which is all that they can do at G = 4. So keys are the rows of a tensor-core product
// and heads its few columns,
//     S^T [128 keys, N] = K Q^T,   O^T [d, N] = V^T P^T,
// and the codes go from the cache to the tensor core as they are: K and V tiles come by TMA
// and are operands without any conversion.
//
// 8 bits: a product of kind f8f6f4 takes 8-bit operands on both sides, so the queries and the
// weights are written as sums of e4m3 numbers, in columns of their own:
//     q = 2^e (q1 + 2^-5 q2 + 2^-10 q3),   q1 = e4m3(2^-e q), q2 = e4m3(2^5 (2^-e q - q1)), ...
// with 2^e such that the row's largest is in [128, 256). An e4m3 holds 4 significant bits: a
// remainder is at most 2^-4 of the power of two below its number, so 32 times it at most 256, and takes the
// next 5 bits. Two parts hold the 8 bits of a bf16 number and three the 11 of an fp16 number exactly, down to 2^-22
// and 2^-27 of the row's largest. (The columns are there
// anyway: N is at least 16.) Weights are three parts, at most 2^-9 2^-5 = 2^-14 off, relative; their sums are
// of the 32-bit weights. Where a weight is far below the largest, the error is absolute, 2^-26 of that one.
// A page's scales are factors of its keys: that of K multiplies the score, that of V
// the weight ahead of its rounding. So that the weight times scale stays in e4m3's range whatever the
// scales are, the running reference that is subtracted is of score + log2(scale of V), not of the score.
// The sum of the weights has the same reference, less 36 (kShift): in it the largest weight is 2^(36 - up) to 2^(37 - up) for a
// scale of 2^up, so that at scales of up to 2^128 weights down to 2^-34 of the largest are numbers of 32 bits, and the sum of
// 2^26 weights at 2^-60 (2^123) is one too. Scales of V below 2^-60, the least that appending sets, count as 2^-60 in it.
// References of different pages may so be 2^188 apart with equal weights: a sum is brought from one to the other by two factors
// of half the way, here and in the merge (what O holds at the lower one is then nothing next to the other).
//
// 16 bits: the operands in the storage type, a weight as the sum of two such numbers (the second one's columns are
// there anyway too), 2^-16 off in bf16, 2^-22 in fp16 (held times 2^7, its second part times 2^11: weights down to 2^-21 of
// the largest in fp16's normal range), neither of them below 0, so that infinite values stay infinite. With weights of one part (two in bf16 over e4m3) the outputs of few keys, which do not
// average their errors, were up to 8 % further from the definition than the output's rounding leaves them. The times are the same
// (48 sequences of up to 8192 keys: within 1 %) but for many heads on a kv head, 256 sequences, bf16, 8 on one: e4m3 42.1 ->
// 36.4 us at head_dim 64 (two CTAs per SM in the place of four), 45.8 -> 49.5 at 160, 16 bits 36.4 -> 37.5 at 64; 32 on one
// 126 -> 117, 139 -> 166 (spills) and 107 -> 111, 16 bits at 128 115 -> 123, at 160 161 -> 177.
//
// Work: a unit is (sequence, kv head, up to eight of its query heads, sixteen over wide 16-bit
// rows: unit_heads in attn_paged.cu) of ceil(len / 128) key tiles. The tiles of all units, in one
// line, are cut into equal ranges, one per CTA, whatever the lengths are; a CTA's
// stay in a unit is a segment with a partial result (reference, sum, O), joined by the merge.
// Where the cache has few tiles per sequence (is_direct in attn_paged.cu) a CTA takes a whole unit and
// writes its rows: no range to find, no partial results, one launch.
// The lengths are device data: each CTA sums them itself. Tiles go from the newest key down.
// A tile is 128 keys from up to eight pages: a lane of the loading warp for each 16 of them finds
// the page one tile ahead, copies its rows by TMA and its scales by cp.async. A page id outside
// the pool becomes a coordinate outside the tensor map, which fills with zeros; its keys are
// masked. The last tile is copied in boxes of 16 keys, up to the product's step; rows behind
// its end that the cache holds are cleared: 0 times what an unused entry holds need not be 0.
// 7 warps: loading; MMA issue; four of softmax, a thread per key; queries.
// Measured and bound: 96 sequences of up to 16384 keys, 32/8 x 128 heads, e4m3: 153-156 us (6.5 TB/s, 0.95-0.97 of
// the copy rate); 8 of up to 32771, 16 x 128, 16 bits: 150 us (6.7 TB/s). Below some 100 MB the fixed
// parts show: launch 2.4 us, the first tile's chain (lengths, table, tile, scores, softmax, product) 3, the
// CTAs' ends apart 2, merge 3 (32 of up to 4099 keys, 32/8 x 128: 22.4 us for 14.1 of bytes). Three CTAs per SM at head_dim 128: 24.3.
#pragma once

#include <cuda_fp8.h>

#include "attn_paged.h"

namespace blk {

namespace {

constexpr int kThreads = 224;
constexpr int kTK = 128;
constexpr float kLog2e = 1.4426950408889634f;
// The queries' warp waits for a buffer as long as its segment takes, up to 2^19 tiles. A tile takes 3.1 us where all CTAs
// share the memory's 6.5 TB/s (16 bits, head_dim 128: 64 KB, 304 CTAs), so 1.6 s, which is near the limit of the other waits.
constexpr unsigned long long kTileLimitNs = 20000;

template <typename T, bool E8, int D, int GP>
struct Cfg {
    static constexpr int kElem = E8 ? 1 : 2;
    // slices of a row: 128 bytes each (128-byte swizzle), then one of 64 (64-byte swizzle).
    // head_dim 160: its last slice is part zeros, which TMA writes
    static constexpr int kWide = E8 ? D / 128 : (D + 63) / 64;
    static constexpr int kNarrow = E8 && D % 128 ? 1 : 0;
    static constexpr int kRow = 128 * kWide + 64 * kNarrow;
    static constexpr int kTile = kTK * kRow;
    static constexpr int kStepKeys = 32 / kElem;  // keys of a product's step: 32 bytes of P
    static constexpr bool kF16 = dt_traits<T>::mma_fmt == 0;
    static constexpr int kQParts = !E8 ? 1 : kF16 ? 3 : 2, kPParts = E8 ? 3 : 2;  // of queries, of weights
    // each part, next to the one before it, is held times this
    static constexpr int kUp = E8 ? 32 : kF16 ? 2048 : 256;
    static constexpr int kQUsed = kQParts * GP, kPUsed = kPParts * GP;  // columns with something in them
    static constexpr int columns(int used) { return used <= 16 ? 16 : 32; }
    static constexpr int kNS = columns(kQUsed), kNO = columns(kPUsed);
    // ... and the operands' rows for them in groups of 8; what follows in shared
    // memory makes up the rest (columns do not mix, and none of the rest is read)
    static constexpr int kQRows = (kQUsed + 7) / 8 * 8, kPRows = (kPUsed + 7) / 8 * 8;
    static constexpr int loads(int used) { return used == 3 ? 4 : used == 12 ? 16 : used; }
    static constexpr int kLdS = loads(kQUsed), kLdO = loads(kPUsed);
    static constexpr int kBlocks = D > 128 ? 2 : 1;  // of O's rows: 128 and 64
    // (each buffer at a multiple of the swizzle's 1024 bytes)
    static constexpr int kQBytes = (kQRows * kRow + 1023) / 1024 * 1024, kPBytes = kPRows * 128 * kElem;
    static constexpr int kHeads = GP > 8 ? GP : 8;  // that the small arrays have room for
    static constexpr int kFixed =
        2 * kQBytes + 2 * kPBytes + 8 * 2 * 8 * 4 + 4 * kHeads * 4 * 4 + 2 * kHeads * 4 + 512 + 16;
    // two CTAs per SM, so that one's chain of scores, softmax and product fills the
    // other's gaps; four where tiles are short, one where three of them do not fit twice (16 x 64, e4m3, by four, three and
    // two: 256 sequences of up to 1000 keys 46.1, 48.9 and 63.3 us, 48 of up to 8192 56.4, 52.2 and 60.7; 16/4 x 64: 23.9, 24.8 and
    // 24.8, 24.2, 23.7 and 24.4; with eight heads on a kv head four spilled, 42.8 us for the 36.1 of two)
    static constexpr int fit(int ctas) { return (228 * 1024 / ctas - 2048 - 64 - kFixed) / kTile; }
    static constexpr int kCtas = E8 && D == 64 && kNO == 16 ? 4 : fit(2) < 3 ? 1 : 2;
    static constexpr int kFit = fit(kCtas);
    static constexpr int kSlots = kFit < 6 ? kFit : 6;
    static_assert(kSlots >= 3 && kSlots <= 6, "a ring of tiles, and the scales' ring of eight");
    static constexpr int kOffQ = kSlots * kTile;
    static constexpr int kOffP = kOffQ + 2 * kQBytes;
    static constexpr int kOffScale = kOffP + 2 * kPBytes;    // [8 tiles][K, V][8 groups of 16 keys]
    static constexpr int kOffMax = kOffScale + 8 * 2 * 8 * 4;    // [2][kHeads][4]
    static constexpr int kOffSum = kOffMax + 2 * kHeads * 4 * 4;  // [2][kHeads][4]
    static constexpr int kOffMul = kOffSum + 2 * kHeads * 4 * 4;  // [2][kHeads]
    static constexpr int kOffBar = kOffMul + 2 * kHeads * 4;
    static constexpr int kOffSlot = kOffBar + 512;
    static constexpr int kSmem = kOffSlot + 16 + 1024;  // + alignment slack
    static_assert(kCtas * (kSmem + 1024 + 64) <= 228 * 1024, "shared memory of an SM");
    // TMEM: S^T twice (by tile), O^T twice (by segment)
    static constexpr uint32_t kColO = 2 * kNS;
    static constexpr uint32_t kCols = 2 * kNS + 2 * kBlocks * kNO <= 128 ? 128 : 256;
    static_assert(2 * kNS + 2 * kBlocks * kNO <= static_cast<int>(kCols) && kCtas * kCols <= 512, "TMEM");
    // weights are at most 2^threshold times this: 2^8 in e4m3, 2^15 in fp16
    static constexpr float kTop = E8 || kF16 ? 128.f : 1.f;
    static constexpr float kBack = E8 ? 1.f / (1ull << 36) : 1.f, kShift = E8 ? 36.f : 0.f;  // 2^-shift
    static constexpr float kThreshold = E8 ? 1.f : 8.f;  // log2 of the largest weight before a rescale
};

template <int N>
__device__ __forceinline__ void ld_cols(uint32_t taddr, uint32_t (&r)[N]) {
    if constexpr (N == 1)
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];\n\t"
                     "tcgen05.wait::ld.sync.aligned;" : "=r"(r[0]) : "r"(taddr) : "memory");
    else if constexpr (N == 2)
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x2.b32 {%0, %1}, [%2];\n\t"
                     "tcgen05.wait::ld.sync.aligned;"
                     : "=r"(r[0]), "=r"(r[1]) : "r"(taddr) : "memory");
    else if constexpr (N == 4)
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];\n\t"
                     "tcgen05.wait::ld.sync.aligned;"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(taddr) : "memory");
    else if constexpr (N == 8)
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n\t"
                     "tcgen05.wait::ld.sync.aligned;"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
                       "=r"(r[6]), "=r"(r[7]) : "r"(taddr) : "memory");
    else if constexpr (N == 16)
        tmem_ld16(taddr, r);
    else if constexpr (N == 24)  // (the first load must not overwrite the second's address)
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, "
                     "%13, %14, %15}, [%24];\n\t"
                     "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%16, %17, %18, %19, %20, %21, %22, %23}, [%25];\n\t"
                     "tcgen05.wait::ld.sync.aligned;"
                     : "=&r"(r[0]), "=&r"(r[1]), "=&r"(r[2]), "=&r"(r[3]), "=&r"(r[4]), "=&r"(r[5]), "=&r"(r[6]),
                       "=&r"(r[7]), "=&r"(r[8]), "=&r"(r[9]), "=&r"(r[10]), "=&r"(r[11]), "=&r"(r[12]), "=&r"(r[13]),
                       "=&r"(r[14]), "=&r"(r[15]), "=&r"(r[16]), "=&r"(r[17]), "=&r"(r[18]), "=&r"(r[19]), "=&r"(r[20]),
                       "=&r"(r[21]), "=&r"(r[22]), "=&r"(r[23]) : "r"(taddr), "r"(taddr + 16) : "memory");
    else
        tmem_ld32(taddr, r);
}
template <int N>
__device__ __forceinline__ void st_cols(uint32_t taddr, const uint32_t (&r)[N]) {
    if constexpr (N == 1)
        asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" ::"r"(taddr), "r"(r[0])
                     : "memory");
    else if constexpr (N == 2)
        asm volatile("tcgen05.st.sync.aligned.32x32b.x2.b32 [%0], {%1, %2};" ::"r"(taddr), "r"(r[0]),
                     "r"(r[1]) : "memory");
    else if constexpr (N == 4)
        asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};" ::"r"(taddr),
                     "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]) : "memory");
    else if constexpr (N == 8)
        asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
                     ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]),
                     "r"(r[6]), "r"(r[7]) : "memory");
    else if constexpr (N == 16)
        tmem_st16_nowait(taddr, r);
    else if constexpr (N == 24) {
        asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
                     "%12, %13, %14, %15, %16};"
                     ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]),
                     "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
                     "r"(r[15]) : "memory");
        asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
                     ::"r"(taddr + 16), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]),
                     "r"(r[22]), "r"(r[23]) : "memory");
    } else
        tmem_st32_nowait(taddr, r);
    tmem_st_wait();
}

// max over the warp's lanes: floats as integers of the same order
__device__ __forceinline__ float warp_max(float v) {
    int i = __float_as_int(v);
    i = i < 0 ? i ^ 0x7fffffff : i;
    i = __reduce_max_sync(0xffffffffu, i);
    return __int_as_float(i < 0 ? i ^ 0x7fffffff : i);
}

// Descriptor of `off` (in 16 bytes) behind the one of d, added in the low word (the
// address is its field and does not carry out of it).
__device__ __forceinline__ uint64_t desc_at(uint64_t d, uint32_t off) {
    uint32_t lo, hi;
    asm("mov.b64 {%0, %1}, %2;" : "=r"(lo), "=r"(hi) : "l"(d));
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(lo + off), "r"(hi));
    return r;
}

// Two numbers to e4m3 codes and back.
__device__ __forceinline__ uint32_t to_codes(float x, float y) {
    return __nv_cvt_float2_to_fp8x2(make_float2(x, y), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ float2 of_codes(uint32_t c) {
    return __half22float2(
        __half2(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(c), __NV_E4M3)));
}
// The numbers' parts, each remainder times 32: c[i] holds the codes of part i of both.
template <int PARTS>
__device__ __forceinline__ void split_parts(float x, float y, uint32_t (&c)[PARTS]) {
#pragma unroll
    for (int i = 0; i < PARTS; ++i) {
        c[i] = to_codes(x, y);
        if (i + 1 < PARTS) {
            const float2 f = of_codes(c[i]);
            x = (x - f.x) * 32.f;
            y = (y - f.y) * 32.f;
        }
    }
}
// Two numbers of at least 0 as sums of two 16-bit ones, the first towards zero, the remainder times UP. The second is never 0
// (least: the type's least number): both parts times an infinity are that infinity, and their sum is.
template <typename T, int UP>
__device__ __forceinline__ void split_16(float x, float y, uint32_t (&c)[2]) {
    constexpr bool f16 = dt_traits<T>::mma_fmt == 0;
    constexpr float least = f16 ? 0x1p-24f : 0x1p-126f;
    if (f16) asm("cvt.rz.f16x2.f32 %0, %1, %2;" : "=r"(c[0]) : "f"(y), "f"(x));
    else asm("cvt.rz.bf16x2.f32 %0, %1, %2;" : "=r"(c[0]) : "f"(y), "f"(x));
    const float2 f = dt_traits<T>::unpack2(c[0]);
    c[1] = dt_traits<T>::pack2(fmaxf((x - f.x) * UP, least), fmaxf((y - f.y) * UP, least));
}
__device__ __forceinline__ void st_byte(uint32_t at, uint32_t v) {
    asm volatile("st.shared.b8 [%0], %1;" ::"r"(at), "r"(v) : "memory");
}
__device__ __forceinline__ void st_half(uint32_t at, uint32_t v) {
    asm volatile("st.shared.b16 [%0], %1;" ::"r"(at), "h"(static_cast<uint16_t>(v)) : "memory");
}

// 4 bytes to shared memory, with nothing waited for ...
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
// ... and an arrival once this thread's copies so far are there.
__device__ __forceinline__ void arrive_behind_copies(uint32_t bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

template <int SLOTS>
struct Bars {
    uint32_t at;
    static constexpr int kBytes = 208 + 16 * SLOTS;
    __device__ __forceinline__ uint32_t q_full(int i) const { return at + 8u * i; }
    __device__ __forceinline__ uint32_t q_empty(int i) const { return at + 16u + 8u * i; }
    __device__ __forceinline__ uint32_t s_full(int i) const { return at + 32u + 8u * i; }
    __device__ __forceinline__ uint32_t s_free(int i) const { return at + 48u + 8u * i; }
    __device__ __forceinline__ uint32_t p_full(int i) const { return at + 64u + 8u * i; }
    __device__ __forceinline__ uint32_t pv_done(int i) const { return at + 80u + 8u * i; }
    __device__ __forceinline__ uint32_t o_free(int i) const { return at + 96u + 8u * i; }
    __device__ __forceinline__ uint32_t max_full() const { return at + 112u; }
    __device__ __forceinline__ uint32_t sum_full() const { return at + 120u; }
    __device__ __forceinline__ uint32_t drain() const { return at + 128u; }
    __device__ __forceinline__ uint32_t range_full() const { return at + 136u; }
    __device__ __forceinline__ uint32_t scale_full(int i) const { return at + 144u + 8u * i; }
    __device__ __forceinline__ uint32_t full(int i) const { return at + 208u + 8u * i; }
    __device__ __forceinline__ uint32_t empty(int i) const { return at + 208u + 8u * (SLOTS + i); }
    __device__ __forceinline__ void init() const {
        for (int i = 0; i < 2; ++i) {
            mbar_init(q_full(i), 1);
            mbar_init(q_empty(i), 1 + 4);  // the products', and the softmax warps' with the factors
            mbar_init(s_full(i), 1);
            mbar_init(s_free(i), 4);
            mbar_init(p_full(i), 4);
            mbar_init(pv_done(i), 1);
            mbar_init(o_free(i), 4);
        }
        mbar_init(max_full(), 4);
        mbar_init(sum_full(), 4);
        mbar_init(drain(), 1);
        mbar_init(range_full(), 4);
        for (int i = 0; i < 8; ++i) mbar_init(scale_full(i), 8);
        for (int i = 0; i < SLOTS; ++i) {
            mbar_init(full(i), 1);
            mbar_init(empty(i), 1);
        }
    }
};

__device__ __forceinline__ int len_of(const PagedArgs& a, int b) {
    return min(max(a.c.lens[b], 0), a.c.max_pages << a.c.page_log2);
}

// A CTA's segments: tiles [t, t + n) of unit (b, u), key tiles first ..
// first + n - 1 of the unit; t counts all units' tiles.
struct Segments {
    int64_t t, end;
    int b, u, first, n, len, it;
    bool valid;
    __device__ __forceinline__ void set() {
        valid = t < end;
        if (!valid) return;
        const int left = (len + kTK - 1) / kTK - first;
        n = static_cast<int>(min(static_cast<int64_t>(left), end - t));
    }
    // base: tiles ahead of sequence b0's first unit; the range starts in b0, of length l0
    __device__ __forceinline__ void start(int64_t lo, int64_t hi, int b0, int64_t base, int l0) {
        t = lo;
        end = hi;
        it = 0;
        b = b0;
        valid = t < end;
        if (!valid) return;
        len = l0;
        const int nt = (len + kTK - 1) / kTK;
        // (from its sequence's first tile: units * 2^24 tiles at most, by lengths in 31 bits)
        const int64_t in = t - base;
        u = in < (int64_t(1) << 31) ? static_cast<int>(static_cast<uint32_t>(in) / static_cast<uint32_t>(nt))
                                    : static_cast<int>(in / nt);
        first = static_cast<int>(in - static_cast<int64_t>(u) * nt);
        set();
    }
    __device__ __forceinline__ void next(const PagedArgs& a) {
        t += n;
        ++it;
        first = 0;
        if (t < end && ++u == a.units) {
            u = 0;
            do {
                len = len_of(a, ++b);
            } while (len == 0);
        }
        set();
    }
};

// The tiles of a CTA's segments in turn.
struct Tile {
    int t, it, b, u, row, keys;  // running number, segment; first key, keys from there on
    bool first, last;            // of its segment
};
struct Tiles {
    Segments c;
    int t = 0, i = 0;
    __device__ __forceinline__ bool next(const PagedArgs& a, Tile& x) {
        if (!c.valid) return false;
        x.t = t++;
        x.it = c.it;
        x.b = c.b;
        x.u = c.u;
        x.row = (c.first + c.n - 1 - i) * kTK;
        x.keys = c.len - x.row;
        x.first = i == 0;
        x.last = ++i == c.n;
        if (x.last) {
            c.next(a);
            i = 0;
        }
        return true;
    }
};

// The range of CTA `me` among W tiles: as many CTAs as there are tiles, if those are fewer (the merge
// counts on every CTA of a unit's span having some of it).
__device__ __forceinline__ void cut(int64_t W, int64_t& lo, int64_t& hi) {
    const int64_t ctas = min(static_cast<int64_t>(gridDim.x), W), me = blockIdx.x;
    if (me >= ctas) {
        lo = hi = 0;
    } else if (W < (1 << 21)) {  // (me + 1 is at most 2^10: 32 bits)
        const uint32_t n = static_cast<uint32_t>(ctas), w = static_cast<uint32_t>(W);
        lo = static_cast<uint32_t>(me) * w / n;
        hi = (static_cast<uint32_t>(me) + 1) * w / n;
    } else {
        lo = me * W / ctas;
        hi = (me + 1) * W / ctas;
    }
}

// This CTA's range of tiles, by the four softmax warps: tiles [lo, hi), the first in sequence
// b0, `base` tiles ahead of that sequence.
struct Range {
    int64_t lo, hi, base;
    int b0;
    int64_t sum[4];
};
__device__ __forceinline__ void find_range(const PagedArgs& a, Range& out, uint32_t range_full) {
    const int t = static_cast<int>(threadIdx.x) - 64, lane = t & 31, w = t / 32;
    // thread t sums the tiles of a run of sequences
    const int per = (a.c.B + 127) / 128;
    const int b_lo = min(t * per, a.c.B), b_hi = min(b_lo + per, a.c.B);
    int64_t mine = 0;
    for (int b = b_lo; b < b_hi; ++b) mine += (len_of(a, b) + kTK - 1) / kTK;
    int64_t upto = mine;  // inclusive sum over the warp's threads, then over all
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += v;
    }
    if (lane == 31) out.sum[w] = upto;
    // (all four warps come here before any wait that can give up)
    asm volatile("bar.sync 1, 128;" ::: "memory");
    int64_t before = upto - mine, total = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (i < w) before += out.sum[i];
        total += out.sum[i];
    }
    const int64_t W = total * a.units, me = blockIdx.x;
    int64_t lo, hi;
    cut(W, lo, hi);
    if (t == 0) {
        out.lo = lo;
        out.hi = hi;
    }
    // the thread whose run holds the first tile finds its sequence
    if (lo < hi && before * a.units <= lo && lo < (before + mine) * a.units) {
        int64_t base = before * a.units;
        int b = b_lo;
        for (;; ++b) {
            const int64_t nt = (len_of(a, b) + kTK - 1) / kTK * static_cast<int64_t>(a.units);
            if (lo < base + nt) break;
            base += nt;
        }
        out.b0 = b;
        out.base = base;
    }
    if (me == 0) {
        int64_t c = before;
        for (int b = b_lo; b < b_hi; ++b) {
            a.cum[b] = c;
            c += (len_of(a, b) + kTK - 1) / kTK;
        }
        if (t == 0) a.cum[a.c.B] = total;
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(range_full);
}

// The same for up to 128 sequences, by each warp for itself: four lengths a lane, read once and passed
// between lanes, no barrier and no shared memory (with find_range a CTA has its range 1.45 us behind its
// start and its first copies out 3.2 us behind it; with this a call of 23.0 us takes 22.4).
constexpr int kFewSequences = 128;
__device__ __forceinline__ void warp_range(const PagedArgs& a, int lane, bool first_warp, Segments& c) {
    const int per = (a.c.B + 31) / 32, b0 = lane * per;
    int len[4], mine = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        len[k] = k < per && b0 + k < a.c.B ? len_of(a, b0 + k) : 0;
        mine += (len[k] + kTK - 1) / kTK;
    }
    int upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += v;
    }
    const int before = upto - mine, total = __shfl_sync(0xffffffffu, upto, 31);
    int64_t lo, hi;
    cut(static_cast<int64_t>(total) * a.units, lo, hi);
    if (blockIdx.x == 0 && first_warp) {
        int64_t sum = before;
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (k < per && b0 + k < a.c.B) {
                a.cum[b0 + k] = sum;
                sum += (len[k] + kTK - 1) / kTK;
            }
        if (lane == 0) a.cum[a.c.B] = total;
    }
    // the lane whose sequences hold the first tile, and which of them
    const int64_t mul = a.units;
    const bool here = lo < hi && before * mul <= lo && lo < upto * mul;
    int b = 0, l = 0;
    int64_t base = before * mul;
    bool found = false;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int64_t nt = (len[k] + kTK - 1) / kTK * mul;
        if (!found && lo < base + nt) {
            found = true;
            b = b0 + k;
            l = len[k];
        }
        if (!found) base += nt;
    }
    const unsigned who = __ballot_sync(0xffffffffu, here);
    const int src = who ? __ffs(who) - 1 : 0;
    b = __shfl_sync(0xffffffffu, b, src);
    l = __shfl_sync(0xffffffffu, l, src);
    base = __shfl_sync(0xffffffffu, base, src);
    c.start(lo, hi, b, base, l);
}

template <typename T, bool E8, int D, int GP>
__device__ __forceinline__ void paged_body(const PagedArgs& a, const PagedMaps& tm, Tiles tiles,
                                           uint8_t* smem, uint32_t tmem, int warp, int lane) {
    using C = Cfg<T, E8, D, GP>;
    constexpr int kSlots = C::kSlots, NS = C::kNS, NO = C::kNO;
    const uint32_t sKV = smem_u32(smem);
    const uint32_t sQ = sKV + C::kOffQ, sP = sKV + C::kOffP;
    const Bars<kSlots> bar{sKV + C::kOffBar};
    float* scales = reinterpret_cast<float*>(smem + C::kOffScale);
    float* red_max = reinterpret_cast<float*>(smem + C::kOffMax);
    float* red_sum = reinterpret_cast<float*>(smem + C::kOffSum);
    float* factors = reinterpret_cast<float*>(smem + C::kOffMul);
    const int lg = a.c.page_log2;
    bool ok = true;
    if (warp == 0) {
        const uint64_t pol = l2_evict_first_policy();
        int r = 0;  // tiles of K and V on their way so far
        Tile x, y;
        // the page of this lane's 16 keys, -1: none
        auto find_page = [&](const Tile& z) -> int {
            const int at = z.row + 16 * lane;
            if (lane >= 8 || 16 * lane >= z.keys) return -1;
            const int p = a.c.table[static_cast<int64_t>(z.b) * a.c.max_pages + (at >> lg)];
            return p >= 0 && p < a.c.pages ? p : -1;
        };
        bool have = tiles.next(a, x), more = false;
        int page = have ? find_page(x) : -1, page_next = -1;
        while (have) {
            more = tiles.next(a, y);
            if (more) page_next = find_page(y);
            const int g = x.u / a.groups;
            const bool whole = x.keys >= kTK;
            const int rows = whole ? kTK : (x.keys + C::kStepKeys - 1) / C::kStepKeys * C::kStepKeys;
            // boxes of a page's rows, or of 16
            const int box = whole ? min(kTK, 1 << lg) : 16;
            const bool mine = lane < 8 && (16 * lane) % box == 0 && 16 * lane < rows;
            const int from = (x.row + 16 * lane) & ((1 << lg) - 1);
            for (int kv = 0; kv < 2; ++kv, ++r) {
                const int sl = r % kSlots;
                ok = __all_sync(0xffffffffu, mbar_wait(bar.empty(sl), ((r / kSlots) & 1) ^ 1u, a.err));
                if (!ok) break;
                if (kv == 0 && lane < 8) {
                    // the scales of these 16 keys; negative: they are masked. The ring's
                    // entry was read ahead of the product that has freed this slot
                    float* dst = scales + (x.t & 7) * 16 + lane;
                    if (E8 && page >= 0) {
                        const int64_t at = static_cast<int64_t>(page) * a.c.Hk + g;
                        cp_async4(smem_u32(dst), a.c.k_scale + at);
                        cp_async4(smem_u32(dst + 8), a.c.v_scale + at);
                        arrive_behind_copies(bar.scale_full(x.t & 7));
                    } else {
                        dst[0] = page >= 0 ? 1.f : -1.f;
                        dst[8] = 1.f;
                        mbar_arrive(bar.scale_full(x.t & 7));
                    }
                }
                if (lane == 0) mbar_expect_tx(bar.full(sl), rows * C::kRow);
                __syncwarp();
                if (mine) {
                    const uint32_t dst = sKV + sl * C::kTile;
                    const CUtensorMap* m = tm.m[kv][whole ? 0 : 1];
                    const int p = page >= 0 ? page : a.c.pages;  // outside: zeros
#pragma unroll
                    for (int s = 0; s < C::kWide; ++s)
                        tma_load_4d_hint(dst + s * kTK * 128 + lane * 16 * 128, m, bar.full(sl),
                                         s * 128 / C::kElem, from, g, p, pol);
                    if (C::kNarrow)
                        tma_load_4d_hint(dst + C::kWide * kTK * 128 + lane * 16 * 64, m + 1, bar.full(sl),
                                         C::kWide * 128, from, g, p, pol);
                }
            }
            if (!ok) break;
            x = y;
            page = page_next;
            have = more;
        }
        // whatever the others met, no copy lands behind this block's end
        cp_async_commit();
        cp_async_wait<0>();
        for (int i = r > kSlots ? r - kSlots : 0; i < r; ++i)
            mbar_wait(bar.full(i % kSlots), (i / kSlots) & 1, a.err);
    } else if (warp == 1) {
        if (lane == 0) {
            constexpr uint32_t fmt = E8 ? 0 : dt_traits<T>::mma_fmt;  // e4m3 is 0 too
            constexpr uint32_t idesc_s = make_idesc_f16(fmt, kTK, NS, false);
            // A MN-major
            constexpr uint32_t idesc_o = make_idesc_f16(fmt, D == 64 ? 64 : 128, NO, false) | (1u << 15);
            constexpr uint32_t idesc_o2 = make_idesc_f16(fmt, 64, NO, false) | (1u << 15);
            constexpr uint32_t kSlotStep = C::kTile >> 4;
            // offsets in 16 bytes of the narrow slices, and of V's second block of rows
            constexpr uint32_t kNarrowK = (C::kWide * kTK * 128) >> 4;
            constexpr uint32_t kNarrowQ = (C::kWide * C::kQRows * 128) >> 4;
            constexpr uint32_t kSecond = (D > 128 ? (E8 ? 1 : 2) * kTK * 128 : 0) >> 4;
            const uint64_t dk0 = make_sdesc_sw128(sKV, 16, 1024), dk0n = make_sdesc_sw64(sKV, 16, 512);
            const uint64_t dv0 = make_sdesc_sw128(sKV, kTK * 128, 1024);
            const uint64_t dq0 = make_sdesc_sw128(sQ, 16, 1024), dq0n = make_sdesc_sw64(sQ, 16, 512);
            const uint64_t dp0 = make_sdesc_sw128(sP, 16, 1024);
            auto mma = [&](uint32_t d, uint64_t da, uint64_t db, uint32_t idesc, uint32_t acc) {
                if (E8) tc_mma_f8_ss(d, da, db, idesc, acc);
                else tc_mma_ss(d, da, db, idesc, acc);
            };
            // S^T = K Q^T: the keys and (first tile) queries are there, and the
            // softmax has read the S buffer's last tile
            auto s_ready = [&](const Tile& x) {
                const int r = 2 * x.t;
                return mbar_test(bar.full(r % kSlots), (r / kSlots) & 1) &&
                       (!x.first || mbar_test(bar.q_full(x.it & 1), (x.it >> 1) & 1)) &&
                       (x.t < 2 || mbar_test(bar.s_free(x.t & 1), ((x.t >> 1) - 1) & 1));
            };
            auto issue_s = [&](const Tile& x) {
                tc_fence_after();
                const int sl = 2 * x.t % kSlots;
                const uint32_t k = sl * kSlotStep, q = (x.it & 1) * (C::kQBytes >> 4);
#pragma unroll
                for (int ks = 0; ks < D * C::kElem / 32; ++ks) {
                    const uint32_t in = (ks % 4) * 2;
                    if (ks / 4 < C::kWide)
                        mma(tmem + NS * (x.t & 1), desc_at(dk0, k + (ks / 4) * ((kTK * 128) >> 4) + in),
                            desc_at(dq0, q + (ks / 4) * ((C::kQRows * 128) >> 4) + in), idesc_s, ks > 0 ? 1u : 0u);
                    else
                        mma(tmem + NS * (x.t & 1), desc_at(dk0n, k + kNarrowK + in),
                            desc_at(dq0n, q + kNarrowQ + in), idesc_s, ks > 0 ? 1u : 0u);
                }
                tc_commit(bar.s_full(x.t & 1));
                tc_commit(bar.empty(sl));
                if (x.last) tc_commit(bar.q_empty(x.it & 1));
            };
            // O^T += V^T P^T: the values and P are there, and (first tile) the O
            // buffer's last segment has been read out
            auto pv_ready = [&](const Tile& x) {
                const int r = 2 * x.t + 1;
                return mbar_test(bar.full(r % kSlots), (r / kSlots) & 1) &&
                       mbar_test(bar.p_full(x.t & 1), (x.t >> 1) & 1) &&
                       (!x.first || x.it < 2 || mbar_test(bar.o_free(x.it & 1), ((x.it >> 1) - 1) & 1));
            };
            auto issue_pv = [&](const Tile& x) {
                tc_fence_after();
                const int sl = (2 * x.t + 1) % kSlots;
                const uint32_t v = sl * kSlotStep, p = (x.t & 1) * (C::kPBytes >> 4);
                const uint32_t o = tmem + C::kColO + C::kBlocks * NO * (x.it & 1);
                const int steps = (min(x.keys, kTK) + C::kStepKeys - 1) / C::kStepKeys;
#pragma unroll
                for (int ks = 0; ks < kTK / C::kStepKeys; ++ks) {
                    if (ks >= steps) continue;
                    const uint64_t dp = desc_at(dp0, p + (ks / 4) * ((C::kPRows * 128) >> 4) + (ks % 4) * 2);
                    const uint32_t acc = !x.first || ks > 0 ? 1u : 0u;
                    constexpr uint32_t kStep = (C::kStepKeys * 128) >> 4;
                    if (C::kWide > 0)
                        mma(o, desc_at(dv0, v + ks * kStep), dp, idesc_o, acc);
                    else  // 64-byte rows
                        mma(o, desc_at(dk0n, v + ks * (kStep / 2)), dp, idesc_o, acc);
                    if (C::kBlocks > 1) {
                        if (C::kNarrow)
                            mma(o + NO, desc_at(dk0n, v + kSecond + ks * (kStep / 2)), dp, idesc_o2, acc);
                        else
                            mma(o + NO, desc_at(dv0, v + kSecond + ks * kStep), dp, idesc_o2, acc);
                    }
                }
                tc_commit(bar.pv_done(x.t & 1));
                tc_commit(bar.empty(sl));
            };
            Tile now, nxt;
            bool have = tiles.next(a, now), more = true, s_out = false, pv_out = false;
            bool ahead = false;  // S of nxt is out
            if (have) more = tiles.next(a, nxt);
            uint64_t t0 = globaltimer_ns();
            for (uint32_t spin = 1; have; ++spin) {
                bool did = false;
                if (!s_out) {
                    if (s_ready(now)) {
                        issue_s(now);
                        s_out = did = true;
                    }
                } else if (more && !ahead && s_ready(nxt)) {
                    issue_s(nxt);
                    ahead = did = true;
                }
                if (s_out && !pv_out && pv_ready(now)) {
                    issue_pv(now);
                    pv_out = did = true;
                }
                if (pv_out) {  // on to the next tile
                    have = more;
                    now = nxt;
                    s_out = ahead;
                    pv_out = ahead = false;
                    if (more) more = tiles.next(a, nxt);
                }
                if (did) {
                    spin = 0;
                } else if (spin == 1) {
                    t0 = globaltimer_ns();
                } else if ((spin & 63u) == 0u && globaltimer_ns() - t0 > kWaitLimitNs) {
                    report_error(a.err, DEV_ERR_TIMEOUT);
                    break;
                }
            }
            // ... and no product
            tc_commit(bar.drain());
            mbar_wait(bar.drain(), 0, a.err);
        }
    } else if (warp == 6) {
        // queries: rows of the operand are part * GP + head
        Segments& c = tiles.c;
        constexpr int kPairs = (D + 63) / 64;  // of neighbouring dims, per lane
        unsigned long long tiles_of[2] = {0, 0};  // the buffers' segments
        while (ok && c.valid) {
            const int qb = c.it & 1;
            const int g = c.u / a.groups, h0 = g * a.G + (c.u - g * a.groups) * GP;
            const int heads = min(GP, (g + 1) * a.G - h0);
            float2 f[GP][kPairs];
#pragma unroll
            for (int h = 0; h < GP; ++h) {
                const T* q = static_cast<const T*>(a.q) + c.b * a.qs[0] + (h0 + h) * a.qs[1];
#pragma unroll
                for (int i = 0; i < kPairs; ++i) {
                    const int p = lane + 32 * i;
                    f[h][i] = h < heads && 2 * p < D
                                  ? dt_traits<T>::unpack2(*reinterpret_cast<const uint32_t*>(q + 2 * p))
                                  : make_float2(0.f, 0.f);
                }
            }
            ok = __all_sync(0xffffffffu, mbar_wait_inl(bar.q_empty(qb), ((c.it >> 1) & 1) ^ 1u, a.err,
                                                       kWaitLimitNs + tiles_of[qb] * kTileLimitNs));
            if (!ok) break;
            tiles_of[qb] = c.n;
            const uint32_t dst = sQ + qb * C::kQBytes;
#pragma unroll
            for (int h = 0; h < GP; ++h) {
                float down = 1.f, up = 1.f;
                if (E8) {
                    uint32_t most = 0;
#pragma unroll
                    for (int i = 0; i < kPairs; ++i) {
                        const uint32_t x = __float_as_uint(f[h][i].x) & 0x7fffffffu;
                        const uint32_t y = __float_as_uint(f[h][i].y) & 0x7fffffffu;
                        if (x < 0x7f800000u) most = max(most, x);
                        if (y < 0x7f800000u) most = max(most, y);
                    }
                    most = __reduce_max_sync(0xffffffffu, most);
                    const int e = most ? max(static_cast<int>(most >> 23) - 127 - 7, -100) : 0;
                    down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
                    up = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
                }
                if (lane == 0) factors[qb * C::kHeads + h] = up * a.scale * kLog2e;
#pragma unroll
                for (int i = 0; i < kPairs; ++i) {
                    const int col = 2 * (lane + 32 * i) * C::kElem;  // byte of the row
                    if (2 * (lane + 32 * i) >= D) continue;
                    uint32_t c8[C::kQParts];
                    if (E8) {
                        split_parts<C::kQParts>(f[h][i].x * down, f[h][i].y * down, c8);
                        // an infinity is no code: a NaN, as its scores' softmax is
                        if (isinf(f[h][i].x)) c8[0] |= 0x7fu;
                        if (isinf(f[h][i].y)) c8[0] |= 0x7f00u;
                    } else {
                        c8[0] = dt_traits<T>::pack2(f[h][i].x, f[h][i].y);
                    }
#pragma unroll
                    for (int s = 0; s < C::kQParts; ++s) {
                        const int n = s * GP + h;
                        uint32_t at;
                        if (col < 128 * C::kWide)
                            at = dst + (col / 128) * C::kQRows * 128 + n * 128 + ((col & 127) ^ ((n & 7) << 4));
                        else
                            at = dst + C::kWide * C::kQRows * 128 + n * 64 +
                                 ((col - 128 * C::kWide) ^ (((n >> 1) & 3) << 4));
                        if (E8)
                            asm volatile("st.shared.b16 [%0], %1;" ::"r"(at),
                                         "h"(static_cast<uint16_t>(c8[s])) : "memory");
                        else
                            asm volatile("st.shared.b32 [%0], %1;" ::"r"(at), "r"(c8[s]) : "memory");
                    }
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar.q_full(qb));
            c.next(a);
        }
    } else {
        Segments& c = tiles.c;
        const int quarter = warp & 3;
        const int key = quarter * 32 + lane;  // TMEM lane: key of a tile
        const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
        const uint32_t tS = tmem + lane_off, tO = tmem + lane_off + C::kColO;
        int t = 0;
        // a segment's O is in TMEM until its last PV has completed: read out
        // behind the next segment's first tile
        bool pend = false;
        int pend_t = 0, pend_buf = 0, pend_heads = 0;
        int64_t pend_rec = 0;
        auto read_out = [&]() -> bool {
            if (!mbar_wait(bar.pv_done(pend_t & 1), (pend_t >> 1) & 1, a.err)) return false;
            tc_fence_after();
            uint32_t o[C::kBlocks][C::kLdO];
#pragma unroll
            for (int mb = 0; mb < C::kBlocks; ++mb)
                ld_cols<C::kLdO>(tO + NO * (C::kBlocks * pend_buf + mb), o[mb]);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar.o_free(pend_buf));
            float inv[GP];
            if (a.direct) {  // (the only segment: its sums are the first)
#pragma unroll
                for (int h = 0; h < GP; ++h) {
                    const float4 w = *reinterpret_cast<const float4*>(red_sum + h * 4);
                    const float sum = (w.x + w.y) + (w.z + w.w);
                    inv[h] = sum == 0.f ? 0.f : 1.f / (sum * (C::kTop * C::kBack));
                }
            }
#pragma unroll
            for (int mb = 0; mb < C::kBlocks; ++mb) {
                // a block of 64 rows takes 16 lanes of each quarter
                const bool half = D == 64 || mb == 1;
                const int dim = half ? mb * 128 + quarter * 16 + lane : key;
                if ((!half || lane < 16) && dim < D) {
#pragma unroll
                    for (int h = 0; h < GP; ++h) {
                        float v = fmaf(__uint_as_float(o[mb][GP + h]), 1.f / static_cast<float>(C::kUp),
                                       __uint_as_float(o[mb][h]));
                        if (C::kPParts > 2)
                            v = fmaf(__uint_as_float(o[mb][(C::kPParts - 1) * GP + h]), 1.f / static_cast<float>(C::kUp * C::kUp), v);
                        if (!a.direct) {
                            a.po[(pend_rec * GP + h) * D + dim] = v * (1.f / (C::kTop * C::kBack));
                        } else if (h < pend_heads) {
                            const uint16_t bits =
                                static_cast<uint16_t>(dt_traits<T>::pack2(v * inv[h], 0.f));
                            static_cast<uint16_t*>(a.o)[(pend_rec + h) * D + dim] = bits;
                        }
                    }
                }
                __syncwarp();
            }
            return true;
        };
        while (ok && c.valid) {
            float m[GP], l[GP], slope[GP], mul[GP];
            if (!(ok = mbar_wait(bar.q_full(c.it & 1), (c.it >> 1) & 1, a.err))) break;
            const int g = c.u / a.groups, h0 = g * a.G + (c.u - g * a.groups) * GP;
#pragma unroll
            for (int h = 0; h < GP; ++h) {
                m[h] = -INFINITY;
                l[h] = 0.f;
                mul[h] = factors[(c.it & 1) * C::kHeads + h];
                slope[h] = 0.f;
                if (a.alibi) {
                    const int hq = min(h0 + h, a.H - 1);
                    slope[h] = kLog2e * (a.slopes ? a.slopes[hq]
                                                  : exp2f(-8.0f * static_cast<float>(hq + 1) /
                                                          static_cast<float>(a.H)));
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(bar.q_empty(c.it & 1));
            for (int i = 0; i < c.n; ++i, ++t) {
                const int row = (c.first + c.n - 1 - i) * kTK;
                const int keys = c.len - row;
                if (!mbar_wait(bar.scale_full(t & 7), (t >> 3) & 1, a.err) ||
                    !mbar_wait(bar.s_full(t & 1), (t >> 1) & 1, a.err)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                uint32_t r[C::kLdS];
                ld_cols<C::kLdS>(tS + NS * (t & 1), r);
                const float ks = scales[(t & 7) * 16 + key / 16];
                const float vs = scales[(t & 7) * 16 + 8 + key / 16];
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar.s_free(t & 1));
                const bool seen = key < keys && !(ks < 0.f);
                const float back = static_cast<float>(row + key - (c.len - 1));
                // the scale of V is at most 2^up
                const int up = static_cast<int>((__float_as_uint(vs) + 0x7fffffu) >> 23) - 127;
                const float shift = E8 ? static_cast<float>(max(up, -60)) - C::kShift : 0.f;
                float s[GP];
                float* rm = red_max + (t & 1) * 4 * C::kHeads;
#pragma unroll
                for (int h = 0; h < GP; ++h) {
                    float v = __uint_as_float(r[h]);
                    if (C::kQParts > 1) v = fmaf(__uint_as_float(r[GP + h]), 1.f / 32, v);
                    if (C::kQParts > 2)
                        v = fmaf(__uint_as_float(r[(C::kQParts - 1) * GP + h]), 1.f / 1024, v);
                    s[h] = seen ? fmaf(v, E8 ? mul[h] * ks : mul[h], slope[h] * back) : -INFINITY;
                    const float w = warp_max(s[h] + shift);
                    if (lane == h) rm[h * 4 + quarter] = w;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(bar.max_full());
                if (!mbar_wait(bar.max_full(), t & 1, a.err)) {
                    ok = false;
                    break;
                }
                // the same decision in every thread
                // (8 bits: half of the way, since references may lie further apart than a number is small)
                constexpr float kWay = E8 ? 0.5f : 1.f;
                float corr[GP];
                bool moved = false;
#pragma unroll
                for (int h = 0; h < GP; ++h) {
                    const float4 w = *reinterpret_cast<const float4*>(rm + h * 4);
                    const float mx = fmaxf(fmaxf(w.x, w.y), fmaxf(w.z, w.w));
                    corr[h] = 1.f;
                    if (mx > m[h] + C::kThreshold) {
                        corr[h] = ex2_approx(kWay * (m[h] - mx));
                        m[h] = mx;
                        moved = true;
                    }
                }
                // P^T buffer t & 1 was read by the PV of tile t - 2
                if (t > 1 && !mbar_wait(bar.pv_done(t & 1), ((t >> 1) - 1) & 1, a.err)) {
                    ok = false;
                    break;
                }
                float p[GP];
#pragma unroll
                for (int h = 0; h < GP; ++h) {
                    // (nothing seen so far: 0, not a NaN)
                    p[h] = ex2_approx(s[h] - (m[h] == -INFINITY ? 0.f : m[h]));
                    l[h] = fmaf(E8 ? l[h] * corr[h] : l[h], corr[h], p[h]);
                }
                const uint32_t p_buf = sP + (t & 1) * C::kPBytes;
                const float top = E8 ? vs * (C::kTop * C::kBack) : C::kTop;
                constexpr int kStep = GP > 1 ? 2 : 1;
#pragma unroll
                for (int h = 0; h < GP; h += kStep) {
                    uint32_t c[C::kPParts];
                    const float x = p[h] * top, y = GP > 1 ? p[h + kStep - 1] * top : 0.f;
                    if constexpr (E8) split_parts<C::kPParts>(x, y, c);
                    else split_16<T, C::kUp>(x, y, c);
#pragma unroll
                    for (int q = 0; q < C::kPParts; ++q)
#pragma unroll
                        for (int e = 0; e < kStep; ++e) {
                            const int n = q * GP + h + e;
                            if constexpr (E8)
                                st_byte(p_buf + n * 128 + (key ^ ((n & 7) << 4)), c[q] >> (8 * e));
                            else
                                st_half(p_buf + (key / 64) * C::kPRows * 128 + n * 128 +
                                            (((key & 63) * 2) ^ ((n & 7) << 4)),
                                        c[q] >> (16 * e));
                        }
                }
                if (keys < kTK && (keys & 15) && quarter == 0) {
                    // values behind the tile's end, up to the next copied box
                    const int rv = 2 * t + 1, sl = rv % kSlots;
                    if (!mbar_wait(bar.full(sl), (rv / kSlots) & 1, a.err)) {
                        ok = false;
                        break;
                    }
                    const int n = 16 - (keys & 15);
                    const uint32_t at = sKV + sl * C::kTile;
#pragma unroll
                    for (int w = 0; w < C::kWide; ++w)
                        for (int x = lane; x < 8 * n; x += 32)
                            st_shared_v4(at + w * kTK * 128 + keys * 128 + x * 16, 0u, 0u, 0u, 0u);
                    if (C::kNarrow)
                        for (int x = lane; x < 4 * n; x += 32)
                            st_shared_v4(at + C::kWide * kTK * 128 + keys * 64 + x * 16, 0u, 0u, 0u, 0u);
                }
                fence_proxy_async_smem();
                if (i > 0 && moved) {
                    if (!mbar_wait(bar.pv_done((t - 1) & 1), ((t - 1) >> 1) & 1, a.err)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    if (E8)
#pragma unroll
                        for (int h = 0; h < GP; ++h) corr[h] *= corr[h];
#pragma unroll
                    for (int mb = 0; mb < C::kBlocks; ++mb) {
                        uint32_t o[C::kLdO];
                        const uint32_t col = tO + NO * (C::kBlocks * (c.it & 1) + mb);
                        ld_cols<C::kLdO>(col, o);
#pragma unroll
                        for (int n = 0; n < C::kPUsed; ++n)
                            o[n] = __float_as_uint(__uint_as_float(o[n]) * corr[n % GP]);
                        st_cols<C::kLdO>(col, o);
                    }
                    tc_fence_before();
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(bar.p_full(t & 1));
                if (pend) {
                    ok = read_out();
                    pend = false;
                    if (!ok) break;
                }
            }
            if (!ok) break;
            // Keys seen, each with a score of -inf: no softmax (0 / 0) unless another segment has a finite one. Whether any is
            // seen is looked up again (kept from tile to tile: 127 us for 122, 256 sequences, 32 heads on one). Over
            // e4m3 such a score is NaN: the queries' operand has no infinity, and codes are none.
            if (!E8) {
                bool none = false;
#pragma unroll
                for (int h = 0; h < GP; ++h) none = none || m[h] == -INFINITY;
                if (none) {
                    bool any = false;
                    for (int i = 0; i < c.n && !any; ++i) {
                        const int at = (c.first + i) * kTK + key;
                        if (at >= c.len) break;
                        const int page = a.c.table[static_cast<int64_t>(c.b) * a.c.max_pages + (at >> lg)];
                        any = page >= 0 && page < a.c.pages;
                    }
#pragma unroll
                    for (int h = 0; h < GP; ++h)
                        if (any && m[h] == -INFINITY && l[h] == 0.f) l[h] = a.direct ? NAN : 1.f;
                }
            }
            // the segment's result
#pragma unroll
            for (int h = 0; h < GP; ++h) {
                float v = l[h];
#pragma unroll
                for (int x = 16; x > 0; x >>= 1) v += __shfl_xor_sync(0xffffffffu, v, x);
                if (lane == h) red_sum[((c.it & 1) * C::kHeads + h) * 4 + quarter] = v;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(bar.sum_full());
            if (!mbar_wait(bar.sum_full(), c.it & 1, a.err)) {
                ok = false;
                break;
            }
            const int64_t rec = static_cast<int64_t>(blockIdx.x) +
                                (static_cast<int64_t>(c.b) * a.units + c.u);
            pend = true;
            pend_t = t - 1;
            pend_buf = c.it & 1;
            pend_rec = a.direct ? static_cast<int64_t>(c.b) * a.H + h0 : rec;
            pend_heads = (g + 1) * a.G - h0;
            if (!a.direct && quarter == 0 && lane < GP) {
                const float4 w = *reinterpret_cast<const float4*>(red_sum + ((c.it & 1) * C::kHeads + lane) * 4);
                float mh = m[0];
#pragma unroll
                for (int h = 1; h < GP; ++h)
                    if (lane == h) mh = m[h];
                a.pm[rec * GP + lane] = make_float2(mh, (w.x + w.y) + (w.z + w.w));
            }
            c.next(a);
        }
        if (ok && pend) ok = read_out();
    }
}

template <typename T, bool E8, int D, int GP>
__global__ void __launch_bounds__(kThreads, (Cfg<T, E8, D, GP>::kCtas))
    paged_kernel(const __grid_constant__ PagedMapSet tm, const __grid_constant__ PagedArgs a) {
    using C = Cfg<T, E8, D, GP>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ Range range;
    uint8_t* smem = align_1024(smem_raw);
    const Bars<C::kSlots> bar{smem_u32(smem) + C::kOffBar};
    static_assert(Bars<C::kSlots>::kBytes <= 512, "barrier space");
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffSlot);
    const int warp = threadIdx.x / 32;
    const int lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        bar.init();
        fence_barrier_init();
        for (int i = 0; i < 4; ++i) tma_prefetch_desc(&tm.m[i / 2][i % 2][C::kWide ? 0 : 1]);
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(tmem_slot), C::kCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    if (a.pdl) pdl_wait();
    Tiles tiles;
    bool ok = true;
    if (a.direct) {
        // a unit per CTA, whole
        const int b = static_cast<int>(blockIdx.x) / a.units, u = static_cast<int>(blockIdx.x) - b * a.units;
        const int len = len_of(a, b), nt = (len + kTK - 1) / kTK;
        tiles.c.start(static_cast<int64_t>(u) * nt, static_cast<int64_t>(u + 1) * nt, b, 0, len);
        if (nt == 0) {  // no key: zero rows
            const int g = u / a.groups, h0 = g * a.G + (u - g * a.groups) * GP;
            const int n = min(GP, (g + 1) * a.G - h0) * (D / 8);
            uint4* o = reinterpret_cast<uint4*>(static_cast<T*>(a.o) + (static_cast<int64_t>(b) * a.H + h0) * D);
            for (int i = threadIdx.x; i < n; i += kThreads) o[i] = make_uint4(0u, 0u, 0u, 0u);
        }
    } else if (a.c.B <= kFewSequences) {
        warp_range(a, lane, warp == 2, tiles.c);
    } else {
        if (warp >= 2 && warp < 6) find_range(a, range, bar.range_full());
        ok = mbar_wait(bar.range_full(), 0, a.err);
        if (ok) tiles.c.start(range.lo, range.hi, range.b0, range.base,
                              range.lo < range.hi ? len_of(a, range.b0) : 0);
    }
    if (ok) {
        const PagedMaps maps{{{tm.m[0][0], tm.m[0][1]}, {tm.m[1][0], tm.m[1][1]}}};
        paged_body<T, E8, D, GP>(a, maps, tiles, smem, tmem, warp, lane);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, C::kCols);
    if (a.pdl) pdl_launch_dependents();
}

template <typename T, bool E8, int D, int GP>
cudaError_t launch_paged_g(const PagedMapSet& tm, PagedArgs& a, int sms, cudaStream_t s) {
    using C = Cfg<T, E8, D, GP>;
    auto kern = paged_kernel<T, E8, D, GP>;
    const cudaError_t e = set_smem_attr_once(reinterpret_cast<const void*>(kern), C::kSmem);
    if (e != cudaSuccess) return e;
    const int64_t room = static_cast<int64_t>(a.c.max_pages) << a.c.page_log2;
    const int64_t most = static_cast<int64_t>(a.c.B) * a.units * ((room + kTK - 1) / kTK);
    int64_t grid = C::kCtas * sms;
    grid = grid < kPagedMaxGrid ? grid : kPagedMaxGrid;
    grid = a.direct ? static_cast<int64_t>(a.c.B) * a.units : grid < most ? grid : most;
    a.grid = static_cast<int>(grid);
    return launch_pdl(a.pdl != 0, kern, dim3(a.grid), dim3(kThreads), C::kSmem, s, tm,
                      static_cast<const PagedArgs&>(a));
}

template <typename T, bool E8, int D>
cudaError_t launch_paged_d(const PagedMapSet& tm, PagedArgs& a, int sms, cudaStream_t s) {
    switch (a.GP) {
        case 1: return launch_paged_g<T, E8, D, 1>(tm, a, sms, s);
        case 4: return launch_paged_g<T, E8, D, 4>(tm, a, sms, s);
        case 8: return launch_paged_g<T, E8, D, 8>(tm, a, sms, s);
        default:
            if constexpr (!E8 && D >= 128)
                if (a.GP == 16) return launch_paged_g<T, E8, D, 16>(tm, a, sms, s);
            return cudaErrorInvalidValue;
    }
}

template <typename T, bool E8>
cudaError_t launch_paged_t(const PagedMapSet& tm, PagedArgs& a, int sms, cudaStream_t s) {
    switch (a.c.d) {
        case 64: return launch_paged_d<T, E8, 64>(tm, a, sms, s);
        case 128: return launch_paged_d<T, E8, 128>(tm, a, sms, s);
        case 160: return launch_paged_d<T, E8, 160>(tm, a, sms, s);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace

}  // namespace blk
