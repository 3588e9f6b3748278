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
// Work: a team of threads takes one page's new rows of one head of K or V, so that the page's
// largest value is found and used in one place, without atomics: each thread holds
// its turned values in registers between the two. Blocks of queries take a
// group of heads and reuse the angles. The number of pages that a sequence
// touches is device data: sequence b's items are numbers floor(cu[b] / size) + 2 b and
// up, which leaves room for floor(n / size) + 2 items, enough for n tokens from any
// offset; surplus blocks end at once.
// To read and write: the new rows, their codes and scales, once. Measured and bound: the queries' part
// by those bytes, the keys' and values' in 8 bits by instructions and latency per row at 0.6 of the copy
// rate; 27595 tokens of 32/8 x 128 heads with queries 100 us (6.2 TB/s), 5713 of 32 x 64 24.5 us (4.7
// TB/s); a step of 16 sequences 4 us.
#include <cuda_fp8.h>

#include <algorithm>
#include <cmath>
#include <type_traits>

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
    int tokens, H;             // query heads
    int kv_log2, q_log2;       // tokens of an item, of keys and values and of queries
    unsigned kv_items, q_items;
    int team, teams;           // threads of an item of keys or values and head, and such teams
    int kv_rows;               // rows that a team takes in a round
    int64_t head_hop[2], cache_hop;  // elements from a team's head to its next one, of k, v and the cache
    int kv_per, kv_groups;     // heads of K and V per block (K's, then V's), and blocks of them
    int q_per;                 // query heads per block
    int pdl;
};

// The new rows of one item: of a sequence's positions j 2^lg .. (j + 1) 2^lg - 1 for some j.
struct ItemRows {
    int b, n;          // sequence, rows
    int64_t row, pos;  // of the first: row of k, v and q, position
};

__device__ __forceinline__ int start_of(const AppendArgs& a, int b) {
    return min(max(a.cu[b], 0), a.tokens);
}

// Rows of item i, in every thread of a warp alike; false: none.
__device__ __forceinline__ bool rows_of(const AppendArgs& a, int64_t i, int lg, int lane, ItemRows& r) {
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
    const int64_t j = (p0 >> lg) + at;
    const int64_t lo = max(p0, j << lg), hi = min(end, (j + 1) << lg);
    if (at < 0 || lo >= hi) return false;
    r.n = static_cast<int>(hi - lo);
    r.row = c0 + lo;
    r.pos = lo;
    return true;
}

__device__ __forceinline__ float max_abs(float a, float b, float c) {
    float r;
    asm("max.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ float if_finite(float x) {
    x = fabsf(x);
    return x < INFINITY ? x : 0.f;
}

// The smallest power of two of at least 2^-60 with which a number takes at most 448 = 1.75 * 2^8.
__device__ __forceinline__ float scale_for(float most) {
    const int e = static_cast<int>((__float_as_uint(most) + 0x1fffffu) >> 23) - 127 - 8;
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

// A block's heads of queries of an item: threads by head, token and unit.
template <typename T, int VP>
__device__ __forceinline__ void turn_queries(const AppendArgs& a, const ItemRows& r, const Unit<VP>& at,
                                             const uint64_t* plan, int group, int place, int rows) {
    using Raw = typename RawPiece<VP>::type;
    const float m = a.turn.plan.amplitude;
    const int side = min(rows, 1 << a.q_log2);       // tokens side by side
    const int step = rows / side;                    // and heads
    const int h0 = group * a.q_per, h1 = min(h0 + a.q_per, a.H);
    if (place >= side * step) return;
    for (int k = place % side; k < r.n; k += side) {
        Angles<VP> ang;
        if (at.turned) {
            uint64_t turns[VP];
#pragma unroll
            for (int i = 0; i < VP; ++i)
                turns[i] = VP == 1 || i < VP / 2 ? plan[at.p0 + i] : plan[at.p1 + i - VP / 2];
            ang.set(turns, a.positions ? a.positions[r.row + k] : static_cast<int>(r.pos + k), m, m);
        }
        const T* x = static_cast<const T*>(a.x[2]) + (r.row + k) * a.xs[2][1];
        T* y = static_cast<T*>(a.q_out) + (r.row + k) * a.qs[1];
        // several heads' loads on their way at a time
        constexpr int kHeads = VP == 8 ? 2 : 4;
        for (int h = h0 + place / side; h < h1; h += kHeads * step) {
            Raw raw[kHeads][2];
#pragma unroll
            for (int i = 0; i < kHeads; ++i)
                if (h + i * step < h1) {
                    raw[i][0] = load_raw<T, VP>(x + (h + i * step) * a.xs[2][0] + at.a);
                    raw[i][1] = load_raw<T, VP>(x + (h + i * step) * a.xs[2][0] + at.b);
                }
#pragma unroll
            for (int i = 0; i < kHeads; ++i)
                if (h + i * step < h1) {
                    float p[VP], q[VP];
                    unpack_raw<T, VP>(raw[i][0], p);
                    unpack_raw<T, VP>(raw[i][1], q);
                    if (at.turned) ang.turn(p, q, a.turn.plan.interleaved);
                    store_piece(y + (h + i * step) * a.qs[0] + at.a, p);
                    store_piece(y + (h + i * step) * a.qs[0] + at.b, q);
                }
        }
    }
}

// A block has teams of threads: a team takes one item and head at a time, its threads so many that IT
// rounds of them hold the rows. What a block needs to know of its item (the search, the length, the
// table) is a chain of dependent loads, which its teams and heads share: with a block of one warp for
// each page and head, 5713 tokens of 32 x 64 heads took 47 us, with teams 34, and 24.5 with the steps
// below.
// ROUNDS (8 bits): for pages of more values than 512 threads hold: 256 read the rows twice (a variant of its own,
// since its registers would be the other's spills).
template <typename T, bool E8, int VP, int IT, bool ROUNDS>
__global__ void __launch_bounds__(IT * VP > 8 ? 768 : 1024) kv_append_kernel(const __grid_constant__ AppendArgs a) {
    static_assert(E8 || !ROUNDS, "16-bit items fit a block");
    __shared__ float most[2][32];
    extern __shared__ float4 angles[];
    __shared__ uint64_t plan[kMaxRotaryPairs];
    const int d = a.c.d, units = d / (2 * VP);
    const int lane = threadIdx.x & 31;
    // blocks of keys and values, the longest, come first, then those of queries (side by side:
    // 118 us for 112 in the large case, the tail being one of the former)
    const unsigned kv_blocks = a.kv_items * a.kv_groups;
    const bool is_q = blockIdx.x >= kv_blocks;
    const unsigned of = is_q ? a.q_items : a.kv_items, nth = is_q ? blockIdx.x - kv_blocks : blockIdx.x;
    const int group = nth / of, item = nth - group * of;
    // queries: threads by head, token and unit; else by team, token and unit
    const int threads = is_q ? blockDim.x : a.team;
    const int team = is_q ? 0 : threadIdx.x / a.team;
    const int tid = is_q ? threadIdx.x : threadIdx.x % a.team;
    const int u = tid % units, place = tid / units;
    const int rows = threads / units;
    const Unit<VP> at(u, d, a.turn.plan.pairs, a.turn.plan.interleaved);
    for (int i = threadIdx.x; i < a.turn.plan.pairs; i += blockDim.x) plan[i] = a.turn.plan.turns[i];
    const float m = a.turn.plan.amplitude;
    __syncthreads();
    if (a.pdl) pdl_wait();
    ItemRows r;
    if (!rows_of(a, item, is_q ? a.q_log2 : a.kv_log2, lane, r)) return;
    using Raw = typename RawPiece<VP>::type;

    // cosines and sines of the rows, for all the block's heads of keys: plane j of a unit's pairs
    // 2 j and 2 j + 1 (VP 1: of its pair)
    const int turned_units = a.turn.plan.pairs / VP, cells = r.n * turned_units;
    constexpr int kPlanes = VP > 1 ? VP / 2 : 1;
    auto make_table = [&]() {
        for (int i = threadIdx.x; i < cells * kPlanes; i += blockDim.x) {
            const int cell = i / kPlanes, j = i - cell * kPlanes;
            const int k = cell / turned_units;
            const Unit<VP> of(cell - k * turned_units, d, a.turn.plan.pairs, a.turn.plan.interleaved);
            const int pair = VP == 1 ? of.p0 : 2 * j < VP / 2 ? of.p0 + 2 * j : of.p1 + 2 * j - VP / 2;
            const int pos = a.positions ? a.positions[r.row + k] : static_cast<int>(r.pos + k);
            float c0, s0, c1, s1;
            turn_cos_sin(plan[pair], pos, c0, s0);
            if constexpr (VP > 1) {
                turn_cos_sin(plan[pair + 1], pos, c1, s1);
                angles[j * cells + cell] = make_float4(c0 * m, s0 * m, c1 * m, s1 * m);
            } else {
                reinterpret_cast<float2*>(angles)[cell] = make_float2(c0 * m, s0 * m);
            }
        }
        __syncthreads();
    };
    // ... two pairs at a time
    auto turn_by_table = [&](int cell, float (&x)[VP], float (&y)[VP]) {
        if constexpr (VP > 1) {
            if (a.turn.plan.interleaved) {
#pragma unroll
                for (int j = 0; j < kPlanes; ++j) {
                    const float4 f = angles[j * cells + cell];
                    float(&z)[VP] = j < kPlanes / 2 ? x : y;
                    turn_pair(z[4 * j % VP], z[4 * j % VP + 1], f.x, f.y);
                    turn_pair(z[4 * j % VP + 2], z[4 * j % VP + 3], f.z, f.w);
                }
            } else {
#pragma unroll
                for (int j = 0; j < kPlanes; ++j) {
                    const float4 f = angles[j * cells + cell];
                    turn_pair(x[2 * j], y[2 * j], f.x, f.y);
                    turn_pair(x[2 * j + 1], y[2 * j + 1], f.z, f.w);
                }
            }
        } else {
            const float2 f = reinterpret_cast<const float2*>(angles)[cell];
            turn_pair(x[0], y[0], f.x, f.y);
        }
    };

    if (is_q) {
        turn_queries<T, VP>(a, r, at, plan, group, place, rows);
        return;
    }

    // a page of the sequence's that is not there takes nothing
    const int64_t column = r.pos >> a.c.page_log2;
    if (column >= a.c.max_pages) return;
    const int page = a.c.table[static_cast<int64_t>(r.b) * a.c.max_pages + column];
    if (page < 0 || page >= a.c.pages) return;
    const int in_page = static_cast<int>(r.pos & ((1 << a.c.page_log2) - 1));  // the first row's place
    const int team_warps = a.team / 32;
    // (What is the same for all blocks is read from the arguments at each use: registers hold less, fewer
    // are spilled. 27595 tokens of 32/8 x 128: 101.4 -> 100.3 us; 3020 of 16 x 64, 16 bits: 9.41 -> 9.33.)
    const int first = group * a.kv_per, end = min(first + a.kv_per, 2 * a.c.Hk);
    const int64_t head_size = static_cast<int64_t>(d) << a.c.page_log2;
    // This thread's rows: the others' values are zeros, which change no largest one, and are not
    // stored. (With everything of a row behind its condition the branches were a tenth of the kernel.)
    bool on[IT];
    int cell[IT];
#pragma unroll
    for (int i = 0; i < IT; ++i) {
        const int k = place + i * a.kv_rows;
        on[i] = place < a.kv_rows && k < r.n;
        cell[i] = min(k, r.n - 1) * turned_units + u;
    }
    const int gap = at.b - at.a;
    const int chunks = (r.n + a.kv_rows * IT - 1) / (a.kv_rows * IT);
    // The largest of x over the team (a round of its own barrier; entries alternate between rounds).
    int odd = 0;
    auto of_team = [&](float x) {
        x = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(x)));
        if (team_warps > 1) {
            if (lane == 0) most[odd][threadIdx.x / 32] = x;
            asm volatile("bar.sync %0, %1;" ::"r"(1 + team), "r"(a.team) : "memory");
            x = most[odd][team * team_warps + (lane < team_warps ? lane : 0)];
            x = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(x)));
            odd ^= 1;
        } else {
            __syncwarp();  // every lane has read the scale
        }
        return x;
    };
    // Heads s0 + team, s0 + team + teams, ... < s1 of K or of V.
    auto append = [&](auto values, int s0, int s1) {
        constexpr bool kValues = decltype(values)::value;
        s0 += team;
        if (s0 >= s1) return;
        // (the values' pieces lie where the keys' do)
        const bool turned = at.turned && !kValues;
        // (offsets in a head fit 32 bits: token strides are below 2^24)
        const T* x = static_cast<const T*>(a.x[kValues]) + s0 * a.xs[kValues][0] + r.row * a.xs[kValues][1];
        const int64_t base = page * a.c.page_stride + s0 * head_size + in_page * d;
        uint8_t* codes = static_cast<uint8_t*>(kValues ? a.c.v : a.c.k) + base;
        T* cache = static_cast<T*>(kValues ? a.c.v : a.c.k) + base;
        float* scale = (kValues ? a.c.v_scale : a.c.k_scale) + static_cast<int64_t>(page) * a.c.Hk + s0;
        constexpr bool kAhead = VP > 1;  // the next head's loads behind this one's (VP 1: too many registers)
        Raw raw[IT][2];
        int from[IT], to[IT];
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            const int k = place + i * a.kv_rows;  // (where there is no such row: a number that is not used)
            from[i] = static_cast<int>(static_cast<uint32_t>(k) * static_cast<uint32_t>(a.xs[kValues][1])) + at.a;
            to[i] = k * d + at.a;
            raw[i][0] = Raw{};
            raw[i][1] = Raw{};
        }
        auto fetch = [&](int ahead) {
#pragma unroll
            for (int i = 0; i < IT; ++i)
                if (on[i]) {
                    raw[i][0] = load_raw<T, VP>(x + from[i]);
                    raw[i][1] = load_raw<T, VP>(x + from[i] + gap);
                }
            x += a.head_hop[kValues];
            // ... and the head after it to the L2 cache (25.2 -> 24.0 us, 109.5 -> 106.9; in 16
            // bits, where blocks are more, it gains nothing)
#pragma unroll
            for (int i = 0; i < IT; ++i)
                if (E8 && on[i] && ahead > 0) {
                    asm volatile("prefetch.global.L2 [%0];" ::"l"(x + from[i]));
                    asm volatile("prefetch.global.L2 [%0];" ::"l"(x + from[i] + gap));
                }
        };
        // Values of rounds c IT .. of a head, for pages of more rows than IT rounds take.
        auto rounds = [&](int c, float (&v)[IT][2][VP], bool (&in)[IT]) {
#pragma unroll
            for (int i = 0; i < IT; ++i) {
                const int k = place + (c * IT + i) * a.kv_rows;
                in[i] = place < a.kv_rows && k < r.n;
                raw[i][0] = Raw{};
                raw[i][1] = Raw{};
                if (in[i]) {
                    raw[i][0] = load_raw<T, VP>(x + k * static_cast<int>(a.xs[kValues][1]) + at.a);
                    raw[i][1] = load_raw<T, VP>(x + k * static_cast<int>(a.xs[kValues][1]) + at.b);
                }
            }
#pragma unroll
            for (int i = 0; i < IT; ++i) {
                unpack_raw<T, VP>(raw[i][0], v[i][0]);
                unpack_raw<T, VP>(raw[i][1], v[i][1]);
                const int k = min(place + (c * IT + i) * a.kv_rows, r.n - 1);
                if (turned) turn_by_table(k * turned_units + u, v[i][0], v[i][1]);
            }
        };
        // The page's scale, set by its largest value; what it holds at another one is brought to it.
        auto set_scale = [&](float top, float held) {
            const float now = fmaxf(scale_for(top), held);
            if (tid == 0) *scale = now;
            if (in_page > 0 && held < now) {
                const float by = held / now;
                uint4* old = reinterpret_cast<uint4*>(codes - in_page * d);
                for (int i = tid; i < in_page * (d / 16); i += a.team) {
                    uint4 o = old[i];
                    o.x = rescaled(o.x, by);
                    o.y = rescaled(o.y, by);
                    o.z = rescaled(o.z, by);
                    o.w = rescaled(o.w, by);
                    old[i] = o;
                }
            }
            return 1.0f / now;
        };
        if constexpr (ROUNDS) {
            // the largest first, then the rows again (from the L2 cache), turned again
            for (int s = s0; s < s1; s += a.teams) {
                float v[IT][2][VP];
                bool in[IT];
                const float held = in_page > 0 ? *scale : 0.f;
                float top = 0.f;
                for (int finite = 0; finite < 2; ++finite) {
                    for (int c = 0; c < chunks; ++c) {
                        rounds(c, v, in);
#pragma unroll
                        for (int i = 0; i < IT; ++i)
#pragma unroll
                            for (int e = 0; e < VP; ++e)
                                top = finite ? fmaxf(top, fmaxf(if_finite(v[i][0][e]), if_finite(v[i][1][e])))
                                             : max_abs(top, v[i][0][e], v[i][1][e]);
                    }
                    top = of_team(top);
                    if (top < INFINITY) break;
                    top = 0.f;
                }
                const float inv = set_scale(top, held);
                for (int c = 0; c < chunks; ++c) {
                    rounds(c, v, in);
#pragma unroll
                    for (int i = 0; i < IT; ++i) {
                        if (!in[i]) continue;
                        const int at_row = (place + (c * IT + i) * a.kv_rows) * d;
                        store_codes<VP>(codes + at_row + at.a, v[i][0], inv);
                        store_codes<VP>(codes + at_row + at.b, v[i][1], inv);
                    }
                }
                x += a.head_hop[kValues];
                codes += a.cache_hop;
                scale += a.teams;
            }
            return;
        }
        if (kAhead) fetch(s1 - s0 - a.teams);
        for (int s = s0; s < s1; s += a.teams) {
            if (!kAhead) fetch(0);
            float v[IT][2][VP];
#pragma unroll
            for (int i = 0; i < IT; ++i) {
                unpack_raw<T, VP>(raw[i][0], v[i][0]);
                unpack_raw<T, VP>(raw[i][1], v[i][1]);
            }
            if (kAhead && s + a.teams < s1) fetch(s1 - s - 2 * a.teams);
            float held = 0.f;
            if (E8 && in_page > 0) held = *scale;  // (a page's first row begins its scale anew)
            float top = 0.f;
#pragma unroll
            for (int i = 0; i < IT; ++i) {
                if (turned) turn_by_table(cell[i], v[i][0], v[i][1]);
                if constexpr (E8) {
#pragma unroll
                    for (int e = 0; e < VP; ++e) top = max_abs(top, v[i][0][e], v[i][1][e]);  // (NaN: passed over)
                }
            }
            if constexpr (E8) {
                top = of_team(top);
                if (top == INFINITY) {  // the largest finite one, then
                    top = 0.f;
#pragma unroll
                    for (int i = 0; i < IT; ++i) {
#pragma unroll
                        for (int e = 0; e < VP; ++e)
                            top = fmaxf(top, fmaxf(if_finite(v[i][0][e]), if_finite(v[i][1][e])));
                    }
                    top = of_team(top);
                }
                const float inv = set_scale(top, held);
#pragma unroll
                for (int i = 0; i < IT; ++i)
                    if (on[i]) {
                        store_codes<VP>(codes + to[i], v[i][0], inv);
                        store_codes<VP>(codes + to[i] + gap, v[i][1], inv);
                    }
                codes += a.cache_hop;
                scale += a.teams;
            } else {
#pragma unroll
                for (int i = 0; i < IT; ++i)
                    if (on[i]) {
                        store_piece(cache + to[i], v[i][0]);
                        store_piece(cache + to[i] + gap, v[i][1]);
                    }
                cache += a.cache_hop;
            }
        }
    };
    if (first < a.c.Hk) {
        make_table();
        append(std::false_type{}, first, min(end, a.c.Hk));
    }
    if (end > a.c.Hk) append(std::true_type{}, max(first - a.c.Hk, 0), end - a.c.Hk);
}

template <typename T, bool E8, int VP, int IT, bool ROUNDS>
cudaError_t launch_variant(const AppendArgs& a, unsigned blocks, int threads, cudaStream_t s) {
    auto kern = kv_append_kernel<T, E8, VP, IT, ROUNDS>;
    const int table = (1 << a.kv_log2) * a.turn.plan.pairs * 8;
    if (table > 46 * 1024) {  // (with the static 1.3 KB, more than a launch has without asking)
        const cudaError_t e = set_smem_attr_once(reinterpret_cast<const void*>(kern), 128 * 1024);
        if (e != cudaSuccess) return e;
    }
    return launch_pdl(a.pdl != 0, kern, dim3(blocks), dim3(threads), table, s, a);
}

template <typename T, bool E8, int VP>
cudaError_t launch_append(AppendArgs& a, int sms, cudaStream_t s) {
    // 32 values per thread at a time; in 16 bits, where no value waits for the page's largest,
    // 16 (10.6 -> 9.4 us for 3020 tokens of 16 x 64)
    constexpr int IT = E8 ? (VP == 8 ? 2 : VP == 4 ? 4 : 16) : VP == 8 ? 1 : VP == 4 ? 4 : 16;
    const int units = a.c.d / (2 * VP);
    // An item of keys and values is a page, whose largest value is one; in 16 bits at most 32 tokens
    // (16 prompts of 994 tokens, 16 x 128, pages of 128: 76 us with items of a page, 64 with these)
    constexpr int kLog2 = 5;
    a.kv_log2 = E8 ? a.c.page_log2 : std::min(a.c.page_log2, kLog2);
    a.team = (units * (((1 << a.kv_log2) + IT - 1) / IT) + 31) / 32 * 32;
    static_assert(E8 || 256 / (2 * VP) * (((1 << kLog2) + IT - 1) / IT) <= 512, "16-bit items are not read in rounds");
    const bool rounds = a.team > 512;
    if (rounds) a.team = 256;
    const int teams = a.team >= 256 ? 1 : 256 / a.team, threads = teams * a.team;
    a.teams = teams;
    a.kv_rows = a.team / units;
    for (int i = 0; i < 2; ++i) a.head_hop[i] = teams * a.xs[i][0];
    a.cache_hop = static_cast<int64_t>(teams) * a.c.d << a.c.page_log2;
    const int64_t B = a.c.B;
    const int64_t kv_items = a.cu ? (a.tokens >> a.kv_log2) + 2 * B : B;
    // Heads of a block: about so many as make one round of blocks, since what is ahead of a block's
    // first load is a chain of latencies; sixteen in turn at most. In 8 bits, where a block takes
    // longest, not above one round: the second one would be the tail (5713 tokens of 32 x 64, eight heads in
    // turn for a team for six: 25.4 -> 24.6 us; in 16 bits, 3020 tokens of 16 x 64: 9.4 -> 10.8).
    const int64_t blocks = static_cast<int64_t>(sms) * std::max(1, (IT * VP > 8 ? 768 : 1024) / threads);
    const int64_t slots = 2 * a.c.Hk, there = a.cu ? (a.tokens >> a.kv_log2) + B : B;
    const int64_t side_by_side = teams * std::max<int64_t>(1, blocks / there);
    const int64_t turns = E8 ? (slots + side_by_side - 1) / side_by_side : kv_items * slots / (teams * blocks);
    const int64_t loops = std::min<int64_t>(16, std::max<int64_t>(1, turns));
    a.kv_per = static_cast<int>(teams * loops);
    a.kv_groups = static_cast<int>((slots + a.kv_per - 1) / a.kv_per);
    const int64_t kv_blocks = kv_items * a.kv_groups;
    // Queries, an item: as many tokens as a block has threads for; heads: four at least for a thread
    // (its loads on their way), so that there are six blocks per SM or so, 32 at most. (In a launch of
    // their own, with fewer registers, they no longer fill what the others leave: 16 prompts of 994
    // tokens, 32 x 64: 69 us for 55.)
    for (a.q_log2 = 3; units << (a.q_log2 + 1) <= threads && a.q_log2 < 7;) ++a.q_log2;
    const int64_t q_items = a.cu ? (a.tokens >> a.q_log2) + 2 * B : B;
    const int64_t step = std::max(1, threads / units >> a.q_log2);  // heads side by side
    const int64_t heads = q_items * a.H / step;
    const int64_t per = heads < 4 * sms ? 1 : std::min<int64_t>(32, (heads / (6 * sms) + 4) / 4 * 4);
    a.q_per = static_cast<int>(step * per);
    const int64_t all = kv_blocks + q_items * ((a.H + a.q_per - 1) / a.q_per);
    if (all > 0x7fffffff) return cudaErrorInvalidConfiguration;
    a.kv_items = static_cast<unsigned>(kv_items);
    a.q_items = static_cast<unsigned>(q_items);
    if constexpr (E8)
        if (rounds) return launch_variant<T, E8, VP, IT, true>(a, static_cast<unsigned>(all), threads, s);
    return launch_variant<T, E8, VP, IT, false>(a, static_cast<unsigned>(all), threads, s);
}
template <typename T, bool E8>
cudaError_t launch_append_w(AppendArgs& a, int sms, cudaStream_t s) {
    switch (turn_width(a.turn.plan.pairs)) {
        case 8: return launch_append<T, E8, 8>(a, sms, s);
        case 4: return launch_append<T, E8, 4>(a, sms, s);
        default: return launch_append<T, E8, 1>(a, sms, s);
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
    // (a unit's tiles are then 2^19 at most, by which attn_paged.cuh counts and sets a wait's limit)
    REQUIRE(d->max_pages * d->page_tokens <= (int64_t(1) << 26), "max_pages * page_tokens out of range");
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
        REQUIRE(i > 1 || strides[i][1] < (int64_t(1) << 24), "token strides of k and v must be below 2^24");
    }
    REQUIRE(!q || places_apart(d->n_heads, d->tokens, d->q_out_head_stride, d->q_out_token_stride, a.c.d),
            "an output's strides make it overlap itself");
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
    const bool e8 = d->cache.kind == BLK_CACHE_E4M3;
    const cudaError_t e =
        dt == BLK_F16 ? (e8 ? launch_append_w<__half, true>(a, sms, cs)
                            : launch_append_w<__half, false>(a, sms, cs))
                      : (e8 ? launch_append_w<__nv_bfloat16, true>(a, sms, cs)
                            : launch_append_w<__nv_bfloat16, false>(a, sms, cs));
    return e == cudaSuccess ? BLK_OK
                            : report_error_status(BLK_ECUDA, "append launch: %s", cudaGetErrorString(e));
}
