// Rotary positions by a plan (blk_rope_plan): what rope_pos.cu and kv_append.cu share.
//
// A plan holds each pair's angle per position in units of 2^-64 of a turn, as a
// 64-bit whole number. position * turns, modulo 2^64, is then the angle modulo one
// turn without any rounding, for every 32-bit position (and negative ones): the
// product of a float loses the fraction of a turn at far positions, and the FP64
// unit, at 2 lanes per SM, is too slow for an angle per token and pair. The
// whole number's upper bits are the quarter turn that the angle is nearest to, the rest, at
// most an eighth of a turn either way, goes to a float and to the Taylor series of sine (to
// x^9) and cosine (to x^8), whose first terms left out are 1.8e-9 and 2.5e-8 there: with
// the 32-bit steps, a turned value is at most 2^-22 (|x| + |y|) off, 2^-23.5 at the most in 600000 pairs (by
// the hardware's sine and cosine 2^-21.3, no faster, and codes of an 8-bit cache moved to their neighbours).
//
// A thread works on a unit: VP pairs of one token, read as two pieces of VP
// elements. The pieces of neighbouring units lie side by side, so that a warp's access is
// whole lines of memory. Half layout: pair j is (j, j + pairs); a unit's pieces are VP dims
// of the first half and their partners. Interleaved: pair j is (2j, 2j + 1); a unit has a piece
// (VP / 2 pairs) in each half of the span. Units behind the turned part have one in each half of
// the rest, which they pass on. (Two pieces next to each other, 32 bytes per thread: half sectors
// at a time.)
// VP is 8 (16-byte accesses) where the span is a multiple of 16, 4 where it is one of
// 8 (40 of 160 dims), else 1.
#pragma once

#include "internal.h"

namespace blk {

struct TurnArgs {
    blk_rope_plan plan;  // pairs 0: nothing is turned
    int inverse;
};

// A piece as it lies in memory, and its numbers.
template <int VP> struct RawPiece;
template <> struct RawPiece<8> { using type = uint4; };
template <> struct RawPiece<4> { using type = uint2; };
template <> struct RawPiece<1> { using type = uint16_t; };

template <typename T, int VP>
__device__ __forceinline__ typename RawPiece<VP>::type load_raw(const T* p) {
    return *reinterpret_cast<const typename RawPiece<VP>::type*>(p);
}
template <typename T, int VP>
__device__ __forceinline__ void unpack_raw(const typename RawPiece<VP>::type& r, float (&f)[VP]) {
    if constexpr (VP == 1) {
        f[0] = dt_traits<T>::unpack2(r).x;
    } else {
        uint32_t w[VP / 2];
        w[0] = r.x;
        w[1] = r.y;
        if constexpr (VP == 8) {
            w[2] = r.z;
            w[3] = r.w;
        }
#pragma unroll
        for (int i = 0; i < VP / 2; ++i) {
            const float2 x = dt_traits<T>::unpack2(w[i]);
            f[2 * i] = x.x;
            f[2 * i + 1] = x.y;
        }
    }
}
template <typename T, int VP>
__device__ __forceinline__ void load_piece(const T* p, float (&f)[VP]) {
    unpack_raw<T, VP>(load_raw<T, VP>(p), f);
}

template <typename T, int VP>
__device__ __forceinline__ void store_piece(T* p, const float (&f)[VP]) {
    if constexpr (VP == 8) {
        store8(p, f);
    } else if constexpr (VP == 4) {
        *reinterpret_cast<uint2*>(p) =
            make_uint2(dt_traits<T>::pack2(f[0], f[1]), dt_traits<T>::pack2(f[2], f[3]));
    } else {
        const uint16_t u = static_cast<uint16_t>(dt_traits<T>::pack2(f[0], 0.f));
        *reinterpret_cast<uint16_t*>(p) = u;
    }
}

// Unit u of a head of d dims: where its two pieces lie, and whether it is turned; the first
// pair of the first and of the second half of its pairs.
template <int VP>
struct Unit {
    int a, b, p0, p1;
    bool turned;
    __device__ __forceinline__ Unit(int u, int d, int pairs, int interleaved) {
        turned = u * VP < pairs;
        if (turned) {
            a = u * VP;
            b = pairs + a;
            p0 = interleaved ? u * (VP / 2) : u * VP;
            p1 = interleaved ? (pairs + u * VP) / 2 : u * VP + VP / 2;
            if (VP == 1 && interleaved) {  // a pair by itself
                a = 2 * u;
                b = a + 1;
                p0 = u;
            }
        } else {
            a = pairs + u * VP;  // span + (u - pairs / VP) VP
            b = a + (d / 2 - pairs);
            p0 = p1 = 0;
        }
    }
};

// Cosine and sine of one pair's angle at a position.
__device__ __forceinline__ void turn_cos_sin(uint64_t turns, int pos, float& c, float& s) {
    const uint32_t t = static_cast<uint32_t>(
        (turns * static_cast<uint64_t>(static_cast<int64_t>(pos)) + 0x80000000ull) >> 32);
    const uint32_t quarter = (t + 0x20000000u) >> 30;
    const float x = static_cast<float>(static_cast<int32_t>(t - (quarter << 30))) *
                    (6.28318530717958648f / 4294967296.0f);
    const float z = x * x;
    float u = fmaf(z, 1.f / 362880, -1.f / 5040);
    u = fmaf(z, u, 1.f / 120);
    u = fmaf(z, u, -1.f / 6);
    u = fmaf(z * x, u, x);  // sine
    float w = fmaf(z, 1.f / 40320, -1.f / 720);
    w = fmaf(z, w, 1.f / 24);
    w = fmaf(z, w, -0.5f);
    w = fmaf(z, w, 1.f);  // cosine
    // a quarter turn on: (c, s) -> (-s, c)
    c = quarter & 1 ? u : w;
    s = quarter & 1 ? w : u;
    if ((quarter + 1) & 2) c = -c;
    if (quarter & 2) s = -s;
}

__device__ __forceinline__ void turn_pair(float& x, float& y, float c, float s) {
    const float x0 = x;
    x = fmaf(x0, c, -(y * s));
    y = fmaf(y, c, x0 * s);
}

// Turns a unit's pieces a and b: pair i by (c[i], s[i]).
template <int VP>
__device__ __forceinline__ void turn_unit(float (&a)[VP], float (&b)[VP], int interleaved,
                                          const float (&c)[VP], const float (&s)[VP]) {
    if (VP > 1 && interleaved) {
#pragma unroll
        for (int i = 0; i < VP / 2; ++i) {
            turn_pair(a[2 * i], a[2 * i + 1], c[i], s[i]);
            turn_pair(b[2 * i], b[2 * i + 1], c[VP / 2 + i], s[VP / 2 + i]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < VP; ++i) turn_pair(a[i], b[i], c[i], s[i]);
    }
}

// A unit's cosines and sines at a position, times the amplitude (sign: the same, or its
// negative to turn back), for several heads.
template <int VP>
struct Angles {
    float c[VP], s[VP];
    __device__ __forceinline__ void set(const uint64_t (&turns)[VP], int pos, float amplitude, float sign) {
#pragma unroll
        for (int i = 0; i < VP; ++i) {
            float cs, sn;
            turn_cos_sin(turns[i], pos, cs, sn);
            c[i] = cs * amplitude;
            s[i] = sn * sign;
        }
    }
    __device__ __forceinline__ void turn(float (&a)[VP], float (&b)[VP], int interleaved) const {
        turn_unit<VP>(a, b, interleaved, c, s);
    }
};

// The widest pieces that a span and a head allow.
inline int turn_width(int pairs) { return pairs % 8 == 0 ? 8 : pairs % 4 == 0 ? 4 : 1; }

// Whether the heads and tokens of an output [heads][tokens][d] each have a place of their own: the shorter
// stride holds a head, the longer one all that the shorter one reaches.
inline bool places_apart(int64_t heads, int64_t tokens, int64_t head_stride, int64_t token_stride, int64_t d) {
    if (heads <= 1) return tokens <= 1 || token_stride >= d;
    if (tokens <= 1) return head_stride >= d;
    const bool inner_heads = head_stride < token_stride;
    const int64_t inner = inner_heads ? head_stride : token_stride, outer = inner_heads ? token_stride : head_stride;
    return inner >= d && (outer - d) / inner >= (inner_heads ? heads : tokens) - 1;
}

// blk_rope_plan_init fills `check` with this: a call refuses a plan that it did not make.
constexpr int32_t kPlanMade = 0x524f5045;
inline bool plan_made(const blk_rope_plan* p, int64_t head_dim) {
    return p->check == kPlanMade && p->pairs >= 1 && p->pairs <= 128 && 2 * p->pairs <= head_dim &&
           (p->interleaved == 0 || p->interleaved == 1);
}

}  // namespace blk
