// Rotary positions by a plan (blk_rope_plan): what rope_pos.cu and kv_append.cu share.
//
// A plan holds each pair's angle per position in units of 2^-64 of a turn, as a
// 64-bit whole number. position * turns, modulo 2^64, is then the angle modulo one
// turn without any rounding, for every 32-bit position (and negative ones): the
// product of a float loses the fraction of a turn at far positions, and the FP64
// unit, at 2 lanes per SM, is too slow for an angle per token and pair. The
// upper 32 bits go to a float (24 bits, at most 2^-25 of half a turn off) and to
// the sine and cosine of the hardware (absolute error 2^-20.9 in half a turn
// either way: 1/900 of the half step of fp16).
//
// A thread works on a unit: VP pairs of one token, read as two pieces of VP
// elements. Half layout: pair j is (j, j + pairs); the pieces are VP dims
// of the first half and their partners. Interleaved: pair j is (2j, 2j + 1); the
// pieces lie side by side. Units behind the turned part pass two pieces on.
// VP is 8 (16-byte accesses) where the span is a multiple of 16, 4 where it is one of
// 8 (40 of 160 dims), else 1.
#pragma once

#include "internal.h"

namespace blk {

struct TurnArgs {
    blk_rope_plan plan;  // pairs 0: nothing is turned
    int inverse;
};

template <typename T, int VP>
__device__ __forceinline__ void load_piece(const T* p, float (&f)[VP]) {
    if constexpr (VP == 8) {
        load8(p, f);
    } else if constexpr (VP == 4) {
        const uint2 u = *reinterpret_cast<const uint2*>(p);
        const float2 x = dt_traits<T>::unpack2(u.x), y = dt_traits<T>::unpack2(u.y);
        f[0] = x.x;
        f[1] = x.y;
        f[2] = y.x;
        f[3] = y.y;
    } else {
        f[0] = dt_traits<T>::to_f(p[0]);
    }
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

// Unit u of a head: where its two pieces lie, and whether it is turned.
template <int VP>
struct Unit {
    int a, b;
    bool turned;
    __device__ __forceinline__ Unit(int u, int pairs, int interleaved) {
        turned = u * VP < pairs;
        if (interleaved || !turned) {
            a = 2 * u * VP;  // (behind the span: 2 pairs + 2 VP (u - pairs / VP))
            b = a + VP;
        } else {
            a = u * VP;
            b = pairs + a;
        }
    }
};

// Cosines and sines of a unit's pairs at a position, times the amplitude.
template <int VP>
struct Angles {
    float c[VP], s[VP];
    __device__ __forceinline__ void set(const uint64_t (&turns)[VP], int pos, float amplitude,
                                        float sign) {
#pragma unroll
        for (int i = 0; i < VP; ++i) {
            const uint64_t t = turns[i] * static_cast<uint64_t>(static_cast<int64_t>(pos));
            // half turns in [-1, 1], to radians
            const float x = static_cast<float>(static_cast<int32_t>((t + 0x80000000ull) >> 32)) *
                            (3.14159265358979f / 2147483648.0f);
            float sn, cs;
            __sincosf(x, &sn, &cs);
            c[i] = cs * amplitude;
            s[i] = sn * sign;  // sign: +- amplitude
        }
    }
    __device__ __forceinline__ void turn(float (&a)[VP], float (&b)[VP], int interleaved) const {
        if (VP > 1 && interleaved) {
#pragma unroll
            for (int i = 0; i < VP / 2; ++i) {
                pair(a[2 * i], a[2 * i + 1], i);
                pair(b[2 * i], b[2 * i + 1], VP / 2 + i);
            }
        } else {
#pragma unroll
            for (int i = 0; i < VP; ++i) pair(a[i], b[i], i);
        }
    }

private:
    __device__ __forceinline__ void pair(float& x, float& y, int i) const {
        const float x0 = x;
        x = fmaf(x0, c[i], -(y * s[i]));
        y = fmaf(y, c[i], x0 * s[i]);
    }
};

// The widest pieces that a span and a head allow.
inline int turn_width(int pairs) { return pairs % 8 == 0 ? 8 : pairs % 4 == 0 ? 4 : 1; }

// blk_rope_plan_init fills `check` with this: a call refuses a plan that it did not make.
constexpr int32_t kPlanMade = 0x524f5045;
inline bool plan_made(const blk_rope_plan* p, int64_t head_dim) {
    return p->check == kPlanMade && p->pairs >= 1 && p->pairs <= 128 && 2 * p->pairs <= head_dim &&
           (p->interleaved == 0 || p->interleaved == 1);
}

}  // namespace blk
