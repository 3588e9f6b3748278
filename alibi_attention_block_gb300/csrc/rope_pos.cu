// K4p: rotary at given positions, on packed queries and keys (blk_rope_positions),
// and the plan that it and the paged cache's append take (blk_rope_plan_init).
//
//   (x_i, x_j) -> m (x_i cos a - x_j sin a, x_j cos a + x_i sin a), a = position * theta'
//
// The rotary of nnterp "stablelm" 03 Notes at positions from device memory;
// angles and units: turn.cuh. Bound by bytes: each element is read and written
// once (in place, the turned part only). A block takes a run of tokens and a
// group of heads: a thread keeps its unit's angles in registers over the
// group, so that a sine and cosine serve several heads. 16384 tokens of 32 + 8 x 128 heads:
// 54 us (6.2 TB/s, 0.91 of the copy rate); 24 tokens 2.2 us.
#include <cmath>
#include <cstring>

#include "turn.cuh"

namespace blk {

namespace {

constexpr int kThreads = 128;

struct RopePosArgs {
    TurnArgs turn;
    const void* x[2];  // q, k
    void* y[2];
    int64_t xs[2][2], ys[2][2];  // strides of heads and tokens, in elements
    const int32_t* positions;
    int tokens, heads[2], d;
    int per;      // heads per block
    int in_place[2];
    int pdl;
};

template <typename T, int VP>
__global__ void __launch_bounds__(kThreads) rope_pos_kernel(const __grid_constant__ RopePosArgs a) {
    const int units = a.d / (2 * VP);
    const int rows = kThreads / units;  // tokens of a block
    const int u = threadIdx.x % units;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * rows + threadIdx.x / units;
    if (threadIdx.x >= rows * units || t >= a.tokens) return;
    const Unit<VP> at(u, a.d, a.turn.plan.pairs, a.turn.plan.interleaved);
    uint64_t turns[VP];
#pragma unroll
    for (int i = 0; i < VP; ++i)
        turns[i] = !at.turned                 ? 0
                   : VP == 1 || i < VP / 2 ? a.turn.plan.turns[at.p0 + i]
                                              : a.turn.plan.turns[at.p1 + i - VP / 2];
    if (a.pdl) pdl_wait();
    Angles<VP> ang;
    if (at.turned) {
        const float m = a.turn.plan.amplitude;
        ang.set(turns, a.positions[t], m, a.turn.inverse ? -m : m);
    }
    const int h0 = blockIdx.y * a.per, h1 = min(h0 + a.per, a.heads[0] + a.heads[1]);
#pragma unroll 4
    for (int h = h0; h < h1; ++h) {
        const int w = h >= a.heads[0];
        if (!at.turned && a.in_place[w]) continue;
        const int64_t n = w ? h - a.heads[0] : h;
        const T* x = static_cast<const T*>(a.x[w]) + n * a.xs[w][0] + t * a.xs[w][1];
        T* y = static_cast<T*>(a.y[w]) + n * a.ys[w][0] + t * a.ys[w][1];
        float p[VP], q[VP];
        load_piece(x + at.a, p);
        load_piece(x + at.b, q);
        if (at.turned) ang.turn(p, q, a.turn.plan.interleaved);
        store_piece(y + at.a, p);
        store_piece(y + at.b, q);
    }
}

template <typename T>
cudaError_t launch_rope_pos(const RopePosArgs& a, dim3 grid, int vp, cudaStream_t s) {
    switch (vp) {
        case 8: return launch_pdl(a.pdl != 0, rope_pos_kernel<T, 8>, grid, dim3(kThreads), 0, s, a);
        case 4: return launch_pdl(a.pdl != 0, rope_pos_kernel<T, 4>, grid, dim3(kThreads), 0, s, a);
        default: return launch_pdl(a.pdl != 0, rope_pos_kernel<T, 1>, grid, dim3(kThreads), 0, s, a);
    }
}

#define REQUIRE(cond, ...)                                                      \
    do {                                                                        \
        if (!(cond)) return report_error_status(BLK_EINVAL, __VA_ARGS__);       \
    } while (0)

}  // namespace

}  // namespace blk

using namespace blk;

extern "C" {

blk_status blk_rope_plan_init(const blk_rope_desc* d, blk_rope_plan* plan) {
    REQUIRE(d && plan, "desc or plan is NULL");
    REQUIRE(d->span >= 2 && d->span % 2 == 0 && d->span <= 256, "span must be even and in [2, 256]");
    REQUIRE(std::isfinite(d->base) && d->base >= 1.0, "base must be finite and >= 1");
    REQUIRE(d->interleaved == 0 || d->interleaved == 1, "interleaved must be 0 or 1");
    REQUIRE(d->scaling >= BLK_ROPE_PLAIN && d->scaling <= BLK_ROPE_BY_PARTS, "unknown scaling");
    REQUIRE(std::isfinite(d->amplitude) && d->amplitude > 0.f, "amplitude must be finite and > 0");
    const bool scaled = d->scaling != BLK_ROPE_PLAIN;
    REQUIRE(!scaled || (std::isfinite(d->factor) && d->factor >= 1.0), "factor must be finite and >= 1");
    if (d->scaling == BLK_ROPE_BY_PARTS)
        REQUIRE(std::isfinite(d->original_len) && d->original_len > 0.0 && std::isfinite(d->beta_slow) &&
                    std::isfinite(d->beta_fast) && d->beta_fast > d->beta_slow,
                "by parts: original_len must be > 0 and beta_fast > beta_slow");
    std::memset(plan, 0, sizeof(*plan));
    const double two_pi = 6.283185307179586476925286766559;
    for (int j = 0; j < d->span / 2; ++j) {
        double theta = std::pow(d->base, -2.0 * j / d->span);
        if (d->scaling == BLK_ROPE_LINEAR) theta /= d->factor;
        if (d->scaling == BLK_ROPE_BY_PARTS) {
            const double turns = d->original_len * theta / two_pi;
            double keep = (turns - d->beta_slow) / (d->beta_fast - d->beta_slow);
            keep = keep < 0.0 ? 0.0 : keep > 1.0 ? 1.0 : keep;
            theta = keep * theta + (1.0 - keep) * theta / d->factor;
        }
        plan->turns[j] = static_cast<uint64_t>(std::ldexp(theta / two_pi, 64) + 0.5);
    }
    plan->pairs = d->span / 2;
    plan->interleaved = d->interleaved;
    plan->amplitude = d->amplitude;
    plan->check = kPlanMade;
    return BLK_OK;
}

blk_status blk_rope_positions(const blk_rope_pos_desc* d, const blk_rope_plan* plan, const void* q,
                              const void* k, const int32_t* positions, void* q_out, void* k_out,
                              blk_dtype dt, blk_stream_t s) {
    REQUIRE(dt == BLK_F16 || dt == BLK_BF16, "dtype must be BLK_F16 or BLK_BF16");
    REQUIRE(d, "desc is NULL");
    REQUIRE(plan, "plan is NULL");
    REQUIRE(d->tokens >= 1 && d->tokens <= (int64_t(1) << 30), "tokens out of range");
    REQUIRE(d->head_dim >= 16 && d->head_dim % 16 == 0 && d->head_dim <= 256,
            "head_dim must be a multiple of 16 in [16, 256]");
    REQUIRE(plan_made(plan, d->head_dim), "plan was not made by blk_rope_plan_init, or its span is above head_dim");
    REQUIRE(d->n_heads >= 1 && d->n_heads <= 16384, "n_heads out of range");
    REQUIRE(d->n_k_heads >= 0 && d->n_k_heads <= 16384 && (d->n_k_heads > 0) == (k != nullptr) &&
                (k != nullptr) == (k_out != nullptr),
            "k, k_out and n_k_heads go together");
    REQUIRE(d->inverse == 0 || d->inverse == 1, "inverse must be 0 or 1");
    REQUIRE(q && q_out, "q or q_out is NULL");
    REQUIRE(positions && (reinterpret_cast<uintptr_t>(positions) & 3u) == 0,
            "positions must be a 4-byte aligned device pointer");
    const void* ptrs[4] = {q, q_out, k, k_out};
    const int64_t strides[4][2] = {{d->q_head_stride, d->q_token_stride},
                                   {d->q_out_head_stride, d->q_out_token_stride},
                                   {d->k_head_stride, d->k_token_stride},
                                   {d->k_out_head_stride, d->k_out_token_stride}};
    for (int i = 0; i < (k ? 4 : 2); ++i) {
        REQUIRE((reinterpret_cast<uintptr_t>(ptrs[i]) & 15u) == 0, "tensors must be 16-byte aligned");
        for (int j = 0; j < 2; ++j)
            REQUIRE(strides[i][j] >= 0 && strides[i][j] % 8 == 0 && strides[i][j] <= (int64_t(1) << 40),
                    "strides must be multiples of 8 elements");
    }
    REQUIRE(places_apart(d->n_heads, d->tokens, d->q_out_head_stride, d->q_out_token_stride, d->head_dim) &&
                (!k || places_apart(d->n_k_heads, d->tokens, d->k_out_head_stride, d->k_out_token_stride, d->head_dim)),
            "an output's strides make it overlap itself");
    RopePosArgs a{};
    a.turn.plan = *plan;
    a.turn.inverse = d->inverse;
    for (int w = 0; w < 2; ++w) {
        a.x[w] = ptrs[2 * w];
        a.y[w] = const_cast<void*>(ptrs[2 * w + 1]);
        for (int j = 0; j < 2; ++j) {
            a.xs[w][j] = strides[2 * w][j];
            a.ys[w][j] = strides[2 * w + 1][j];
        }
        a.in_place[w] = a.x[w] == a.y[w];
        REQUIRE(!a.in_place[w] || !a.x[w] || (a.xs[w][0] == a.ys[w][0] && a.xs[w][1] == a.ys[w][1]),
                "an output in place has the input's strides");
    }
    a.positions = positions;
    a.tokens = static_cast<int>(d->tokens);
    a.heads[0] = static_cast<int>(d->n_heads);
    a.heads[1] = static_cast<int>(d->n_k_heads);
    a.d = static_cast<int>(d->head_dim);
    int sms = 0;
    unsigned* err = nullptr;
    const blk_status st = current_device_info(&sms, &err);
    if (st != BLK_OK) return st;
    const cudaStream_t cs = reinterpret_cast<cudaStream_t>(s);
    a.pdl = pdl_allowed(cs);
    const int vp = turn_width(plan->pairs);
    const int64_t rows = kThreads / (a.d / (2 * vp));
    const int64_t tiles = (d->tokens + rows - 1) / rows, heads = d->n_heads + d->n_k_heads;
    // heads per block: so many that there are about 32 blocks per SM, in whole fours, a thread's
    // loads in flight (4093 tokens of 32 + 32 x 64: one each 20.0 us, four 14.3; 16000 of 32 + 8 x
    // 160: forty 84, eight to twelve 72); one where tokens are few
    int64_t per = (tiles * heads / (32 * sms) + 3) / 4 * 4;
    if (tiles * heads >= 4 * sms) per = per < 4 ? 4 : per;
    per = per < 1 ? 1 : per > heads ? heads : per;
    a.per = static_cast<int>(per);
    const dim3 grid(static_cast<unsigned>(tiles), static_cast<unsigned>((heads + per - 1) / per));
    const cudaError_t e = dt == BLK_F16 ? launch_rope_pos<__half>(a, grid, vp, cs)
                                        : launch_rope_pos<__nv_bfloat16>(a, grid, vp, cs);
    return e == cudaSuccess ? BLK_OK
                            : report_error_status(BLK_ECUDA, "rope launch: %s", cudaGetErrorString(e));
}

}  // extern "C"
