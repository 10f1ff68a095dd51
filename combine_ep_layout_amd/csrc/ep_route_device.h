// The router on the device: what ep_route.hip's kernels and the layer for a few
// tokens (ep_tokens.hip) share.  Not installed; callers use include/ep_layout.h.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ep_layout.h"
#include "ep_wave.h"

namespace epk {

struct RouteArgs {
    const void* logits;         // [T, ld] fp32 or bf16
    int64_t ld;
    int32_t T;
    int32_t E;
    int32_t K;
    int32_t bf16;
    int32_t sigmoid;
    int32_t normalize;
    float scale;
    const float* bias;          // [E] or null
    int32_t* idx;               // [T, K]
    float* weights;             // [T, K]
    const int32_t* chosen;      // backward
    const float* grad_weights;
    void* grad_logits;          // [T, grad_ld], the logits' type
    int64_t grad_ld;
};

// Checks what every call on logits shares; fills what they need.
ep_status check_route(const void* logits, int64_t ld, int32_t T, int32_t E, int32_t K, uint32_t flags, float scale,
                      RouteArgs& a);
hipError_t launch_route(const RouteArgs& a, hipStream_t stream);

namespace {

constexpr int kRouteMaxExperts = 1024;
constexpr int kRouteMaxTopK = 32;
constexpr int kRouteMaxTokens = 1 << 25;    // a wave each: the grid stays below 2^32 threads


// NaN closes the expert as -inf does; +inf is the largest finite logit.
__device__ __forceinline__ float clean(float v) {
    return v != v ? -__builtin_inff() : fminf(v, 3.402823466e38f);
}
__device__ __forceinline__ float load_logit(const RouteArgs& a, int64_t at) {
    return clean(a.bf16 ? __uint_as_float((uint32_t)((const uint16_t*)a.logits)[at] << 16) : ((const float*)a.logits)[at]);
}

// A lane's logits of token t: experts `lane`, lane + LANES, ...; -inf past the
// last.  The type is asked for once, or every load would wait for the last.
template <int LANES, int N>
__device__ __forceinline__ void load_row(const RouteArgs& a, int t, int lane, bool real, float (&l)[N]) {
    const int64_t at = t * a.ld + lane;
    if (a.bf16) {
        uint32_t v[N];
#pragma unroll
        for (int i = 0; i < N; ++i)
            v[i] = real && i * LANES + lane < a.E ? ((const uint16_t*)a.logits)[at + i * LANES] : 0xFF80u;
#pragma unroll
        for (int i = 0; i < N; ++i) l[i] = clean(__uint_as_float(v[i] << 16));
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
            l[i] = real && i * LANES + lane < a.E ? ((const float*)a.logits)[at + i * LANES] : -__builtin_inff();
#pragma unroll
        for (int i = 0; i < N; ++i) l[i] = clean(l[i]);
    }
}

// Unsigned integers in the order of the floating-point values; -0 and +0 are
// one value.
__device__ __forceinline__ uint32_t ordered(float v) {
    const uint32_t b = __float_as_uint(v + 0.0f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ uint64_t ordered(double v) {
    const uint64_t b = (uint64_t)__double_as_longlong(v + 0.0);
    return b >> 63 ? ~b : b | 0x8000000000000000ull;
}

__device__ __forceinline__ float unordered(uint32_t k) {
    return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}

template <int CTRL>
__device__ __forceinline__ uint32_t dpp_u32(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, true);
}
// Moves of a wave-wide reduction: within rows of 16 lanes, then across rows;
// lanes without a source get 0, and the last lane ends with the result.
template <int CTRL>
__device__ __forceinline__ uint32_t max_step(uint32_t v) {
    const uint32_t o = dpp_u32<CTRL>(v);
    return o > v ? o : v;
}
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
    v = max_step<0x111>(v);         // row_shr:1, 2, 4, 8
    v = max_step<0x112>(v);
    v = max_step<0x114>(v);
    v = max_step<0x118>(v);
    v = max_step<0x142>(v);         // row_bcast:15, 31
    v = max_step<0x143>(v);
    return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}
// The same moves for a sum (lanes without a source add 0, and always in the
// same order) and for a maximum of floats above -inf.
template <int CTRL, int ROWS = 0xF>
__device__ __forceinline__ float dpp_f32(float v) {
    return __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v), CTRL, ROWS, 0xF, true));
}
__device__ __forceinline__ float last_lane(float v) {
    return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(v), 63));
}
__device__ __forceinline__ float wave_sum(float v) {
    v += dpp_f32<0x111>(v);
    v += dpp_f32<0x112>(v);
    v += dpp_f32<0x114>(v);
    v += dpp_f32<0x118>(v);
    v += dpp_f32<0x142, 0xA>(v);        // into rows 1 and 3
    v += dpp_f32<0x143, 0xC>(v);        // into rows 2 and 3
    return last_lane(v);
}
// The same over a row of 16 lanes, each of which gets the result (rotations).
__device__ __forceinline__ uint32_t row_max(uint32_t v) {
    v = max_step<0x128>(v);         // row_ror:8, 4, 2, 1
    v = max_step<0x124>(v);
    v = max_step<0x122>(v);
    return max_step<0x121>(v);
}
__device__ __forceinline__ float row_sum(float v) {
    v += dpp_f32<0x128>(v);
    v += dpp_f32<0x124>(v);
    v += dpp_f32<0x122>(v);
    return v + dpp_f32<0x121>(v);
}

// The lanes that share a token.
struct Wave {
    static constexpr int kLanes = 64;
    __device__ static uint32_t max(uint32_t v) { return wave_max(v); }
    __device__ static float sum(float v) { return wave_sum(v); }
};
struct Row {
    static constexpr int kLanes = 16;
    __device__ static uint32_t max(uint32_t v) { return row_max(v); }
    __device__ static float sum(float v) { return row_sum(v); }
};
template <class L>
__device__ __forceinline__ float max_f32(float v) { return unordered(L::max(ordered(v))); }

__device__ __forceinline__ float sigmoid(float x) { return 1.0f / (1.0f + expf(-x)); }

// Weights of the chosen experts, one a lane (lanes below K with an open
// expert; `on`), before the scale.
//   l: the lane's chosen logit; top, sum: maximum of the row's open logits and
//   sum of exp(l - top) over them (softmax without normalising only).
template <class L>
__device__ __forceinline__ float chosen_weight(const RouteArgs& a, bool on, float l, float top, float sum) {
    if (!a.sigmoid && !a.normalize) return on ? expf(l - top) / sum : 0.0f;
    const float s = a.sigmoid && on ? sigmoid(l) : 0.0f;
    if (!a.normalize) return s;
    const float m = max_f32<L>(on ? l : -__builtin_inff());
    const float e = on ? expf(l - m) : 0.0f;
    const float total = L::sum(a.sigmoid ? s : e), ratio = L::sum(e);
    // far below zero the sigmoid is exp(l), and only its ratios are left
    if (a.sigmoid && total > 0x1p-60f) return s / total;
    return on ? e / ratio : 0.0f;
}

// Maximum and sum of exp over the row's open experts.
template <class L, int N>
__device__ __forceinline__ void row_softmax(const float (&l)[N], float& top, float& sum) {
    top = -__builtin_inff();
#pragma unroll
    for (int i = 0; i < N; ++i) top = fmaxf(top, l[i]);
    top = max_f32<L>(top);
    sum = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) sum += l[i] > -__builtin_inff() ? expf(l[i] - top) : 0.0f;
    sum = L::sum(sum);
}

// One token's choice by a wave: lane k < K gets the k-th chosen expert (-1: none
// is left) and its weight after the scale.
// N: experts of a lane.  BIASED: ordered by sigmoid(logit) + bias in double,
// where two scores next to each other need more than fp32 holds; otherwise by
// the logits themselves, which the scores follow exactly.
template <int N, bool BIASED>
__device__ __forceinline__ void route_token(const RouteArgs& a, int t, int lane, int& mine, float& weight) {
    float l[N];
    uint32_t hi[N], lo[BIASED ? N : 1];         // keys; 0: closed or taken
    load_row<kWave>(a, t, lane, true, l);
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const bool open = l[i] > -__builtin_inff();
        if constexpr (BIASED) {
            const int e = i * kWave + lane;
            const double s = 1.0 / (1.0 + exp(-(double)l[i])) + (double)(e < a.E ? a.bias[e] : 0.0f);
            // a bias of -inf or NaN closes the expert
            const uint64_t k = open && s > -__builtin_inf() ? ordered(s) : 0;
            hi[i] = (uint32_t)(k >> 32);
            lo[i] = (uint32_t)k;
        } else {
            hi[i] = open ? ordered(l[i]) : 0u;
        }
    }
    float top = 0.0f, sum = 1.0f;
    if (!a.sigmoid && !a.normalize) row_softmax<Wave>(l, top, sum);

    mine = -1;
    float mine_l = 0.0f;        // lane k: the k-th chosen logit
    for (int k = 0; k < a.K; ++k) {
        // the lane's best expert left: its key, slot and (BIASED) logit
        uint32_t best = 0, best_lo = 0;
        int slot = 0;
        float best_l = 0.0f;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            bool more = hi[i] > best;
            if constexpr (BIASED) more = more || (hi[i] == best && lo[i] > best_lo);
            best = more ? hi[i] : best;
            slot = more ? i : slot;
            if constexpr (BIASED) {
                best_lo = more ? lo[i] : best_lo;
                best_l = more ? l[i] : best_l;
            }
        }
        const uint32_t win = wave_max(best);
        if (win == 0) break;                    // no expert is left
        bool is = best == win;
        if constexpr (BIASED) {
            const uint32_t win_lo = wave_max(is ? best_lo : 0u);        // every lane takes part
            is = is && best_lo == win_lo;
        }
        // the lowest expert of those that have the key; mostly there is one
        const uint64_t who = __ballot(is);
        int e;
        if ((who & (who - 1)) == 0) {
            const int owner = __builtin_ctzll(who);
            e = __builtin_amdgcn_readlane(slot, owner) * kWave + owner;
        } else {
            e = 0xFFFF - (int)wave_max(is ? 0xFFFFu - (uint32_t)(slot * kWave + lane) : 0u);
        }
        float le = unordered(win);
        if constexpr (BIASED)
            le = __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(best_l), e & (kWave - 1)));
        const bool owner = lane == (e & (kWave - 1));
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const bool taken = owner && i == slot;
            hi[i] = taken ? 0u : hi[i];
            if constexpr (BIASED) lo[i] = taken ? 0u : lo[i];
        }
        if (lane == k) {
            mine = e;
            mine_l = le;
        }
    }
    const float w = chosen_weight<Wave>(a, mine >= 0, mine_l, top, sum);
    weight = mine >= 0 ? a.scale * w : 0.0f;
}

}  // namespace
}  // namespace epk
