// gfx950 kernels of the router, and their C entry points: scores of every
// expert -> the top_k experts of each token and their weights (the inputs of
// ep_layout), and the gradient of the logits from that of the weights.
//
// One wave a token, four tokens a workgroup; lane l holds experts l, l + 64,
// ... of the row, so every load of the row is contiguous over the wave.  The
// choice takes top_k rounds; a round is a maximum over the wave of one key a
// lane (its best expert left), by data-parallel-primitive moves without LDS.
// Keys order as the scores do and never tie: the expert's number breaks ties,
// the lowest first.  The whole row stays in registers, so the kernel reads it
// once; at these sizes (a few MB) it is bound by the rounds' latency.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ep_layout.h"
#include "ep_ranges.h"
#include "ep_route_device.h"

namespace epk {
namespace {

constexpr int kRouteWaves = 4;              // tokens of a workgroup
// From here on four tokens a wave: 16384 tokens of 256 experts, top 8, take 9.7
// us so and 12.4 with a wave a token, 8192 take 6.5 and 7.5, 4096 take 5.7 and 5.2.
constexpr int kRowsTokens = 8192;

template <int N, bool BIASED>
__global__ void __launch_bounds__(kRouteWaves * kWave)
route_kernel(RouteArgs a) {
    const int lane = threadIdx.x & (kWave - 1);
    const int t = blockIdx.x * kRouteWaves + __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    if (t >= a.T) return;
    int mine;
    float weight;
    route_token<N, BIASED>(a, t, lane, mine, weight);
    if (lane < a.K) {
        a.idx[(int64_t)t * a.K + lane] = mine;
        a.weights[(int64_t)t * a.K + lane] = weight;
    }
}

// The same for many tokens, four a wave: 16 lanes hold a token's experts, N
// each, so that a round's maximum costs four moves for four tokens instead of
// six for one (the instructions of the rounds bound the kernel then).
template <int N>
__global__ void __launch_bounds__(kRouteWaves * kWave)
route_rows_kernel(RouteArgs a) {
    constexpr int L = Row::kLanes;
    const int sub = threadIdx.x & (L - 1);
    const int t = (int)(blockIdx.x * (kRouteWaves * kWave / L) + threadIdx.x / L);
    const bool real = t < a.T;              // lanes past the last token stay for the moves
    uint32_t key[N];
    float top = 0.0f, sum = 1.0f;
    {
        float l[N];
        load_row<L>(a, t, sub, real, l);
#pragma unroll
        for (int i = 0; i < N; ++i) key[i] = l[i] > -__builtin_inff() ? ordered(l[i]) : 0u;
        if (!a.sigmoid && !a.normalize) row_softmax<Row>(l, top, sum);
    }
    int mine = -1;              // lane k of a row: the k-th chosen expert and its logit
    float mine_l = 0.0f;
    for (int k = 0; k < a.K; ++k) {
        uint32_t best = 0;
#pragma unroll
        for (int i = 0; i < N; ++i) best = key[i] > best ? key[i] : best;
        const uint32_t win = row_max(best);
        // the lowest expert that has this key
        int slot = N;
#pragma unroll
        for (int i = N - 1; i >= 0; --i) slot = key[i] == win ? i : slot;
        const uint32_t last = row_max(slot < N ? 0xFFFFu - (uint32_t)(slot * L + sub) : 0u);
        const int e = 0xFFFF - (int)last;
        const int clear = (e & (L - 1)) == sub ? e / L : N;
#pragma unroll
        for (int i = 0; i < N; ++i) key[i] = i == clear ? 0u : key[i];
        if (sub == k && win != 0) {         // 0: no expert is left
            mine = e;
            mine_l = unordered(win);
        }
    }
    const float w = chosen_weight<Row>(a, mine >= 0, mine_l, top, sum);
    if (real && sub < a.K) {
        a.idx[(int64_t)t * a.K + sub] = mine;
        a.weights[(int64_t)t * a.K + sub] = mine >= 0 ? a.scale * w : 0.0f;
    }
}

// Gradient of the logits.  With q the weights before the scale, w = scale q:
//   normalised        dl_i = scale q_i (gw_i - sum_j q_j gw_j), times 1 - s_i
//                     with sigmoid scores; zero for experts not chosen
//   softmax, whole    dl_e = p_e (scale gw_e [e chosen] - scale sum_j q_j gw_j)
//   sigmoid, whole    dl_i = scale gw_i s_i (1 - s_i)
template <int N>
__global__ void __launch_bounds__(kRouteWaves * kWave)
route_backward_kernel(RouteArgs a) {
    const int lane = threadIdx.x & (kWave - 1);
    const int t = blockIdx.x * kRouteWaves + __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    if (t >= a.T) return;
    int mine = lane < a.K ? a.chosen[(int64_t)t * a.K + lane] : -1;
    if (mine < -1 || mine >= a.E) mine = -1;
    const float gw = mine >= 0 ? a.grad_weights[(int64_t)t * a.K + lane] * a.scale : 0.0f;
    const float l = mine >= 0 ? load_logit(a, t * a.ld + mine) : 0.0f;
    const bool on = mine >= 0 && l > -__builtin_inff();
    const bool whole = !a.sigmoid && !a.normalize;
    float row[N], top = 0.0f, sum = 1.0f;
    if (whole) {
        load_row<kWave>(a, t, lane, true, row);
        row_softmax<Wave>(row, top, sum);
    }
    const float q = chosen_weight<Wave>(a, on, l, top, sum);
    const float g = on ? gw : 0.0f;
    const float dot = wave_sum(q * g);
    float d;
    if (a.normalize) d = q * (g - dot) * (a.sigmoid ? sigmoid(-l) : 1.0f);
    else d = a.sigmoid ? g * q * sigmoid(-l) : q * g;
    if (!on) d = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i)
        row[i] = whole && row[i] > -__builtin_inff() ? -dot * (expf(row[i] - top) / sum) : 0.0f;
    // the chosen experts' own terms, in slot order
    for (int k = 0; k < a.K; ++k) {
        const int e = __builtin_amdgcn_readlane(mine, k);
        if (e < 0) continue;
        const float v = __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(d), k));
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (e == i * kWave + lane) row[i] += v;
    }
    const int64_t at = t * a.grad_ld + lane;
    if (a.bf16) {
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (i * kWave + lane < a.E) ((__bf16*)a.grad_logits)[at + i * kWave] = (__bf16)row[i];
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (i * kWave + lane < a.E) ((float*)a.grad_logits)[at + i * kWave] = row[i];
    }
}

template <int N>
void launch_n(const RouteArgs& a, bool backward, hipStream_t stream) {
    const int grid = (a.T + kRouteWaves - 1) / kRouteWaves, threads = kRouteWaves * kWave;
    if (backward) route_backward_kernel<N><<<grid, threads, 0, stream>>>(a);
    else if (a.bias) route_kernel<N, true><<<grid, threads, 0, stream>>>(a);
    else route_kernel<N, false><<<grid, threads, 0, stream>>>(a);
}

template <int N>
void launch_rows(const RouteArgs& a, hipStream_t stream) {
    constexpr int kTokens = kRouteWaves * kWave / Row::kLanes;
    route_rows_kernel<N><<<(a.T + kTokens - 1) / kTokens, kRouteWaves * kWave, 0, stream>>>(a);
}

hipError_t launch(const RouteArgs& a, bool backward, hipStream_t stream) {
    if (!backward && !a.bias && a.T >= kRowsTokens && a.K <= Row::kLanes && a.E <= 256) {
        if (a.E <= 64) launch_rows<4>(a, stream);
        else if (a.E <= 128) launch_rows<8>(a, stream);
        else launch_rows<16>(a, stream);
        return hipGetLastError();
    }
    if (a.E <= 64) launch_n<1>(a, backward, stream);
    else if (a.E <= 128) launch_n<2>(a, backward, stream);
    else if (a.E <= 256) launch_n<4>(a, backward, stream);
    else if (a.E <= 512) launch_n<8>(a, backward, stream);
    else launch_n<16>(a, backward, stream);
    return hipGetLastError();
}

constexpr uint32_t kRouteFlags = EP_ROUTE_BF16 | EP_ROUTE_SIGMOID | EP_ROUTE_NORMALIZE;

}  // namespace

ep_status check_route(const void* logits, int64_t ld, int32_t T, int32_t E, int32_t K, uint32_t flags,
                      float scale, RouteArgs& a) {
    if (flags & ~kRouteFlags) return EP_ERR_INVALID_ARGUMENT;
    if (T < 0 || E < 1 || K < 1 || K > E || ld < E || scale != scale) return EP_ERR_INVALID_ARGUMENT;
    if (E > kRouteMaxExperts || K > kRouteMaxTopK || T > kRouteMaxTokens) return EP_ERR_UNSUPPORTED;
    if (T > 0 && (!logits || !aligned(logits, (flags & EP_ROUTE_BF16) ? 2 : 4))) return EP_ERR_INVALID_ARGUMENT;
    a.logits = logits;
    a.ld = ld;
    a.T = T;
    a.E = E;
    a.K = K;
    a.bf16 = (flags & EP_ROUTE_BF16) ? 1 : 0;
    a.sigmoid = (flags & EP_ROUTE_SIGMOID) ? 1 : 0;
    a.normalize = (flags & EP_ROUTE_NORMALIZE) ? 1 : 0;
    a.scale = scale;
    return EP_OK;
}

hipError_t launch_route(const RouteArgs& a, hipStream_t stream) { return launch(a, false, stream); }

}  // namespace epk

extern "C" {

ep_status ep_route(const void* logits, int64_t logits_ld, int32_t num_tokens, int32_t num_experts, int32_t top_k,
                   uint32_t flags, const float* bias, float scale, int32_t* topk_idx, float* topk_weights,
                   hipStream_t stream) {
    epk::RouteArgs a{};
    const ep_status st = epk::check_route(logits, logits_ld, num_tokens, num_experts, top_k, flags, scale, a);
    if (st != EP_OK) return st;
    // the order of softmax scores is that of the logits: a bias is for sigmoid scores
    if (bias && !a.sigmoid) return EP_ERR_UNSUPPORTED;
    if (num_tokens == 0) return EP_OK;
    if (!topk_idx || !topk_weights || !epk::aligned(topk_idx, 4) || !epk::aligned(topk_weights, 4) ||
        !epk::aligned(bias, 4))
        return EP_ERR_INVALID_ARGUMENT;
    const epk::Rows in(logits, logits_ld, num_experts, num_tokens, a.bf16 ? 2 : 4), idx(topk_idx, top_k, top_k, num_tokens, 4),
        weights(topk_weights, top_k, top_k, num_tokens, 4), biases(bias, num_experts, num_experts, 1, 4);
    if (epk::share(idx, in) || epk::share(weights, in) || epk::share(idx, weights) ||
        (bias && (epk::share(idx, biases) || epk::share(weights, biases))))
        return EP_ERR_INVALID_ARGUMENT;
    a.bias = bias;
    a.idx = topk_idx;
    a.weights = topk_weights;
    return epk::launch(a, false, stream) == hipSuccess ? EP_OK : EP_ERR_HIP;
}

ep_status ep_route_backward(const void* logits, int64_t logits_ld, int32_t num_tokens, int32_t num_experts,
                            int32_t top_k, uint32_t flags, float scale, const int32_t* topk_idx,
                            const float* grad_weights, void* grad_logits, int64_t grad_ld, hipStream_t stream) {
    epk::RouteArgs a{};
    const ep_status st = epk::check_route(logits, logits_ld, num_tokens, num_experts, top_k, flags, scale, a);
    if (st != EP_OK) return st;
    if (grad_ld < num_experts) return EP_ERR_INVALID_ARGUMENT;
    if (num_tokens == 0) return EP_OK;
    if (!topk_idx || !grad_weights || !grad_logits || !epk::aligned(topk_idx, 4) ||
        !epk::aligned(grad_weights, 4) || !epk::aligned(grad_logits, a.bf16 ? 2 : 4))
        return EP_ERR_INVALID_ARGUMENT;
    const epk::Rows out(grad_logits, grad_ld, num_experts, num_tokens, a.bf16 ? 2 : 4);
    if (epk::share(out, epk::Rows(logits, logits_ld, num_experts, num_tokens, a.bf16 ? 2 : 4)) ||
        epk::share(out, epk::Rows(topk_idx, top_k, top_k, num_tokens, 4)) ||
        epk::share(out, epk::Rows(grad_weights, top_k, top_k, num_tokens, 4)))
        return EP_ERR_INVALID_ARGUMENT;
    a.chosen = topk_idx;
    a.grad_weights = grad_weights;
    a.grad_logits = grad_logits;
    a.grad_ld = grad_ld;
    return epk::launch(a, true, stream) == hipSuccess ? EP_OK : EP_ERR_HIP;
}

}  // extern "C"
