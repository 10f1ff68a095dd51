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

namespace epk {
namespace {

constexpr int kWave = 64;
constexpr int kRouteWaves = 4;              // tokens of a workgroup
// From here on four tokens a wave: 16384 tokens of 256 experts, top 8, take 9.7
// us so and 12.4 with a wave a token, 8192 take 6.5 and 7.5, 4096 take 5.7 and 5.2.
constexpr int kRowsTokens = 8192;
constexpr int kRouteMaxExperts = 1024;
constexpr int kRouteMaxTopK = 32;
constexpr int kRouteMaxTokens = 1 << 25;    // a wave each: the grid stays below 2^32 threads

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

// N: experts of a lane.  BIASED: ordered by sigmoid(logit) + bias in double,
// where two scores next to each other need more than fp32 holds; otherwise by
// the logits themselves, which the scores follow exactly.
template <int N, bool BIASED>
__global__ void __launch_bounds__(kRouteWaves * kWave)
route_kernel(RouteArgs a) {
    const int lane = threadIdx.x & (kWave - 1);
    const int t = blockIdx.x * kRouteWaves + __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    if (t >= a.T) return;
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

    int mine = -1;              // lane k: the k-th chosen expert and its logit
    float mine_l = 0.0f;
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
    if (lane < a.K) {
        a.idx[(int64_t)t * a.K + lane] = mine;
        a.weights[(int64_t)t * a.K + lane] = mine >= 0 ? a.scale * w : 0.0f;
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

bool aligned(const void* p, int n) { return ((uintptr_t)p & (uintptr_t)(n - 1)) == 0; }

// n rows of `width` bytes, `ld` bytes apart.
struct Rows {
    uintptr_t at;
    __int128 ld, width, n;
    Rows(const void* p, int64_t ld_, int64_t width_, int64_t n_, int size)
        : at((uintptr_t)p), ld((__int128)ld_ * size), width((__int128)width_ * size), n(n_) {
        if (n == 1 || ld == width) {            // one piece
            width *= n;
            ld = width;
            n = 1;
        }
    }
    __int128 row(__int128 i) const { return (__int128)at + i * ld; }
    // whether a row shares a byte with [p, q)
    bool meets(__int128 p, __int128 q) const {
        const __int128 i = p < row(0) + width ? 0 : (p - row(0) - width) / ld + 1;      // the first row that ends behind p
        return i < n && row(i) < q;
    }
    bool meets_row(const Rows& o, __int128 i) const { return meets(o.row(i), o.row(i) + o.width); }
};

// Whether two arrays share a byte: column slices of one buffer lie between each
// other's rows and share none.
bool share(const Rows& a, const Rows& b) {
    if (a.row(a.n - 1) + a.width <= b.at || b.row(b.n - 1) + b.width <= a.at) return false;
    // equal strides: where rows i and j meet, rows i - m and j - m do, and with m the smaller one is row 0
    if (a.ld == b.ld) return a.meets_row(b, 0) || b.meets_row(a, 0);
    const Rows& few = a.n < b.n ? a : b;
    const Rows& many = a.n < b.n ? b : a;
    for (__int128 i = 0; i < few.n; ++i)
        if (many.meets_row(few, i)) return true;
    return false;
}

// Checks that both calls share; fills what both need.
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

}  // namespace
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
