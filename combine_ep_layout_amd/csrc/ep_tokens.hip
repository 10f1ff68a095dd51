// gfx950 kernels of a whole MoE layer for a few tokens, and their C entry point.
//
//     y_t = sum_k w_tk Wd[e] a,  a = act(Wg[e] x_t) * (Wu[e] x_t),  e = e_tk
//
// Two launches: the choice of the experts with the gate and up products and the
// activation, then the down products with the weighted sum.  No rows move: the
// experts' matrices are the bytes that count, and every matrix that a token
// uses is read once.
//
// A workgroup takes 16 rows of a matrix and shares the summed index out to its
// eight waves, so that all of the chip's compute units read at once however few
// the experts are.  A wave's product is a matrix instruction with 16 rows of
// the weights on one side and up to 16 tokens of the expert on the other: the
// weights go from memory to the registers in the instruction's own layout,
// several steps ahead, with no pass through LDS, and further tokens of the same
// expert cost no bytes.  The waves' sums meet in LDS, in a fixed order.
//
// Weights are bf16, or 4-bit codes (e2m1) with an exponent byte for each 32 of
// them: two codes become two bf16 values, exactly, in one instruction, so the
// products, sums and roundings are those of bf16 weights.  a is rounded to bf16
// once, as the operand of the down product; y is rounded once.  All sums are
// fp32, the weights w_tk included.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ep_act.h"
#include "ep_layout.h"
#include "ep_ranges.h"
#include "ep_route_device.h"

namespace epk {
namespace {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kWaves = 8;
constexpr int kThreads = kWaves * kWave;
constexpr int kRows = 16;                   // rows of a matrix that a workgroup takes
constexpr int kMaxTokens = 64;
constexpr int kMaxSlots = kMaxTokens * kRouteMaxTopK;
constexpr int kMaxExperts = kRouteMaxExperts;
constexpr int kMaxUsed = kMaxExperts + kMaxSlots / 16;
constexpr int kMaxWidth = 1 << 16;          // hidden, inter
constexpr int64_t kMaxMatrix = 1 << 29;     // hidden * inter of one expert
// An offset past every buffer, also with a row's own offset added: such a lane loads zeros.
constexpr uint32_t kOutOfRange = 0x80000000u;

struct TokensArgs {
    const __bf16* x;            // [T, x_ld]
    int64_t x_ld;
    int32_t T, K, E, H, I;
    int32_t act;
    RouteArgs route;            // logits, when routed here
    int32_t route_here;
    int32_t* idx;               // [T, K]
    float* weights;             // [T, K]
    const void* w_gate_up;      // [E, 2I, H]
    const uint8_t* s_gate_up;   // [E, 2I, H / 32]
    const void* w_down;         // [E, H, I]
    const uint8_t* s_down;      // [E, H, I / 32]
    __bf16* a;                  // [T * K, I]
    __bf16* y;                  // [T, H]
};

__device__ __forceinline__ int uni(int v) { return __builtin_amdgcn_readfirstlane(v); }

typedef __amdgpu_buffer_rsrc_t Buffer;
__device__ __forceinline__ Buffer buffer(const void* base, int64_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc((void*)base, 0, (int)(uint32_t)bytes, 0x00020000);
}
__device__ __forceinline__ u32x4 load16(Buffer b, uint32_t lane, int at) {
    return __builtin_amdgcn_raw_buffer_load_b128(b, (int)lane, at, 0);
}

// The weights' forms.  A step is what one 16-byte load of each lane's row covers
// (bf16: two loads); lane l holds row l % 16 and the summed indices of its
// quarter q = l / 16, in kFrags fragments of 8.
struct Bf16Weights {
    static constexpr int kStep = 64, kFrags = 2;
    struct Regs { u32x4 v[2]; };
    struct Matrix { Buffer w; };
    // rows x n of expert e, from row `first`
    __device__ static Matrix open(const void* w, const uint8_t*, int64_t e, int64_t each, int64_t first, int64_t rows, int n) {
        return {buffer((const __bf16*)w + (e * each + first) * n, rows * n * 2)};
    }
    // summed index of fragment f inside a step
    __device__ static int k_of(int q, int f) { return f * 32 + q * 8; }
    struct Lane { uint32_t at; };
    __device__ static Lane lane(int row, int rows, int n, int q) {
        return {row < rows ? (uint32_t)row * (uint32_t)n * 2u + q * 16 : kOutOfRange};
    }
    // left: summed indices from this step on
    __device__ static Regs load(const Matrix& m, const Lane& l, int step, int left, int q) {
        Regs r;
#pragma unroll
        for (int f = 0; f < 2; ++f) r.v[f] = load16(m.w, k_of(q, f) < left ? l.at + f * 64 : kOutOfRange, step * (kStep * 2));
        return r;
    }
    __device__ static bf16x8 fragment(const Regs& r, int f) { return __builtin_bit_cast(bf16x8, r.v[f]); }
};

struct Mxfp4Weights {
    static constexpr int kStep = 128, kFrags = 4;
    struct Regs { u32x4 v; uint32_t scale; };
    struct Matrix { Buffer w, s; };
    __device__ static Matrix open(const void* w, const uint8_t* s, int64_t e, int64_t each, int64_t first, int64_t rows, int n) {
        const int64_t at = e * each + first;
        return {buffer((const uint8_t*)w + at * (n / 2), rows * (n / 2)), buffer(s + at * (n / 32), rows * (n / 32))};
    }
    __device__ static int k_of(int q, int f) { return q * 32 + f * 8; }
    struct Lane { uint32_t at, scale; };
    __device__ static Lane lane(int row, int rows, int n, int q) {
        return row < rows ? Lane{(uint32_t)row * (uint32_t)(n / 2) + q * 16, (uint32_t)row * (uint32_t)(n / 32) + q}
                          : Lane{kOutOfRange, kOutOfRange};
    }
    __device__ static Regs load(const Matrix& m, const Lane& l, int step, int left, int q) {
        const bool in = q * 32 < left;
        Regs r;
        r.v = load16(m.w, in ? l.at : kOutOfRange, step * (kStep / 2));
        r.scale = __builtin_amdgcn_raw_buffer_load_b8(m.s, (int)(in ? l.scale : kOutOfRange), step * (kStep / 32), 0);
        return r;
    }
    __device__ static bf16x8 fragment(const Regs& r, int f) {
        const float s = __uint_as_float(r.scale << 23);
        union { bf16x2 p[4]; bf16x8 v; } u;
        u.p[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(r.v[f], s, 0);
        u.p[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(r.v[f], s, 1);
        u.p[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(r.v[f], s, 2);
        u.p[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(r.v[f], s, 3);
        return u.v;
    }
};

// The tokens' slots by expert, made by every workgroup for itself from the
// choice of the experts: no launch of its own, no counters in memory.
struct Slots {
    int16_t expert[kMaxSlots];              // -1: none
    int16_t rank[kMaxSlots];                // among the expert's slots, -1: none
    float weight[kMaxSlots];
    int32_t count[kMaxExperts];             // then the expert's first place, and its slots << 16
    int16_t used[kMaxUsed];                 // experts with a slot, ascending
    int32_t start[kMaxUsed + 1];            // their first places
    int16_t sorted[kMaxSlots];
    int32_t n_used;
};

// ROUTE: the choice is made here, a wave a token.  CHUNK: an expert with more
// slots than this is listed several times, the slots in their order (which one
// is listed where decides which waves share its sums).
template <bool ROUTE, int CHUNK>
__device__ __forceinline__ void find_slots(const TokensArgs& a, Slots& s) {
    const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = uni(tid / kWave);
    const int S = a.T * a.K;
    for (int e = tid; e < a.E; e += kThreads) s.count[e] = 0;
    if (ROUTE) {
        if (wave < a.T) {
            int mine;
            float weight;
            if (a.route.bias) route_token<4, true>(a.route, wave, lane, mine, weight);
            else route_token<4, false>(a.route, wave, lane, mine, weight);
            if (lane < a.K) {
                const int at = wave * a.K + lane;
                s.expert[at] = (int16_t)mine;
                s.weight[at] = weight;
                if (blockIdx.x == 0) {
                    a.idx[at] = mine;
                    a.weights[at] = weight;
                }
            }
        }
    } else {
        for (int i = tid; i < S; i += kThreads) {
            const int e = a.idx[i];
            s.expert[i] = (int16_t)(e >= 0 && e < a.E ? e : -1);
            s.weight[i] = a.weights[i];
        }
    }
    __syncthreads();
    // An expert that a token names twice is one product with both weights.
    for (int i = tid; i < S; i += kThreads) {
        const int e = s.expert[i], t = i / a.K, end = (t + 1) * a.K;
        int rank = -1;
        if (e >= 0) {
            bool first = true;
            for (int j = t * a.K; j < i; ++j) first = first && s.expert[j] != e;
            if (first) rank = atomicAdd(&s.count[e], 1);        // in any order
        }
        s.rank[i] = (int16_t)rank;
        if (rank >= 0)
            for (int j = i + 1; j < end; ++j)
                if (s.expert[j] == e) s.weight[i] += s.weight[j];
    }
    __syncthreads();
    if (wave == 0) {
        const int per = (a.E + kWave - 1) / kWave;
        int used = 0, slots = 0;
#pragma unroll 1
        for (int i = 0; i < per; ++i) {
            const int e = lane * per + i, n = e < a.E ? s.count[e] : 0;
            used += (n + CHUNK - 1) / CHUNK;
            slots += n;
        }
        int before = used << 16 | slots;            // at most kMaxUsed and 2048
#pragma unroll
        for (int d = 1; d < kWave; d <<= 1) {
            const int o = __shfl_up(before, d);
            if (lane >= d) before += o;
        }
        if (lane == kWave - 1) {
            s.n_used = before >> 16;
            s.start[before >> 16] = before & 0xFFFF;
        }
        before -= used << 16 | slots;
        int u = before >> 16, p = before & 0xFFFF;
#pragma unroll 1
        for (int i = 0; i < per; ++i) {
            const int e = lane * per + i, n = e < a.E ? s.count[e] : 0;
            if (n > 0) s.count[e] = p | n << 16;
            for (int k = 0; k < n; k += CHUNK) {
                s.used[u] = (int16_t)e;
                s.start[u++] = p + k;
            }
            p += n;
        }
    }
    __syncthreads();
    for (int i = tid; i < S; i += kThreads)
        if (s.rank[i] >= 0) s.sorted[(s.count[s.expert[i]] & 0xFFFF) + s.rank[i]] = (int16_t)i;
    __syncthreads();
    if constexpr (CHUNK < kMaxTokens) {
        for (int i = tid; i < S; i += kThreads) {
            if (s.rank[i] < 0) continue;
            const int p = s.count[s.expert[i]] & 0xFFFF, n = s.count[s.expert[i]] >> 16;
            int before = 0;
            for (int j = p; j < p + n; ++j) before += s.sorted[j] < i;
            s.rank[i] = (int16_t)before;
        }
        __syncthreads();
        for (int i = tid; i < S; i += kThreads)
            if (s.rank[i] >= 0) s.sorted[(s.count[s.expert[i]] & 0xFFFF) + s.rank[i]] = (int16_t)i;
        __syncthreads();
    }
}

// What a wave loads for one step: M matrices' parts and NT tiles of 16 tokens.
template <class W, int M, int NT>
struct Stage {
    typename W::Regs w[M];
    u32x4 x[NT][W::kFrags];
};

// x_at: the lane's token's offset in bytes, or kOutOfRange.
template <class W, int M, int NT>
__device__ __forceinline__ void load_stage(Stage<W, M, NT>& s, const typename W::Matrix (&m)[M], const typename W::Lane& l,
                                           Buffer x, const uint32_t (&x_at)[NT], int step, int left, int q) {
    // The buffers' range is checked less the common offset, which therefore stays inside.
    step = left > 0 ? step : 0;
#pragma unroll
    for (int i = 0; i < M; ++i) s.w[i] = W::load(m[i], l, step, left, q);
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int f = 0; f < W::kFrags; ++f)
            s.x[j][f] = load16(x, W::k_of(q, f) < left ? x_at[j] + W::k_of(q, f) * 2 : kOutOfRange, step * (W::kStep * 2));
}

template <class W, int M, int NT>
__device__ __forceinline__ void multiply(const Stage<W, M, NT>& s, f32x4 (&c)[M][NT]) {
#pragma unroll
    for (int f = 0; f < W::kFrags; ++f)
#pragma unroll
        for (int i = 0; i < M; ++i) {
            const bf16x8 w = W::fragment(s.w[i], f);
#pragma unroll
            for (int j = 0; j < NT; ++j)
                c[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, __builtin_bit_cast(bf16x8, s.x[j][f]), c[i][j], 0, 0, 0);
        }
}

// Gate and up rows [tile * 16, + 16) of expert e, for n of the sorted slots.
template <class W, int NT>
__device__ __forceinline__ void up_item(const TokensArgs& a, const Slots& s, float* red, int e, int first, int n, int tile) {
    constexpr int D = NT == 1 ? 4 : 2;          // steps that a wave loads ahead
    const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = uni(tid / kWave), q = lane >> 4;
    const int r0 = tile * kRows;
    const typename W::Matrix m[2] = {W::open(a.w_gate_up, a.s_gate_up, e, 2 * (int64_t)a.I, 0, a.I, a.H),
                                     W::open(a.w_gate_up, a.s_gate_up, e, 2 * (int64_t)a.I, a.I, a.I, a.H)};
    const typename W::Lane l = W::lane(r0 + (lane & 15), a.I, a.H, q);
    const Buffer x = buffer(a.x, ((int64_t)(a.T - 1) * a.x_ld + a.H) * 2);
    uint32_t x_at[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        const int i = j * 16 + (lane & 15);
        x_at[j] = i < n ? (uint32_t)(s.sorted[first + i] / a.K) * (uint32_t)a.x_ld * 2u : kOutOfRange;
    }
    const int steps = (a.H + W::kStep - 1) / W::kStep, mine = (steps - wave + kWaves - 1) / kWaves;
    f32x4 c[2][NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) c[0][j] = c[1][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    Stage<W, 2, NT> stage[D];
    auto load = [&](int slot, int i) {
        const int step = wave + i * kWaves;
        load_stage<W, 2, NT>(stage[slot], m, l, x, x_at, step, a.H - step * W::kStep, q);
    };
#pragma unroll
    for (int d = 0; d < D; ++d) {
        load(d, d);
        __builtin_amdgcn_sched_barrier(0);      // in this order, or the loop's first wait would be for all of them
    }
#pragma unroll 1
    for (int i = 0; i < mine; i += D) {
#pragma unroll
        for (int d = 0; d < D; ++d) {
            multiply<W, 2, NT>(stage[d], c);
            load(d, i + d + D);
            __builtin_amdgcn_sched_barrier(0);
        }
    }
    // lane l holds rows 4 (l / 16) + 0..3 of its slot l % 16
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        if (j * 16 >= n) break;
        f32x4* const to = (f32x4*)red + wave * 128 + lane;
        to[0] = c[0][j];
        to[64] = c[1][j];
        __syncthreads();
        if (tid < 256) {
            float g = 0.f, up = 0.f;
#pragma unroll
            for (int w = 0; w < kWaves; ++w) {
                g += red[w * 512 + tid];
                up += red[w * 512 + 256 + tid];
            }
            const int i = j * 16 + ((tid >> 2) & 15), r = r0 + (tid >> 6) * 4 + (tid & 3);
            if (i < n && r < a.I) a.a[(int64_t)s.sorted[first + i] * a.I + r] = (__bf16)(act_value(g, a.act) * up);
        }
        __syncthreads();
    }
}

// MANY: an expert may have more than 16 tokens.  Two tiles of them are the most
// that the registers hold; a third and fourth are another pass over the weights.
template <class W, bool MANY, bool ROUTE>
__global__ void __launch_bounds__(kThreads, 4) tokens_up_kernel(TokensArgs a) {
    __shared__ Slots s;
    __shared__ __attribute__((aligned(16))) float red[kWaves * 512];
    find_slots<ROUTE, kMaxTokens>(a, s);
    const int tiles = (a.I + kRows - 1) / kRows, items = uni(s.n_used) * tiles;
    for (int i = blockIdx.x; i < items; i += gridDim.x) {
        const int u = i / tiles, tile = i - u * tiles;
        const int e = uni(s.used[u]), first = uni(s.start[u]), n = uni(s.start[u + 1]) - first;
        if (!MANY || n <= 16) up_item<W, 1>(a, s, red, e, first, n, tile);
        else
            for (int k = 0; k < n; k += 32) up_item<W, 2>(a, s, red, e, first + k, n - k < 32 ? n - k : 32, tile);
    }
}

// Columns [tile * 16, + 16) of y.  A wave takes an eighth of the used experts'
// steps, one after another; sums: [wave][token][16].  An expert's further tokens
// past 16 read its rows again, out of the L2 where they just were.
template <class W, int TOKENS>
__device__ __forceinline__ void down_item(const TokensArgs& a, const Slots& s, float (&sums)[kWaves][TOKENS][kRows], int tile) {
    constexpr int D = 4, NT = 1;
    const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = uni(tid / kWave), q = lane >> 4;
    const int steps = (a.I + W::kStep - 1) / W::kStep, units = uni(s.n_used) * steps;
    const int begin = (int)((int64_t)units * wave / kWaves), end = (int)((int64_t)units * (wave + 1) / kWaves);
    const typename W::Lane l = W::lane(tile * kRows + (lane & 15), a.H, a.I, q);
    const Buffer x = buffer(a.a, (int64_t)a.T * a.K * a.I * 2);
    Stage<W, 1, NT> stage[D];
    f32x4 c[1][NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) c[0][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    // where the loads are, and where the products are
    int load_u = begin / steps, load_step = begin - load_u * steps;
    int u = load_u, step = load_step;
    typename W::Matrix m[1] = {};
    uint32_t x_at[NT];
    auto open = [&] {
        const int e = uni(s.used[load_u]), first = uni(s.start[load_u]), n = uni(s.start[load_u + 1]) - first;
        m[0] = W::open(a.w_down, a.s_down, e, a.H, 0, a.H, a.I);
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            const int i = j * 16 + (lane & 15);
            x_at[j] = i < n ? (uint32_t)s.sorted[first + i] * (uint32_t)a.I * 2u : kOutOfRange;
        }
    };
    auto load = [&](int slot, int i) {
        // past the wave's last step: nothing (every lane out of range)
        load_stage<W, 1, NT>(stage[slot], m, l, x, x_at, load_step, i < end ? a.I - load_step * W::kStep : 0, q);
        if (++load_step == steps) {
            load_step = 0;
            if (i + 1 < end) {
                ++load_u;
                open();
            }
        }
    };
    if (begin < end) {
        open();
#pragma unroll
        for (int d = 0; d < D; ++d) {
            load(d, begin + d);
            __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll 1
        for (int i = begin; i < end; i += D) {
#pragma unroll
            for (int d = 0; d < D; ++d) {
                multiply<W, 1, NT>(stage[d], c);
                load(d, i + d + D);
                __builtin_amdgcn_sched_barrier(0);
                if (i + d < end && (++step == steps || i + d + 1 == end)) {
                    // the expert's part is done: every token has it once
                    const int first = uni(s.start[u]), n = uni(s.start[u + 1]) - first;
#pragma unroll
                    for (int j = 0; j < NT; ++j) {
                        const int k = j * 16 + (lane & 15);
                        if (k < n) {
                            const int slot = s.sorted[first + k];
                            const float w = s.weight[slot];
                            f32x4* const to = (f32x4*)&sums[wave][slot / a.K][q * 4];
                            f32x4 v = *to;
#pragma unroll
                            for (int r = 0; r < 4; ++r) v[r] = __builtin_fmaf(w, c[0][j][r], v[r]);
                            *to = v;
                        }
                        c[0][j] = f32x4{0.f, 0.f, 0.f, 0.f};
                    }
                    step = 0;
                    ++u;
                }
            }
        }
    }
    __syncthreads();
    for (int i = tid; i < a.T * kRows; i += kThreads) {
        const int t = i / kRows, r = i & (kRows - 1);
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            v += sums[w][t][r];
            sums[w][t][r] = 0.f;
        }
        if (tile * kRows + r < a.H) a.y[(int64_t)t * a.H + tile * kRows + r] = (__bf16)v;
    }
    __syncthreads();
}

template <class W, int TOKENS>
__global__ void __launch_bounds__(kThreads, 4) tokens_down_kernel(TokensArgs a) {
    __shared__ Slots s;
    __shared__ __attribute__((aligned(16))) float sums[kWaves][TOKENS][kRows];
    for (int i = threadIdx.x; i < kWaves * TOKENS * kRows; i += kThreads) (&sums[0][0][0])[i] = 0.f;
    find_slots<false, TOKENS == 16 ? kMaxTokens : 16>(a, s);        // of 16 tokens no expert has more
    const int tiles = (a.H + kRows - 1) / kRows;
    for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x) down_item<W, TOKENS>(a, s, sums, tile);
}

// From so many tokens on, or past 256 experts, the choice has a launch of its own:
// a workgroup would have to make more than its waves can at once.
constexpr int kRouteHereTokens = kWaves;
static_assert(kRouteHereTokens <= 16, "no expert has more");
constexpr int kRouteHereExperts = 256;

template <class W, bool MANY>
hipError_t launch(const TokensArgs& a, int num_cu, hipStream_t stream) {
    const int most = 2 * num_cu;            // two workgroups of a compute unit
    const int64_t used = (int64_t)a.T * a.K < a.E ? (int64_t)a.T * a.K : a.E;
    const int64_t up = used * ((a.I + kRows - 1) / kRows), down = (a.H + kRows - 1) / kRows;
    const int g1 = (int)(up < most ? up : most), g2 = (int)(down < most ? down : most);
    bool here = false;
    if constexpr (!MANY) {
        here = a.route_here;
        if (here) tokens_up_kernel<W, MANY, true><<<g1, kThreads, 0, stream>>>(a);
    }
    if (!here) tokens_up_kernel<W, MANY, false><<<g1, kThreads, 0, stream>>>(a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    tokens_down_kernel<W, MANY ? kMaxTokens : 16><<<g2, kThreads, 0, stream>>>(a);
    return hipGetLastError();
}

template <class W>
hipError_t launch(const TokensArgs& a, int num_cu, hipStream_t stream) {
    return a.T <= 16 ? launch<W, false>(a, num_cu, stream) : launch<W, true>(a, num_cu, stream);
}

constexpr uint32_t kRouteFlags = EP_ROUTE_BF16 | EP_ROUTE_SIGMOID | EP_ROUTE_NORMALIZE;

}  // namespace
}  // namespace epk

extern "C" ep_status ep_moe_tokens(const ep_moe_tokens_args* p, hipStream_t stream) {
    using namespace epk;
    if (!p) return EP_ERR_INVALID_ARGUMENT;
    const int32_t T = p->num_tokens, K = p->top_k, E = p->num_experts, H = p->hidden, I = p->inter;
    if (p->flags & ~(EP_MOE_MXFP4 | kRouteFlags)) return EP_ERR_INVALID_ARGUMENT;
    const bool four = p->flags & EP_MOE_MXFP4;
    const int32_t unit = four ? 32 : 8;
    if (T < 0 || E < 1 || K < 1 || H <= 0 || I <= 0 || H % unit != 0 || I % unit != 0 ||
        p->x_ld < H || p->x_ld % 8 != 0 || (p->activation != EP_ACT_SILU && p->activation != EP_ACT_GELU))
        return EP_ERR_INVALID_ARGUMENT;
    TokensArgs a{};
    if (p->logits) {
        const ep_status st = check_route(p->logits, p->logits_ld, T, E, K, p->flags & kRouteFlags, p->scale, a.route);
        if (st != EP_OK) return st;
        if (p->bias && !a.route.sigmoid) return EP_ERR_UNSUPPORTED;
    } else if (T > 0 && ((p->flags & kRouteFlags) || p->bias)) {       // without tokens logits may be null
        return EP_ERR_INVALID_ARGUMENT;
    }
    if (T > kMaxTokens || E > kMaxExperts || K > kRouteMaxTopK || H > kMaxWidth || I > kMaxWidth || (int64_t)H * I > kMaxMatrix ||
        p->x_ld > ((int64_t)1 << 23))
        return EP_ERR_UNSUPPORTED;
    if (T == 0) return EP_OK;
    if (!p->x || !p->topk_idx || !p->topk_weights || !p->w_gate_up || !p->w_down || !p->act || !p->y || !aligned(p->x, 16) ||
        !aligned(p->topk_idx, 4) || !aligned(p->topk_weights, 4) || !aligned(p->bias, 4) || !aligned(p->w_gate_up, 16) ||
        !aligned(p->w_down, 16) || !aligned(p->act, 16) || !aligned(p->y, 16) ||
        four != (p->gate_up_scales != nullptr) || four != (p->down_scales != nullptr))
        return EP_ERR_INVALID_ARGUMENT;
    // nothing that is written shares memory with anything else
    const int64_t S = (int64_t)T * K, m = (int64_t)E * H * I;
    const Rows flat[] = {Rows(p->act, S * I, S * I, 1, 2), Rows(p->y, (int64_t)T * H, (int64_t)T * H, 1, 2),
                         Rows(p->topk_idx, S, S, 1, 4), Rows(p->topk_weights, S, S, 1, 4),
                         Rows(p->x, p->x_ld, H, T, 2), Rows(p->w_gate_up, four ? m : 4 * m, four ? m : 4 * m, 1, 1),
                         Rows(p->w_down, four ? m / 2 : 2 * m, four ? m / 2 : 2 * m, 1, 1)};
    for (int i = 0; i < 4; ++i) {
        for (int j = i + 1; j < 7; ++j)
            if (share(flat[i], flat[j])) return EP_ERR_INVALID_ARGUMENT;
        if (p->logits && share(flat[i], Rows(p->logits, p->logits_ld, E, T, a.route.bf16 ? 2 : 4))) return EP_ERR_INVALID_ARGUMENT;
        if (p->bias && share(flat[i], Rows(p->bias, E, E, 1, 4))) return EP_ERR_INVALID_ARGUMENT;
        if (four && (share(flat[i], Rows(p->gate_up_scales, m / 16, m / 16, 1, 1)) ||
                     share(flat[i], Rows(p->down_scales, m / 32, m / 32, 1, 1))))
            return EP_ERR_INVALID_ARGUMENT;
    }
    int device = 0, num_cu = 0;
    if (hipGetDevice(&device) != hipSuccess ||
        hipDeviceGetAttribute(&num_cu, hipDeviceAttributeMultiprocessorCount, device) != hipSuccess || num_cu <= 0)
        return EP_ERR_HIP;
    a.x = (const __bf16*)p->x;
    a.x_ld = p->x_ld;
    a.T = T;
    a.K = K;
    a.E = E;
    a.H = H;
    a.I = I;
    a.act = p->activation == EP_ACT_GELU ? kActGelu : kActSilu;
    a.idx = p->topk_idx;
    a.weights = p->topk_weights;
    a.w_gate_up = p->w_gate_up;
    a.s_gate_up = p->gate_up_scales;
    a.w_down = p->w_down;
    a.s_down = p->down_scales;
    a.a = (__bf16*)p->act;
    a.y = (__bf16*)p->y;
    if (p->logits) {
        a.route.bias = p->bias;
        a.route.idx = p->topk_idx;
        a.route.weights = p->topk_weights;
        a.route_here = T <= kRouteHereTokens && E <= kRouteHereExperts;
        if (!a.route_here && launch_route(a.route, stream) != hipSuccess) return EP_ERR_HIP;
    }
    const hipError_t e = four ? launch<Mxfp4Weights>(a, num_cu, stream) : launch<Bf16Weights>(a, num_cu, stream);
    return e == hipSuccess ? EP_OK : EP_ERR_HIP;
}
