// gfx950 kernels of a whole MoE layer for a few tokens, and their C entry point.
//
//     y_t = sum_k w_tk Wd[e] a,  a = act(Wg[e] x_t) * (Wu[e] x_t),  e = e_tk
//
// Two launches: the choice of the experts with the gate and up products and the
// activation, then the down products with the weighted sum.  No rows move: the
// experts' matrices are the bytes that count.  A matrix that a token uses is read
// once for 32 of its expert's tokens in the gate and up products, once for 16 in
// the down product, and again for further ones.
//
// A workgroup takes 16 to 64 rows of a matrix and shares the summed index out to
// its waves, so that all of the chip's compute units read at once however few
// the experts are.  A wave's product is a matrix instruction with 16 rows of
// the weights on one side and up to 16 tokens of the expert on the other, so
// further tokens of the same expert cost no bytes of theirs.  The waves' sums meet
// in LDS, in a fixed order.
//
// Weights are bf16, or 4-bit codes (e2m1) with an exponent byte for each 32 of
// them: two codes become two bf16 values, exactly, in one instruction, so the
// products, sums and roundings are those of bf16 weights.  a is rounded to bf16
// once, as the operand of the down product; y is rounded once.  All sums are
// fp32, the weights w_tk included.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ep_act.h"
#include "ep_gemm.h"
#include "ep_layout.h"
#include "ep_ranges.h"
#include "ep_route_device.h"
#include "ep_tokens_shape.h"

namespace epk {
namespace {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kWaves = kTokensWaves;
constexpr int kThreads = kWaves * kWave;
constexpr int kRows = kTokensRows;
constexpr int kMaxTokens = 64;
constexpr int kMaxSlots = kMaxTokens * kRouteMaxTopK;
constexpr int kMaxExperts = kRouteMaxExperts;
constexpr int kMaxUsed = kMaxExperts + kMaxSlots / 16;
constexpr int kMaxWidth = 1 << 16;          // hidden, inter
constexpr int64_t kMaxMatrix = 1 << 29;     // hidden * inter of one expert
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

typedef __amdgpu_buffer_rsrc_t Buffer;
__device__ __forceinline__ Buffer buffer(const void* base, int64_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc((void*)base, 0, (int)(uint32_t)bytes, 0x00020000);
}
__device__ __forceinline__ u32x4 load16(Buffer b, uint32_t lane, int at) {
    return __builtin_amdgcn_raw_buffer_load_b128(b, (int)lane, at, 0);
}

// The weights' forms.  A step is 64 (bf16) or 128 (4-bit) summed indices of a
// row, four steps are a group; lane l holds row l % 16 and the indices of its
// quarter q = l / 16 in kFrags fragments of 8.
// kUpTiles: row tiles of a wave in the gate and up products.  Two share what is
// loaded of the tokens, which beside 4-bit weights is as many bytes as the
// weights (64 tokens: 267 us, 338 with one); beside bf16 weights it is little, and
// two workgroups of a compute unit that hide each other's ends are worth more
// (24 experts of 2056 x 1000: 38 us, 43).  kUpWaves: waves of a SIMD so.  With two
// tiles a wave a workgroup may take four, half of its waves two of them: longer
// shares, fewer ends (ep_tokens_shape.h).
struct Bf16Weights {
    static constexpr int kStep = 64, kFrags = 2, kTileBytes = 0, kUpTiles = 1, kUpWaves = 4;
    struct Regs { u32x4 v[2]; };
    struct Scales {};
    struct Matrix { Buffer w; };
    // rows x n of expert e, from row `first` of each
    __device__ static Matrix open(const void* w, const uint8_t*, int64_t e, int64_t each, int64_t first, int64_t rows, int n) {
        return {buffer((const __bf16*)w + (e * each + first) * n, rows * n * 2)};
    }
    // summed index of fragment f inside a step
    __device__ static int k_of(int q, int f) { return f * 32 + q * 8; }
    struct Lane { uint32_t at; };
    // of the tile of rows from `first` on
    __device__ static Lane lane(int first, int rows, int n, int lane) {
        const int row = first + (lane & 15), q = lane >> 4;
        return {row < rows ? (uint32_t)row * (uint32_t)n * 2u + q * 16 : kOutOfRange};
    }
    // left: summed indices from this step on
    __device__ static void load(Regs& r, const Matrix& m, const Lane& l, int step, int left, int lane, uint32_t) {
#pragma unroll
        for (int f = 0; f < 2; ++f) r.v[f] = load16(m.w, k_of(lane >> 4, f) < left ? l.at + f * 64 : kOutOfRange, step * (kStep * 2));
    }
    __device__ static void take(Regs&, lds_char*, int) {}
    __device__ static Scales load_scales(const Matrix&, const Lane&, int, int) { return {}; }
    __device__ static void settle(Scales&) {}
    __device__ static float scale_of(const Scales&, const Lane&, int, int, int) { return 1.0f; }
    __device__ static bf16x8 fragment(const Regs& r, float, int f) {
        return __builtin_bit_cast(bf16x8, r.v[f]);
    }
};

struct Mxfp4Weights {
    static constexpr int kStep = 128, kFrags = 4, kTileBytes = kRows * 64, kUpTiles = 2, kUpWaves = 2;
    struct Regs { u32x4 v; };
    // a row's bytes of a group: four of each step (one for each quarter)
    struct Scales { u32x4 v; uint32_t more; int over; };
    struct Matrix { i32x4 w; Buffer s; int bytes; };
    __device__ static Matrix open(const void* w, const uint8_t* s, int64_t e, int64_t each, int64_t first, int64_t rows, int n) {
        const int64_t at = e * each + first;
        return {make_rsrc((const uint8_t*)w + at * (n / 2)), buffer(s + at * (n / 32), rows * (n / 32)),
                (int)(rows * (n / 32))};
    }
    __device__ static int k_of(int q, int f) { return q * 32 + f * 8; }
    struct Lane { uint32_t at, scale, shift; };
    // The codes go through LDS, whole lines a load: lane l loads row l / 4 of the tile,
    // the piece that lets eight rows be read together from different banks.
    __device__ static int piece(int lane) { return (lane & 3) ^ (lane >> 3 & 3); }
    __device__ static Lane lane(int first, int rows, int n, int lane) {
        const int row = first + lane / 4, own = first + (lane & 15);
        const uint32_t s = (uint32_t)own * (uint32_t)(n / 32);
        Lane l{kOutOfRange, kOutOfRange, 0};
        if (row < rows) l.at = (uint32_t)row * (uint32_t)(n / 2) + piece(lane) * 16;
        if (own < rows) {
            l.scale = s & ~3u;
            l.shift = s & 3u;
        }
        return l;
    }
    __device__ static void load(Regs&, const Matrix& m, const Lane& l, int step, int left, int lane, uint32_t lds) {
        load_to_lds(uni((int)lds), l.at != kOutOfRange && piece(lane) * 32 < left ? l.at + (uint32_t)step * (kStep / 2) : kOutOfRange, m.w);
    }
    __device__ static void take(Regs& r, lds_char* tile, int lane) {
        r.v = *(__attribute__((address_space(3))) u32x4*)(tile + (lane & 15) * 64 + ((lane >> 4) ^ (lane >> 1 & 3)) * 16);
    }
    // 16 bytes from the row's dword on, for rows that start inside a dword 4 more.
    // A matrix has a multiple of 32 bytes; its last row's last load comes from
    // further up instead of reaching past them, by `over` (4, 8 or 12).
    __device__ static Scales load_scales(const Matrix& m, const Lane& l, int step, int n) {
        Scales s;
        const uint32_t at = l.scale + (uint32_t)step * 4;
        const bool in = l.scale != kOutOfRange && at < (uint32_t)m.bytes;
        s.over = in && at + 16 > (uint32_t)m.bytes ? (int)(at + 16 - (uint32_t)m.bytes) : 0;
        s.v = load16(m.s, in ? at - s.over : kOutOfRange, 0);
        s.more = 0;
        if ((n & 127) != 0) s.more = __builtin_amdgcn_raw_buffer_load_b32(m.s, (int)(in ? at + 16 : kOutOfRange), 0, 0);
        return s;
    }
    // ready to be used: the words where they belong
    __device__ static void settle(Scales& s) {
        if (__ballot(s.over != 0) == 0) return;
        if (s.over & 4) s.v = u32x4{s.v[1], s.v[2], s.v[3], 0};
        if (s.over & 8) s.v = u32x4{s.v[2], s.v[3], 0, 0};
    }
    // d: the step inside its group.  A byte past the row may be anything.
    __device__ static float scale_of(const Scales& s, const Lane& l, int d, int left, int q) {
        const uint32_t four = __builtin_amdgcn_alignbyte(d < 3 ? s.v[d < 3 ? d + 1 : 3] : s.more, s.v[d], l.shift);
        return __uint_as_float(q * 32 < left ? (four >> (8 * q) & 0xFFu) << 23 : 0u);
    }
    __device__ static bf16x8 fragment(const Regs& r, float scale, int f) {
        union { bf16x2 p[4]; bf16x8 v; } u;
        u.p[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(r.v[f], scale, 0);
        u.p[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(r.v[f], scale, 1);
        u.p[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(r.v[f], scale, 2);
        u.p[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(r.v[f], scale, 3);
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
            if (a.E <= kWave) {
                if (a.route.bias) route_token<1, true>(a.route, wave, lane, mine, weight);
                else route_token<1, false>(a.route, wave, lane, mine, weight);
            } else {
                if (a.route.bias) route_token<4, true>(a.route, wave, lane, mine, weight);
                else route_token<4, false>(a.route, wave, lane, mine, weight);
            }
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
    if (a.T == 1) {             // the slots themselves, by one wave
        if (wave == 0) {
            const int e = lane < a.K ? s.expert[lane] : -1;
            float w = lane < a.K ? s.weight[lane] : 0.0f;
            bool first = e >= 0;
            for (int j = 0; j < a.K; ++j) {
                const int other = __builtin_amdgcn_readlane(e, j);
                const float more = __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(w), j));
                if (other == e && j < lane) first = false;
                if (other == e && j > lane) w += more;          // this lane's own sum, of slots that are no first ones
            }
            const uint64_t who = __ballot(first);
            const int u = __builtin_popcountll(who & ((1ull << lane) - 1)), n = __builtin_popcountll(who);
            if (first) {
                s.used[u] = (int16_t)e;
                s.start[u] = u;
                s.sorted[u] = (int16_t)lane;
                s.weight[lane] = w;
            }
            if (lane == 0) {
                s.n_used = n;
                s.start[n] = n;
            }
        }
        __syncthreads();
        return;
    }
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

// Bytes of LDS of a wave: a step of M tiles of weights (in 4 bits) and NT tiles of tokens.
template <class W, int M, int NT>
constexpr int kStepBytes = M * W::kTileBytes + NT * kRows * W::kStep * 2;

// A wave's stream of steps, one loaded ahead; a group's scales are loaded a group
// ahead.  More steps ahead cost (one token in bf16: 131 us, 142 with four) or bring
// nothing (64 tokens in 4 bits, gate and up: 246 us, 245 with two).
// In the instruction's own layout each lane's 16 bytes lie in a line of their own.
// The tokens' values, as many bytes as 4-bit weights have, go through LDS instead,
// loaded in whole lines (64 tokens in 4 bits: gate and up 264 -> 243 us, down
// 160 -> 137), and the codes, too (223 and 130; the vector cache's address unit
// busy for 102 M cycles instead of 116 M in gate and up).
// bf16 weights stay in registers: their LDS would leave one workgroup a compute unit.
template <class W, int M, int NT>
struct Stream {
    // The tokens' pieces of 16 bytes: of a row, and rows that a load of 1 KiB covers.
    static constexpr int kPieces = W::kStep / 8, kEach = kWave / kPieces, kLoads = kRows / kEach;
    typename W::Regs w[M];
    bf16x8 v[NT][W::kFrags];
    typename W::Scales scales[M], ahead[M];
    uint32_t x_at[NT][kLoads];      // the lane's piece of a load's rows, or kOutOfRange
    i32x4 x;
    int n;                          // rows with a token
    lds_char* lds;

    // row(i): offset in bytes of the i-th token
    template <class F>
    __device__ __forceinline__ void set_tokens(const void* base, int count, int lane, F row) {
        x = make_rsrc(base);
        n = count;
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int k = 0; k < kLoads; ++k) {
                const int i = j * kRows + k * kEach + lane / kPieces;
                x_at[j][k] = i < n ? row(i) + piece(lane + k * kWave) * 16 : kOutOfRange;
            }
    }
    // which piece of a row a lane loads: those of eight rows that are read together lie in different banks
    __device__ __forceinline__ static int piece(int lane) { return (lane % kPieces) ^ (lane / kPieces & 7); }
    // left: summed indices from this step on; <= 0: nothing (every lane out of range)
    __device__ __forceinline__ void load(const typename W::Matrix (&m)[M], const typename W::Lane (&l)[M], int step, int left, int lane) {
        // The buffers' range is checked less the common offset, which therefore stays inside.
        step = left > 0 ? step : 0;
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");          // what is there is read
        const uint32_t at = (uint32_t)(uintptr_t)lds;
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int k = 0; k < kLoads; ++k) {
                if (j * kRows + k * kEach >= n) continue;           // what is there belongs to no token
                const bool in = piece(lane + k * kWave) * 8 < left;
                load_to_lds(uni((int)at + M * W::kTileBytes + (j * kLoads + k) * 1024),
                            in && x_at[j][k] != kOutOfRange ? x_at[j][k] + (uint32_t)step * (W::kStep * 2) : kOutOfRange, x);
            }
#pragma unroll
        for (int i = 0; i < M; ++i) W::load(w[i], m[i], l[i], step, left, lane, at + i * W::kTileBytes);
        __builtin_amdgcn_sched_barrier(0);
    }
    // No load into LDS outlives the workgroup.
    __device__ __forceinline__ static void end() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }
    __device__ __forceinline__ void load_scales(const typename W::Matrix (&m)[M], const typename W::Lane (&l)[M], int step, int n) {
#pragma unroll
        for (int i = 0; i < M; ++i) ahead[i] = W::load_scales(m[i], l[i], step, n);
        __builtin_amdgcn_sched_barrier(0);
    }
    __device__ __forceinline__ void next_group() {
#pragma unroll
        for (int i = 0; i < M; ++i) {
            scales[i] = ahead[i];
            W::settle(scales[i]);
        }
    }
    // The step in LDS to registers.
    __device__ __forceinline__ void take(int lane) {
        const int q = lane >> 4, r = lane & 15;
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
#pragma unroll
        for (int i = 0; i < M; ++i) W::take(w[i], lds + i * W::kTileBytes, lane);
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int f = 0; f < W::kFrags; ++f)
                v[j][f] = *(__attribute__((address_space(3))) bf16x8*)(lds + M * W::kTileBytes + (j * kRows + r) * (W::kStep * 2) +
                                                                       ((W::k_of(q, f) / 8) ^ (r & 7)) * 16);
    }
    __device__ __forceinline__ void multiply(int d, const typename W::Lane (&l)[M], int left, int lane, f32x4 (&c)[M][NT]) const {
        float scale[M];
#pragma unroll
        for (int i = 0; i < M; ++i) scale[i] = W::scale_of(scales[i], l[i], d, left, lane >> 4);
#pragma unroll
        for (int f = 0; f < W::kFrags; ++f)
#pragma unroll
            for (int i = 0; i < M; ++i) {
                const bf16x8 u = W::fragment(w[i], scale[i], f);
#pragma unroll
                for (int j = 0; j < NT; ++j) c[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(u, v[j][f], c[i][j], 0, 0, 0);
            }
    }
    // A step's products, and next()'s loads: those into LDS before the products, those
    // into the registers that these are made of behind them.
    template <class F>
    __device__ __forceinline__ void step(int d, const typename W::Lane (&l)[M], int left, int lane, f32x4 (&c)[M][NT], F next) {
        take(lane);
        if constexpr (W::kTileBytes > 0) next();
        multiply(d, l, left, lane, c);
        if constexpr (W::kTileBytes == 0) next();
    }
};

// R row tiles of gate and up rows from r0 on, of expert e, for n of the sorted slots.
struct UpItem {
    int e, first, n, r0;
};

// A wave's share of an item: an eighth of the summed index.
template <class W, int R, int NT, int GROUPS>
struct UpShare {
    static constexpr int M = 2 * R, kParts = kWaves / GROUPS;
    typename W::Matrix m[M];
    typename W::Lane l[M];
    int begin, end, H;
    Stream<W, M, NT> stream;

    __device__ __forceinline__ int left(int i) const { return i < end ? H - i * W::kStep : 0; }

    // Puts the first steps' loads on their way.
    __device__ __forceinline__ void start(const TokensArgs& a, const Slots& s, const UpItem& t, int wave, int lane) {
        const typename W::Matrix gate = W::open(a.w_gate_up, a.s_gate_up, t.e, 2 * (int64_t)a.I, 0, a.I, a.H);
        const typename W::Matrix up = W::open(a.w_gate_up, a.s_gate_up, t.e, 2 * (int64_t)a.I, a.I, a.I, a.H);
#pragma unroll
        for (int i = 0; i < M; ++i) {
            m[i] = i & 1 ? up : gate;
            l[i] = W::lane(t.r0 + (wave / kParts * R + (i >> 1)) * kRows, a.I, a.H, lane);
        }
        stream.set_tokens(a.x, t.n, lane, [&](int i) { return (uint32_t)(s.sorted[t.first + i] / a.K) * (uint32_t)a.x_ld * 2u; });
        H = a.H;
        const int steps = (H + W::kStep - 1) / W::kStep;
        begin = steps * (wave % kParts) / kParts;
        end = steps * (wave % kParts + 1) / kParts;
        if (begin == end) return;
        stream.load_scales(m, l, begin, H);
        stream.load(m, l, begin, left(begin), lane);
    }
    __device__ __forceinline__ void run(int lane, f32x4 (&c)[M][NT]) {
#pragma unroll
        for (int i = 0; i < M; ++i)
#pragma unroll
            for (int j = 0; j < NT; ++j) c[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
        for (int i = begin; i < end; i += 4) {
            stream.next_group();
#pragma unroll
            for (int d = 0; d < 4; ++d) {
                stream.step(d, l, left(i + d), lane, c, [&] {
                    if (d == 0) stream.load_scales(m, l, i + 4 < end ? i + 4 : i, H);
                    stream.load(m, l, i + d + 1, left(i + d + 1), lane);
                });
            }
        }
        stream.end();
    }
};

// The waves' sums, the activation and the store of an item.
template <int R, int NT, int GROUPS>
__device__ __forceinline__ void up_finish(const TokensArgs& a, const Slots& s, float* red, const UpItem& t, int wave, int lane,
                                          const f32x4 (&c)[2 * R][NT]) {
    const int tid = threadIdx.x;
    // lane l holds rows 4 (l / 16) + 0..3 of its slot l % 16
#pragma unroll
    for (int k = 0; k < R; ++k)
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            if (j * 16 >= t.n) break;
            f32x4* const to = (f32x4*)red + wave * 128 + lane;
            to[0] = c[2 * k][j];
            to[64] = c[2 * k + 1][j];
            __syncthreads();
            if (tid < 256 * GROUPS) {
                constexpr int kParts = kWaves / GROUPS;
                const int group = tid >> 8, at = tid & 255;
                float g = 0.f, u = 0.f;
#pragma unroll
                for (int w = 0; w < kParts; ++w) {
                    g += red[(group * kParts + w) * 512 + at];
                    u += red[(group * kParts + w) * 512 + 256 + at];
                }
                const int i = j * 16 + ((at >> 2) & 15), r = t.r0 + (group * R + k) * kRows + (at >> 6) * 4 + (at & 3);
                if (i < t.n && r < a.I) a.a[(int64_t)s.sorted[t.first + i] * a.I + r] = (__bf16)(act_value(g, a.act) * u);
            }
            __syncthreads();
        }
}

template <class W, int R, int NT, int GROUPS>
__device__ __forceinline__ void up_item(const TokensArgs& a, const Slots& s, float* red, lds_char* tokens, const UpItem& t) {
    const int lane = threadIdx.x & (kWave - 1), wave = uni(threadIdx.x / kWave);
    UpShare<W, R, NT, GROUPS> share;
    f32x4 c[2 * R][NT];
    share.stream.lds = tokens + wave * kStepBytes<W, 2 * R, NT>;
    share.start(a, s, t, wave, lane);
    share.run(lane, c);
    up_finish<R, NT, GROUPS>(a, s, red, t, wave, lane, c);
}

template <class W, int R, bool MANY>
constexpr size_t kUpLds = kWaves * kStepBytes<W, 2 * R, MANY ? 2 : 1> + kWaves * 512 * sizeof(float) + sizeof(Slots);

// MANY: an expert may have more than 16 tokens.  Two tiles of them are the most
// that the registers hold; a third and fourth are another pass over the weights
// (the same 8 experts: 32 tokens fetch them once, 108 us, 64 twice, 192).
template <class W, int R, int GROUPS, bool MANY, bool ROUTE>
__global__ void __launch_bounds__(kThreads, W::kUpWaves) tokens_up_kernel(TokensArgs a) {
    extern __shared__ __attribute__((aligned(1024))) char smem[];
    lds_char* const tokens = (lds_char*)smem;
    float* const red = (float*)(smem + kWaves * kStepBytes<W, 2 * R, MANY ? 2 : 1>);
    Slots& s = *(Slots*)(red + kWaves * 512);
    find_slots<ROUTE, kMaxTokens>(a, s);
    constexpr int kSide = GROUPS * R * kRows;
    const int tiles = (a.I + kSide - 1) / kSide, items = uni(s.n_used) * tiles;
    for (int i = blockIdx.x; i < items; i += gridDim.x) {
        const int u = i / tiles, first = uni(s.start[u]);
        const UpItem t{uni(s.used[u]), first, uni(s.start[u + 1]) - first, (i - u * tiles) * kSide};
        if (!MANY || t.n <= 16) up_item<W, R, 1, GROUPS>(a, s, red, tokens, t);
        else
            for (int k = 0; k < t.n; k += 32) up_item<W, R, 2, GROUPS>(a, s, red, tokens, {t.e, first + k, t.n - k < 32 ? t.n - k : 32, t.r0});
    }
}

// R row tiles of columns of y from c0 on.  A wave takes an eighth of the used experts'
// groups, one after another; sums: [wave][token][columns].  An expert's further
// tokens past 16 read its rows again, and not out of the L2: with 8 experts of
// 7168 x 2048 (bf16) that every token chooses, 32 and 64 tokens fetch 2 and 4
// times the bytes of 16 (95 and 167 us, 60).
template <class W, int R, int TOKENS>
__device__ __forceinline__ void down_item(const TokensArgs& a, const Slots& s, float (&sums)[kWaves][TOKENS][R * kRows], lds_char* tokens, int c0) {
    constexpr int M = R, kSide = M * kRows;
    const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = uni(tid / kWave), q = lane >> 4;
    const int groups = (a.I + 4 * W::kStep - 1) / (4 * W::kStep), units = uni(s.n_used) * groups;
    const int begin = (int)((int64_t)units * wave / kWaves), end = (int)((int64_t)units * (wave + 1) / kWaves);
    typename W::Lane l[M];
#pragma unroll
    for (int i = 0; i < M; ++i) l[i] = W::lane(c0 + i * kRows, a.H, a.I, lane);
    Stream<W, M, 1> stream;
    stream.lds = tokens + wave * kStepBytes<W, R, 1>;
    f32x4 c[M][1];
#pragma unroll
    for (int i = 0; i < M; ++i) c[i][0] = f32x4{0.f, 0.f, 0.f, 0.f};
    typename W::Matrix m[M] = {};
    auto open = [&](int u) {
        const int e = uni(s.used[u]), first = uni(s.start[u]), n = uni(s.start[u + 1]) - first;
        const typename W::Matrix w = W::open(a.w_down, a.s_down, e, a.H, 0, a.H, a.I);
#pragma unroll
        for (int i = 0; i < M; ++i) m[i] = w;
        stream.set_tokens(a.a, n, lane, [&](int i) { return (uint32_t)s.sorted[first + i] * (uint32_t)a.I * 2u; });
    };
    if (begin < end) {
        int u = begin / groups, g = begin - u * groups;         // where the products are
        open(u);
        stream.load_scales(m, l, g * 4, a.I);
        stream.load(m, l, g * 4, a.I - g * 4 * W::kStep, lane);
#pragma unroll 1
        for (int i = begin; i < end; ++i) {
            // the next group: of this expert, or of the next one
            const bool more = i + 1 < end;
            const int next_g = g + 1 == groups ? 0 : g + 1;
            stream.next_group();
#pragma unroll
            for (int d = 0; d < 4; ++d) {
                stream.step(d, l, a.I - (g * 4 + d) * W::kStep, lane, c, [&] {
                    if (d < 3) {
                        stream.load(m, l, g * 4 + d + 1, a.I - (g * 4 + d + 1) * W::kStep, lane);
                    } else {
                        if (more && next_g == 0) open(u + 1);
                        stream.load_scales(m, l, more ? next_g * 4 : 0, a.I);
                        stream.load(m, l, next_g * 4, more ? a.I - next_g * 4 * W::kStep : 0, lane);
                    }
                });
            }
            if (next_g == 0 || !more) {
                // the expert's part is done: every token has it once
                const int first = uni(s.start[u]), n = uni(s.start[u + 1]) - first, k = lane & 15;
                if (k < n) {
                    const int slot = s.sorted[first + k];
                    const float w = s.weight[slot];
#pragma unroll
                    for (int t = 0; t < M; ++t) {
                        f32x4* const to = (f32x4*)&sums[wave][slot / a.K][t * kRows + q * 4];
                        f32x4 v = *to;
#pragma unroll
                        for (int r = 0; r < 4; ++r) v[r] = __builtin_fmaf(w, c[t][0][r], v[r]);
                        *to = v;
                    }
                }
#pragma unroll
                for (int t = 0; t < M; ++t) c[t][0] = f32x4{0.f, 0.f, 0.f, 0.f};
                ++u;
            }
            g = next_g;
        }
        stream.end();
    }
    __syncthreads();
    for (int i = tid; i < a.T * kSide; i += kThreads) {
        const int t = i / kSide, r = i % kSide;
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            v += sums[w][t][r];
            sums[w][t][r] = 0.f;
        }
        if (c0 + r < a.H) a.y[(int64_t)t * a.H + c0 + r] = (__bf16)v;
    }
    __syncthreads();
}

// The sums follow the slots: past 64 KiB together with many tokens.
template <class W, int R, int TOKENS>
constexpr size_t kDownLds = kWaves * kStepBytes<W, R, 1> + sizeof(float) * kWaves * TOKENS * R * kRows + sizeof(Slots);

template <class W, int R, int TOKENS>
__global__ void __launch_bounds__(kThreads, 4 / R) tokens_down_kernel(TokensArgs a) {
    extern __shared__ __attribute__((aligned(1024))) char smem[];
    constexpr int kSide = R * kRows;
    float (&sums)[kWaves][TOKENS][kSide] = *(float (*)[kWaves][TOKENS][kSide])(smem + kWaves * kStepBytes<W, R, 1>);
    Slots& s = *(Slots*)(smem + kWaves * kStepBytes<W, R, 1> + sizeof(sums));
    for (int i = threadIdx.x; i < kWaves * TOKENS * kSide; i += kThreads) (&sums[0][0][0])[i] = 0.f;
    find_slots<false, TOKENS == 16 ? kMaxTokens : 16>(a, s);        // of 16 tokens no expert has more
    const int tiles = (a.H + kSide - 1) / kSide;
    for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x) down_item<W, R, TOKENS>(a, s, sums, (lds_char*)smem, tile * kSide);
}

hipError_t launch_with(void (*kernel)(TokensArgs), const TokensArgs& a, int grid, size_t lds, hipStream_t stream) {
    if (lds > 64 * 1024) {
        const hipError_t e = hipFuncSetAttribute((const void*)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
        if (e != hipSuccess) return e;
    }
    kernel<<<grid, kThreads, lds, stream>>>(a);
    return hipGetLastError();
}

template <class W, int R, int GROUPS, bool MANY>
hipError_t launch_up(const TokensArgs& a, int64_t items, int num_cu, hipStream_t stream) {
    const int most = W::kUpWaves / 2 * num_cu;          // what the registers let run at once
    const int grid = (int)(items < most ? items : most);
    constexpr size_t lds = kUpLds<W, R, MANY>;
    if constexpr (!MANY)
        if (a.route_here) return launch_with(tokens_up_kernel<W, R, GROUPS, MANY, true>, a, grid, lds, stream);
    return launch_with(tokens_up_kernel<W, R, GROUPS, MANY, false>, a, grid, lds, stream);
}

template <class W, int R, int TOKENS>
hipError_t launch_down(const TokensArgs& a, int64_t items, int num_cu, hipStream_t stream) {
    const int most = 2 / R * num_cu, grid = (int)(items < most ? items : most);
    return launch_with(tokens_down_kernel<W, R, TOKENS>, a, grid, kDownLds<W, R, TOKENS>, stream);
}

template <class W, bool MANY>
hipError_t launch(const TokensArgs& a, const TokensShape& f, int num_cu, hipStream_t stream) {
    constexpr int kTokens = MANY ? kMaxTokens : 16;
    hipError_t e = hipSuccess;
    if (f.up_tiles == 1) {
        e = launch_up<W, 1, 1, MANY>(a, f.up_items, num_cu, stream);
    } else if constexpr (W::kUpTiles > 1) {
        e = f.up_groups == 2 ? launch_up<W, W::kUpTiles, 2, MANY>(a, f.up_items, num_cu, stream)
                             : launch_up<W, W::kUpTiles, 1, MANY>(a, f.up_items, num_cu, stream);
    }
    if (e != hipSuccess) return e;
    return f.down_tiles == 2 ? launch_down<W, 2, kTokens>(a, f.down_items, num_cu, stream)
                             : launch_down<W, 1, kTokens>(a, f.down_items, num_cu, stream);
}

template <class W>
hipError_t launch(TokensArgs& a, int num_cu, hipStream_t stream) {
    const TokensShape f = tokens_shape({a.T, a.K, a.E, a.H, a.I, W::kUpTiles, num_cu});
    a.route_here = a.route.logits && f.route_here;
    if (a.route.logits && !a.route_here) {
        const hipError_t e = launch_route(a.route, stream);
        if (e != hipSuccess) return e;
    }
    return f.many ? launch<W, true>(a, f, num_cu, stream) : launch<W, false>(a, f, num_cu, stream);
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
        !aligned(p->gate_up_scales, 16) || !aligned(p->down_scales, 16) ||
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
    }
    const hipError_t e = four ? launch<Mxfp4Weights>(a, num_cu, stream) : launch<Bf16Weights>(a, num_cu, stream);
    return e == hipSuccess ? EP_OK : EP_ERR_HIP;
}
