// gfx950 kernels that orthogonalise matrices by Newton-Schulz products, and of
// the optimiser step on it, with their C entry points.
//
// A matrix U, laid as m x n with m <= n (a tall one transposed), becomes
//     X = U / (|U| + eps),  then `steps` times  X = a X + P X,
//     G = X X^T,  P = b G + c G G,
// which takes every singular value through a s + b s^3 + c s^5 and leaves the
// singular vectors: with the usual coefficients those above 1/500 of the norm
// end between 0.7 and 1.2.  G and P are symmetric, so only the tiles on and below
// the diagonal are computed: m^2 n + m^3 + 2 m^2 n operations a step.
//
// The products run on the matrix cores in fp16 with fp32 sums.  fp16 and not
// bf16: everything here is bounded (|X| <= 1.2 in the 2-norm), so powers of two
// put the values into fp16's range for good, and its 11 bits leave results 1.6e-3
// off in the norm where bf16 makes 1.1e-2.  X itself is kept as two fp16 values,
// hi and 2^-11 lo: the first steps multiply small singular values by a = 3.4 each, and
// with them whatever rounding X had; the products see hi alone, where a rounding
// is no more than its share of P X (matrices of rank 16 in noise-free form:
// 4e-4 instead of 4.5e-2).  In the last two steps X = (a - k) X + (P + k I) X with
// k = -(b l + c l^2), l the mean of G's diagonal: the same, but where singular values have
// come near 1 P + k I is small and its rounding with it (noise of 512 x 1792: 9.6e-4
// before the result's own rounding instead of 1.7e-3).  Earlier it would put the
// rounding of hi, k times it, among the singular values that are still small.
//
// One launch serves all matrices of a list: their shapes and addresses travel
// in the kernel's arguments.  Step by step: the norms (with the momentum), the
// split into hi and lo, then three products each; the last one writes the
// results, or updates the parameters, from its registers.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>
#include <atomic>
#include <new>
#include <vector>

#include "ep_gemm.h"
#include "ep_layout.h"
#include "ep_muon_shape.h"
#include "ep_ranges.h"

namespace epk {
namespace {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

constexpr int kProblems = kMuonProblems;
constexpr int kMaxSide = 1 << 16;
constexpr int64_t kMaxMatrix = 1 << 29;     // values: a matrix of fp16 stays below 2 GiB
constexpr int kGroupM = 8;                  // row tiles that share their column tiles' loads
// Powers of two that G and P are held at: G's least entries, 1 / (m sqrt(n)) of
// the first step, are normal numbers, and |P| <= |b| + |c| is far from 65504.
constexpr float kGramScale = 1024.0f;
constexpr float kLow = 2048.0f;             // lo is held at this many times its value
constexpr int kPartials = 256;              // sums of squares of a matrix at most
constexpr int kThreads = 256;
constexpr int kSplit = 64;                  // side of a tall matrix's tile in the split
constexpr int kUnit = 512;                  // pieces of 8 values in a unit of the split: such a tile

// `batch` matrices of one shape.  The workspace holds, each for all of them:
// hi (two, by turns), lo [m, ld_n], g, p [m, ld_m] in fp16, and the partial sums.
struct Problem {
    const void* x;              // the gradient, or what is orthogonalised
    float* momentum;            // null: x alone
    void* param;                // fp32 or bf16 [rows, cols]; the result (bf16) without momentum
    __bf16* copy;               // may be null
    char* ws;
    int32_t m, n, ld_m, ld_n;
    int32_t batch;
    int32_t begin, mats;        // the matrices that a product is for
    int32_t tall;               // x and param are [n, m]
    int32_t partials;           // of a matrix
    float scale;                // the power of two that X is held at
    float step;                 // learning rate times the shape's factor

    // whether pieces of 8 values, of a matrix and of a row of x, start at whole 16 bytes
    __device__ bool even() const { return ((int64_t)m * n & 7) == 0; }
    __device__ bool even_rows() const { return ((tall ? m : n) & 7) == 0; }
    __host__ __device__ int64_t x_size() const { return (int64_t)m * ld_n; }
    __host__ __device__ int64_t g_size() const { return (int64_t)m * ld_m; }
    __device__ _Float16* hi(int turn) const { return (_Float16*)ws + turn * batch * x_size(); }
    __device__ _Float16* lo() const { return (_Float16*)ws + 2 * batch * x_size(); }
    __device__ _Float16* g() const { return (_Float16*)ws + 3 * batch * x_size(); }
    __device__ _Float16* p() const { return (_Float16*)ws + 3 * batch * x_size() + batch * g_size(); }
    __device__ double* sums() const { return (double*)((_Float16*)ws + 3 * batch * x_size() + 2 * batch * g_size()); }
    // k of the shifted steps, where the sums were (read before)
    __device__ float& shift(int mat) const { return *(float*)(sums() + (int64_t)mat * partials); }
    // bytes of one matrix; a multiple of 16, since the leading dimensions are multiples of 8
    __host__ int64_t ws_each() const { return 6 * x_size() + 4 * g_size() + (int64_t)partials * 8; }
};

struct GroupArgs {
    int32_t count;
    int32_t turn;               // which hi is read
    int32_t shifted;            // one of the last two steps
    int32_t x_bf16, param_bf16, nesterov;
    float a, b, c;
    float mu, rest_mu;          // momentum
    float eps;
    float decay;
    int32_t first[kProblems + 1];           // first tile (or workgroup) of each problem
    Problem p[kProblems];
};
static_assert(sizeof(GroupArgs) <= 4096, "kernel arguments");

// The problem that item i belongs to.
__device__ __forceinline__ int find_problem(const GroupArgs& a, int i) {
    const int lane = threadIdx.x & (kWave - 1);
    return __builtin_popcountll(__ballot(lane < a.count && a.first[lane] <= i)) - 1;
}

// Eight values, or with even false the first `left` of them and zeros.
__device__ __forceinline__ void load8(const float* x, int64_t i, bool even, int left, float (&v)[8]) {
    if (even) {
        const f32x4 lo = *(const f32x4*)(x + i), hi = *(const f32x4*)(x + i + 4);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            v[q] = lo[q];
            v[4 + q] = hi[q];
        }
    } else {
#pragma unroll
        for (int q = 0; q < 8; ++q) v[q] = q < left ? x[i + q] : 0.0f;
    }
}
__device__ __forceinline__ void load8(const __bf16* x, int64_t i, bool even, int left, float (&v)[8]) {
    if (even) {
        const bf16x8 b = *(const bf16x8*)(x + i);
#pragma unroll
        for (int q = 0; q < 8; ++q) v[q] = (float)b[q];
    } else {
#pragma unroll
        for (int q = 0; q < 8; ++q) v[q] = q < left ? (float)x[i + q] : 0.0f;
    }
}
__device__ __forceinline__ void load8(bool bf16, const void* x, int64_t i, bool even, int left, float (&v)[8]) {
    if (bf16) load8((const __bf16*)x, i, even, left, v);
    else load8((const float*)x, i, even, left, v);
}
__device__ __forceinline__ void store8(float* x, int64_t i, bool even, int left, const float (&v)[8]) {
    if (even) {
        *(f32x4*)(x + i) = f32x4{v[0], v[1], v[2], v[3]};
        *(f32x4*)(x + i + 4) = f32x4{v[4], v[5], v[6], v[7]};
    } else {
#pragma unroll
        for (int q = 0; q < 8; ++q)
            if (q < left) x[i + q] = v[q];
    }
}
__device__ __forceinline__ void store8(__bf16* x, int64_t i, bool even, int left, const float (&v)[8]) {
    if (even) {
        bf16x8 b;
#pragma unroll
        for (int q = 0; q < 8; ++q) b[q] = (__bf16)v[q];
        *(bf16x8*)(x + i) = b;
    } else {
#pragma unroll
        for (int q = 0; q < 8; ++q)
            if (q < left) x[i + q] = (__bf16)v[q];
    }
}

// The update's value from the gradient and the new momentum.
__device__ __forceinline__ float mix(const GroupArgs& a, float g, float m) {
    return a.nesterov ? a.rest_mu * g + a.mu * m : m;
}

// Sum over the workgroup, the same in every thread.
__device__ __forceinline__ double block_sum(double v, double* part) {
#pragma unroll
    for (int d = kWave / 2; d >= 1; d >>= 1) v += __shfl_xor(v, d);
    if ((threadIdx.x & (kWave - 1)) == 0) part[threadIdx.x / kWave] = v;
    __syncthreads();
    return (part[0] + part[1]) + (part[2] + part[3]);
}

// The momentum, and the sums of squares of the update, in double: neither tiny
// nor huge gradients leave its range.
__global__ void __launch_bounds__(kThreads) muon_sums_kernel(GroupArgs a) {
    __shared__ double part[kThreads / kWave];
    const int i = find_problem(a, blockIdx.x), tid = threadIdx.x;
    const Problem& p = a.p[i];
    const int local = blockIdx.x - a.first[i], mat = local / p.partials, k = local - mat * p.partials;
    const int64_t n = (int64_t)p.m * p.n, at = mat * n, step = (int64_t)p.partials * kThreads * 8;
    const bool even = p.even();
    double sum = 0.0;
#pragma unroll 2
    for (int64_t j = ((int64_t)k * kThreads + tid) * 8; j < n; j += step) {
        const int left = n - j < 8 ? (int)(n - j) : 8;
        float u[8];
        load8(a.x_bf16, p.x, at + j, even, left, u);
        if (p.momentum) {
            float m[8];
            load8(p.momentum, at + j, even, left, m);
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                m[q] = a.mu * m[q] + a.rest_mu * u[q];
                u[q] = mix(a, u[q], m[q]);
            }
            store8(p.momentum, at + j, even, left, m);
        }
#pragma unroll
        for (int q = 0; q < 8; ++q) sum += (double)u[q] * (double)u[q];
    }
    sum = block_sum(sum, part);
    if (tid == 0) p.sums()[local] = sum;
}

__device__ __forceinline__ void split(float v, _Float16& hi, _Float16& lo) {
    hi = (_Float16)v;
    lo = (_Float16)((v - (float)hi) * kLow);
}
__device__ __forceinline__ void split8(const float (&v)[8], f16x8& hi, f16x8& lo) {
#pragma unroll
    for (int q = 0; q < 8; ++q) {
        _Float16 h, l;
        split(v[q], h, l);
        hi[q] = h;
        lo[q] = l;
    }
}

// Units of a matrix in the split.
__host__ __device__ inline int64_t split_units(int m, int ld_n, bool tall) {
    return tall ? (int64_t)((m + kSplit - 1) / kSplit) * ((ld_n + kSplit - 1) / kSplit) : ((int64_t)m * (ld_n / 8) + kUnit - 1) / kUnit;
}

// X over its norm, as hi and lo, tall matrices turned through LDS; columns past n
// are zeros.  per: units of a workgroup.
__global__ void __launch_bounds__(kThreads) muon_split_kernel(GroupArgs a, int per) {
    __shared__ float tile[kSplit][kSplit + 1];
    __shared__ double part[kThreads / kWave];
    const int i = find_problem(a, blockIdx.x), tid = threadIdx.x;
    const Problem& p = a.p[i];
    const int64_t units = split_units(p.m, p.ld_n, p.tall);
    const int blocks = (int)((units + per - 1) / per), local = blockIdx.x - a.first[i], mat = local / blocks;
    double sum = 0.0;
    for (int k = tid; k < p.partials; k += kThreads) sum += p.sums()[mat * p.partials + k];
    const double norm = sqrt(block_sum(sum, part));
    const double s = norm == 0.0 ? 0.0 : (double)p.scale / (norm + (double)a.eps);       // a matrix of zeros stays one
    const int64_t at = (int64_t)mat * p.m * p.n;
    _Float16* const hi = p.hi(0) + mat * p.x_size();
    _Float16* const lo = p.lo() + mat * p.x_size();
    const bool even = p.even() && p.even_rows();
    // a piece of a row of x: pieces past its end are zeros
    auto load = [&](int64_t from, int left, float (&u)[8]) {
        if (left <= 0) {
#pragma unroll
            for (int q = 0; q < 8; ++q) u[q] = 0.0f;
            return;
        }
        load8(a.x_bf16, p.x, from, even, left, u);
        if (p.momentum) {
            float m[8];
            load8(p.momentum, from, even, left, m);
#pragma unroll
            for (int q = 0; q < 8; ++q) u[q] = mix(a, u[q], m[q]);
        }
#pragma unroll
        for (int q = 0; q < 8; ++q) u[q] = (float)((double)u[q] * s);
    };
    const int64_t first = (int64_t)(local - mat * blocks) * per, last = first + per < units ? first + per : units;
    if (!p.tall) {
        const int64_t pieces = (int64_t)p.m * (p.ld_n / 8);
        const int row = p.ld_n / 8;
#pragma unroll 2
        for (int64_t j = first * kUnit + tid; j < last * kUnit && j < pieces; j += kThreads) {
            const int r = (int)(j / row), c = (int)(j - (int64_t)r * row) * 8;
            float u[8];
            load(at + (int64_t)r * p.n + c, p.n - c, u);
            f16x8 h, l;
            split8(u, h, l);
            *(f16x8*)(hi + j * 8) = h;
            *(f16x8*)(lo + j * 8) = l;
        }
        return;
    }
    const int across = (p.ld_n + kSplit - 1) / kSplit;
    for (int64_t t = first; t < last; ++t) {
        const int r0 = (int)(t / across) * kSplit, c0 = (int)(t % across) * kSplit;
#pragma unroll
        for (int k = 0; k < kUnit / kThreads; ++k) {
            const int j = k * kThreads + tid, y = j / (kSplit / 8), x = j % (kSplit / 8) * 8;
            float u[8];
            load(at + (int64_t)(c0 + y) * p.m + r0 + x, c0 + y < p.n ? p.m - r0 - x : 0, u);
#pragma unroll
            for (int q = 0; q < 8; ++q) tile[y][x + q] = u[q];
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kUnit / kThreads; ++k) {
            const int j = k * kThreads + tid, y = j / (kSplit / 8), x = j % (kSplit / 8) * 8;
            if (r0 + y < p.m && c0 + x < p.ld_n) {
                float u[8];
#pragma unroll
                for (int q = 0; q < 8; ++q) u[q] = tile[x + q][y];
                f16x8 h, l;
                split8(u, h, l);
                const int64_t to = (int64_t)(r0 + y) * p.ld_n + c0 + x;
                *(f16x8*)(hi + to) = h;
                *(f16x8*)(lo + to) = l;
            }
        }
        __syncthreads();
    }
}

// BM x BN tiles, WM x WN of it to each wave, ST LDS tiles of each operand.
template <int OP_, int BM_, int BN_, int WM_, int WN_, int ST_, bool PIPELINED>
struct Shape {
    static constexpr int OP = OP_, BM = BM_, BN = BN_, WM = WM_, WN = WN_, BK = 64, ST = ST_;
    static constexpr int kWaves = (BM / WM) * (BN / WN);
    static constexpr int kThreads = kWaves * kWave;
    static constexpr int kStageBytes = (BM + BN) * BK * 2;
    static constexpr bool kPipelined = PIPELINED;
    static constexpr bool kAStrided = false, kBStrided = is_update(OP), kF16 = true;
    using A = Loader<BM, BK, kAStrided, kWaves>;
    using B = Loader<BN, BK, kBStrided, kWaves>;
    static constexpr int kLoads = A::kLoads + B::kLoads;
    static constexpr size_t kLds = (size_t)ST * kStageBytes;
};

// The eight sums of a lane out of two fragments, consecutive along the side that
// its sums lie on; lane l's first is at eight_at(l) of the fragments' places.
__device__ __forceinline__ void eight(const f32x4& v0, const f32x4& v1, float (&o)[8]) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v0[q]), __float_as_uint(v1[q]), false, false);
        o[q] = __uint_as_float(r[0]);
        o[4 + q] = __uint_as_float(r[1]);
    }
}
__device__ __forceinline__ int eight_at(int lane) { return (lane & 16) + (lane >> 5) * 8; }

// Eight consecutive results, or `left` of them: bf16, or the parameters' step and
// their copy.  old: the parameters.
__device__ __forceinline__ void write_results(const GroupArgs& a, const Problem& p, int64_t at, bool even, int left,
                                              const float (&old)[8], float (&v)[8]) {
    const float back = 1.0f / p.scale;          // a power of two
    if (p.momentum) {
#pragma unroll
        for (int q = 0; q < 8; ++q) v[q] = old[q] * a.decay - p.step * (v[q] * back);
        if (a.param_bf16) store8((__bf16*)p.param, at, even, left, v);
        else store8((float*)p.param, at, even, left, v);
        if (p.copy) store8(p.copy, at, even, left, v);
    } else {
#pragma unroll
        for (int q = 0; q < 8; ++q) v[q] *= back;
        store8((__bf16*)p.param, at, even, left, v);
    }
}

// k, from G's diagonal, by every wave for itself.
__device__ __forceinline__ float shift_of(const GroupArgs& a, const Problem& p, int mat, int lane) {
    const _Float16* const g = p.g() + mat * p.g_size();
    float sum = 0.0f;
#pragma unroll 4
    for (int r = lane; r < p.m; r += kWave) sum += (float)g[(int64_t)r * (p.ld_m + 1)];
#pragma unroll
    for (int d = kWave / 2; d >= 1; d >>= 1) sum += __shfl_xor(sum, d);
    const float l = fminf(sum / ((float)p.m * kGramScale), 1.0f);
    return -(a.b * l + a.c * (l * l));
}

// Floats of a column of 32 rows in LDS: 4 more spread the columns over the banks.
constexpr int kTurnRow = 36;

// G's or P's tile and, off the diagonal, its mirror image.
template <int OP, int MF, int NF>
__device__ __forceinline__ void finish_square(const GroupArgs& a, const Problem& p, int mat, int r_at, int c_at, bool mirror, int lane,
                                              float k, const f32x4 (&acc)[MF][NF]) {
    const _Float16* const g = p.g() + mat * p.g_size();
    _Float16* const out = (OP == kGram ? p.g() : p.p()) + mat * p.g_size();
#pragma unroll
    for (int i = 0; i < MF; ++i) {
        const int r = r_at + i * 16 + (lane & 15);
        const bool real = r < p.m;
#pragma unroll
        for (int j = 0; j < NF; j += 2) {
            float v[8];
            eight(acc[i][j], acc[i][j + 1], v);         // every lane takes part
            const int c = c_at + j * 16 + eight_at(lane);
            if (r >= p.ld_m || c >= p.ld_m) continue;
            f16x8 w;
            if constexpr (OP == kGram) {
                const float s = kGramScale / (p.scale * p.scale);
#pragma unroll
                for (int q = 0; q < 8; ++q) w[q] = (_Float16)(v[q] * s);
            } else {
                f16x8 old = {0, 0, 0, 0, 0, 0, 0, 0};
                if (real) old = *(const f16x8*)(g + (int64_t)r * p.ld_m + c);
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    w[q] = (_Float16)(a.b * (float)old[q] + a.c * (v[q] * (1.0f / kGramScale)) +
                                      (c + q == r && real ? k * kGramScale : 0.0f));
            }
            if (real) *(f16x8*)(out + (int64_t)r * p.ld_m + c) = w;
            if (mirror)
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    if (c + q < p.m) out[(int64_t)(c + q) * p.ld_m + r] = w[q];
        }
    }
}

// The next X's tile, or the results'.  The sums go through LDS (the wave's own
// part of it), 32 rows at a time, so that a load or store covers whole lines of
// several rows (the last product of 8 matrices of 7168 x 2048, bf16 copies: 723 us;
// 810 with 64 bytes of 16 rows each).  What it moves is not hidden: the compute
// units reach it together, and the next tile's loads wait for the stores (16
// matrices of 2048 x 7168, the next X: 1127 us, 769 without memory, 840 without
// the stores alone).
template <int OP, int MF, int NF>
__device__ __forceinline__ void finish_update(const GroupArgs& a, const Problem& p, int mat, int r_at, int c_at, int lane, float k,
                                              float* lds, const f32x4 (&acc)[MF][NF]) {
    constexpr int kPieces = NF * 2, kRowsAt = kWave / kPieces, kBatch = 32 / kRowsAt;      // pieces of 8 values of a row
    constexpr int kLine = NF * 16 + 4;          // 4 more spread the rows over the banks
    static_assert(MF % 2 == 0 && NF % 2 == 0, "32 rows");
    const _Float16* const hi = p.hi(a.turn) + mat * p.x_size();
    _Float16* const lo = p.lo() + mat * p.x_size();
    const int64_t result = (int64_t)mat * p.m * p.n;
    const bool even = p.even() && p.even_rows();
    const int x = lane % kPieces * 8, c = c_at + x;
    // a wave's LDS accesses keep their order; the fence is for the compiler
    auto fence = [] {
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    };
#pragma unroll
    for (int b = 0; b < MF; b += 2) {
        const int r0 = r_at + b * 16 + lane / kPieces;
        f16x8 h[kBatch], l[kBatch];
        float old[kBatch][8];
#pragma unroll
        for (int t = 0; t < kBatch; ++t) {
            const int r = r0 + t * kRowsAt;
            h[t] = l[t] = f16x8{0, 0, 0, 0, 0, 0, 0, 0};
            if (r < p.m && c < p.ld_n) {
                h[t] = *(const f16x8*)(hi + (int64_t)r * p.ld_n + c);
                l[t] = *(const f16x8*)(lo + (int64_t)r * p.ld_n + c);
                if (OP == kLast && p.momentum && c < p.n)
                    load8(a.param_bf16, p.param, result + (int64_t)r * p.n + c, even, p.n - c, old[t]);
            }
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < NF; ++j)
                *(f32x4*)(lds + (i * 16 + (lane & 15)) * kLine + j * 16 + (lane >> 4) * 4) = acc[b + i][j];
        fence();
        float v[kBatch][8];
#pragma unroll
        for (int t = 0; t < kBatch; ++t) {
            const float* const from = lds + (t * kRowsAt + lane / kPieces) * kLine + x;
            const f32x4 s0 = *(const f32x4*)from, s1 = *(const f32x4*)(from + 4);
#pragma unroll
            for (int q = 0; q < 8; ++q)
                v[t][q] = (a.a - k) * ((float)h[t][q] + (float)l[t][q] * (1.0f / kLow)) + (q < 4 ? s0[q] : s1[q - 4]) * (1.0f / kGramScale);
        }
        fence();
        if constexpr (OP == kLastTall) {
            // [column][row]
#pragma unroll
            for (int t = 0; t < kBatch; ++t)
#pragma unroll
                for (int q = 0; q < 8; ++q) lds[(x + q) * kTurnRow + t * kRowsAt + lane / kPieces] = v[t][q];
            fence();
            const int y = lane % 4 * 8, r = r_at + b * 16 + y;
#pragma unroll
            for (int x0 = 0; x0 < NF * 16; x0 += kWave / 4) {
                const int column = x0 + lane / 4;
                const f32x4 s0 = *(const f32x4*)(lds + column * kTurnRow + y), s1 = *(const f32x4*)(lds + column * kTurnRow + y + 4);
                float w[8] = {s0[0], s0[1], s0[2], s0[3], s1[0], s1[1], s1[2], s1[3]}, before[8] = {};
                if (r < p.m && c_at + column < p.n) {
                    const int64_t at = result + (int64_t)(c_at + column) * p.m + r;
                    if (p.momentum) load8(a.param_bf16, p.param, at, even, p.m - r, before);
                    write_results(a, p, at, even, p.m - r, before, w);
                }
            }
            fence();
        } else {
#pragma unroll
            for (int t = 0; t < kBatch; ++t) {
                const int r = r0 + t * kRowsAt;
                if constexpr (OP == kNext) {
                    if (r >= p.m || c >= p.ld_n) continue;
                    f16x8 nh, nl;
                    split8(v[t], nh, nl);
                    const int64_t at = (int64_t)r * p.ld_n + c;
                    *(f16x8*)(p.hi(a.turn ^ 1) + mat * p.x_size() + at) = nh;
                    *(f16x8*)(lo + at) = nl;
                } else {
                    if (r >= p.m || c >= p.n) continue;
                    write_results(a, p, result + (int64_t)r * p.n + c, even, p.n - c, old[t], v[t]);
                }
            }
        }
    }
}

template <class S>
__global__ void __launch_bounds__(S::kThreads) muon_gemm_kernel(GroupArgs a) {
    extern __shared__ __attribute__((aligned(1024))) char smem[];
    constexpr int OP = S::OP, BM = S::BM, BN = S::BN, WM = S::WM, WN = S::WN;
    lds_char* lds = (lds_char*)smem;
    const int tid = threadIdx.x, lane = tid & 63, wave = uni(tid >> 6), block = blockIdx.x, G = gridDim.x;
    // Workgroup b runs on XCD b mod 8: consecutive tiles, which share rows and
    // columns, go to one XCD and its L2.
    const int first = (G % kXcds == 0) ? (block % kXcds) * (G / kXcds) + block / kXcds : block;
    const int total = a.first[a.count];
    for (int t = first; t < total; t += G) {
        const int i = uni(find_problem(a, t));
        const Problem& p = a.p[i];
        const int per = (int)tiles_of<BM, BN>(OP, p.m, p.ld_n), local = t - a.first[i];
        const int mat = p.begin + local / per, in = local % per;
        int mt, nt;
        if constexpr (is_update(OP)) {
            const int tiles_m = (p.m + BM - 1) / BM, tiles_n = (p.ld_n + BN - 1) / BN;
            const int grp = in / (kGroupM * tiles_n), rest = in - grp * kGroupM * tiles_n;
            const int rows = tiles_m - grp * kGroupM < kGroupM ? tiles_m - grp * kGroupM : kGroupM;
            nt = rest / rows;
            mt = grp * kGroupM + rest - nt * rows;
        } else {
            // the largest mt with mt (mt + 1) / 2 <= in
            mt = (int)((sqrtf(8.0f * (float)in + 1.0f) - 1.0f) * 0.5f);
            while (mt * (mt + 1) / 2 > in) --mt;
            while ((mt + 1) * (mt + 2) / 2 <= in) ++mt;
            nt = in - mt * (mt + 1) / 2;
        }
        mt = uni(mt);
        nt = uni(nt);
        const int m0 = mt * BM, n0 = nt * BN;
        const int K = OP == kGram ? p.ld_n : p.m;
        const _Float16* const x = p.hi(a.turn) + mat * p.x_size();
        const _Float16* const left = OP == kGram ? x : (OP == kPoly ? p.g() : p.p()) + mat * p.g_size();
        const _Float16* const right = OP == kPoly ? left : x;
        const uint32_t a_ld = (uint32_t)(OP == kGram ? p.ld_n : p.ld_m) * 2, b_ld = (uint32_t)(OP == kPoly ? p.ld_m : p.ld_n) * 2;
        typename S::A la;
        typename S::B lb;
        // rows and columns past the matrix are out of the buffers' range: zeros
        la.init(left + (int64_t)m0 * (a_ld / 2), a_ld, wave, lane, [&](int r) { return m0 + r < p.m ? (uint32_t)r * a_ld : kOutOfRange; });
        if constexpr (is_update(OP))
            lb.init(right, b_ld, wave, lane,
                    [&](int c) { return n0 / 8 + c < p.ld_n / 8 ? (uint32_t)(n0 / 8 + c) * 16u : kOutOfRange; });
        else
            lb.init(right + (int64_t)n0 * (b_ld / 2), b_ld, wave, lane,
                    [&](int r) { return n0 + r < p.m ? (uint32_t)r * b_ld : kOutOfRange; });
        // the last tile's reads are done before its LDS is filled again
        wait_loads<0>();
        __builtin_amdgcn_s_barrier();
        constexpr int kAcross = BN / WN;
        const int r = wave / kAcross * WM, c = wave % kAcross * WN;
        auto done = [&](const f32x4 (&acc)[WM / 16][WN / 16]) {
            float k = 0.0f;
            if (OP != kGram && a.shifted) {
                k = OP == kPoly ? shift_of(a, p, mat, lane) : p.shift(mat);
                if (OP == kPoly && in == 0 && tid == 0) p.shift(mat) = k;
            }
            if constexpr (is_update(OP)) {
                // the tiles in LDS are done with, and zeros past the last one have arrived
                wait_loads<0>();
                __builtin_amdgcn_s_barrier();
                static_assert(sizeof(float) * WN * kTurnRow <= S::kLds / S::kWaves && sizeof(float) * 32 * (WN + 4) <= S::kLds / S::kWaves,
                              "LDS of a wave");
                float* const own = (float*)smem + wave * (int)(S::kLds / S::kWaves / sizeof(float));
                finish_update<OP, WM / 16, WN / 16>(a, p, mat, m0 + r, n0 + c, lane, k, own, acc);
            } else {
                finish_square<OP, WM / 16, WN / 16>(a, p, mat, m0 + r, n0 + c, mt != nt, lane, k, acc);
            }
        };
        if constexpr (S::kPipelined) pipelined_tile<S, WM / 16, WN / 16>(la, lb, K, r, c, wave, lane, lds, done);
        else plain_tile<S>(la, lb, K, r, c, wave, lane, lds, done);
    }
    wait_loads<0>();        // no load into LDS outlives the workgroup
}

template <int OP> using Wide = Shape<OP, 256, 256, 128, 64, 2, true>;
template <int OP> using Middle = Shape<OP, 128, 128, 64, 64, 2, false>;
template <int OP> using Small = Shape<OP, 64, 64, 32, 32, 4, false>;

template <class S>
int64_t set_tiles(GroupArgs& a) {
    int64_t total = 0;
    for (int i = 0; i < a.count; ++i) {
        a.first[i] = (int32_t)total;
        total += a.p[i].mats * tiles_of<S::BM, S::BN>(S::OP, a.p[i].m, a.p[i].ld_n);
    }
    a.first[a.count] = (int32_t)total;
    return total;
}

// Where a call runs.
struct Place {
    int device, num_cu;
    hipStream_t stream;
};

template <class S>
hipError_t launch_shape(GroupArgs& a, const Place& at) {
    const int64_t tiles = set_tiles<S>(a), most = (int64_t)at.num_cu * (int64_t)(kLdsBytes / S::kLds);
    if (tiles == 0) return hipSuccess;
    static std::atomic<uint64_t> allowed{0};            // devices that know of the LDS
    const uint64_t bit = at.device < 64 ? (uint64_t)1 << at.device : 0;
    if (!(allowed.load(std::memory_order_relaxed) & bit)) {
        const hipError_t e = hipFuncSetAttribute((const void*)muon_gemm_kernel<S>, hipFuncAttributeMaxDynamicSharedMemorySize, (int)S::kLds);
        if (e != hipSuccess) return e;
        allowed.fetch_or(bit, std::memory_order_relaxed);
    }
    muon_gemm_kernel<S><<<(int)(tiles < most ? tiles : most), S::kThreads, S::kLds, at.stream>>>(a);
    return hipGetLastError();
}

template <int OP>
hipError_t launch_product(GroupArgs& a, const Place& at) {
    MuonSizes sizes[kProblems];
    for (int i = 0; i < a.count; ++i) sizes[i] = {a.p[i].m, a.p[i].ld_n, a.p[i].mats};
    const MuonShape f = muon_shape(OP, a.count, sizes, at.num_cu);
    if (f.small) return launch_shape<Small<OP>>(a, at);
    GroupArgs part = a;
    auto take = [&](bool wide) {
        part.count = 0;
        for (int i = 0; i < a.count; ++i) {
            const int mats = wide ? f.wide_mats[i] : a.p[i].mats - f.wide_mats[i];
            if (mats == 0) continue;
            Problem& q = part.p[part.count++] = a.p[i];
            q.begin += wide ? 0 : f.wide_mats[i];
            q.mats = mats;
        }
    };
    take(true);
    const hipError_t e = launch_shape<Wide<OP>>(part, at);
    if (e != hipSuccess) return e;
    take(false);
    return launch_shape<Middle<OP>>(part, at);
}

// The last products of the wide or of the tall problems.
template <int OP>
hipError_t launch_last(const GroupArgs& a, const Place& at) {
    GroupArgs some = a;
    some.count = 0;
    for (int i = 0; i < a.count; ++i)
        if (a.p[i].tall == (OP == kLastTall)) some.p[some.count++] = a.p[i];
    return some.count ? launch_product<OP>(some, at) : hipSuccess;
}

hipError_t run_group(GroupArgs& a, int steps, const Place& at) {
    int64_t blocks = 0;
    for (int i = 0; i < a.count; ++i) {
        a.first[i] = (int32_t)blocks;
        blocks += (int64_t)a.p[i].batch * a.p[i].partials;
    }
    a.turn = 0;
    muon_sums_kernel<<<(int)blocks, kThreads, 0, at.stream>>>(a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    // fewer units a workgroup where there are few
    int per = 8;
    for (;; per /= 4) {
        blocks = 0;
        for (int i = 0; i < a.count; ++i) {
            a.first[i] = (int32_t)blocks;
            const Problem& p = a.p[i];
            blocks += (int64_t)p.batch * ((split_units(p.m, p.ld_n, p.tall) + per - 1) / per);
        }
        if (per < 4 || blocks >= 4 * at.num_cu) break;
    }
    muon_split_kernel<<<(int)blocks, kThreads, 0, at.stream>>>(a, per);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    for (int s = 0; s < steps; ++s) {
        a.shifted = s + 2 >= steps;
        if ((e = launch_product<kGram>(a, at)) != hipSuccess) return e;
        if ((e = launch_product<kPoly>(a, at)) != hipSuccess) return e;
        if (s + 1 < steps) e = launch_product<kNext>(a, at);
        else if ((e = launch_last<kLast>(a, at)) == hipSuccess) e = launch_last<kLastTall>(a, at);
        if (e != hipSuccess) return e;
        a.turn ^= 1;
    }
    return hipSuccess;
}

int up8(int v) { return (v + 7) / 8 * 8; }

// One matrix of a shape (batch 1).
Problem problem_of(int32_t rows, int32_t cols) {
    Problem p{};
    p.tall = rows > cols;
    p.m = p.tall ? cols : rows;
    p.n = p.tall ? rows : cols;
    p.ld_m = up8(p.m);
    p.ld_n = up8(p.n);
    p.batch = 1;
    const int64_t n = (int64_t)rows * cols, chunks = (n + 8191) / 8192;
    p.partials = (int)(chunks < kPartials ? (chunks + 1) / 2 * 2 : kPartials);      // even: 16 bytes
    p.scale = exp2f(roundf(0.5f * log2f((float)p.n)));
    return p;
}

ep_status check_shape(int64_t batch, int32_t rows, int32_t cols) {
    if (batch < 0 || rows < 0 || cols < 0) return EP_ERR_INVALID_ARGUMENT;
    if (rows > kMaxSide || cols > kMaxSide || (int64_t)rows * cols > kMaxMatrix || batch > (1 << 20)) return EP_ERR_UNSUPPORTED;
    return EP_OK;
}

// What a call would like to have: everything at once up to 4 GiB, and room for
// the largest matrix in any case.
constexpr int64_t kLikedBytes = (int64_t)4 << 30;

struct Shapes {
    int64_t batch;
    int32_t rows, cols;
};

int64_t workspace_of(const std::vector<Shapes>& shapes) {
    int64_t all = 0, largest = 0;
    for (const Shapes& s : shapes) {
        if (s.batch == 0 || s.rows == 0 || s.cols == 0) continue;
        const int64_t each = problem_of(s.rows, s.cols).ws_each();
        largest = each > largest ? each : largest;
        const int64_t room = kLikedBytes - all;
        all += s.batch <= room / each ? s.batch * each : room;
    }
    return all > largest ? all : largest;
}

// Problems put into groups as the workspace and the launches hold them, and run.
struct Runner {
    GroupArgs a{};
    char* ws;
    int64_t bytes, used = 0;
    int64_t blocks = 0;         // of a launch, at most
    int steps;
    Place at;

    hipError_t flush() {
        hipError_t e = a.count ? run_group(a, steps, at) : hipSuccess;
        a.count = 0;
        used = blocks = 0;
        return e;
    }
    // size of param and copy in bytes a value, x as the flags say
    hipError_t add(Problem p, int64_t batch, int64_t x_size, int64_t param_size) {
        const int64_t each = p.ws_each(), n = (int64_t)p.m * p.n;
        const int64_t blocks_each = muon_blocks_of(p.m, p.ld_n, p.partials);
        for (int64_t done = 0; done < batch;) {
            const int64_t fit = muon_fit(bytes - used, each, blocks, blocks_each);
            if (a.count == kProblems || fit < 1) {
                const hipError_t e = flush();
                if (e != hipSuccess) return e;
                continue;
            }
            const int64_t k = batch - done < fit ? batch - done : fit;
            Problem& q = a.p[a.count++] = p;
            q.batch = q.mats = (int32_t)k;
            q.begin = 0;
            q.x = (const char*)p.x + done * n * x_size;
            if (p.momentum) q.momentum = p.momentum + done * n;
            q.param = (char*)p.param + done * n * param_size;
            if (p.copy) q.copy = p.copy + done * n;
            q.ws = ws + used;
            used += k * each;
            blocks += k * blocks_each;
            done += k;
        }
        return hipSuccess;
    }
};

bool here(Place& at) {
    return hipGetDevice(&at.device) == hipSuccess &&
           hipDeviceGetAttribute(&at.num_cu, hipDeviceAttributeMultiprocessorCount, at.device) == hipSuccess && at.num_cu > 0;
}

bool fine(const double (&c)[3]) { return std::isfinite(c[0]) && std::isfinite(c[1]) && std::isfinite(c[2]); }

}  // namespace
}  // namespace epk

extern "C" {

int64_t ep_muon_workspace_bytes(const ep_muon_tensor* tensors, int32_t count) {
    using namespace epk;
    if (count < 0 || (count > 0 && !tensors)) return -1;
    try {
        std::vector<Shapes> shapes;
        shapes.reserve((size_t)count);
        for (int32_t i = 0; i < count; ++i) {
            if (check_shape(tensors[i].batch, tensors[i].rows, tensors[i].cols) != EP_OK) return -1;
            shapes.push_back({tensors[i].batch, tensors[i].rows, tensors[i].cols});
        }
        return workspace_of(shapes);
    } catch (const std::bad_alloc&) {
        return -1;
    }
}

ep_status ep_orthogonalize(const void* x, int64_t batch, int32_t rows, int32_t cols, int32_t steps,
                           const double coefficients[3], double eps, uint32_t flags, void* workspace,
                           int64_t workspace_bytes, void* out, hipStream_t stream) {
    using namespace epk;
    if (flags & ~EP_MUON_GRAD_BF16) return EP_ERR_INVALID_ARGUMENT;
    const ep_status st = check_shape(batch, rows, cols);
    if (st != EP_OK) return st;
    if (steps < 1 || steps > 100 || !(eps >= 0) || !std::isfinite(eps)) return EP_ERR_INVALID_ARGUMENT;
    double k[3] = {3.4445, -4.775, 2.0315};
    if (coefficients)
        for (int i = 0; i < 3; ++i) k[i] = coefficients[i];
    if (!fine(k)) return EP_ERR_INVALID_ARGUMENT;
    if (batch == 0 || rows == 0 || cols == 0) return EP_OK;
    const bool bf16 = flags & EP_MUON_GRAD_BF16;
    const Problem one = problem_of(rows, cols);
    const int64_t n = batch * rows * cols, xs = bf16 ? 2 : 4;
    if (!x || !out || !workspace || !aligned(x, 16) || !aligned(out, 16) || !aligned(workspace, 16) ||
        workspace_bytes < one.ws_each())
        return EP_ERR_INVALID_ARGUMENT;
    const Rows rx(x, n, n, 1, (int)xs), ro(out, n, n, 1, 2), rw(workspace, workspace_bytes, workspace_bytes, 1, 1);
    if (share(rx, ro) || share(rx, rw) || share(ro, rw)) return EP_ERR_INVALID_ARGUMENT;
    Runner run;
    run.ws = (char*)workspace;
    run.bytes = workspace_bytes;
    run.steps = steps;
    run.at.stream = stream;
    if (!here(run.at)) return EP_ERR_HIP;
    run.a.x_bf16 = bf16;
    run.a.a = (float)k[0];
    run.a.b = (float)k[1];
    run.a.c = (float)k[2];
    run.a.eps = (float)eps;
    Problem p = one;
    p.x = x;
    p.param = out;
    if (run.add(p, batch, xs, 2) != hipSuccess || run.flush() != hipSuccess) return EP_ERR_HIP;
    return EP_OK;
}

ep_status ep_muon(const ep_muon_tensor* tensors, int32_t count, const ep_muon_config* cfg, void* workspace,
                  int64_t workspace_bytes, hipStream_t stream) {
    using namespace epk;
    if (!cfg || count < 0 || (count > 0 && !tensors)) return EP_ERR_INVALID_ARGUMENT;
    if (cfg->flags & ~(EP_MUON_PARAM_BF16 | EP_MUON_GRAD_BF16 | EP_MUON_NESTEROV)) return EP_ERR_INVALID_ARGUMENT;
    const double k[3] = {cfg->a, cfg->b, cfg->c};
    if (!(cfg->momentum >= 0 && cfg->momentum < 1 && cfg->eps >= 0 && cfg->scale >= 0) || !std::isfinite(cfg->eps) ||
        !std::isfinite(cfg->scale) || !std::isfinite(cfg->lr) || !std::isfinite(cfg->weight_decay) || !fine(k) || cfg->steps < 1 ||
        cfg->steps > 100)
        return EP_ERR_INVALID_ARGUMENT;
    const bool pb = cfg->flags & EP_MUON_PARAM_BF16, gb = cfg->flags & EP_MUON_GRAD_BF16;
    const int64_t ps = pb ? 2 : 4, gs = gb ? 2 : 4;
    auto none = [](const ep_muon_tensor& t) { return t.batch == 0 || t.rows == 0 || t.cols == 0; };
    bool any = false;
    try {
        std::vector<Range> ranges;
        ranges.reserve((size_t)count * 4 + 1);
        auto put = [&](const void* p, int64_t n, bool w) {
            if (p) ranges.push_back({(uintptr_t)p, (uintptr_t)p + (uintptr_t)n, w});
        };
        for (int32_t i = 0; i < count; ++i) {
            const ep_muon_tensor& t = tensors[i];
            const ep_status st = check_shape(t.batch, t.rows, t.cols);
            if (st != EP_OK) return st;
            if (t.copy && pb) return EP_ERR_UNSUPPORTED;        // bf16 parameters are their own copy
            if (none(t)) continue;
            any = true;
            if (!t.param || !t.grad || !t.momentum || !aligned(t.param, 16) || !aligned(t.grad, 16) ||
                !aligned(t.momentum, 16) || !aligned(t.copy, 16) || workspace_bytes < problem_of(t.rows, t.cols).ws_each())
                return EP_ERR_INVALID_ARGUMENT;
            const int64_t n = t.batch * t.rows * t.cols;
            put(t.param, n * ps, true);
            put(t.grad, n * gs, false);
            put(t.momentum, n * 4, true);
            put(t.copy, n * 2, true);
        }
        if (!any) return EP_OK;
        if (!workspace || !aligned(workspace, 16)) return EP_ERR_INVALID_ARGUMENT;
        put(workspace, workspace_bytes, true);
        std::sort(ranges.begin(), ranges.end());
        if (shared(ranges)) return EP_ERR_INVALID_ARGUMENT;
    } catch (const std::bad_alloc&) {
        return EP_ERR_OUT_OF_MEMORY;
    }
    Runner run;
    run.ws = (char*)workspace;
    run.bytes = workspace_bytes;
    run.steps = cfg->steps;
    run.at.stream = stream;
    if (!here(run.at)) return EP_ERR_HIP;
    GroupArgs& a = run.a;
    a.x_bf16 = gb;
    a.param_bf16 = pb;
    a.nesterov = (cfg->flags & EP_MUON_NESTEROV) != 0;
    a.a = (float)cfg->a;
    a.b = (float)cfg->b;
    a.c = (float)cfg->c;
    a.mu = (float)cfg->momentum;
    a.rest_mu = (float)(1.0 - cfg->momentum);
    a.eps = (float)cfg->eps;
    a.decay = (float)(1.0 - cfg->lr * cfg->weight_decay);
    for (int32_t i = 0; i < count; ++i) {
        const ep_muon_tensor& t = tensors[i];
        if (none(t)) continue;
        Problem p = problem_of(t.rows, t.cols);
        p.x = t.grad;
        p.momentum = t.momentum;
        p.param = t.param;
        p.copy = (__bf16*)t.copy;
        p.step = (float)(cfg->lr * (cfg->scale > 0 ? cfg->scale : 0.2 * sqrt((double)p.n)));
        if (run.add(p, t.batch, gs, ps) != hipSuccess) return EP_ERR_HIP;
    }
    return run.flush() == hipSuccess ? EP_OK : EP_ERR_HIP;
}

}  // extern "C"
