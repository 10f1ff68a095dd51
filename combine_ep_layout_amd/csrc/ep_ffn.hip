// gfx950 kernels of the experts' gated feed-forward over the dispatched pool,
// and of its backward pass.
//
// For a real pool row x of expert e (I = intermediate size):
//     g = x Wg^T,  u = x Wu^T,  a = act(g) * u,  o = a Wd^T
// and, for the gradient do of o,
//     da = do Wd,  dg = da * u * act'(g),  du = da * act(g)
//     dx = dg Wg + du Wu,  dWg = dg^T x,  dWu = du^T x,  dWd = do^T a
// summed over the rows of the expert.  These are six products over the
// experts' row regions, so one kernel serves them all, a grouped matrix
// product on the matrix cores (16x16x32 bf16, fp32 sums): it differs in which
// operands have the summed index contiguous in memory and in what it does
// with the finished tile (the activation and the product, their derivatives,
// or a rounding).
//
// a, dg and du are rounded to bf16, once each: they are operands of the next
// products, whose matrix instructions take bf16 (in fp32 the rate would be a
// sixteenth).  With independent roundings of at most half a step, 2^-8, that
// makes results 2.3e-3 of their norm off where one rounding alone makes 1.7e-3.
// g and u stay fp32, since nothing multiplies them on the matrix cores.
//
// Operands go from memory straight into LDS (16 bytes a lane, no registers),
// ST tiles of 32 or 64 summed indices deep.  Where the summed index is contiguous a
// fragment is one ds_read_b128; where it is not, the tile keeps the memory's
// order and two transposing reads (ds_read_b64_tr_b16) make the fragment, so
// no operand is transposed in memory.  Both layouts are swizzled by permuting
// which 16 bytes a lane fetches, since the load itself fills LDS linearly
// (SQ_LDS_BANK_CONFLICT counts none in any product).
//
// What bounds it, measured on MI355X at 32 experts of 2048 rows, 7168 x 2048:
// 1.05 (gradient of the activation) to 1.31 PFLOP/s (pool gradient).  By the
// counters the matrix cores are busy in 48-63 % of the cycles, at 1.9-2.0 GHz,
// and a compute unit reads 17-21 bytes a cycle out of L2.  In variants with the
// rest left out, a 256 x 256 tile's matrix instructions run at 1.95 PFLOP/s, with
// the LDS reads at 1.64-1.76, and the loads (64 KiB for 64 summed indices) keep
// pace with 1.95-2.1, 26 bytes a cycle.  So both need most of the time, and two
// tiles in LDS hide only part of a load's latency.  Few rows are bound by the
// weights' bytes instead: 5.7-5.8 TB/s.
#include <hip/hip_runtime.h>
#include <stdint.h>
#include <utility>

#include "ep_act.h"
#include "ep_ffn.h"
#include "ep_ffn_shape.h"
#include "ep_gemm.h"

namespace epk {
namespace {


constexpr int kMaxExperts = 1024;
constexpr int kGroupM = 8;                  // row tiles that share their column tiles' loads

constexpr bool a_strided(int op) { return op == kWeightGrad; }
constexpr bool b_strided(int op) { return op == kActGrad || op == kRowGrad || op == kWeightGrad; }

__device__ __forceinline__ bf16x4 round4(const f32x4& v) {
    bf16x4 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = (__bf16)v[i];
    return r;
}

// BM x BN tiles, WM x WN of it to each wave, ST LDS tiles of each operand, BK
// summed indices deep.
template <int OP_, int BM_, int BN_, int WM_, int WN_, int BK_, int ST_, bool PIPELINED = false>
struct Shape {
    static constexpr int OP = OP_, BM = BM_, BN = BN_, WM = WM_, WN = WN_, BK = BK_, ST = ST_;
    static constexpr int kWaves = (BM / WM) * (BN / WN);
    static constexpr int kThreads = kWaves * kWave;
    static constexpr int kStageBytes = (BM + BN) * BK * 2;
    static constexpr int kCols = OP == kUp ? BN / 2 : BN;       // output columns of a tile
    // kUp: gate columns and then their up columns, in groups of this many
    static constexpr int kPair = 32;
    static constexpr bool kPipelined = PIPELINED;
    static constexpr bool kAStrided = a_strided(OP), kBStrided = b_strided(OP), kF16 = false;
    using A = Loader<BM, BK, a_strided(OP), kWaves>;
    using B = Loader<BN, BK, b_strided(OP), kWaves>;
    static constexpr int kLoads = A::kLoads + B::kLoads;
    static constexpr size_t kTileLds = (size_t)ST * kStageBytes;
    // the scan of the row tiles follows the operands' tiles
    static size_t lds(int E) { return kTileLds + (OP == kWeightGrad ? 0 : (size_t)(E + 1) * sizeof(int)); }
};

// One tile of one expert.
struct Tile {
    int e, cnt, m0, n0;
    int64_t region;             // the expert's first pool row
};

// A row's values of a fragment pair, columns c0.. of the first and c1.. of the
// second (16 each), rounded to bf16.  Lane l holds row l % 16 and columns
// 4 (l / 16) + 0..3; the lanes of odd rows of 16 trade their first half for the
// even ones' second, so that each stores 16 bytes.
__device__ __forceinline__ void store_pair(__bf16* out, int c0, int c1, int cols, int lane, const f32x4& v0, const f32x4& v1) {
    union { bf16x4 h[2]; uint32_t w[4]; i32x4 q; } x;
    x.h[0] = round4(v0);
    x.h[1] = round4(v1);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const auto r = __builtin_amdgcn_permlane16_swap(x.w[i], x.w[2 + i], false, false);
        x.w[i] = r[0];
        x.w[2 + i] = r[1];
    }
    const int c = ((lane & 16) ? c1 : c0) + (lane >> 5) * 8;
    if (c < cols) *(i32x4*)(out + c) = x.q;
}
__device__ __forceinline__ void store_one(__bf16* out, int c, int cols, const f32x4& v) {
    if (c < cols) *(bf16x4*)(out + c) = round4(v);
}

// Writes a wave's part of the finished tile: rows from r_at, tile columns from c_at.
template <class S, int MF, int NF>
__device__ __forceinline__ void finish(const GemmArgs& p, const Tile& t, int r_at, int c_at, int lane,
                                       const f32x4 (&acc)[MF][NF]) {
    constexpr int OP = S::OP;
    const int r0 = t.m0 + r_at + (lane & 15), c_in = (lane >> 4) * 4;
    const int rows = OP == kWeightGrad ? p.M : t.cnt;
#pragma unroll
    for (int i = 0; i < MF; ++i) {
        const int r = r0 + i * 16;
        // lanes of a row past the end take part in the exchange, but not in the stores
        const int cols = r < rows ? p.N : 0;
        if constexpr (OP == kUp) {
            // fragments j, j + 1: 16 gate columns and their up columns
            __bf16* out = (__bf16*)p.c + (t.region + r) * (int64_t)p.N;
            f32x4 v[NF / 2];
#pragma unroll
            for (int j = 0; j < NF / 2; ++j)
#pragma unroll
                for (int q = 0; q < 4; ++q) v[j][q] = act_value(acc[i][2 * j][q], p.act) * acc[i][2 * j + 1][q];
            const int c = t.n0 + (c_at >> 1);
            if constexpr (NF == 2) {
                store_one(out, c + c_in, cols, v[0]);
            } else {
#pragma unroll
                for (int j = 0; j < NF / 2; j += 2) store_pair(out, c + j * 16, c + j * 16 + 16, cols, lane, v[j], v[j + 1]);
            }
            if (p.save) {
                float* save = (float*)p.save + (t.region + r) * (int64_t)(2 * p.N);
#pragma unroll
                for (int j = 0; j < NF / 2; ++j)
                    if (c + j * 16 + c_in < cols) {
                        *(f32x4*)(save + c + j * 16 + c_in) = acc[i][2 * j];
                        *(f32x4*)(save + p.N + c + j * 16 + c_in) = acc[i][2 * j + 1];
                    }
            }
        } else if constexpr (OP == kActGrad) {
            const float* saved = (const float*)p.save + (t.region + r) * (int64_t)(2 * p.N);
            __bf16* out = (__bf16*)p.c + (t.region + r) * (int64_t)(2 * p.N);
            f32x4 dg[NF], du[NF];
#pragma unroll
            for (int j = 0; j < NF; ++j) {
                const int c = t.n0 + c_at + j * 16 + c_in;
                f32x4 g{0.f, 0.f, 0.f, 0.f}, u = g;
                if (c < cols) {
                    g = *(const f32x4*)(saved + c);
                    u = *(const f32x4*)(saved + p.N + c);
                }
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    float value, slope;
                    act_both(g[q], p.act, value, slope);
                    dg[j][q] = acc[i][j][q] * u[q] * slope;
                    du[j][q] = acc[i][j][q] * value;
                }
            }
#pragma unroll
            for (int j = 0; j < NF; j += 2) {
                const int c = t.n0 + c_at + j * 16;
                store_pair(out, c, c + 16, cols, lane, dg[j], dg[j + 1]);
                store_pair(out + p.N, c, c + 16, cols, lane, du[j], du[j + 1]);
            }
        } else {
            const int64_t at = OP == kWeightGrad ? ((int64_t)t.e * p.M + r) * p.N : (t.region + r) * (int64_t)p.N;
            if (OP == kWeightGrad && p.out_f32) {
#pragma unroll
                for (int j = 0; j < NF; ++j) {
                    const int c = t.n0 + c_at + j * 16 + c_in;
                    if (c >= cols) continue;
                    f32x4* o = (f32x4*)((float*)p.c + at + c);
                    f32x4 v = acc[i][j];
                    if (p.accumulate) {
                        const f32x4 old = *o;
#pragma unroll
                        for (int q = 0; q < 4; ++q) v[q] += old[q];
                    }
                    *o = v;
                }
            } else {
#pragma unroll
                for (int j = 0; j < NF; j += 2)
                    store_pair((__bf16*)p.c + at, t.n0 + c_at + j * 16, t.n0 + c_at + j * 16 + 16, cols, lane, acc[i][j], acc[i][j + 1]);
            }
        }
    }
}

// All tiles of a product that fall to workgroup `block` of G.
template <class S>
__device__ __forceinline__ void run_product(const GemmArgs& p, int block, int G, char* smem) {
    constexpr int OP = S::OP, BM = S::BM, BN = S::BN, WM = S::WM, WN = S::WN;
    constexpr bool BS = b_strided(OP);
    lds_char* lds = (lds_char*)smem;
    int* s_pref = (int*)(smem + S::ST * S::kStageBytes);
    const int tid = threadIdx.x, lane = tid & 63, wave = uni(tid >> 6);
    const int tiles_n = (p.N + S::kCols - 1) / S::kCols;

    int total;
    if constexpr (OP == kWeightGrad) {
        total = p.E * ((p.M + BM - 1) / BM) * tiles_n;
    } else {
        // row tiles before each expert: an exclusive scan of its rows' tiles
        for (int e = tid; e < p.E; e += S::kThreads) s_pref[e + 1] = (p.counts[e] + BM - 1) / BM;
        if (tid == 0) s_pref[0] = 0;
        __syncthreads();
        if (wave == 0) {
            int sum = 0;
            const int per = (p.E + kWave - 1) / kWave;
#pragma unroll 1
            for (int i = 0; i < per; ++i) {
                const int e = lane * per + i;
                sum += e < p.E ? s_pref[e + 1] : 0;
            }
            int incl = sum;
            for (int d = 1; d < kWave; d <<= 1) {
                const int o = __shfl_up(incl, d);
                if (lane >= d) incl += o;
            }
            int run = incl - sum;
#pragma unroll 1
            for (int i = 0; i < per; ++i) {
                const int e = lane * per + i;
                if (e < p.E) {
                    run += s_pref[e + 1];
                    s_pref[e + 1] = run;
                }
            }
        }
        __syncthreads();
        total = uni(s_pref[p.E]) * tiles_n;
    }

    // Workgroup b runs on XCD b mod 8: consecutive tiles, which share rows and
    // columns, go to one XCD and its L2.
    const int per_xcd = G / kXcds;
    const int first = (G % kXcds == 0) ? (block % kXcds) * per_xcd + block / kXcds : block;

    for (int n = first; n < total; n += G) {
        Tile t;
        int mt, nt;
        {
            int local, tiles_m;
            if constexpr (OP == kWeightGrad) {
                tiles_m = (p.M + BM - 1) / BM;
                t.e = n / (tiles_m * tiles_n);
                local = n - t.e * tiles_m * tiles_n;
            } else {
                const int key = n / tiles_n;
                int lo = 0, hi = p.E;               // s_pref[lo] <= key < s_pref[hi]
                while (hi - lo > 1) {
                    const int mid = (lo + hi) >> 1;
                    if (s_pref[mid] <= key) lo = mid;
                    else hi = mid;
                }
                t.e = uni(lo);
                const int before = uni(s_pref[t.e]);
                tiles_m = uni(s_pref[t.e + 1]) - before;
                local = n - before * tiles_n;
            }
            const int grp = local / (kGroupM * tiles_n);
            const int in = local - grp * kGroupM * tiles_n;
            const int rows = tiles_m - grp * kGroupM < kGroupM ? tiles_m - grp * kGroupM : kGroupM;
            nt = in / rows;
            mt = grp * kGroupM + in - nt * rows;
        }
        t.cnt = uni(p.counts[t.e]);
        t.region = (int64_t)uni(p.offsets[t.e]) * p.block_m;
        t.m0 = mt * BM;
        t.n0 = nt * S::kCols;
        const int K = OP == kWeightGrad ? t.cnt : p.K;

        typename S::A la;
        typename S::B lb;
        const uint32_t a_ldb = (uint32_t)p.a_ld * 2, b_ldb = (uint32_t)p.b_ld * 2;
        // Rows past the region and columns past the matrix are out of the
        // buffers' range: zeros that cost no bytes, and that are not stored.
        auto chunk = [](int c, int n) { return c < (n >> 3) ? (uint32_t)c * 16u : kOutOfRange; };
        if constexpr (OP == kWeightGrad) {
            la.init((const char*)p.a + t.region * a_ldb, a_ldb, wave, lane, [&](int c) { return chunk((t.m0 >> 3) + c, p.M); });
            lb.init((const char*)p.b + t.region * b_ldb, b_ldb, wave, lane, [&](int c) { return chunk((t.n0 >> 3) + c, p.N); });
        } else {
            const int left = t.cnt - t.m0;
            la.init((const char*)p.a + (t.region + t.m0) * a_ldb, a_ldb, wave, lane,
                    [&](int r) { return r < left ? (uint32_t)r * a_ldb : kOutOfRange; });
            const char* b = (const char*)p.b + (int64_t)t.e * p.b_expert * 2;
            if constexpr (OP == kUp) {
                lb.init(b, b_ldb, wave, lane, [&](int r) {
                    constexpr int P = S::kPair;
                    const int j = r % P, up = j >= P / 2;
                    const int c = t.n0 + r / P * (P / 2) + j % (P / 2);
                    return c < p.N ? (uint32_t)(up ? p.N + c : c) * b_ldb : kOutOfRange;
                });
            } else if constexpr (!BS) {
                lb.init(b, b_ldb, wave, lane, [&](int r) { return t.n0 + r < p.N ? (uint32_t)(t.n0 + r) * b_ldb : kOutOfRange; });
            } else {
                lb.init(b, b_ldb, wave, lane, [&](int c) { return chunk((t.n0 >> 3) + c, p.N); });
            }
        }

        // the last tile's reads are done before its LDS is filled again
        wait_loads<0>();
        __builtin_amdgcn_s_barrier();
        constexpr int kAcross = BN / WN;
        const int r = wave / kAcross * WM, c = wave % kAcross * WN;
        auto whole = [&](const f32x4 (&acc)[WM / 16][WN / 16]) { finish<S, WM / 16, WN / 16>(p, t, r, c, lane, acc); };
        if constexpr (S::kPipelined) {
            static_assert(BM == 2 * WM, "two rows of waves");
            // a tile whose lower half or three quarters have no rows is shared
            // out by columns alone
            if (OP != kWeightGrad && t.cnt - t.m0 <= WM / 2) {
                const int c = wave * (WN / 2);
                pipelined_tile<S, WM / 32, WN / 32>(la, lb, K, 0, c, wave, lane, lds, [&](const f32x4 (&acc)[WM / 32][WN / 32]) {
                    finish<S, WM / 32, WN / 32>(p, t, 0, c, lane, acc);
                });
            } else if (OP != kWeightGrad && t.cnt - t.m0 <= WM) {
                const int c = wave * (WN / 2);
                pipelined_tile<S, WM / 16, WN / 32>(la, lb, K, 0, c, wave, lane, lds, [&](const f32x4 (&acc)[WM / 16][WN / 32]) {
                    finish<S, WM / 16, WN / 32>(p, t, 0, c, lane, acc);
                });
            } else {
                pipelined_tile<S, WM / 16, WN / 16>(la, lb, K, r, c, wave, lane, lds, whole);
            }
        } else {
            plain_tile<S>(la, lb, K, r, c, wave, lane, lds, whole);
        }
    }
    wait_loads<0>();        // no load into LDS outlives the workgroup
}

template <class S>
__global__ void __launch_bounds__(S::kThreads) ffn_gemm_kernel(GemmArgs p) {
    extern __shared__ __attribute__((aligned(1024))) char smem[];
    run_product<S>(p, blockIdx.x, gridDim.x, smem);
}

// The three products that follow the activation's gradient, for problems of
// less than a round of tiles each: nothing is gained by their order then, and
// two launches are saved (forward and backward of 8 experts of 256 x 512, 256
// rows: 32 us, 52 with six launches of the larger shapes).
struct AfterArgs {
    GemmArgs rows, gate_up, down;
    int32_t grid_rows, grid_gate_up;        // workgroups of the first two
};
template <class R, class W>
__global__ void __launch_bounds__(R::kThreads) ffn_after_kernel(AfterArgs a) {
    static_assert(R::kThreads == W::kThreads, "one launch");
    extern __shared__ __attribute__((aligned(1024))) char smem[];
    const int b = blockIdx.x, n1 = a.grid_rows, n2 = n1 + a.grid_gate_up;
    if (b < n1) run_product<R>(a.rows, b, n1, smem);
    else if (b < n2) run_product<W>(a.gate_up, b - n1, n2 - n1, smem);
    else run_product<W>(a.down, b - n2, (int)gridDim.x - n2, smem);
}

template <class K>
hipError_t allow_lds(K* kernel, size_t lds) {
    return hipFuncSetAttribute((const void*)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
}

FfnSizes sizes(const GemmArgs& p) { return {p.E, p.slots, p.M, p.N, p.num_cu}; }

template <class S>
int grid_of(const GemmArgs& p) {
    const int64_t tiles = ffn_tile_count((FfnOp)S::OP, {S::BM, S::BN}, sizes(p)), most = (int64_t)p.num_cu * (int64_t)(kLdsBytes / S::lds(p.E));
    return (int)(tiles < most ? tiles : most);
}

template <class S>
hipError_t launch(const GemmArgs& p, hipStream_t stream) {
    const int grid = grid_of<S>(p);
    if (grid == 0) return hipSuccess;
    static_assert(S::kTileLds + (kMaxExperts + 1) * sizeof(int) <= kLdsBytes, "LDS of a compute unit");
    hipError_t e = allow_lds(ffn_gemm_kernel<S>, S::lds(p.E));
    if (e != hipSuccess) return e;
    ffn_gemm_kernel<S><<<grid, S::kThreads, S::lds(p.E), stream>>>(p);
    return hipGetLastError();
}

// The tiles' shapes (ep_ffn_shape.h, with the rule that chooses).
template <int OP, FfnShape KIND, int WM, int WN, int ST, bool PIPELINED = false>
using Tiles = Shape<OP, kFfnTiles[KIND].m, kFfnTiles[KIND].n, WM, WN, 64, ST, PIPELINED>;
template <int OP> using Wide = Tiles<OP, kWide, 128, 64, 2, true>;
template <int OP> using Middle = Tiles<OP, kMiddle, 64, 64, 2>;
template <int OP> using Low = Tiles<OP, kLow, 64, 32, 3>;
template <int OP> using Small = Tiles<OP, kSmall, 32, 32, 4>;
template <int OP> using Few = Tiles<OP, kFew, 16, 32, 4>;

template <int OP>
hipError_t launch_rows(const GemmArgs& p, hipStream_t stream) {
    switch (ffn_rows_shape((FfnOp)OP, sizes(p))) {
        case kWide: return launch<Wide<OP>>(p, stream);
        case kMiddle: return launch<Middle<OP>>(p, stream);
        case kSmall: return launch<Small<OP>>(p, stream);
        case kLow: return launch<Low<OP>>(p, stream);
        default: return launch<Few<OP>>(p, stream);
    }
}

hipError_t launch_weight_grad(const GemmArgs& p, hipStream_t stream) {
    if (ffn_weight_grad_shape(sizes(p)) == kWide) return launch<Wide<kWeightGrad>>(p, stream);
    return launch<Middle<kWeightGrad>>(p, stream);
}

hipError_t launch_after(const GemmArgs& rows, const GemmArgs& gate_up, const GemmArgs& down, hipStream_t stream) {
    using R = Small<kRowGrad>;
    using W = Middle<kWeightGrad>;
    AfterArgs a{rows, gate_up, down, grid_of<R>(rows), grid_of<W>(gate_up)};
    const int grid = a.grid_rows + a.grid_gate_up + grid_of<W>(down);
    const size_t lds = R::lds(rows.E) > W::lds(rows.E) ? R::lds(rows.E) : W::lds(rows.E);
    hipError_t e = allow_lds(ffn_after_kernel<R, W>, lds);
    if (e != hipSuccess) return e;
    ffn_after_kernel<R, W><<<grid, R::kThreads, lds, stream>>>(a);
    return hipGetLastError();
}

GemmArgs rows_of(const FfnArgs& f) {
    GemmArgs p{};
    p.counts = f.counts;
    p.offsets = f.offsets;
    p.E = f.E;
    p.block_m = f.block_m;
    p.slots = f.slots;
    p.num_cu = f.num_cu;
    p.act = f.act;
    return p;
}

}  // namespace

hipError_t launch_ffn(const FfnArgs& f, hipStream_t stream) {
    GemmArgs p = rows_of(f);
    p.a = f.pool;
    p.a_ld = f.H;
    p.b = f.w_gate_up;
    p.b_ld = f.H;
    p.b_expert = (int64_t)2 * f.I * f.H;
    p.c = f.act_rows;
    p.save = f.gate_up;
    p.N = f.I;
    p.K = f.H;
    hipError_t e = launch_rows<kUp>(p, stream);
    if (e != hipSuccess) return e;
    p.a = f.act_rows;
    p.a_ld = f.I;
    p.b = f.w_down;
    p.b_ld = f.I;
    p.b_expert = (int64_t)f.I * f.H;
    p.c = f.out;
    p.save = nullptr;
    p.N = f.H;
    p.K = f.I;
    return launch_rows<kDown>(p, stream);
}

hipError_t launch_ffn_backward(const FfnArgs& f, hipStream_t stream) {
    GemmArgs p = rows_of(f);
    // gradients of gate and up
    p.a = f.grad_out;
    p.a_ld = f.H;
    p.b = f.w_down;
    p.b_ld = f.I;
    p.b_expert = (int64_t)f.I * f.H;
    p.c = f.grad_gate_up;
    p.save = f.gate_up;
    p.N = f.I;
    p.K = f.H;
    hipError_t e = launch_rows<kActGrad>(p, stream);
    if (e != hipSuccess) return e;
    p.save = nullptr;
    GemmArgs rows = p, gate_up = p, down = p;
    rows.a = f.grad_gate_up;
    rows.a_ld = 2 * f.I;
    rows.b = f.w_gate_up;
    rows.b_ld = f.H;
    rows.b_expert = (int64_t)2 * f.I * f.H;
    rows.c = f.grad_pool;
    rows.N = f.H;
    rows.K = 2 * f.I;
    gate_up.a = f.grad_gate_up;
    gate_up.a_ld = 2 * f.I;
    gate_up.b = f.pool;
    gate_up.b_ld = f.H;
    gate_up.c = f.grad_w_gate_up;
    gate_up.M = 2 * f.I;
    gate_up.N = f.H;
    down.a = f.grad_out;
    down.a_ld = f.H;
    down.b = f.act_rows;
    down.b_ld = f.I;
    down.c = f.grad_w_down;
    down.M = f.H;
    down.N = f.I;
    gate_up.out_f32 = down.out_f32 = f.grad_f32;
    gate_up.accumulate = down.accumulate = f.accumulate;
    if (rows.c && gate_up.c && down.c && ffn_after_in_one(sizes(rows), sizes(gate_up), sizes(down)))
        return launch_after(rows, gate_up, down, stream);
    if (rows.c && (e = launch_rows<kRowGrad>(rows, stream)) != hipSuccess) return e;
    if (gate_up.c && (e = launch_weight_grad(gate_up, stream)) != hipSuccess) return e;
    if (down.c) e = launch_weight_grad(down, stream);
    return e;
}

}  // namespace epk
