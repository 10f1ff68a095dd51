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
// Operands go from memory straight into LDS (16 bytes a lane, no registers),
// ST tiles of 64 summed indices deep.  Where the summed index is contiguous a
// fragment is one ds_read_b128; where it is not, the tile keeps the memory's
// order and two transposing reads (ds_read_b64_tr_b16) make the fragment, so
// no operand is transposed in memory.  Both layouts are swizzled by permuting
// which 16 bytes a lane fetches, since the load itself fills LDS linearly.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ep_ffn.h"

namespace epk {
namespace {

typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) char lds_char;

constexpr int kWave = 64;
constexpr int BK = 64;                      // summed indices of one LDS tile
constexpr uint32_t kOutOfRange = 0x80000000u;   // offset past every buffer's range: such a lane loads zeros
constexpr int kMaxExperts = 1024;
constexpr int kXcds = 8;
constexpr int kGroupM = 8;                  // row tiles that share their column tiles' loads

// The products.
enum Op { kUp, kDown, kActGrad, kRowGrad, kWeightGrad };

constexpr bool a_strided(int op) { return op == kWeightGrad; }
constexpr bool b_strided(int op) { return op == kActGrad || op == kRowGrad || op == kWeightGrad; }

__device__ __forceinline__ int uni(int v) { return __builtin_amdgcn_readfirstlane(v); }

// 1 KiB from memory to LDS: lane l's 16 bytes at base + voff to lds + 16 l.
// Not visible to the compiler's wait counting: the pipeline waits by itself.
__device__ __forceinline__ void load_to_lds(uint32_t lds, uint32_t voff, const i32x4& rsrc) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
                 ::"s"(lds), "v"(voff), "s"(rsrc) : "memory");
}

__device__ __forceinline__ i32x4 make_rsrc(const void* base) {
    const uint64_t b = (uint64_t)(uintptr_t)base;
    i32x4 r;
    r[0] = uni((int)(uint32_t)b);
    r[1] = uni((int)(uint32_t)(b >> 32));
    r[2] = 0x7FFFFFFF;
    r[3] = 0x00020000;
    return r;
}

// Waits until at most N of this wave's loads into LDS are in flight and all of
// its LDS reads have returned: what a barrier after it orders.
template <int N>
__device__ __forceinline__ void wait_loads() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(N) : "memory");
}

// Swizzle of a strided tile's row k: which pair of 16-byte chunks (16 columns)
// goes where.  A transposing read touches rows 4h..4h+3 of four row groups 8
// apart, so these bits spread its lanes over the banks.
template <int R>
__device__ __forceinline__ int strided_swizzle(int k) {
    constexpr int mask = (R / 16 < 8 ? R / 16 : 8) - 1;
    return ((k & 3) | ((k >> 1) & 4)) & mask;
}

// Loads of one operand's LDS tile by one wave.
//   STRIDED false: R rows of 64 summed values; true: 64 rows of R columns.
template <int R, bool STRIDED, int WAVES>
struct Loader {
    static constexpr int kTotal = R / 8;                              // 1 KiB loads of a tile
    static constexpr int kLoads = kTotal / WAVES > 0 ? kTotal / WAVES : 1;   // each wave's
    uint32_t voff[kLoads];
    int k[kLoads];              // summed index of the lane's first value inside the tile
    i32x4 rsrc;
    uint64_t base, step;

    __device__ __forceinline__ static int load_index(int wave, int i) {
        // more waves than loads: some repeat another wave's load, to the same place
        return (wave * kLoads + i) % kTotal;
    }
    // row(r): offset in bytes of tile row r (or, STRIDED, of column chunk r of 8)
    template <class F>
    __device__ __forceinline__ void init(const void* p, uint32_t ld_bytes, int wave, int lane, F row) {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int g = load_index(wave, i);
            if constexpr (!STRIDED) {
                const int r = lane >> 3, c = (lane & 7) ^ r;
                voff[i] = row(g * 8 + r) + c * 16;
                k[i] = c * 8;
            } else {
                constexpr int kRows = 512 / R;
                const int kk = g * kRows + lane / (R / 8), c = lane % (R / 8);
                const int src = (((c >> 1) ^ strided_swizzle<R>(kk)) << 1) | (c & 1);
                voff[i] = (uint32_t)kk * ld_bytes + row(src);
                k[i] = kk;
            }
        }
        base = (uint64_t)(uintptr_t)p;
        step = STRIDED ? (uint64_t)ld_bytes * BK : BK * 2;
    }
    // rem: summed indices left from this tile on (may be <= 0: zeros)
    __device__ __forceinline__ void issue(uint32_t lds, int wave, int rem) {
        rsrc = make_rsrc((const void*)(uintptr_t)base);
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
            load_to_lds(uni(lds + load_index(wave, i) * 1024), k[i] < rem ? voff[i] : kOutOfRange, rsrc);
        base += step;
    }
};

// A fragment for the matrix core: 16 rows (or columns) from `at`, summed
// indices 32 s + 8 (lane / 16) + 0..7.
template <int R, bool STRIDED>
__device__ __forceinline__ bf16x8 fragment(lds_char* tile, int at, int s, int lane) {
    if constexpr (!STRIDED) {
        const int r = at + (lane & 15);
        const int c = (s * 4 + (lane >> 4)) ^ (lane & 7);       // at is a multiple of 16
        return *(__attribute__((address_space(3))) bf16x8*)(tile + r * 128 + c * 16);
    } else {
        const int k = s * 32 + (lane >> 4) * 8 + ((lane & 15) >> 2);
        // rows k and k + 4 have the same swizzle
        lds_char* p = tile + k * (R * 2) + (((at >> 4) ^ strided_swizzle<R>(k)) << 5) + (lane & 3) * 8;
        typedef __attribute__((address_space(3))) s16x4* P;
        const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((P)p);
        const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((P)(p + 4 * R * 2));
        union { s16x4 h[2]; bf16x8 v; } u;
        u.h[0] = lo;
        u.h[1] = hi;
        return u.v;
    }
}

// act(g) and act'(g).  Both activations in fp32; exp and the reciprocal are
// the hardware's (about 1 ulp each), the results are rounded to bf16.
__device__ __forceinline__ float sigmoid_f(float x) {
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(x * -1.44269504088896341f));
}
__device__ __forceinline__ float gelu_inner(float g) {
    return 0.7978845608028654f * (g + 0.044715f * g * g * g);
}
__device__ __forceinline__ float act_value(float g, int kind) {
    // the tanh form of gelu: (1 + tanh z) / 2 = sigmoid(2 z)
    return g * sigmoid_f(kind == kActGelu ? 2.0f * gelu_inner(g) : g);
}
__device__ __forceinline__ void act_both(float g, int kind, float& value, float& slope) {
    if (kind == kActGelu) {
        const float s = sigmoid_f(2.0f * gelu_inner(g));
        value = g * s;
        slope = s + 2.0f * g * s * (1.0f - s) * 0.7978845608028654f * (1.0f + 3 * 0.044715f * g * g);
    } else {
        const float s = sigmoid_f(g);
        value = g * s;
        slope = s * (1.0f + g * (1.0f - s));
    }
}

__device__ __forceinline__ bf16x4 round4(const f32x4& v) {
    bf16x4 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = (__bf16)v[i];
    return r;
}

// BM x BN tiles, WM x WN of it to each wave, ST LDS tiles of each operand.
template <int OP, int BM, int BN, int WM, int WN, int ST>
struct Shape {
    static constexpr int kWaves = (BM / WM) * (BN / WN);
    static constexpr int kThreads = kWaves * kWave;
    static constexpr int kStageBytes = (BM + BN) * BK * 2;
    static constexpr int kCols = OP == kUp ? BN / 2 : BN;       // output columns of a tile
    static constexpr size_t lds() { return (size_t)ST * kStageBytes + (kMaxExperts + 1 + 16) * sizeof(int); }
};

template <int OP, int BM, int BN, int WM, int WN, int ST>
__global__ void __launch_bounds__((Shape<OP, BM, BN, WM, WN, ST>::kThreads))
ffn_gemm_kernel(GemmArgs p) {
    using S = Shape<OP, BM, BN, WM, WN, ST>;
    constexpr bool AS = a_strided(OP), BS = b_strided(OP);
    constexpr int MF = WM / 16, NF = WN / 16;
    extern __shared__ __attribute__((aligned(1024))) char smem[];
    lds_char* lds = (lds_char*)smem;
    int* s_pref = (int*)(smem + ST * S::kStageBytes);
    const int tid = threadIdx.x, lane = tid & 63, wave = uni(tid >> 6);
    const int wm = wave / (BN / WN), wn = wave % (BN / WN);
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
    const int G = gridDim.x, per_xcd = G / kXcds;
    const int first = (G % kXcds == 0) ? (blockIdx.x % kXcds) * per_xcd + blockIdx.x / kXcds : blockIdx.x;

    for (int t = first; t < total; t += G) {
        int e, mt, nt;
        {
            int local, tiles_m;
            if constexpr (OP == kWeightGrad) {
                tiles_m = (p.M + BM - 1) / BM;
                e = t / (tiles_m * tiles_n);
                local = t - e * tiles_m * tiles_n;
            } else {
                const int key = t / tiles_n;
                int lo = 0, hi = p.E;               // s_pref[lo] <= key < s_pref[hi]
                while (hi - lo > 1) {
                    const int mid = (lo + hi) >> 1;
                    if (s_pref[mid] <= key) lo = mid;
                    else hi = mid;
                }
                e = uni(lo);
                const int before = uni(s_pref[e]);
                tiles_m = uni(s_pref[e + 1]) - before;
                local = t - before * tiles_n;
            }
            const int grp = local / (kGroupM * tiles_n);
            const int in = local - grp * kGroupM * tiles_n;
            const int rows = tiles_m - grp * kGroupM < kGroupM ? tiles_m - grp * kGroupM : kGroupM;
            nt = in / rows;
            mt = grp * kGroupM + in - nt * rows;
        }
        const int cnt = uni(p.counts[e]);
        const int64_t region = (int64_t)uni(p.offsets[e]) * p.block_m;
        const int K = OP == kWeightGrad ? cnt : p.K;
        const int m0 = mt * BM, n0 = nt * S::kCols;
        const int nk = (K + BK - 1) / BK;

        Loader<BM, AS, S::kWaves> la;
        Loader<BN, BS, S::kWaves> lb;
        const uint32_t a_ldb = (uint32_t)p.a_ld * 2, b_ldb = (uint32_t)p.b_ld * 2;
        if constexpr (OP == kWeightGrad) {
            // columns past the matrix repeat its last chunk; they are not stored
            const int a_last = (p.M >> 3) - 1, b_last = (p.N >> 3) - 1;
            la.init((const char*)p.a + region * a_ldb, a_ldb, wave, lane, [&](int c) {
                const int g = (m0 >> 3) + c;
                return (uint32_t)(g < a_last ? g : a_last) * 16u;
            });
            lb.init((const char*)p.b + region * b_ldb, b_ldb, wave, lane, [&](int c) {
                const int g = (n0 >> 3) + c;
                return (uint32_t)(g < b_last ? g : b_last) * 16u;
            });
        } else {
            // rows past the region repeat its last row; they are not stored
            const int last = cnt - 1 - m0;
            la.init((const char*)p.a + (region + m0) * a_ldb, a_ldb, wave, lane,
                    [&](int r) { return (uint32_t)(r < last ? r : last) * a_ldb; });
            const char* b = (const char*)p.b + (int64_t)e * p.b_expert * 2;
            if constexpr (OP == kUp) {
                // gate columns, then the up columns that belong to them, per wave
                lb.init(b, b_ldb, wave, lane, [&](int r) {
                    const int j = r % WN, up = j >= WN / 2;
                    int c = n0 + r / WN * (WN / 2) + j % (WN / 2);
                    c = c < p.N ? c : p.N - 1;
                    return (uint32_t)(up ? p.N + c : c) * b_ldb;
                });
            } else if constexpr (!BS) {
                lb.init(b, b_ldb, wave, lane, [&](int r) {
                    const int c = n0 + r;
                    return (uint32_t)(c < p.N ? c : p.N - 1) * b_ldb;
                });
            } else {
                const int b_last = (p.N >> 3) - 1;
                lb.init(b, b_ldb, wave, lane, [&](int c) {
                    const int g = (n0 >> 3) + c;
                    return (uint32_t)(g < b_last ? g : b_last) * 16u;
                });
            }
        }

        const uint32_t lds0 = (uint32_t)(uintptr_t)lds;
        auto issue = [&](int kt) {
            const uint32_t at = lds0 + (uint32_t)(kt % ST) * S::kStageBytes;
            la.issue(at, wave, K - kt * BK);
            lb.issue(at + BM * BK * 2, wave, K - kt * BK);
        };
        constexpr int kLoads = Loader<BM, AS, S::kWaves>::kLoads + Loader<BN, BS, S::kWaves>::kLoads;

        f32x4 acc[MF][NF];
#pragma unroll
        for (int i = 0; i < MF; ++i)
#pragma unroll
            for (int j = 0; j < NF; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

        // the last tile's reads are done before its LDS is filled again
        wait_loads<0>();
        __builtin_amdgcn_s_barrier();
#pragma unroll
        for (int s = 0; s < ST - 1; ++s) issue(s);
#pragma unroll 1
        for (int kt = 0; kt < nk; ++kt) {
            wait_loads<(ST - 2) * kLoads>();            // this wave's loads of tile kt
            __builtin_amdgcn_s_barrier();               // every wave's; tile kt - 1 is read
            issue(kt + ST - 1);
            lds_char* at = lds + (kt % ST) * S::kStageBytes;
#pragma unroll
            for (int s = 0; s < BK / 32; ++s) {
                bf16x8 fa[MF], fb[NF];
#pragma unroll
                for (int j = 0; j < NF; ++j) fb[j] = fragment<BN, BS>(at + BM * BK * 2, wn * WN + j * 16, s, lane);
#pragma unroll
                for (int i = 0; i < MF; ++i) fa[i] = fragment<BM, AS>(at, wm * WM + i * 16, s, lane);
#pragma unroll
                for (int i = 0; i < MF; ++i)
#pragma unroll
                    for (int j = 0; j < NF; ++j)
                        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fb[j], fa[i], acc[i][j], 0, 0, 0);
            }
        }

        // Lane l holds row l % 16 and columns 4 (l / 16) + 0..3 of a fragment.
        const int r0 = m0 + wm * WM + (lane & 15), c_in = (lane >> 4) * 4;
        const int rows = OP == kWeightGrad ? p.M : cnt;
#pragma unroll
        for (int i = 0; i < MF; ++i) {
            const int r = r0 + i * 16;
            if (r >= rows) continue;
            if constexpr (OP == kUp) {
                __bf16* out = (__bf16*)p.c + (region + r) * (int64_t)p.N;
                float* save = p.save ? (float*)p.save + (region + r) * (int64_t)(2 * p.N) : nullptr;
#pragma unroll
                for (int j = 0; j < NF / 2; ++j) {
                    const int c = n0 + wn * (WN / 2) + j * 16 + c_in;
                    if (c >= p.N) continue;
                    const f32x4 g = acc[i][j], u = acc[i][j + NF / 2];
                    f32x4 v;
#pragma unroll
                    for (int q = 0; q < 4; ++q) v[q] = act_value(g[q], p.act) * u[q];
                    *(bf16x4*)(out + c) = round4(v);
                    if (save) {
                        *(f32x4*)(save + c) = g;
                        *(f32x4*)(save + p.N + c) = u;
                    }
                }
            } else if constexpr (OP == kActGrad) {
                const float* saved = (const float*)p.save + (region + r) * (int64_t)(2 * p.N);
                __bf16* out = (__bf16*)p.c + (region + r) * (int64_t)(2 * p.N);
#pragma unroll
                for (int j = 0; j < NF; ++j) {
                    const int c = n0 + wn * WN + j * 16 + c_in;
                    if (c >= p.N) continue;
                    const f32x4 g = *(const f32x4*)(saved + c), u = *(const f32x4*)(saved + p.N + c);
                    f32x4 dg, du;
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        float value, slope;
                        act_both(g[q], p.act, value, slope);
                        dg[q] = acc[i][j][q] * u[q] * slope;
                        du[q] = acc[i][j][q] * value;
                    }
                    *(bf16x4*)(out + c) = round4(dg);
                    *(bf16x4*)(out + p.N + c) = round4(du);
                }
            } else {
                const int64_t at = OP == kWeightGrad ? ((int64_t)e * p.M + r) * p.N : (region + r) * (int64_t)p.N;
#pragma unroll
                for (int j = 0; j < NF; ++j) {
                    const int c = n0 + wn * WN + j * 16 + c_in;
                    if (c >= p.N) continue;
                    if (OP == kWeightGrad && p.out_f32) {
                        f32x4* o = (f32x4*)((float*)p.c + at + c);
                        f32x4 v = acc[i][j];
                        if (p.accumulate) {
                            const f32x4 old = *o;
#pragma unroll
                            for (int q = 0; q < 4; ++q) v[q] += old[q];
                        }
                        *o = v;
                    } else {
                        *(bf16x4*)((__bf16*)p.c + at + c) = round4(acc[i][j]);
                    }
                }
            }
        }
    }
    wait_loads<0>();        // no load into LDS outlives the workgroup
}

template <int OP, int BM, int BN, int WM, int WN, int ST>
hipError_t launch(const GemmArgs& p, int64_t row_tiles, hipStream_t stream) {
    using S = Shape<OP, BM, BN, WM, WN, ST>;
    auto kernel = ffn_gemm_kernel<OP, BM, BN, WM, WN, ST>;
    const int64_t tiles = row_tiles * ((p.N + S::kCols - 1) / S::kCols);
    if (tiles == 0) return hipSuccess;
    static_assert(S::lds() <= 160 * 1024, "LDS of a compute unit");
    hipError_t e = hipFuncSetAttribute((const void*)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, (int)S::lds());
    if (e != hipSuccess) return e;
    const int per_cu = (int)(160 * 1024 / S::lds());
    const int64_t most = (int64_t)p.num_cu * (per_cu < 1 ? 1 : per_cu);
    const int grid = (int)(tiles < most ? tiles : most);
    kernel<<<grid, S::kThreads, S::lds(), stream>>>(p);
    return hipGetLastError();
}

// Row tiles of height bm that the rows of the layout can need at most.
int64_t row_tile_bound(const GemmArgs& p, int bm) {
    const int64_t used = p.slots < p.E ? p.slots : p.E;
    return used + p.slots / bm;
}

template <int OP>
hipError_t launch_rows(const GemmArgs& p, hipStream_t stream) {
    const int64_t mean = (p.slots + p.E - 1) / p.E;
    if (mean > 128) return launch<OP, 256, 256, 128, 64, 2>(p, row_tile_bound(p, 256), stream);
    if (mean > 48) return launch<OP, 128, 128, 64, 64, 2>(p, row_tile_bound(p, 128), stream);
    if (mean > 16) return launch<OP, 64, 128, 64, 32, 3>(p, row_tile_bound(p, 64), stream);
    return launch<OP, 16, 128, 16, 32, 4>(p, row_tile_bound(p, 16), stream);
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
    if (f.grad_pool) {
        p.a = f.grad_gate_up;
        p.a_ld = 2 * f.I;
        p.b = f.w_gate_up;
        p.b_ld = f.H;
        p.b_expert = (int64_t)2 * f.I * f.H;
        p.c = f.grad_pool;
        p.N = f.H;
        p.K = 2 * f.I;
        e = launch_rows<kRowGrad>(p, stream);
        if (e != hipSuccess) return e;
    }
    p.out_f32 = f.grad_f32;
    p.accumulate = f.accumulate;
    if (f.grad_w_gate_up) {
        p.a = f.grad_gate_up;
        p.a_ld = 2 * f.I;
        p.b = f.pool;
        p.b_ld = f.H;
        p.c = f.grad_w_gate_up;
        p.M = 2 * f.I;
        p.N = f.H;
        e = launch<kWeightGrad, 256, 256, 128, 64, 2>(p, (int64_t)f.E * ((p.M + 255) / 256), stream);
        if (e != hipSuccess) return e;
    }
    if (f.grad_w_down) {
        p.a = f.grad_out;
        p.a_ld = f.H;
        p.b = f.act_rows;
        p.b_ld = f.I;
        p.c = f.grad_w_down;
        p.M = f.H;
        p.N = f.I;
        e = launch<kWeightGrad, 256, 256, 128, 64, 2>(p, (int64_t)f.E * ((p.M + 255) / 256), stream);
    }
    return e;
}

}  // namespace epk
