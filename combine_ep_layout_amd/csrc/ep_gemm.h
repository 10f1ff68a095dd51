// The tile of a matrix product on the matrix cores (16x16x32, fp32 sums), from
// memory through LDS, that the experts' feed-forward (ep_ffn.hip) and the
// orthogonalisation (ep_muon.hip) share.  Not installed; callers use
// include/ep_layout.h.
//
// A shape S has the tile's and the waves' sizes BM, BN, WM, WN, the depth BK and
// number ST of its LDS tiles, kStageBytes of one, the loaders A and B with
// kLoads of both, kAStrided and kBStrided (whether the operand's summed index is
// not the contiguous one) and kF16 (fp16 values, else bf16).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>
#include <utility>

#include "ep_wave.h"

namespace epk {
namespace {

typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) char lds_char;

// Offset past every buffer's range, also with a tile's own offset added: such a
// lane loads zeros.
constexpr uint32_t kOutOfRange = 0x80000000u;
constexpr size_t kLdsBytes = 160 * 1024;        // of a compute unit
constexpr int kXcds = 8;

// f(0), ..., f(N - 1) with constant arguments.
template <class F, int... I>
__device__ __forceinline__ void each_of(F&& f, std::integer_sequence<int, I...>) {
    (f(std::integral_constant<int, I>{}), ...);
}
template <int N, class F>
__device__ __forceinline__ void each(F&& f) { each_of(f, std::make_integer_sequence<int, N>{}); }

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
// Swizzle of a contiguous tile's row r, BK values of it: the 16-byte chunks
// that eight rows read together lie in different banks.
template <int BK>
__device__ __forceinline__ int row_swizzle(int r) {
    return BK == 64 ? r & 7 : (r >> 1) & 3;
}

// Loads of one operand's LDS tile, BK summed indices deep, by one wave.
//   STRIDED false: R rows of BK summed values; true: BK rows of R columns.
template <int R, int BK, bool STRIDED, int WAVES>
struct Loader {
    static constexpr int kTotal = R * BK / 512;                       // 1 KiB loads of a tile
    static constexpr int kLoads = kTotal / WAVES > 0 ? kTotal / WAVES : 1;   // each wave's
    uint32_t voff[kLoads];
    int lane_k;                 // summed index of the lane's first value inside a load's part of the tile
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
                constexpr int kChunks = BK / 8;
                const int r = lane / kChunks, c = (lane % kChunks) ^ row_swizzle<BK>(r);
                voff[i] = row(g * (kWave / kChunks) + r) + c * 16;
                lane_k = c * 8;
            } else {
                constexpr int kRows = 512 / R;
                const int kk = g * kRows + lane / (R / 8), c = lane % (R / 8);
                const int src = (((c >> 1) ^ strided_swizzle<R>(kk)) << 1) | (c & 1);
                voff[i] = (uint32_t)kk * ld_bytes + row(src);
                lane_k = lane / (R / 8);
            }
        }
        base = (uint64_t)(uintptr_t)p;
        step = STRIDED ? (uint64_t)ld_bytes * BK : BK * 2;
    }
    // rem: summed indices left from this tile on (may be <= 0: zeros)
    __device__ __forceinline__ void issue_one(int i, uint32_t lds, int wave, int rem, const i32x4& rsrc) const {
        const int g = load_index(wave, i), first = STRIDED ? g * (512 / R) : 0;
        load_to_lds(uni(lds + g * 1024), lane_k < rem - first ? voff[i] : kOutOfRange, rsrc);
    }
    __device__ __forceinline__ void issue(uint32_t lds, int wave, int rem) {
        const i32x4 rsrc = make_rsrc((const void*)(uintptr_t)base);
#pragma unroll
        for (int i = 0; i < kLoads; ++i) issue_one(i, lds, wave, rem, rsrc);
        base += step;
    }
};

// A fragment for the matrix core: 16 rows (or columns) from `at`, summed
// indices 32 s + 8 (lane / 16) + 0..7.
template <int R, int BK, bool STRIDED>
__device__ __forceinline__ bf16x8 fragment(lds_char* tile, int at, int s, int lane) {
    if constexpr (!STRIDED) {
        const int r = at + (lane & 15);
        const int c = (s * 4 + (lane >> 4)) ^ row_swizzle<BK>(lane & 15);       // at is a multiple of 16
        return *(__attribute__((address_space(3))) bf16x8*)(tile + r * (BK * 2) + c * 16);
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

// c += b a^T in the accumulation registers.  Written out, since the compiler
// moves half of those about at every turn of the loop otherwise.  s_nop 1: the states a
// vector instruction's result needs before the matrix core reads it.
template <bool F16>
__device__ __forceinline__ void mfma(f32x4& c, const bf16x8& b, const bf16x8& a) {
    if constexpr (F16) asm volatile("s_nop 1\n\tv_mfma_f32_16x16x32_f16 %0, %1, %2, %0" : "+a"(c) : "v"(b), "v"(a));
    else asm volatile("s_nop 1\n\tv_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(c) : "v"(b), "v"(a));
}
template <bool F16>
__device__ __forceinline__ f32x4 mfma_value(const bf16x8& b, const bf16x8& a, const f32x4& c) {
    typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
    if constexpr (F16)
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, b), __builtin_bit_cast(f16x8, a), c, 0, 0, 0);
    else return __builtin_amdgcn_mfma_f32_16x16x32_bf16(b, a, c, 0, 0, 0);
}
// The states that the matrix core's results need before another instruction
// reads them (18 at most), for a row of fragments.
__device__ __forceinline__ void settle(f32x4 (&c)[2]) {
    asm volatile("s_nop 15\n\ts_nop 3" : "+a"(c[0]), "+a"(c[1]));
}
__device__ __forceinline__ void settle(f32x4 (&c)[4]) {
    asm volatile("s_nop 15\n\ts_nop 3" : "+a"(c[0]), "+a"(c[1]), "+a"(c[2]), "+a"(c[3]));
}

template <int MF, int NF>
struct Fragments {
    bf16x8 a[MF], b[NF];
};

// A wave's MF x NF fragments of a tile, from tile row r_at and column c_at,
// summed over K and handed to done(), in a software pipeline over halves of 32
// summed indices.
// While the matrix core works on one half from registers, the wave reads the
// next half's fragments from LDS; after a tile's second half has been read,
// its LDS takes the loads of the tile after next.  One barrier a tile.
template <class S, int MF, int NF, class Done>
__device__ __forceinline__ void pipelined_tile(typename S::A& la, typename S::B& lb, int K, int r_at, int c_at, int wave,
                                               int lane, lds_char* lds, Done&& done) {
    static_assert(S::BK == 64 && S::ST == 2, "two tiles of two halves");
    constexpr bool AS = S::kAStrided, BS = S::kBStrided;
    constexpr int LA = S::A::kLoads, L = S::kLoads;
    const uint32_t lds0 = (uint32_t)(uintptr_t)lds;
    // an empty sum takes one turn, over zeros: a way around the loop would have
    // the compiler copy the products behind it, before they have settled
    const int nk = K > 0 ? (K + S::BK - 1) / S::BK : 1;
    f32x4 acc[MF][NF];
#pragma unroll
    for (int i = 0; i < MF; ++i)
#pragma unroll
        for (int j = 0; j < NF; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        const uint32_t at = lds0 + s * S::kStageBytes;
        la.issue(at, wave, K - s * S::BK);
        lb.issue(at + S::BM * S::BK * 2, wave, K - s * S::BK);
    }
    Fragments<MF, NF> f0, f1;
    wait_loads<L>();
    __builtin_amdgcn_s_barrier();
    auto read_a = [&](int i, int slot, int s) {
        return fragment<S::BM, S::BK, AS>(lds + slot * S::kStageBytes, r_at + i * 16, s, lane);
    };
    auto read_b = [&](int j, int slot, int s) {
        return fragment<S::BN, S::BK, BS>(lds + slot * S::kStageBytes + S::BM * S::BK * 2, c_at + j * 16, s, lane);
    };
#pragma unroll
    for (int j = 0; j < NF; ++j) f0.b[j] = read_b(j, 0, 0);
#pragma unroll
    for (int i = 0; i < MF; ++i) f0.a[i] = read_a(i, 0, 0);
    // The products of `now`, with the reads of `next` (half s of an LDS tile)
    // and, LOAD, this wave's loads of a tile spread between them: the matrix
    // core takes 16 cycles for a product and an instruction of another kind 4,
    // so one or two behind each product are free.
    auto half = [&](auto load, const Fragments<MF, NF>& now, Fragments<MF, NF>& next, int slot, int s, uint32_t fill, int rem) {
        constexpr bool LOAD = decltype(load)::value;
        const i32x4 ra = make_rsrc((const void*)(uintptr_t)la.base), rb = make_rsrc((const void*)(uintptr_t)lb.base);
        each<MF * NF>([&](auto product) {
            constexpr int n = product, P = MF * NF, F = MF + NF;
            mfma<S::kF16>(acc[n / NF][n % NF], now.b[n % NF], now.a[n / NF]);
            // both end well before the half, so that the last have come when they are needed
            constexpr int R = P * 3 / 4, r0 = n * F / R < F ? n * F / R : F, r1 = (n + 1) * F / R < F ? (n + 1) * F / R : F;
            each<r1 - r0>([&](auto i) {
                constexpr int r = r0 + i;
                if constexpr (r < NF) next.b[r] = read_b(r, slot, s);
                else next.a[r - NF] = read_a(r - NF, slot, s);
            });
            if constexpr (LOAD) {
                constexpr int Q = P / 2, l0 = n * L / Q < L ? n * L / Q : L, l1 = (n + 1) * L / Q < L ? (n + 1) * L / Q : L;
                each<l1 - l0>([&](auto i) {
                    constexpr int l = l0 + i;
                    if constexpr (l < LA) la.issue_one(l, fill, wave, rem, ra);
                    else lb.issue_one(l - LA, fill + S::BM * S::BK * 2, wave, rem, rb);
                });
            }
            __builtin_amdgcn_sched_barrier(0);
        });
        if constexpr (LOAD) {
            la.base += la.step;
            lb.base += lb.step;
        }
    };
#pragma unroll 1
    for (int kt = 0;;) {
        const int slot = kt & 1;
        half(std::false_type{}, f0, f1, slot, 1, 0, 0);
        // this tile's second half has come to registers, and the next tile to
        // LDS; after the barrier that holds for every wave
        wait_loads<0>();
        __builtin_amdgcn_s_barrier();
        half(std::true_type{}, f1, f0, slot ^ 1, 0, lds0 + slot * S::kStageBytes, K - (kt + 2) * S::BK);
        if (++kt >= nk) break;
    }
#pragma unroll
    for (int i = 0; i < MF; ++i) settle(acc[i]);
    done(acc);
}

// The same without the register pipeline, for the lower tiles: those are bound
// by the weights' bytes or by latency, and several workgroups of a compute unit
// hide each other's waits.
template <class S, class Done>
__device__ __forceinline__ void plain_tile(typename S::A& la, typename S::B& lb, int K, int r_at, int c_at, int wave,
                                           int lane, lds_char* lds, Done&& done) {
    constexpr bool AS = S::kAStrided, BS = S::kBStrided;
    constexpr int MF = S::WM / 16, NF = S::WN / 16, ST = S::ST;
    const uint32_t lds0 = (uint32_t)(uintptr_t)lds;
    const int nk = (K + S::BK - 1) / S::BK;
    f32x4 acc[MF][NF];
#pragma unroll
    for (int i = 0; i < MF; ++i)
#pragma unroll
        for (int j = 0; j < NF; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    auto issue = [&](int kt) {
        const uint32_t at = lds0 + (uint32_t)(kt % ST) * S::kStageBytes;
        la.issue(at, wave, K - kt * S::BK);
        lb.issue(at + S::BM * S::BK * 2, wave, K - kt * S::BK);
    };
#pragma unroll
    for (int s = 0; s < ST - 1; ++s) issue(s);
#pragma unroll 1
    for (int kt = 0; kt < nk; ++kt) {
        wait_loads<(ST - 2) * S::kLoads>();         // this wave's loads of tile kt
        __builtin_amdgcn_s_barrier();               // every wave's; tile kt - 1 is read
        issue(kt + ST - 1);
        lds_char* at = lds + (kt % ST) * S::kStageBytes;
#pragma unroll
        for (int s = 0; s < S::BK / 32; ++s) {
            bf16x8 fa[MF], fb[NF];
#pragma unroll
            for (int j = 0; j < NF; ++j) fb[j] = fragment<S::BN, S::BK, BS>(at + S::BM * S::BK * 2, c_at + j * 16, s, lane);
#pragma unroll
            for (int i = 0; i < MF; ++i) fa[i] = fragment<S::BM, S::BK, AS>(at, r_at + i * 16, s, lane);
#pragma unroll
            for (int i = 0; i < MF; ++i)
#pragma unroll
                for (int j = 0; j < NF; ++j)
                    acc[i][j] = mfma_value<S::kF16>(fb[j], fa[i], acc[i][j]);
        }
    }
    done(acc);
}

}  // namespace
}  // namespace epk
