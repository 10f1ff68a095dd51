// gfx950 kernels that turn values into 4-bit codes with an exponent byte for each
// 32 of them, and back, and their C entry points.
//
// Codes are e2m1 (0, 1/2, 1, 3/2, 2, 3, 4, 6 and a sign in bit 3), two a byte,
// the lower index in the lower half; byte b of a block means 2^(b - 127).  A
// block's exponent is the least one under which no value is larger than 6, so
// nothing saturates; values go to the nearest code, ties to the even one.
//
// One pass over memory: a lane takes 8 values (one dword of codes), four lanes a
// block, whose maximum they find with two moves.  The conversions are the
// scaled ones of the hardware, which round so (tests compare every bf16 value).
// Memory's rate bounds both: 64 matrices of 4096 x 7168 go from fp32 in 1797 us
// and from bf16 in 951 (4.7 and 5.0 TB/s), back in 823 (5.8 TB/s); a large copy
// reaches 5.4.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ep_layout.h"
#include "ep_ranges.h"

namespace epk {
namespace {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kThreads = 256;
constexpr int64_t kMaxValues = (int64_t)1 << 38;

template <int CTRL>
__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
    const uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, true);
    return o > v ? o : v;
}

// BF16: the values' type.
template <bool BF16>
__global__ void __launch_bounds__(kThreads) mxfp4_quantize_kernel(const void* values, int64_t n8, uint32_t* codes, uint8_t* scales) {
    // n8 is a multiple of 4, so a block's four lanes stay together
    const int64_t step = (int64_t)gridDim.x * kThreads;
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < n8; i += step) {
        float v[8];
        if constexpr (BF16) {
            const bf16x8 b = __builtin_nontemporal_load((const bf16x8*)values + i);
#pragma unroll
            for (int q = 0; q < 8; ++q) v[q] = (float)b[q];
        } else {
            const f32x4 lo = __builtin_nontemporal_load((const f32x4*)values + 2 * i);
            const f32x4 hi = __builtin_nontemporal_load((const f32x4*)values + 2 * i + 1);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                v[q] = lo[q];
                v[4 + q] = hi[q];
            }
        }
        // magnitudes order as integers, with infinity and NaN above all
        uint32_t top = 0;
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            const uint32_t m = __float_as_uint(v[q]) & 0x7FFFFFFFu;
            top = m > top ? m : top;
        }
        top = quad_max<0xB1>(top);              // quad_perm: the neighbour, then the other pair
        top = quad_max<0x4E>(top);
        // top <= 6 * 2^e = 1.5 * 2^(e + 2): the exponent less 2, and one more past the mantissa of 1.5
        int byte = (int)(top >> 23) - 2 + ((top & 0x7FFFFFu) > 0x400000u ? 1 : 0);
        byte = byte < 0 ? 0 : byte;
        const bool finite = top < 0x7F800000u;
        // 2^(byte - 127); byte 0 is a subnormal float
        const float scale = byte > 0 ? __uint_as_float((uint32_t)byte << 23) : 0x1p-127f;
        uint32_t w = 0;
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[0], v[1], scale, 0);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[2], v[3], scale, 1);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[4], v[5], scale, 2);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[6], v[7], scale, 3);
        // a block with an infinity or a NaN reads as NaN
        codes[i] = finite ? w : 0u;
        if ((threadIdx.x & 3) == 0) scales[i >> 2] = finite ? (uint8_t)byte : (uint8_t)255;
    }
}

__global__ void __launch_bounds__(kThreads) mxfp4_cast_back_kernel(const uint32_t* codes, const uint8_t* scales, int64_t n8, bf16x8* out) {
    const int64_t step = (int64_t)gridDim.x * kThreads;
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < n8; i += step) {
        const uint32_t w = __builtin_nontemporal_load(codes + i), byte = scales[i >> 2];
        const float scale = byte == 0 ? 0x1p-127f : byte == 255 ? __builtin_nanf("") : __uint_as_float(byte << 23);
        union { bf16x2 p[4]; bf16x8 v; } u;
        u.p[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 0);
        u.p[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 1);
        u.p[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 2);
        u.p[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 3);
        __builtin_nontemporal_store(u.v, out + i);
    }
}

int grid_of(int64_t n8) {
    const int64_t g = (n8 + kThreads - 1) / kThreads;
    return (int)(g < 65536 ? g : 65536);
}

// Whether n values have the buffers that a call needs.
ep_status check(const void* values, int64_t size, int64_t n, const void* codes, const void* scales, bool to_codes) {
    if (n < 0 || n % 32 != 0) return EP_ERR_INVALID_ARGUMENT;
    if (n > kMaxValues) return EP_ERR_UNSUPPORTED;
    if (n == 0) return EP_OK;
    if (!values || !codes || !scales || !aligned(values, 16) || !aligned(codes, 16)) return EP_ERR_INVALID_ARGUMENT;
    const Rows v(values, n, n, 1, (int)size), c(codes, n / 2, n / 2, 1, 1), s(scales, n / 32, n / 32, 1, 1);
    if (share(v, c) || share(v, s) || (to_codes && share(c, s))) return EP_ERR_INVALID_ARGUMENT;
    return EP_OK;
}

}  // namespace
}  // namespace epk

extern "C" {

ep_status ep_mxfp4_quantize(const void* values, int64_t n, uint32_t flags, void* codes, uint8_t* scales, hipStream_t stream) {
    using namespace epk;
    if (flags & ~EP_MXFP4_BF16) return EP_ERR_INVALID_ARGUMENT;
    const bool bf16 = flags & EP_MXFP4_BF16;
    const ep_status st = check(values, bf16 ? 2 : 4, n, codes, scales, true);
    if (st != EP_OK || n == 0) return st;
    if (bf16) mxfp4_quantize_kernel<true><<<grid_of(n / 8), kThreads, 0, stream>>>(values, n / 8, (uint32_t*)codes, scales);
    else mxfp4_quantize_kernel<false><<<grid_of(n / 8), kThreads, 0, stream>>>(values, n / 8, (uint32_t*)codes, scales);
    return hipGetLastError() == hipSuccess ? EP_OK : EP_ERR_HIP;
}

ep_status ep_mxfp4_cast_back(const void* codes, const uint8_t* scales, int64_t n, void* out, hipStream_t stream) {
    using namespace epk;
    const ep_status st = check(out, 2, n, codes, scales, false);
    if (st != EP_OK || n == 0) return st;
    mxfp4_cast_back_kernel<<<grid_of(n / 8), kThreads, 0, stream>>>((const uint32_t*)codes, scales, n / 8, (bf16x8*)out);
    return hipGetLastError() == hipSuccess ? EP_OK : EP_ERR_HIP;
}

}  // extern "C"
