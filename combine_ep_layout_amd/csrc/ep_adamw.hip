// gfx950 kernel of the AdamW step over many tensors at once, and its C entry
// point.
//
// Per value, with t the step:
//     m = b1 m + (1 - b1) g,  v = b2 v + (1 - b2) g^2
//     p = p (1 - lr wd) - lr / (1 - b1^t) * m / (sqrt(v) / sqrt(1 - b2^t) + eps)
// The states are fp32, or 8 bits: e4m3fn codes of m and of sqrt(v) with one
// fp32 scale for each 128 values, which the FP8 dispatch's float32 flavour reads:
// with a the block's largest magnitude, scale a * (1/448) and codes of
// x * ((1/a) * 448), one rounded reciprocal instead of two quotients.  The root is stored because its range is half of v's in
// the exponent, which e4m3 spans within a block; a root above zero keeps the
// least code rather than becoming zero, so no step is divided by eps alone.
//
// A pass over memory and nothing else: every value is read once and written
// once.  The tensors' addresses travel in the kernel's arguments, so nothing
// is uploaded and a captured call holds all that it needs; a workgroup finds
// its tensor with one ballot over the tensors' first chunks.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>
#include <algorithm>
#include <new>
#include <vector>

#include "ep_layout.h"

namespace epk {
namespace {

constexpr int kWave = 64;
constexpr int kThreads = 256;
constexpr int kBlock = 128;                 // values of one 8-bit scale
// Values of a workgroup (a multiple of kBlock): two of a thread's vectors, so
// that all of a workgroup's loads are in flight before its first store.  On
// 169.9 M values with bf16 gradients and copies: 836 us with 2048, 858 with 4096,
// 885 with 8192, 947 with 32768 (8-bit states 466, 498, 513, 556); with cached
// instead of non-temporal accesses 919 (533) at 8192.
constexpr int kChunk = 2048;
constexpr int kTensors = 52;                // tensors of a launch: the arguments stay below 4 KiB

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));

struct Tensor {
    void* p;
    const void* g;
    void* m;
    void* v;
    float* m_scale;
    float* v_scale;
    void* copy;
    int64_t n;
};

struct AdamwArgs {
    float beta1, rest1, beta2, rest2, decay, eps;
    float step_size, root_bc2;              // lr / (1 - b1^t), sqrt(1 - b2^t)
    float grad_scale;
    const float* grad_scale_dev;
    const int64_t* step_dev;                // non-null: t is read on the device
    double lr_d, beta1_d, beta2_d;          // what the device's step is made of, as the host's is
    int32_t count;
    int32_t first[kTensors];                // first chunk of each tensor
    Tensor t[kTensors];
};
static_assert(sizeof(AdamwArgs) <= 4096, "kernel arguments");

template <bool BF16>
__device__ __forceinline__ f32x4 load4(const void* p, int64_t i) {
    if constexpr (BF16) {
        const bf16x4 b = __builtin_nontemporal_load((const bf16x4*)((const __bf16*)p + i));
        return f32x4{(float)b[0], (float)b[1], (float)b[2], (float)b[3]};
    } else {
        return __builtin_nontemporal_load((const f32x4*)((const float*)p + i));
    }
}
template <bool BF16>
__device__ __forceinline__ void store4(void* p, int64_t i, const f32x4& v) {
    if constexpr (BF16) {
        const bf16x4 b{(__bf16)v[0], (__bf16)v[1], (__bf16)v[2], (__bf16)v[3]};
        __builtin_nontemporal_store(b, (bf16x4*)((__bf16*)p + i));
    } else {
        __builtin_nontemporal_store(v, (f32x4*)((float*)p + i));
    }
}
template <bool BF16>
__device__ __forceinline__ float load1(const void* p, int64_t i) {
    if constexpr (BF16) return (float)((const __bf16*)p)[i];
    else return ((const float*)p)[i];
}
template <bool BF16>
__device__ __forceinline__ void store1(void* p, int64_t i, float v) {
    if constexpr (BF16) ((__bf16*)p)[i] = (__bf16)v;
    else ((float*)p)[i] = v;
}

struct Scalars {
    float beta1, rest1, beta2, rest2, decay, eps, step_size, root_bc2, grad_scale;
};

__device__ __forceinline__ Scalars scalars(const AdamwArgs& a) {
    Scalars s{a.beta1, a.rest1, a.beta2, a.rest2, a.decay, a.eps, a.step_size, a.root_bc2, a.grad_scale};
    if (a.grad_scale_dev) s.grad_scale *= *a.grad_scale_dev;
    if (a.step_dev) {
        const double t = (double)*a.step_dev;
        s.step_size = (float)(a.lr_d / (1.0 - pow(a.beta1_d, t)));
        s.root_bc2 = (float)sqrt(1.0 - pow(a.beta2_d, t));
    }
    return s;
}

// One value's step; r becomes sqrt(v).
__device__ __forceinline__ float update(const Scalars& s, float p, float g, float& m, float& v, float& r) {
    g *= s.grad_scale;
    m = s.beta1 * m + s.rest1 * g;
    v = s.beta2 * v + s.rest2 * (g * g);
    r = sqrtf(v);               // correctly rounded, as the quotients are: codes next to a tie depend on it
    return p * s.decay - s.step_size * (m / (r / s.root_bc2 + s.eps));
}

// The workgroup's tensor (uniform) and its first value there.
__device__ __forceinline__ int find_tensor(const AdamwArgs& a, int64_t& begin) {
    const int lane = threadIdx.x & (kWave - 1), chunk = blockIdx.x;
    const bool before = lane < a.count && a.first[lane] <= chunk;
    const int i = __builtin_popcountll(__ballot(before)) - 1;
    begin = (int64_t)(chunk - a.first[i]) * kChunk;
    return i;
}

template <bool PB, bool GB>
__global__ void __launch_bounds__(kThreads) adamw_kernel(AdamwArgs a) {
    int64_t begin;
    const Tensor& t = a.t[find_tensor(a, begin)];
    const Scalars s = scalars(a);
    float* const m = (float*)t.m;
    float* const v = (float*)t.v;
    __bf16* const copy = (__bf16*)t.copy;
    const int64_t end = begin + kChunk < t.n ? begin + kChunk : t.n;
    int64_t i = begin + threadIdx.x * 4;
#pragma unroll 2
    for (; i + 4 <= end; i += kThreads * 4) {
        f32x4 pv = load4<PB>(t.p, i);
        const f32x4 gv = load4<GB>(t.g, i);
        f32x4 mv = load4<false>(m, i), vv = load4<false>(v, i);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            float mq = mv[q], vq = vv[q], r;
            pv[q] = update(s, pv[q], gv[q], mq, vq, r);
            mv[q] = mq;
            vv[q] = vq;
        }
        store4<PB>(t.p, i, pv);
        store4<false>(m, i, mv);
        store4<false>(v, i, vv);
        if (copy) store4<true>(copy, i, pv);
    }
    for (; i < end; ++i) {              // the tensor's last one to three values
        float r;
        const float p = update(s, load1<PB>(t.p, i), load1<GB>(t.g, i), m[i], v[i], r);
        store1<PB>(t.p, i, p);
        if (copy) copy[i] = (__bf16)p;
    }
}

__device__ __forceinline__ float max32(float v) {        // over the 32 lanes of a block
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) v = fmaxf(v, __shfl_xor(v, d));
    return v;
}

// Codes of four values of a block (NaN takes no part in the maximum) and its scale.
__device__ __forceinline__ uint32_t encode4(const float (&x)[4], float& scale) {
    float top = fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3])));
    top = fmaxf(max32(top), 448.0f * 0x1p-126f);
    scale = top * (1.0f / 448.0f);
    const float f = (1.0f / top) * 448.0f;
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(x[0] * f, x[1] * f, 0, false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(x[2] * f, x[3] * f, w, true);
    return (uint32_t)w;
}

// 8-bit states: 32 lanes x 4 values a block.
template <bool PB, bool GB>
__global__ void __launch_bounds__(kThreads) adamw_8bit_kernel(AdamwArgs a) {
    int64_t begin;
    const Tensor& t = a.t[find_tensor(a, begin)];
    const Scalars s = scalars(a);
    uint8_t* const mc = (uint8_t*)t.m;
    uint8_t* const vc = (uint8_t*)t.v;
    __bf16* const copy = (__bf16*)t.copy;
    const int64_t end = begin + kChunk < t.n ? begin + kChunk : t.n;
    // every lane of a block runs the same rounds: its maximum needs them all
    for (int64_t at = begin; at < end; at += kThreads * 4) {
        const int64_t i = at + threadIdx.x * 4, block = i / kBlock;
        const int left = (int)(end - i < 4 ? end - i : 4);        // may be below zero
        float pv[4] = {0.f, 0.f, 0.f, 0.f}, gv[4] = {0.f, 0.f, 0.f, 0.f};
        uint32_t mw = 0, vw = 0;
        float ms = 0.f, vs = 0.f;
        if (left > 0) {
            ms = t.m_scale[block];
            vs = t.v_scale[block];
        }
        if (left == 4) {
            const f32x4 p4 = load4<PB>(t.p, i), g4 = load4<GB>(t.g, i);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                pv[q] = p4[q];
                gv[q] = g4[q];
            }
            mw = *(const uint32_t*)(mc + i);
            vw = *(const uint32_t*)(vc + i);
        } else {
#pragma unroll
            for (int q = 0; q < 3; ++q)
                if (q < left) {
                    pv[q] = load1<PB>(t.p, i + q);
                    gv[q] = load1<GB>(t.g, i + q);
                    mw |= (uint32_t)mc[i + q] << (8 * q);
                    vw |= (uint32_t)vc[i + q] << (8 * q);
                }
        }
        float mv[4] = {__builtin_amdgcn_cvt_f32_fp8(mw, 0), __builtin_amdgcn_cvt_f32_fp8(mw, 1),
                       __builtin_amdgcn_cvt_f32_fp8(mw, 2), __builtin_amdgcn_cvt_f32_fp8(mw, 3)};
        float rv[4] = {__builtin_amdgcn_cvt_f32_fp8(vw, 0), __builtin_amdgcn_cvt_f32_fp8(vw, 1),
                       __builtin_amdgcn_cvt_f32_fp8(vw, 2), __builtin_amdgcn_cvt_f32_fp8(vw, 3)};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            mv[q] *= ms;
            const float r = rv[q] * vs;
            float v = r * r;
            pv[q] = update(s, pv[q], gv[q], mv[q], v, rv[q]);
            if (q >= left) mv[q] = rv[q] = 0.0f;        // past the tensor
        }
        mw = encode4(mv, ms);
        vw = encode4(rv, vs);
        // under an infinite scale code 0 reads as NaN, as the block is to read; the least code would be infinity
        const bool finite = vs < __builtin_inff();
#pragma unroll
        for (int q = 0; q < 4; ++q)
            if (finite && rv[q] > 0.0f && ((vw >> (8 * q)) & 0xFFu) == 0) vw |= 1u << (8 * q);
        if (left > 0 && (threadIdx.x & 31) == 0) {
            t.m_scale[block] = ms;
            t.v_scale[block] = vs;
        }
        if (left == 4) {
            const f32x4 p4{pv[0], pv[1], pv[2], pv[3]};
            store4<PB>(t.p, i, p4);
            __builtin_nontemporal_store(mw, (uint32_t*)(mc + i));
            __builtin_nontemporal_store(vw, (uint32_t*)(vc + i));
            if (copy) store4<true>(copy, i, p4);
        } else {
#pragma unroll
            for (int q = 0; q < 3; ++q)
                if (q < left) {
                    store1<PB>(t.p, i + q, pv[q]);
                    mc[i + q] = (uint8_t)(mw >> (8 * q));
                    vc[i + q] = (uint8_t)(vw >> (8 * q));
                    if (copy) copy[i + q] = (__bf16)pv[q];
                }
        }
    }
}

bool aligned(const void* p, int n) { return ((uintptr_t)p & (uintptr_t)(n - 1)) == 0; }

void launch(const AdamwArgs& a, uint32_t flags, int grid, hipStream_t stream) {
    const bool pb = flags & EP_ADAMW_PARAM_BF16, gb = flags & EP_ADAMW_GRAD_BF16;
    if (flags & EP_ADAMW_STATE_8BIT) {
        if (pb && gb) adamw_8bit_kernel<true, true><<<grid, kThreads, 0, stream>>>(a);
        else if (pb) adamw_8bit_kernel<true, false><<<grid, kThreads, 0, stream>>>(a);
        else if (gb) adamw_8bit_kernel<false, true><<<grid, kThreads, 0, stream>>>(a);
        else adamw_8bit_kernel<false, false><<<grid, kThreads, 0, stream>>>(a);
    } else {
        if (pb && gb) adamw_kernel<true, true><<<grid, kThreads, 0, stream>>>(a);
        else if (pb) adamw_kernel<true, false><<<grid, kThreads, 0, stream>>>(a);
        else if (gb) adamw_kernel<false, true><<<grid, kThreads, 0, stream>>>(a);
        else adamw_kernel<false, false><<<grid, kThreads, 0, stream>>>(a);
    }
}

struct Range {
    uintptr_t at, end;
    bool wrote;
    bool operator<(const Range& o) const { return at < o.at; }
};

// Merges the ranges from `from` on, one kind of buffer of every tensor, into
// those before.  A kind mostly lies in memory in the list's order, and is only
// merged then: the checks of 300 tensors take 11.3 us on the host, 12.2 with one
// sort of them all; out of order 15.8 and 15.2.
void merge_in(std::vector<Range>& r, size_t from) {
    const auto mid = r.begin() + (std::ptrdiff_t)from;
    if (!std::is_sorted(mid, r.end())) std::sort(mid, r.end());
    std::inplace_merge(r.begin(), mid, r.end());
}

// Whether a buffer that is written shares memory with another buffer (r in order).
bool shared(const std::vector<Range>& r) {
    uintptr_t any = 0, written = 0;         // furthest end so far, of all and of those written
    for (const Range& x : r) {
        if (x.at < written || (x.wrote && x.at < any)) return true;
        any = std::max(any, x.end);
        if (x.wrote) written = std::max(written, x.end);
    }
    return false;
}

}  // namespace
}  // namespace epk

extern "C" ep_status ep_adamw(const ep_adamw_tensor* tensors, int32_t count, const ep_adamw_config* cfg,
                              hipStream_t stream) {
    using namespace epk;
    if (!cfg || count < 0 || (count > 0 && !tensors)) return EP_ERR_INVALID_ARGUMENT;
    if (cfg->flags & ~(EP_ADAMW_PARAM_BF16 | EP_ADAMW_GRAD_BF16 | EP_ADAMW_STATE_8BIT)) return EP_ERR_INVALID_ARGUMENT;
    if (!(cfg->beta1 >= 0 && cfg->beta1 < 1 && cfg->beta2 >= 0 && cfg->beta2 < 1 && cfg->eps >= 0 &&
          std::isfinite(cfg->eps) && std::isfinite(cfg->lr) && std::isfinite(cfg->weight_decay) &&
          std::isfinite(cfg->grad_scale)) ||
        (!cfg->step_dev && cfg->step < 1) || !aligned(cfg->step_dev, 8) || !aligned(cfg->grad_scale_dev, 4))
        return EP_ERR_INVALID_ARGUMENT;
    const bool eight = cfg->flags & EP_ADAMW_STATE_8BIT, pb = cfg->flags & EP_ADAMW_PARAM_BF16;
    const int64_t ps = pb ? 2 : 4, gs = (cfg->flags & EP_ADAMW_GRAD_BF16) ? 2 : 4, ss = eight ? 1 : 4;
    // a launch's grid stays below 2^32 threads
    constexpr int64_t kMostChunks = (int64_t)1 << 23, kMost = kMostChunks * kChunk;
    try {
        std::vector<Range> ranges;
        ranges.reserve((size_t)count * 7);
        auto add = [&](const void* p, int64_t n, bool w) {
            if (p && n > 0) ranges.push_back({(uintptr_t)p, (uintptr_t)p + (uintptr_t)n, w});
        };
        for (int32_t i = 0; i < count; ++i) {
            const ep_adamw_tensor& t = tensors[i];
            if (t.n < 0) return EP_ERR_INVALID_ARGUMENT;
            if (t.n > kMost) return EP_ERR_UNSUPPORTED;
            if (t.copy && pb) return EP_ERR_UNSUPPORTED;        // bf16 parameters are their own copy
            if (t.n == 0) continue;
            if (!t.param || !t.grad || !t.exp_avg || !t.exp_avg_sq || !aligned(t.param, 16) || !aligned(t.grad, 16) ||
                !aligned(t.exp_avg, 16) || !aligned(t.exp_avg_sq, 16) || !aligned(t.copy, 16))
                return EP_ERR_INVALID_ARGUMENT;
            if (eight ? !t.exp_avg_scale || !t.exp_avg_sq_scale || !aligned(t.exp_avg_scale, 4) ||
                            !aligned(t.exp_avg_sq_scale, 4)
                      : t.exp_avg_scale || t.exp_avg_sq_scale)
                return EP_ERR_INVALID_ARGUMENT;
        }
        auto kind = [&](int64_t size, bool wrote, auto at) {
            const size_t from = ranges.size();
            for (int32_t i = 0; i < count; ++i) add(at(tensors[i]), tensors[i].n * size, wrote);
            merge_in(ranges, from);
        };
        auto scales = [&](auto at) {
            const size_t from = ranges.size();
            for (int32_t i = 0; i < count; ++i) add(at(tensors[i]), (tensors[i].n + kBlock - 1) / kBlock * 4, true);
            merge_in(ranges, from);
        };
        using T = ep_adamw_tensor;
        kind(ps, true, [](const T& t) { return (const void*)t.param; });
        kind(gs, false, [](const T& t) { return t.grad; });
        kind(ss, true, [](const T& t) { return (const void*)t.exp_avg; });
        kind(ss, true, [](const T& t) { return (const void*)t.exp_avg_sq; });
        kind(2, true, [](const T& t) { return (const void*)t.copy; });
        if (eight) {
            scales([](const T& t) { return (const void*)t.exp_avg_scale; });
            scales([](const T& t) { return (const void*)t.exp_avg_sq_scale; });
        }
        const size_t from = ranges.size();
        add(cfg->step_dev, 8, false);
        add(cfg->grad_scale_dev, 4, false);
        merge_in(ranges, from);
        if (shared(ranges)) return EP_ERR_INVALID_ARGUMENT;
    } catch (const std::bad_alloc&) {
        return EP_ERR_OUT_OF_MEMORY;
    }

    AdamwArgs a{};
    a.beta1 = (float)cfg->beta1;
    a.rest1 = (float)(1.0 - cfg->beta1);
    a.beta2 = (float)cfg->beta2;
    a.rest2 = (float)(1.0 - cfg->beta2);
    a.decay = (float)(1.0 - cfg->lr * cfg->weight_decay);
    a.eps = (float)cfg->eps;
    a.lr_d = cfg->lr;
    a.beta1_d = cfg->beta1;
    a.beta2_d = cfg->beta2;
    a.grad_scale = cfg->grad_scale;
    a.grad_scale_dev = cfg->grad_scale_dev;
    a.step_dev = cfg->step_dev;
    const double step = cfg->step_dev ? 1.0 : (double)cfg->step;
    a.step_size = (float)(cfg->lr / (1.0 - pow(cfg->beta1, step)));
    a.root_bc2 = (float)sqrt(1.0 - pow(cfg->beta2, step));
    int32_t i = 0;
    while (i < count) {
        int64_t chunks = 0;
        a.count = 0;
        for (; i < count && a.count < kTensors; ++i) {
            const ep_adamw_tensor& t = tensors[i];
            if (t.n == 0) continue;
            const int64_t c = (t.n + kChunk - 1) / kChunk;
            if (a.count > 0 && chunks + c > kMostChunks) break;
            a.first[a.count] = (int32_t)chunks;
            a.t[a.count++] = {t.param, t.grad, t.exp_avg, t.exp_avg_sq, t.exp_avg_scale, t.exp_avg_sq_scale, t.copy, t.n};
            chunks += c;
        }
        if (a.count == 0) break;
        launch(a, cfg->flags, (int)chunks, stream);
        if (hipGetLastError() != hipSuccess) return EP_ERR_HIP;
    }
    return EP_OK;
}
