// The experts' activations on the device.  Not installed; callers use
// include/ep_layout.h.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace epk {

enum ActKind : int32_t {
    kActSilu = 0,
    kActGelu = 1,               // tanh form
};

namespace {

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
        const float s = sigmoid_f(2.0f * gelu_inner(g)), d = s * (1.0f - s);
        value = g * s;
        // far out, where d is zero, g squared may be infinite
        slope = d > 0.0f ? s + 2.0f * g * d * 0.7978845608028654f * (1.0f + 3 * 0.044715f * g * g) : s;
    } else {
        const float s = sigmoid_f(g);
        value = g * s;
        slope = s * (1.0f + g * (1.0f - s));
    }
}

}  // namespace
}  // namespace epk
