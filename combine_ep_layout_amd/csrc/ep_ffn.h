// Internal interface between the C ABI (ep_api.hip) and the feed-forward
// kernels (ep_ffn.hip).  Not installed; callers use include/ep_layout.h.
#pragma once

#include <stdint.h>
#include <hip/hip_runtime.h>

namespace epk {

enum ActKind : int32_t {
    kActSilu = 0,
    kActGelu = 1,               // tanh form
};

// One grouped product (see ep_ffn.hip).
struct GemmArgs {
    const void* a;              // bf16 rows, leading dimension a_ld (elements)
    const void* b;              // bf16 rows, leading dimension b_ld; weights of expert e at b + e * b_expert
    void* c;
    const void* save;           // fp32 [cap, 2N] pre-activations: written (may be null) or read
    const int32_t* counts;      // [E] rows of each expert
    const int32_t* offsets;     // [E+1] first pool tile of each expert
    int32_t E;
    int32_t block_m;
    int32_t M;                  // rows of a weight gradient
    int32_t N;
    int32_t K;
    int32_t a_ld;
    int32_t b_ld;
    int64_t b_expert;
    int64_t slots;              // num_tokens * top_k: bound on the rows
    int32_t num_cu;
    int32_t act;                // ActKind
    int32_t out_f32;            // weight gradients: fp32 instead of bf16
    int32_t accumulate;         // weight gradients: added to what is there (fp32 only)
};

struct FfnArgs {
    const void* pool;           // bf16 [cap, H]
    const void* w_gate_up;      // bf16 [E, 2I, H]
    const void* w_down;         // bf16 [E, H, I]
    void* act_rows;             // bf16 [cap, I]
    void* gate_up;              // fp32 [cap, 2I]; forward: may be null
    void* out;                  // bf16 [cap, H]
    // backward
    const void* grad_out;       // bf16 [cap, H]
    void* grad_gate_up;         // bf16 [cap, 2I]
    void* grad_pool;            // bf16 [cap, H]; may be null
    void* grad_w_gate_up;       // [E, 2I, H]; may be null
    void* grad_w_down;          // [E, H, I]; may be null
    int32_t grad_f32;
    int32_t accumulate;
    const int32_t* counts;
    const int32_t* offsets;
    int32_t E;
    int32_t block_m;
    int32_t H;
    int32_t I;
    int64_t slots;
    int32_t num_cu;
    int32_t act;
};

hipError_t launch_ffn(const FfnArgs& a, hipStream_t stream);
hipError_t launch_ffn_backward(const FfnArgs& a, hipStream_t stream);

}  // namespace epk
