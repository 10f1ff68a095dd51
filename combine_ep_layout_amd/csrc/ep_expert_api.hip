// C entry points of the experts' feed-forward: host-side argument checks and
// launches.  The handle is the dispatch/combine entry points' own structure,
// so this file is compiled together with theirs.
#include "ep_api.hip"
#include "ep_ffn.h"

namespace {

constexpr int64_t kMaxExpertMatrix = 1 << 29;   // hidden * inter of one expert (its gate and up rows below 2 GiB)

// Whether [p, p + n) and [q, q + m) share a byte (a null pointer shares none).
bool overlap(const void* p, int64_t n, const void* q, int64_t m) {
    const uintptr_t a = (uintptr_t)p, b = (uintptr_t)q;
    return p && q && n > 0 && m > 0 && a < b + (uintptr_t)m && b < a + (uintptr_t)n;
}

// Checks that both feed-forward calls share.
ep_status check_ffn(const ep_handle* h, uint32_t epoch, int32_t hidden, int32_t inter, int32_t activation) {
    if (!h) return EP_ERR_INVALID_ARGUMENT;
    if (hidden <= 0 || hidden % 8 != 0 || inter <= 0 || inter % 8 != 0) return EP_ERR_INVALID_ARGUMENT;
    if (activation != EP_ACT_SILU && activation != EP_ACT_GELU) return EP_ERR_INVALID_ARGUMENT;
    // the kernels' 32-bit offsets inside one expert's matrix
    if (hidden > kMaxHidden || inter > kMaxHidden || (int64_t)hidden * inter > kMaxExpertMatrix)
        return EP_ERR_UNSUPPORTED;
    if (h->T < 0 || epoch != h->epoch || h->lease) return EP_ERR_HANDLE_STATE;
    // a launch goes to the current device
    int current = -1;
    if (hipGetDevice(&current) != hipSuccess) return EP_ERR_HIP;
    return current == h->device ? EP_OK : EP_ERR_INVALID_ARGUMENT;
}

epk::FfnArgs ffn_args(const ep_handle* h, const void* pool, int32_t hidden, const void* w_gate_up,
                      const void* w_down, int32_t inter, int32_t activation) {
    epk::FfnArgs a{};
    a.pool = pool;
    a.w_gate_up = w_gate_up;
    a.w_down = w_down;
    a.counts = h->counts;
    a.offsets = h->offsets;
    a.E = h->cfg.num_experts;
    a.block_m = h->cfg.block_m;
    a.H = hidden;
    a.I = inter;
    a.slots = (int64_t)h->T * h->cfg.top_k;
    a.num_cu = h->num_cu;
    a.act = activation == EP_ACT_GELU ? epk::kActGelu : epk::kActSilu;
    return a;
}

}  // namespace

extern "C" {

ep_status ep_expert_ffn(const ep_handle* h, uint32_t epoch, const void* pool, int32_t hidden,
                        const void* w_gate_up, const void* w_down, int32_t inter, int32_t activation,
                        void* act, float* gate_up, void* out, hipStream_t stream) {
    ep_status st = check_ffn(h, epoch, hidden, inter, activation);
    if (st != EP_OK) return st;
    if (h->T == 0) return EP_OK;
    if (!pool || !w_gate_up || !w_down || !act || !out || !aligned16(pool) || !aligned16(w_gate_up) ||
        !aligned16(w_down) || !aligned16(act) || !aligned16(gate_up) || !aligned16(out))
        return EP_ERR_INVALID_ARGUMENT;
    // the backward pass that gate_up is kept for reads the pool
    if (out == pool && gate_up) return EP_ERR_INVALID_ARGUMENT;
    const int64_t E = h->cfg.num_experts, rows_h = h->cap * hidden * 2, rows_i = h->cap * inter * 2;
    const int64_t wgu = E * inter * hidden * 4, wd = E * inter * hidden * 2, gu = rows_i * 4;
    // out may be the pool itself; nothing else written may be read or written elsewhere
    const struct { const void* p; int64_t n; } read[] = {{pool, rows_h}, {w_gate_up, wgu}, {w_down, wd}},
        wrote[] = {{act, rows_i}, {gate_up, gu}, {out, rows_h}};
    for (int i = 0; i < 3; ++i) {
        for (int j = i + 1; j < 3; ++j)
            if (overlap(wrote[i].p, wrote[i].n, wrote[j].p, wrote[j].n)) return EP_ERR_INVALID_ARGUMENT;
        for (const auto& r : read)
            if (overlap(wrote[i].p, wrote[i].n, r.p, r.n) && !(wrote[i].p == out && r.p == pool && out == pool))
                return EP_ERR_INVALID_ARGUMENT;
    }
    epk::FfnArgs a = ffn_args(h, pool, hidden, w_gate_up, w_down, inter, activation);
    a.act_rows = act;
    a.gate_up = gate_up;
    a.out = out;
    return hip_status(epk::launch_ffn(a, stream));
}

ep_status ep_expert_ffn_backward(const ep_handle* h, uint32_t epoch, const void* grad_out, const void* pool,
                                 int32_t hidden, const void* w_gate_up, const void* w_down, int32_t inter,
                                 int32_t activation, const void* act, const float* gate_up, uint32_t flags,
                                 void* grad_gate_up, void* grad_pool, void* grad_w_gate_up,
                                 void* grad_w_down, hipStream_t stream) {
    ep_status st = check_ffn(h, epoch, hidden, inter, activation);
    if (st != EP_OK) return st;
    if (flags & ~(EP_GRAD_F32 | EP_GRAD_ACCUMULATE)) return EP_ERR_INVALID_ARGUMENT;
    // sums over calls are kept in fp32 only
    if ((flags & EP_GRAD_ACCUMULATE) && !(flags & EP_GRAD_F32)) return EP_ERR_UNSUPPORTED;
    if (!aligned16(grad_w_gate_up) || !aligned16(grad_w_down)) return EP_ERR_INVALID_ARGUMENT;
    if (h->T > 0 && (!grad_out || !pool || !w_gate_up || !w_down || !act || !gate_up || !grad_gate_up ||
                     !aligned16(grad_out) || !aligned16(pool) || !aligned16(w_gate_up) || !aligned16(w_down) ||
                     !aligned16(act) || !aligned16(gate_up) || !aligned16(grad_gate_up) || !aligned16(grad_pool)))
        return EP_ERR_INVALID_ARGUMENT;
    const int64_t E = h->cfg.num_experts, rows_h = h->cap * hidden * 2, rows_i = h->cap * inter * 2;
    const int64_t matrix = E * inter * hidden, size = (flags & EP_GRAD_F32) ? 4 : 2;
    const struct { const void* p; int64_t n; }
        read[] = {{grad_out, rows_h}, {pool, rows_h}, {w_gate_up, matrix * 4}, {w_down, matrix * 2},
                  {act, rows_i}, {gate_up, rows_i * 4}},
        wrote[] = {{grad_gate_up, rows_i * 2}, {grad_pool, rows_h}, {grad_w_gate_up, 2 * matrix * size},
                   {grad_w_down, matrix * size}};
    for (int i = 0; i < 4; ++i) {
        for (int j = i + 1; j < 4; ++j)
            if (overlap(wrote[i].p, wrote[i].n, wrote[j].p, wrote[j].n)) return EP_ERR_INVALID_ARGUMENT;
        for (const auto& r : read)
            if (overlap(wrote[i].p, wrote[i].n, r.p, r.n)) return EP_ERR_INVALID_ARGUMENT;
    }
    epk::FfnArgs a = ffn_args(h, pool, hidden, w_gate_up, w_down, inter, activation);
    a.act_rows = const_cast<void*>(act);
    a.gate_up = const_cast<float*>(gate_up);
    a.grad_out = grad_out;
    a.grad_gate_up = grad_gate_up;
    a.grad_pool = grad_pool;
    a.grad_w_gate_up = grad_w_gate_up;
    a.grad_w_down = grad_w_down;
    a.grad_f32 = (flags & EP_GRAD_F32) ? 1 : 0;
    a.accumulate = (flags & EP_GRAD_ACCUMULATE) ? 1 : 0;
    return hip_status(epk::launch_ffn_backward(a, stream));
}

}  // extern "C"
