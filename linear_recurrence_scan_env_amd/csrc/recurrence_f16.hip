// recurrence_f16.hip -- IEEE half entry points of the gated recurrence.
#include "recurrence.hpp"

using namespace lrs;

extern "C" {

lrs_status lrs_gated_recurrence_f16(int64_t N, int64_t T, int64_t H, int64_t KV, int64_t dk, int64_t dv,
    const lrs_f16* q, const lrs_f16* k, const lrs_f16* v, const lrs_f16* log_decay, const uint8_t* reset,
    const float* initial_state, float scale, lrs_f16* out, float* final_state, const int64_t* strides,
    void* ws, size_t ws_bytes, hipStream_t stream)
{
    return recurrence_entry<f16_t>("lrs_gated_recurrence_f16", N, T, H, KV, dk, dv,
        reinterpret_cast<const f16_t*>(q), reinterpret_cast<const f16_t*>(k),
        reinterpret_cast<const f16_t*>(v), reinterpret_cast<const f16_t*>(log_decay), reset,
        initial_state, scale, reinterpret_cast<f16_t*>(out), final_state, strides, ws, ws_bytes, stream);
}

lrs_status lrs_gated_recurrence_backward_f16(int64_t N, int64_t T, int64_t H, int64_t KV, int64_t dk,
    int64_t dv, const lrs_f16* grad_out, const lrs_f16* q, const lrs_f16* k, const lrs_f16* v,
    const lrs_f16* log_decay, const uint8_t* reset, const float* initial_state,
    const float* grad_final_state, float scale, lrs_f16* grad_q, lrs_f16* grad_k, lrs_f16* grad_v,
    lrs_f16* grad_log_decay, float* grad_initial_state, const int64_t* strides, void* ws, size_t ws_bytes,
    hipStream_t stream)
{
    return recurrence_backward_entry<f16_t>("lrs_gated_recurrence_backward_f16", N, T, H, KV, dk, dv,
        reinterpret_cast<const f16_t*>(grad_out), reinterpret_cast<const f16_t*>(q),
        reinterpret_cast<const f16_t*>(k), reinterpret_cast<const f16_t*>(v),
        reinterpret_cast<const f16_t*>(log_decay), reset, initial_state, grad_final_state, scale,
        reinterpret_cast<f16_t*>(grad_q), reinterpret_cast<f16_t*>(grad_k),
        reinterpret_cast<f16_t*>(grad_v), reinterpret_cast<f16_t*>(grad_log_decay), grad_initial_state,
        strides, ws, ws_bytes, stream);
}

lrs_status lrs_gated_recurrence_step_f16(int64_t N, int64_t H, int64_t KV, int64_t dk, int64_t dv,
    const lrs_f16* q, const lrs_f16* k, const lrs_f16* v, const lrs_f16* log_decay, const uint8_t* reset,
    const float* state, float scale, lrs_f16* out, float* next_state, const int64_t* strides,
    hipStream_t stream)
{
    return recurrence_step_entry<f16_t>("lrs_gated_recurrence_step_f16", N, H, KV, dk, dv,
        reinterpret_cast<const f16_t*>(q), reinterpret_cast<const f16_t*>(k),
        reinterpret_cast<const f16_t*>(v), reinterpret_cast<const f16_t*>(log_decay), reset, state,
        scale, reinterpret_cast<f16_t*>(out), next_state, strides, stream);
}

}  // extern "C"
