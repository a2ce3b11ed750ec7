// recurrence.hip -- workspace size and fp32 entry points of the gated recurrence.
#include "recurrence.hpp"

using namespace lrs;

extern "C" {

size_t lrs_gated_recurrence_workspace_bytes(int64_t num_envs, int64_t seq_len, int64_t heads,
                                            int64_t kv_heads, int64_t key_dim, int64_t value_dim,
                                            int backward)
{
    if (check_recurrence("", num_envs, seq_len, heads, kv_heads, key_dim, value_dim, 1.0f) != LRS_OK)
        return 0;
    return plan_recurrence(num_envs, seq_len, heads, kv_heads, key_dim, value_dim, backward != 0).bytes;
}

lrs_status lrs_gated_recurrence_f32(int64_t N, int64_t T, int64_t H, int64_t KV, int64_t dk, int64_t dv,
    const float* q, const float* k, const float* v, const float* log_decay, const uint8_t* reset,
    const float* initial_state, float scale, float* out, float* final_state, const int64_t* strides,
    void* ws, size_t ws_bytes, hipStream_t stream)
{
    return recurrence_entry<float>("lrs_gated_recurrence_f32", N, T, H, KV, dk, dv,
        q, k,
        v, log_decay, reset,
        initial_state, scale, out, final_state, strides, ws, ws_bytes, stream);
}

lrs_status lrs_gated_recurrence_backward_f32(int64_t N, int64_t T, int64_t H, int64_t KV, int64_t dk,
    int64_t dv, const float* grad_out, const float* q, const float* k, const float* v,
    const float* log_decay, const uint8_t* reset, const float* initial_state,
    const float* grad_final_state, float scale, float* grad_q, float* grad_k, float* grad_v,
    float* grad_log_decay, float* grad_initial_state, const int64_t* strides, void* ws, size_t ws_bytes,
    hipStream_t stream)
{
    return recurrence_backward_entry<float>("lrs_gated_recurrence_backward_f32", N, T, H, KV, dk, dv,
        grad_out, q,
        k, v,
        log_decay, reset, initial_state, grad_final_state, scale,
        grad_q, grad_k,
        grad_v, grad_log_decay, grad_initial_state,
        strides, ws, ws_bytes, stream);
}

lrs_status lrs_gated_recurrence_step_f32(int64_t N, int64_t H, int64_t KV, int64_t dk, int64_t dv,
    const float* q, const float* k, const float* v, const float* log_decay, const uint8_t* reset,
    const float* state, float scale, float* out, float* next_state, const int64_t* strides,
    hipStream_t stream)
{
    return recurrence_step_entry<float>("lrs_gated_recurrence_step_f32", N, H, KV, dk, dv,
        q, k,
        v, log_decay, reset, state,
        scale, out, next_state, strides, stream);
}

}  // extern "C"
