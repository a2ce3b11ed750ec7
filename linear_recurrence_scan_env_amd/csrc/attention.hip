// attention.hip -- workspace sizes and fp32 entry points of the windowed attention.
#include "attention.hpp"

using namespace lrs;

extern "C" {

size_t lrs_windowed_attention_workspace_bytes(int64_t num_envs, int64_t query_steps, int64_t key_steps,
                                              int64_t heads, int64_t kv_heads, int64_t key_dim, int64_t value_dim,
                                              int64_t window, int64_t sinks, int has_reset, int backward)
{
    if (!valid_sizes(num_envs, query_steps) || !valid_sizes(num_envs, key_steps) || key_steps < query_steps ||
        !att_sizes_ok(heads, kv_heads, key_dim, value_dim) || window < 1 || sinks < 0)
        return 0;
    return att_workspace(num_envs, query_steps, key_steps, heads, kv_heads, key_dim, value_dim, window, sinks,
                         has_reset != 0, backward != 0)
        .bytes;
}

size_t lrs_windowed_attention_step_workspace_bytes(int64_t num_envs, int64_t heads, int64_t kv_heads,
                                                   int64_t slots, int64_t sinks, int64_t key_dim, int64_t value_dim)
{
    AttStepArgs x{};
    return fill_step(x, num_envs, heads, kv_heads, slots, sinks, key_dim, value_dim) ? step_workspace(x, num_envs) : 0;
}

lrs_status lrs_windowed_attention_f32(
    int64_t num_envs, int64_t query_steps, int64_t key_steps, int64_t heads, int64_t kv_heads,
    int64_t key_dim, int64_t value_dim, int64_t window, int64_t sinks, const float* q, const float* k,
    const float* v, const uint8_t* reset, float scale, float* out, float* lse, const int64_t* strides,
    void* workspace, size_t workspace_bytes, hipStream_t stream)
{
    return attention_entry<float>(
        "lrs_windowed_attention_f32", num_envs, query_steps, key_steps, heads, kv_heads, key_dim,
        value_dim, window, sinks, q, k, v, reset, scale, out, lse, strides, workspace, workspace_bytes,
        stream);
}

lrs_status lrs_windowed_attention_backward_f32(
    int64_t num_envs, int64_t query_steps, int64_t key_steps, int64_t heads, int64_t kv_heads,
    int64_t key_dim, int64_t value_dim, int64_t window, int64_t sinks, const float* grad_out,
    const float* q, const float* k, const float* v, const uint8_t* reset, const float* out,
    const float* lse, float scale, float* grad_q, float* grad_k, float* grad_v, const int64_t* strides,
    void* workspace, size_t workspace_bytes, hipStream_t stream)
{
    return attention_backward_entry<float>(
        "lrs_windowed_attention_backward_f32", num_envs, query_steps, key_steps, heads, kv_heads,
        key_dim, value_dim, window, sinks, grad_out, q, k, v, reset, out, lse, scale, grad_q, grad_k,
        grad_v, strides, workspace, workspace_bytes, stream);
}

lrs_status lrs_windowed_attention_step_f32(
    int64_t num_envs, int64_t heads, int64_t kv_heads, int64_t slots, int64_t sinks, int64_t key_dim,
    int64_t value_dim, const float* q, const float* k, const float* v, float* key_cache,
    float* value_cache, const int32_t* positions, float scale, float* out, const int64_t* strides,
    void* workspace, size_t workspace_bytes, hipStream_t stream)
{
    return attention_step_entry<float>(
        "lrs_windowed_attention_step_f32", num_envs, heads, kv_heads, slots, sinks, key_dim, value_dim,
        q, k, v, key_cache, value_cache, positions, scale, out, strides, workspace, workspace_bytes,
        stream);
}

lrs_status lrs_windowed_attention_fill_f32(
    int64_t num_envs, int64_t seq_len, int64_t kv_heads, int64_t slots, int64_t sinks, int64_t key_dim,
    int64_t value_dim, const float* k, const float* v, const int32_t* positions, float* key_cache,
    float* value_cache, const int64_t* strides, hipStream_t stream)
{
    return attention_fill_entry<float>(
        "lrs_windowed_attention_fill_f32", num_envs, seq_len, kv_heads, slots, sinks, key_dim,
        value_dim, k, v, positions, key_cache, value_cache, strides, stream);
}

}  // extern "C"
