// attention_bf16.hip -- bfloat16 entry points of the windowed attention.
#include "attention.hpp"

using namespace lrs;

extern "C" {

lrs_status lrs_windowed_attention_bf16(
    int64_t num_envs, int64_t query_steps, int64_t key_steps, int64_t heads, int64_t kv_heads,
    int64_t key_dim, int64_t value_dim, int64_t window, int64_t sinks, const lrs_bf16* q,
    const lrs_bf16* k, const lrs_bf16* v, const uint8_t* reset, float scale, lrs_bf16* out, float* lse,
    const int64_t* strides, void* workspace, size_t workspace_bytes, hipStream_t stream)
{
    return attention_entry<bf16_t>(
        "lrs_windowed_attention_bf16", num_envs, query_steps, key_steps, heads, kv_heads, key_dim,
        value_dim, window, sinks, reinterpret_cast<const bf16_t*>(q),
        reinterpret_cast<const bf16_t*>(k), reinterpret_cast<const bf16_t*>(v), reset, scale,
        reinterpret_cast<bf16_t*>(out), lse, strides, workspace, workspace_bytes, stream);
}

lrs_status lrs_windowed_attention_backward_bf16(
    int64_t num_envs, int64_t query_steps, int64_t key_steps, int64_t heads, int64_t kv_heads,
    int64_t key_dim, int64_t value_dim, int64_t window, int64_t sinks, const lrs_bf16* grad_out,
    const lrs_bf16* q, const lrs_bf16* k, const lrs_bf16* v, const uint8_t* reset, const lrs_bf16* out,
    const float* lse, float scale, lrs_bf16* grad_q, lrs_bf16* grad_k, lrs_bf16* grad_v,
    const int64_t* strides, void* workspace, size_t workspace_bytes, hipStream_t stream)
{
    return attention_backward_entry<bf16_t>(
        "lrs_windowed_attention_backward_bf16", num_envs, query_steps, key_steps, heads, kv_heads,
        key_dim, value_dim, window, sinks, reinterpret_cast<const bf16_t*>(grad_out),
        reinterpret_cast<const bf16_t*>(q), reinterpret_cast<const bf16_t*>(k),
        reinterpret_cast<const bf16_t*>(v), reset, reinterpret_cast<const bf16_t*>(out), lse, scale,
        reinterpret_cast<bf16_t*>(grad_q), reinterpret_cast<bf16_t*>(grad_k),
        reinterpret_cast<bf16_t*>(grad_v), strides, workspace, workspace_bytes, stream);
}

lrs_status lrs_windowed_attention_step_bf16(
    int64_t num_envs, int64_t heads, int64_t kv_heads, int64_t slots, int64_t sinks, int64_t key_dim,
    int64_t value_dim, const lrs_bf16* q, const lrs_bf16* k, const lrs_bf16* v, lrs_bf16* key_cache,
    lrs_bf16* value_cache, const int32_t* positions, float scale, lrs_bf16* out, const int64_t* strides,
    void* workspace, size_t workspace_bytes, hipStream_t stream)
{
    return attention_step_entry<bf16_t>(
        "lrs_windowed_attention_step_bf16", num_envs, heads, kv_heads, slots, sinks, key_dim, value_dim,
        reinterpret_cast<const bf16_t*>(q), reinterpret_cast<const bf16_t*>(k),
        reinterpret_cast<const bf16_t*>(v), reinterpret_cast<bf16_t*>(key_cache),
        reinterpret_cast<bf16_t*>(value_cache), positions, scale, reinterpret_cast<bf16_t*>(out),
        strides, workspace, workspace_bytes, stream);
}

lrs_status lrs_windowed_attention_fill_bf16(
    int64_t num_envs, int64_t seq_len, int64_t kv_heads, int64_t slots, int64_t sinks, int64_t key_dim,
    int64_t value_dim, const lrs_bf16* k, const lrs_bf16* v, const int32_t* positions,
    lrs_bf16* key_cache, lrs_bf16* value_cache, const int64_t* strides, hipStream_t stream)
{
    return attention_fill_entry<bf16_t>(
        "lrs_windowed_attention_fill_bf16", num_envs, seq_len, kv_heads, slots, sinks, key_dim,
        value_dim, reinterpret_cast<const bf16_t*>(k), reinterpret_cast<const bf16_t*>(v), positions,
        reinterpret_cast<bf16_t*>(key_cache), reinterpret_cast<bf16_t*>(value_cache), strides, stream);
}

}  // extern "C"
