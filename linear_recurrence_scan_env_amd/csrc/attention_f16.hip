// attention_f16.hip -- float16 entry points of the windowed attention.
#include "attention.hpp"

using namespace lrs;

extern "C" {

lrs_status lrs_windowed_attention_f16(
    int64_t num_envs, int64_t query_steps, int64_t key_steps, int64_t heads, int64_t kv_heads,
    int64_t key_dim, int64_t value_dim, int64_t window, int64_t sinks, const lrs_f16* q,
    const lrs_f16* k, const lrs_f16* v, const uint8_t* reset, float scale, lrs_f16* out, float* lse,
    const int64_t* strides, void* workspace, size_t workspace_bytes, hipStream_t stream)
{
    return attention_entry<f16_t>(
        "lrs_windowed_attention_f16", num_envs, query_steps, key_steps, heads, kv_heads, key_dim,
        value_dim, window, sinks, reinterpret_cast<const f16_t*>(q), reinterpret_cast<const f16_t*>(k),
        reinterpret_cast<const f16_t*>(v), reset, scale, reinterpret_cast<f16_t*>(out), lse, strides,
        workspace, workspace_bytes, stream);
}

lrs_status lrs_windowed_attention_backward_f16(
    int64_t num_envs, int64_t query_steps, int64_t key_steps, int64_t heads, int64_t kv_heads,
    int64_t key_dim, int64_t value_dim, int64_t window, int64_t sinks, const lrs_f16* grad_out,
    const lrs_f16* q, const lrs_f16* k, const lrs_f16* v, const uint8_t* reset, const lrs_f16* out,
    const float* lse, float scale, lrs_f16* grad_q, lrs_f16* grad_k, lrs_f16* grad_v,
    const int64_t* strides, void* workspace, size_t workspace_bytes, hipStream_t stream)
{
    return attention_backward_entry<f16_t>(
        "lrs_windowed_attention_backward_f16", num_envs, query_steps, key_steps, heads, kv_heads,
        key_dim, value_dim, window, sinks, reinterpret_cast<const f16_t*>(grad_out),
        reinterpret_cast<const f16_t*>(q), reinterpret_cast<const f16_t*>(k),
        reinterpret_cast<const f16_t*>(v), reset, reinterpret_cast<const f16_t*>(out), lse, scale,
        reinterpret_cast<f16_t*>(grad_q), reinterpret_cast<f16_t*>(grad_k),
        reinterpret_cast<f16_t*>(grad_v), strides, workspace, workspace_bytes, stream);
}

lrs_status lrs_windowed_attention_step_f16(
    int64_t num_envs, int64_t heads, int64_t kv_heads, int64_t slots, int64_t sinks, int64_t key_dim,
    int64_t value_dim, const lrs_f16* q, const lrs_f16* k, const lrs_f16* v, lrs_f16* key_cache,
    lrs_f16* value_cache, const int32_t* positions, float scale, lrs_f16* out, const int64_t* strides,
    void* workspace, size_t workspace_bytes, hipStream_t stream)
{
    return attention_step_entry<f16_t>(
        "lrs_windowed_attention_step_f16", num_envs, heads, kv_heads, slots, sinks, key_dim, value_dim,
        reinterpret_cast<const f16_t*>(q), reinterpret_cast<const f16_t*>(k),
        reinterpret_cast<const f16_t*>(v), reinterpret_cast<f16_t*>(key_cache),
        reinterpret_cast<f16_t*>(value_cache), positions, scale, reinterpret_cast<f16_t*>(out), strides,
        workspace, workspace_bytes, stream);
}

lrs_status lrs_windowed_attention_fill_f16(
    int64_t num_envs, int64_t seq_len, int64_t kv_heads, int64_t slots, int64_t sinks, int64_t key_dim,
    int64_t value_dim, const lrs_f16* k, const lrs_f16* v, const int32_t* positions, lrs_f16* key_cache,
    lrs_f16* value_cache, const int64_t* strides, hipStream_t stream)
{
    return attention_fill_entry<f16_t>(
        "lrs_windowed_attention_fill_f16", num_envs, seq_len, kv_heads, slots, sinks, key_dim,
        value_dim, reinterpret_cast<const f16_t*>(k), reinterpret_cast<const f16_t*>(v), positions,
        reinterpret_cast<f16_t*>(key_cache), reinterpret_cast<f16_t*>(value_cache), strides, stream);
}

}  // extern "C"
