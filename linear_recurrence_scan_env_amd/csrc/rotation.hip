// rotation.hip -- workspace size and fp32 entry points of the norm of queries
// and keys with the position rotation.
#include "rotation.hpp"

using namespace lrs;

extern "C" {

size_t lrs_qk_norm_rotation_workspace_bytes(int64_t num_envs, int64_t seq_len, int64_t q_heads,
                                            int64_t k_heads, int64_t dim)
{
    if (!valid_sizes(num_envs, seq_len) || q_heads < 1 || k_heads < 1 || q_heads > 65536 ||
        k_heads > 65536 || dim < 1 || dim > kMaxHeadDim)
        return 0;
    return norm_workspace(num_envs, seq_len, q_heads, k_heads, dim);
}

lrs_status lrs_qk_norm_rotation_f32(int64_t N, int64_t T, int64_t HQ, int64_t HK, int64_t dim,
    int64_t rotary_dim, const float* q, const float* k, const float* q_weight, const float* k_weight,
    const float* table, int64_t max_positions, const int32_t* positions, float eps, int interleaved,
    float* q_out, float* k_out, const int64_t* strides, hipStream_t stream)
{
    return norm_rotation_entry<float>("lrs_qk_norm_rotation_f32", N, T, HQ, HK, dim, rotary_dim,
        q, k,
        q_weight, k_weight, table,
        max_positions, positions, eps, interleaved, q_out,
        k_out, strides, stream);
}

lrs_status lrs_qk_norm_rotation_backward_f32(int64_t N, int64_t T, int64_t HQ, int64_t HK, int64_t dim,
    int64_t rotary_dim, const float* grad_q_out, const float* grad_k_out, const float* q, const float* k,
    const float* q_weight, const float* k_weight, const float* table, int64_t max_positions,
    const int32_t* positions, float eps, int interleaved, float* grad_q, float* grad_k,
    float* grad_q_weight, float* grad_k_weight, const int64_t* strides, void* ws, size_t ws_bytes,
    hipStream_t stream)
{
    return norm_rotation_backward_entry<float>("lrs_qk_norm_rotation_backward_f32", N, T, HQ, HK, dim,
        rotary_dim, grad_q_out, grad_k_out,
        q, k,
        q_weight, k_weight, table,
        max_positions, positions, eps, interleaved, grad_q,
        grad_k, grad_q_weight,
        grad_k_weight, strides, ws, ws_bytes, stream);
}

}  // extern "C"
