// rotation_f16.hip -- IEEE half entry points of the norm of queries and keys with
// the position rotation.
#include "rotation.hpp"

using namespace lrs;

extern "C" {

lrs_status lrs_qk_norm_rotation_f16(int64_t N, int64_t T, int64_t HQ, int64_t HK, int64_t dim,
    int64_t rotary_dim, const lrs_f16* q, const lrs_f16* k, const lrs_f16* q_weight, const lrs_f16* k_weight,
    const float* table, int64_t max_positions, const int32_t* positions, float eps, int interleaved,
    lrs_f16* q_out, lrs_f16* k_out, const int64_t* strides, hipStream_t stream)
{
    return norm_rotation_entry<f16_t>("lrs_qk_norm_rotation_f16", N, T, HQ, HK, dim, rotary_dim,
        reinterpret_cast<const f16_t*>(q), reinterpret_cast<const f16_t*>(k),
        reinterpret_cast<const f16_t*>(q_weight), reinterpret_cast<const f16_t*>(k_weight), table,
        max_positions, positions, eps, interleaved, reinterpret_cast<f16_t*>(q_out),
        reinterpret_cast<f16_t*>(k_out), strides, stream);
}

lrs_status lrs_qk_norm_rotation_backward_f16(int64_t N, int64_t T, int64_t HQ, int64_t HK, int64_t dim,
    int64_t rotary_dim, const lrs_f16* grad_q_out, const lrs_f16* grad_k_out, const lrs_f16* q, const lrs_f16* k,
    const lrs_f16* q_weight, const lrs_f16* k_weight, const float* table, int64_t max_positions,
    const int32_t* positions, float eps, int interleaved, lrs_f16* grad_q, lrs_f16* grad_k,
    lrs_f16* grad_q_weight, lrs_f16* grad_k_weight, const int64_t* strides, void* ws, size_t ws_bytes,
    hipStream_t stream)
{
    return norm_rotation_backward_entry<f16_t>("lrs_qk_norm_rotation_backward_f16", N, T, HQ, HK, dim,
        rotary_dim, reinterpret_cast<const f16_t*>(grad_q_out), reinterpret_cast<const f16_t*>(grad_k_out),
        reinterpret_cast<const f16_t*>(q), reinterpret_cast<const f16_t*>(k),
        reinterpret_cast<const f16_t*>(q_weight), reinterpret_cast<const f16_t*>(k_weight), table,
        max_positions, positions, eps, interleaved, reinterpret_cast<f16_t*>(grad_q),
        reinterpret_cast<f16_t*>(grad_k), reinterpret_cast<f16_t*>(grad_q_weight),
        reinterpret_cast<f16_t*>(grad_k_weight), strides, ws, ws_bytes, stream);
}

}  // extern "C"
