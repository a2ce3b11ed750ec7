// policy_bf16.hip -- bfloat16 entry points of the log probabilities of actions and the
// clipped policy loss.
#include "policy.hpp"

using namespace lrs;

extern "C" {

lrs_status lrs_action_log_probs_bf16(
    int64_t num_envs, int64_t seq_len, int64_t num_actions, const lrs_bf16* logits, const int64_t*
    actions, const uint8_t* mask, float temperature, float* log_probs, float* entropy, float* lse, const
    int64_t* strides, hipStream_t stream)
{
    return action_log_probs_entry<bf16_t>(
        "lrs_action_log_probs_bf16", num_envs, seq_len, num_actions, reinterpret_cast<const
        bf16_t*>(logits), actions, mask, temperature, log_probs, entropy, lse, strides, stream);
}

lrs_status lrs_action_log_probs_backward_bf16(
    int64_t num_envs, int64_t seq_len, int64_t num_actions, const float* grad_log_probs, const float*
    grad_entropy, const lrs_bf16* logits, const int64_t* actions, const uint8_t* mask, float
    temperature, const float* entropy, const float* lse, lrs_bf16* grad_logits, const int64_t* strides,
    hipStream_t stream)
{
    return action_log_probs_backward_entry<bf16_t>(
        "lrs_action_log_probs_backward_bf16", num_envs, seq_len, num_actions, grad_log_probs,
        grad_entropy, reinterpret_cast<const bf16_t*>(logits), actions, mask, temperature, entropy, lse,
        reinterpret_cast<bf16_t*>(grad_logits), strides, stream);
}

lrs_status lrs_policy_loss_bf16(
    int64_t num_envs, int64_t seq_len, int64_t num_actions, const lrs_bf16* logits, const int64_t*
    actions, const float* old_log_probs, const float* advantages, const float* ref_log_probs, const
    uint8_t* mask, float clip, float clip_high, float kl_coef, float entropy_coef, float temperature,
    float* loss, float* log_probs, float* entropy, float* lse, const int64_t* strides, hipStream_t
    stream)
{
    return policy_loss_entry<bf16_t>(
        "lrs_policy_loss_bf16", num_envs, seq_len, num_actions, reinterpret_cast<const bf16_t*>(logits),
        actions, old_log_probs, advantages, ref_log_probs, mask, clip, clip_high, kl_coef, entropy_coef,
        temperature, loss, log_probs, entropy, lse, strides, stream);
}

lrs_status lrs_policy_loss_backward_bf16(
    int64_t num_envs, int64_t seq_len, int64_t num_actions, const float* grad_loss, const lrs_bf16*
    logits, const int64_t* actions, const float* old_log_probs, const float* advantages, const float*
    ref_log_probs, const uint8_t* mask, float clip, float clip_high, float kl_coef, float entropy_coef,
    float temperature, const float* entropy, const float* lse, lrs_bf16* grad_logits, const int64_t*
    strides, hipStream_t stream)
{
    return policy_loss_backward_entry<bf16_t>(
        "lrs_policy_loss_backward_bf16", num_envs, seq_len, num_actions, grad_loss,
        reinterpret_cast<const bf16_t*>(logits), actions, old_log_probs, advantages, ref_log_probs,
        mask, clip, clip_high, kl_coef, entropy_coef, temperature, entropy, lse,
        reinterpret_cast<bf16_t*>(grad_logits), strides, stream);
}

lrs_status lrs_policy_loss_and_gradient_bf16(
    int64_t num_envs, int64_t seq_len, int64_t num_actions, const lrs_bf16* logits, const int64_t*
    actions, const float* old_log_probs, const float* advantages, const float* ref_log_probs, const
    uint8_t* mask, const float* weights, float clip, float clip_high, float kl_coef, float entropy_coef,
    float temperature, float* loss, float* log_probs, float* entropy, lrs_bf16* grad_logits, const
    int64_t* strides, hipStream_t stream)
{
    return policy_loss_and_gradient_entry<bf16_t>(
        "lrs_policy_loss_and_gradient_bf16", num_envs, seq_len, num_actions, reinterpret_cast<const
        bf16_t*>(logits), actions, old_log_probs, advantages, ref_log_probs, mask, weights, clip,
        clip_high, kl_coef, entropy_coef, temperature, loss, log_probs, entropy,
        reinterpret_cast<bf16_t*>(grad_logits), strides, stream);
}

}  // extern "C"
