// policy.hip -- fp32 entry points of the log probabilities of actions and the
// clipped policy loss.
#include "policy.hpp"

using namespace lrs;

extern "C" {

lrs_status lrs_action_log_probs_f32(
    int64_t num_envs, int64_t seq_len, int64_t num_actions, const float* logits, const int64_t* actions,
    const uint8_t* mask, float temperature, float* log_probs, float* entropy, float* lse, const int64_t*
    strides, hipStream_t stream)
{
    return action_log_probs_entry<float>(
        "lrs_action_log_probs_f32", num_envs, seq_len, num_actions, logits, actions, mask, temperature,
        log_probs, entropy, lse, strides, stream);
}

lrs_status lrs_action_log_probs_backward_f32(
    int64_t num_envs, int64_t seq_len, int64_t num_actions, const float* grad_log_probs, const float*
    grad_entropy, const float* logits, const int64_t* actions, const uint8_t* mask, float temperature,
    const float* entropy, const float* lse, float* grad_logits, const int64_t* strides, hipStream_t
    stream)
{
    return action_log_probs_backward_entry<float>(
        "lrs_action_log_probs_backward_f32", num_envs, seq_len, num_actions, grad_log_probs,
        grad_entropy, logits, actions, mask, temperature, entropy, lse, grad_logits, strides, stream);
}

lrs_status lrs_policy_loss_f32(
    int64_t num_envs, int64_t seq_len, int64_t num_actions, const float* logits, const int64_t* actions,
    const float* old_log_probs, const float* advantages, const float* ref_log_probs, const uint8_t*
    mask, float clip, float clip_high, float kl_coef, float entropy_coef, float temperature, float*
    loss, float* log_probs, float* entropy, float* lse, const int64_t* strides, hipStream_t stream)
{
    return policy_loss_entry<float>(
        "lrs_policy_loss_f32", num_envs, seq_len, num_actions, logits, actions, old_log_probs,
        advantages, ref_log_probs, mask, clip, clip_high, kl_coef, entropy_coef, temperature, loss,
        log_probs, entropy, lse, strides, stream);
}

lrs_status lrs_policy_loss_backward_f32(
    int64_t num_envs, int64_t seq_len, int64_t num_actions, const float* grad_loss, const float* logits,
    const int64_t* actions, const float* old_log_probs, const float* advantages, const float*
    ref_log_probs, const uint8_t* mask, float clip, float clip_high, float kl_coef, float entropy_coef,
    float temperature, const float* entropy, const float* lse, float* grad_logits, const int64_t*
    strides, hipStream_t stream)
{
    return policy_loss_backward_entry<float>(
        "lrs_policy_loss_backward_f32", num_envs, seq_len, num_actions, grad_loss, logits, actions,
        old_log_probs, advantages, ref_log_probs, mask, clip, clip_high, kl_coef, entropy_coef,
        temperature, entropy, lse, grad_logits, strides, stream);
}

lrs_status lrs_policy_loss_and_gradient_f32(
    int64_t num_envs, int64_t seq_len, int64_t num_actions, const float* logits, const int64_t* actions,
    const float* old_log_probs, const float* advantages, const float* ref_log_probs, const uint8_t*
    mask, const float* weights, float clip, float clip_high, float kl_coef, float entropy_coef, float
    temperature, float* loss, float* log_probs, float* entropy, float* grad_logits, const int64_t*
    strides, hipStream_t stream)
{
    return policy_loss_and_gradient_entry<float>(
        "lrs_policy_loss_and_gradient_f32", num_envs, seq_len, num_actions, logits, actions,
        old_log_probs, advantages, ref_log_probs, mask, weights, clip, clip_high, kl_coef, entropy_coef,
        temperature, loss, log_probs, entropy, grad_logits, strides, stream);
}

}  // extern "C"
