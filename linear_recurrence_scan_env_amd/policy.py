"""Python binding of the policy operators of liblrs.so: log probabilities of
actions (what log ratios for compute_vtrace and compute_retrace are made of)
and the clipped policy loss with a KL term, with their gradients.

Logits are [num_envs, seq_len, num_actions] (or [seq_len, num_envs,
num_actions], or [tokens, num_actions]), float32, bfloat16 or float16, with any
strides over tokens; the actions' axis must be consecutive.  Everything per
token has the shape of the logits without their last axis: actions are
integers, the rest is float32.  Every call runs on the current stream.

compute_* functions are plain calls; action_log_probs and policy_loss are the
same operators for autograd.
"""
from __future__ import annotations

import torch

from . import api as _api
from .sequence import _F32, _call, _gpu, _ptr, _seq_in, _seq_mask, _seq_out, _strides


class _Tokens:
    """The checked logits and actions of a call, and how its tokens lie."""

    def __init__(self, logits, actions, mask):
        if not isinstance(logits, torch.Tensor):
            raise TypeError("logits must be a torch.Tensor")
        if logits.dim() not in (2, 3):
            raise ValueError(f"logits must have 2 or 3 dimensions, got {logits.dim()}")
        self.axes = (0, 1, None) if logits.dim() == 3 else (0, None, None)
        self.sfx, self.dt, self.dev = _api._suffix(logits, "logits"), logits.dtype, _gpu(logits, "logits")
        self.shape, self.lead = tuple(logits.shape), tuple(logits.shape[:-1])
        self.sizes = (self.lead[0], self.lead[1] if len(self.lead) == 2 else 1, self.shape[-1])
        self.logits = _seq_in(logits, "logits", self.dt, self.shape, None, self.axes)
        if not isinstance(actions, torch.Tensor):
            raise TypeError("actions must be a torch.Tensor")
        if actions.dtype not in (torch.int64, torch.int32, torch.int16, torch.int8, torch.uint8):
            raise TypeError(f"actions must be integers, got {actions.dtype}")
        self.actions = _seq_in(actions.long(), "actions", torch.int64, self.lead, self.dev, self.axes)
        self.mask = _seq_mask(mask, "mask", self.lead, self.dev, self.axes)

    def values(self, x, name, required=True):
        if x is None:
            if required:
                raise ValueError(f"{name} is required")
            return None
        return _seq_in(x, name, _F32, self.lead, self.dev, self.axes)

    def out(self, name):
        return _seq_out(None, name, _F32, self.lead, self.dev, self.axes)

    def grad(self):
        return _seq_out(None, "grad_logits", self.dt, self.shape, self.dev, self.axes)


class _Loss(_Tokens):
    """And those of a loss: what the policy and the reference said, and the coefficients."""

    def __init__(self, logits, actions, old_log_probs, advantages, ref_log_probs, mask, clip, clip_high,
                 kl_coef, entropy_coef, temperature):
        super().__init__(logits, actions, mask)
        self.old = self.values(old_log_probs, "old_log_probs")
        self.adv = self.values(advantages, "advantages")
        self.ref = self.values(ref_log_probs, "ref_log_probs", required=False)
        self.inputs = (self.logits, self.actions, self.old, self.adv, self.ref, self.mask)
        self.coefs = (float(clip), float(clip if clip_high is None else clip_high), float(kl_coef),
                      float(entropy_coef), float(temperature))


def compute_action_log_probs(logits, actions, *, mask=None, temperature=1.0):
    """Log probabilities of the actions taken: returns (log_probs, entropy, lse).

    Per token, with z' = logits / temperature: lse = log sum_v exp(z'_v),
    log_probs = z'_action - lse, entropy = -sum_v p_v log p_v.  Logits of
    -infinity (illegal actions) have probability 0; NaN or +infinity, a token of
    -infinity alone, and an action outside the logits make the token NaN.  Tokens
    where mask is 0 have zeros for all three, whatever their logits hold."""
    k = _Tokens(logits, actions, mask)
    lp, ent, lse = k.out("log_probs"), k.out("entropy"), k.out("lse")
    _call("action_log_probs", k.sfx, k.dev, "compute_action_log_probs",
          *k.sizes, _ptr(k.logits), _ptr(k.actions), _ptr(k.mask), float(temperature), _ptr(lp), _ptr(ent),
          _ptr(lse), _strides(k.logits, k.actions, k.mask, lp, ent, lse))
    return lp.t, ent.t, lse.t


def compute_action_log_probs_backward(grad_log_probs, grad_entropy, logits, actions, entropy, lse, *,
                                      mask=None, temperature=1.0):
    """Gradient of compute_action_log_probs with these inputs and results by the
    logits, in their dtype; grad_log_probs and grad_entropy: 0 if None."""
    k = _Tokens(logits, actions, mask)
    dl = k.values(grad_log_probs, "grad_log_probs", required=False)
    dh = k.values(grad_entropy, "grad_entropy", required=False)
    ent, ls, dz = k.values(entropy, "entropy"), k.values(lse, "lse"), k.grad()
    _call("action_log_probs_backward", k.sfx, k.dev, "compute_action_log_probs_backward",
          *k.sizes, _ptr(dl), _ptr(dh), _ptr(k.logits), _ptr(k.actions), _ptr(k.mask), float(temperature),
          _ptr(ent), _ptr(ls), _ptr(dz), _strides(dl, dh, k.logits, k.actions, k.mask, ent, ls, dz))
    return dz.t


def compute_policy_loss(logits, actions, old_log_probs, advantages, *, ref_log_probs=None, mask=None,
                        clip=0.2, clip_high=None, kl_coef=0.0, entropy_coef=0.0, temperature=1.0):
    """The clipped policy loss of each token: returns (loss, log_probs, entropy, lse).

    With log_probs, entropy and lse as compute_action_log_probs gives them,
    r = exp(log_probs - old_log_probs) and d = ref_log_probs - log_probs,

        loss = -min(r * advantages, clamp(r, 1 - clip, 1 + clip_high) * advantages)
               + kl_coef * (exp(d) - d - 1) - entropy_coef * entropy

    clip_high: clip if None.  ref_log_probs is needed (and read) where kl_coef
    is not 0.  Tokens where mask is 0 have zeros for everything."""
    k = _Loss(logits, actions, old_log_probs, advantages, ref_log_probs, mask, clip, clip_high, kl_coef,
              entropy_coef, temperature)
    out = [k.out(name) for name in ("loss", "log_probs", "entropy", "lse")]
    _call("policy_loss", k.sfx, k.dev, "compute_policy_loss", *k.sizes, *map(_ptr, k.inputs), *k.coefs,
          *map(_ptr, out), _strides(*k.inputs, *out))
    return tuple(x.t for x in out)


def compute_policy_loss_backward(grad_loss, logits, actions, old_log_probs, advantages, entropy, lse, *,
                                 ref_log_probs=None, mask=None, clip=0.2, clip_high=None, kl_coef=0.0,
                                 entropy_coef=0.0, temperature=1.0):
    """Gradient by the logits, in their dtype, of compute_policy_loss with these
    inputs and results, from that of its loss.  Where r is beyond a bound that
    the advantage's sign makes it stop at, the clipped term has no gradient."""
    k = _Loss(logits, actions, old_log_probs, advantages, ref_log_probs, mask, clip, clip_high, kl_coef,
              entropy_coef, temperature)
    g = k.values(grad_loss, "grad_loss")
    ent, ls, dz = k.values(entropy, "entropy"), k.values(lse, "lse"), k.grad()
    _call("policy_loss_backward", k.sfx, k.dev, "compute_policy_loss_backward", *k.sizes, _ptr(g),
          *map(_ptr, k.inputs), *k.coefs, _ptr(ent), _ptr(ls), _ptr(dz), _strides(g, *k.inputs, ent, ls, dz))
    return dz.t


def compute_policy_loss_and_gradient(logits, actions, old_log_probs, advantages, *, weights=None,
                                     ref_log_probs=None, mask=None, clip=0.2, clip_high=None, kl_coef=0.0,
                                     entropy_coef=0.0, temperature=1.0):
    """compute_policy_loss and the gradient of sum(weights * loss) by the logits
    in one pass over them: returns (loss, log_probs, entropy, grad_logits), ready
    for logits.backward(grad_logits).  weights: per token (1 / tokens for the
    mean, times the loss scale in float16), 1 if None; loss is without them."""
    k = _Loss(logits, actions, old_log_probs, advantages, ref_log_probs, mask, clip, clip_high, kl_coef,
              entropy_coef, temperature)
    w = k.values(weights, "weights", required=False)
    out = [k.out(name) for name in ("loss", "log_probs", "entropy")] + [k.grad()]
    _call("policy_loss_and_gradient", k.sfx, k.dev, "compute_policy_loss_and_gradient", *k.sizes,
          *map(_ptr, k.inputs), _ptr(w), *k.coefs, *map(_ptr, out), _strides(*k.inputs, w, *out))
    return tuple(x.t for x in out)


# ----------------------------------------------------------------- autograd

class _ActionLogProbs(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, actions, mask, temperature):
        lp, ent, lse = compute_action_log_probs(logits, actions, mask=mask, temperature=temperature)
        ctx.save_for_backward(logits, actions, mask, ent, lse)
        ctx.temperature = temperature
        ctx.set_materialize_grads(False)
        return lp, ent

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad_lp, grad_ent):
        logits, actions, mask, ent, lse = ctx.saved_tensors
        grad = compute_action_log_probs_backward(grad_lp, grad_ent, logits, actions, ent, lse, mask=mask,
                                                 temperature=ctx.temperature)
        return grad, None, None, None


def action_log_probs(logits, actions, *, mask=None, temperature=1.0):
    """compute_action_log_probs for autograd: returns (log_probs, entropy), both
    differentiable in the logits.  In graphs as policy_loss is."""
    return _ActionLogProbs.apply(logits, actions, mask, temperature)


class _PolicyLoss(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, actions, old_log_probs, advantages, ref_log_probs, mask, coefs):
        loss, lp, ent, lse = compute_policy_loss(logits, actions, old_log_probs, advantages,
                                                 ref_log_probs=ref_log_probs, mask=mask, **coefs)
        ctx.save_for_backward(logits, actions, old_log_probs, advantages, ref_log_probs, mask, ent, lse)
        ctx.coefs = coefs
        ctx.mark_non_differentiable(lp, ent)
        return loss, lp, ent

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad_loss, _lp, _ent):
        logits, actions, old, adv, ref, mask, ent, lse = ctx.saved_tensors
        grad = compute_policy_loss_backward(grad_loss, logits, actions, old, adv, ent, lse,
                                            ref_log_probs=ref, mask=mask, **ctx.coefs)
        return grad, None, None, None, None, None, None


def policy_loss(logits, actions, old_log_probs, advantages, *, ref_log_probs=None, mask=None, clip=0.2,
                clip_high=None, kl_coef=0.0, entropy_coef=0.0, temperature=1.0):
    """compute_policy_loss for autograd: returns (loss, log_probs, entropy), the
    loss differentiable in the logits, the others for the record.  To capture
    both directions into a graph, call the compute_ functions, or first drop
    every eager result of the same logits: torch does not capture a backward
    pass beside those."""
    coefs = dict(clip=clip, clip_high=clip_high, kl_coef=kl_coef, entropy_coef=entropy_coef,
                 temperature=temperature)
    return _PolicyLoss.apply(logits, actions, old_log_probs, advantages, ref_log_probs, mask, coefs)
