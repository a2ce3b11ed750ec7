"""The attention policy example: it runs, acting by single steps agrees with the rollout
computed at once, and the gradients of its loss are those of the same formulas in
torch operations."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def plain_losses(policy, obs, first, positions, act, old, scaled, value_target):
    """The same loss from elementary operations in 64 bits on the CPU."""
    import attention_policy as ex
    import attention_reference as ref
    p = {k: v.detach().double().cpu().requires_grad_() for k, v in policy.named_parameters()}
    lin = lambda x, name: x @ p[name + ".weight"].t() + p[name + ".bias"]  # noqa: E731
    obs, old, scaled, value_target = (x.double().cpu() for x in (obs, old, scaled, value_target))
    act, positions = act.cpu(), positions.cpu().long()
    mem = policy.memory
    x = torch.tanh(lin(obs, "embed"))
    q, k, v = (t.unflatten(-1, (-1, mem.dim)) for t in lin(x, "memory.into").split(mem.sizes, -1))
    cos, sin = mem.table.double().cpu()[positions].unsqueeze(2).chunk(2, -1)
    rot = cos.shape[-1]

    def prepared(y, w):
        y = y / (y.square().mean(-1, keepdim=True) + 1e-6).sqrt() * w
        a, b = y[..., :rot], y[..., rot:2 * rot]
        return torch.cat([a * cos - b * sin, b * cos + a * sin, y[..., 2 * rot:]], -1)
    q, k = prepared(q, p["memory.q_weight"]), prepared(k, p["memory.k_weight"])
    k, v = (t.repeat_interleave(q.shape[2] // mem.kv, 2) for t in (k, v))
    ok = ref.seen(obs.shape[1], obs.shape[1], ex.WINDOW, ex.SINKS, first.cpu())[:, None]
    s = torch.einsum("nihd,njhd->nhij", q, k) * mem.dim ** -0.5
    y = torch.einsum("nhij,njhd->nihd", torch.softmax(s.masked_fill(~ok, -torch.inf), -1), v)
    y = lin(x + lin(y.flatten(-2), "memory.back"), "heads")
    logp = torch.log_softmax(y[..., :ex.CUES], -1)
    lp = logp.gather(-1, act[..., None])[..., 0]
    r = torch.exp(lp - old)
    loss = -torch.minimum(r * scaled, r.clamp(0.8, 1.2) * scaled) + 0.01 * (logp.exp() * logp).sum(-1)
    loss = loss.mean() + 0.5 * (y[..., ex.CUES] - value_target).square().mean()
    loss.backward()
    return loss.item(), {k: v.grad for k, v in p.items()}, lp


def test_runs_and_acting_agrees_with_training():
    import attention_policy as ex
    history, drift = ex.main(["--updates", "3", "--envs", "64", "--steps", "40", "--quiet"])
    assert len(history) == 3 and all(0 <= h <= 1 for h in history)
    # both compute the same float32 formulas in another order of sums over 32 and 64 elements
    assert drift < 1e-4


def test_gradients():
    import attention_policy as ex
    import linear_recurrence_scan_env_amd as lrs
    torch.manual_seed(1)
    device = torch.device("cuda")
    policy = ex.Policy().to(device)
    env = ex.Recall(8, device, 1)
    obs, first, positions, act, old, rew, done = ex.rollout(policy, env, 30)
    with torch.no_grad():  # off the policy that acted, by up to a factor of 1.35: some ratios are clipped
        old = old + 0.3 * torch.linspace(-1, 1, old.numel(), device=device).view_as(old)
    loss, now = ex.losses(policy, obs, first, positions, act, old, rew, done)
    loss.backward()
    with torch.no_grad():
        value = policy.heads(policy.memory(policy.observe(obs), first, positions))[..., ex.CUES]
        adv = lrs.compute_gae(rew, value, done, 0.95, 0.9, bootstrap_value=value[:, -1])
        scaled = (adv - adv.mean()) / (adv.std() + 1e-6)
    want, grads, lp = plain_losses(policy, obs, first, positions, act, old, scaled, adv + value)
    assert (now.double().cpu() - lp).abs().max() < 1e-4
    assert abs(loss.item() - want) < 1e-4 * (1 + abs(want))
    assert set(grads) == {k for k, _ in policy.named_parameters()}
    for name, p in policy.named_parameters():
        g = grads[name]
        # float32 through six layers of sums of up to 128 terms: 128 * 6 * 2^-24 is 5e-5 of the size
        assert (p.grad.double().cpu() - g).norm() <= 2e-4 * g.norm() + 1e-7, name
