"""A policy whose memory is attention, on rollouts: windowed attention over the last
steps and the first step of each episode, trained with the clipped policy loss on
advantages from compute_gae.

The task is that of recurrent_policy.py: the first observation of an episode shows
a cue, and at its last step, up to twelve steps on, the action that matches the cue
is rewarded.  The window is shorter than that: only the first step of an episode,
which stays visible, tells.

    acting    one compute_qk_norm_rotation and one compute_windowed_attention_step
              over the caches of all environments (positions within episodes say
              where each stands; nothing is cleared when an episode ends), and
              compute_action_log_probs of what was done;
    training  several passes over the rollout: qk_norm_rotation and
              windowed_attention (autograd) with episode starts as resets,
              policy_loss on advantages from compute_gae.

    python examples/attention_policy.py [--updates 40] [--envs 256] [--steps 64]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
from recurrent_policy import CUES, Recall, lrs  # noqa: E402

WINDOW, SINKS = 4, 1


class AttentionLayer(torch.nn.Module):
    """Query and key heads, normed and rotated by the position within the episode, into the
    windowed attention; query heads share key heads."""

    def __init__(self, width, heads=4, kv_heads=2, head_dim=32, max_positions=512):
        super().__init__()
        self.kv, self.dim = kv_heads, head_dim
        self.sizes = [heads * head_dim, kv_heads * head_dim, kv_heads * head_dim]
        self.into = torch.nn.Linear(width, sum(self.sizes))
        self.back = torch.nn.Linear(heads * head_dim, width)
        self.q_weight = torch.nn.Parameter(torch.ones(head_dim))
        self.k_weight = torch.nn.Parameter(torch.ones(head_dim))
        self.register_buffer("table", lrs.rotary_table(max_positions, head_dim // 2, device="cpu"))

    def caches(self, num_envs, device):
        shape = (num_envs, SINKS + WINDOW, self.kv, self.dim)
        return torch.zeros(shape, device=device), torch.zeros(shape, device=device)

    def parts(self, x):
        """[..., width] -> q, k, v [..., heads, dim], views of one projection."""
        return (t.unflatten(-1, (-1, self.dim)) for t in self.into(x).split(self.sizes, -1))

    def forward(self, x, reset, positions):
        """A rollout [num_envs, seq_len, width] whose rows begin with an episode."""
        q, k, v = self.parts(x)
        q, k = lrs.qk_norm_rotation(q, k, self.q_weight, self.k_weight, self.table, positions)
        y = lrs.windowed_attention(q, k, v, window=WINDOW, sinks=SINKS, reset=reset)
        return x + self.back(y.flatten(-2))

    @torch.no_grad()
    def step(self, x, positions, caches):
        """One step of every environment; the caches are updated in place."""
        q, k, v = self.parts(x[:, None])
        q, k = lrs.compute_qk_norm_rotation(q, k, self.q_weight, self.k_weight, self.table, positions[:, None])
        y = lrs.compute_windowed_attention_step(q[:, 0], k[:, 0], v[:, 0], *caches, positions, sinks=SINKS)
        return x + self.back(y.flatten(-2))


class Policy(torch.nn.Module):
    def __init__(self, width=64):
        super().__init__()
        self.embed = torch.nn.Linear(CUES + 2, width)
        self.memory = AttentionLayer(width)
        self.heads = torch.nn.Linear(width, CUES + 1)  # action logits and the value

    def observe(self, obs):
        return torch.tanh(self.embed(obs))


@torch.no_grad()
def rollout(policy, env, steps):
    """Acts `steps` steps from new episodes; everything as [num_envs, steps, ...]."""
    env.begin(torch.ones(env.n, dtype=torch.bool, device=env.device))
    env.step.zero_()
    caches = policy.memory.caches(env.n, env.device)
    rows = []
    for _ in range(steps):
        o, f, p = env.observation(), env.first, env.step
        y = policy.heads(policy.memory.step(policy.observe(o), p, caches))
        a = torch.distributions.Categorical(logits=y[:, :CUES]).sample()
        lp, _, _ = lrs.compute_action_log_probs(y[:, :CUES], a)
        r, d = env.act(a)
        rows.append((o, f, p, a, lp, r, d))
    return [torch.stack(x, 1) for x in zip(*rows)]


def losses(policy, obs, first, positions, act, old, rew, done):
    """The loss of a rollout, and the log probabilities that the policy now gives its actions."""
    y = policy.heads(policy.memory(policy.observe(obs), first, positions))
    logits, value = y[..., :CUES], y[..., CUES]
    # the rollout's end is cut off: the value of its last step stands in for what follows
    adv = lrs.compute_gae(rew, value.detach(), done, 0.95, 0.9, bootstrap_value=value[:, -1].detach())
    scaled = (adv - adv.mean()) / (adv.std() + 1e-6)
    loss, now, _ = lrs.policy_loss(logits, act, old, scaled, clip=0.2, entropy_coef=0.01)
    return loss.mean() + 0.5 * (value - adv - value.detach()).square().mean(), now


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--updates", type=int, default=40)
    ap.add_argument("--passes", type=int, default=4)
    ap.add_argument("--envs", type=int, default=256)
    ap.add_argument("--steps", type=int, default=64)
    ap.add_argument("--seed", type=int, default=0)
    ap.add_argument("--quiet", action="store_true")
    args = ap.parse_args(argv)
    torch.manual_seed(args.seed)
    device = torch.device("cuda")
    policy = Policy().to(device)
    opt = torch.optim.Adam(policy.parameters(), lr=1e-3)
    env = Recall(args.envs, device, args.seed)
    history, drift = [], 0.0
    for update in range(args.updates):
        obs, first, positions, act, old, rew, done = rollout(policy, env, args.steps)
        for i in range(args.passes):
            loss, now = losses(policy, obs, first, positions, act, old, rew, done)
            if i == 0:  # acting and training agree
                drift = max(drift, (now - old).abs().max().item())
            opt.zero_grad()
            loss.backward()
            torch.nn.utils.clip_grad_norm_(policy.parameters(), 1.0)
            opt.step()
        history.append((rew.sum() / done.sum().clamp(min=1)).item())
        if not args.quiet and (update % 10 == 0 or update == args.updates - 1):
            print(f"update {update:3d}  recalled {history[-1]:.3f} of episodes (chance {1 / CUES:.2f})", flush=True)
    return history, drift


if __name__ == "__main__":
    main()
