"""The sequence operators from their definitions, in 64 bits on the CPU: the
gated recurrence step by step, its gradients by the reverse recursion, and the
norm of queries and keys with rotation.  Inputs are torch tensors of any float
type, [N, T, heads, dim]; results are float64."""
import torch


def gated_recurrence(q, k, v, g, reset=None, h0=None, scale=None):
    q, k, v, g = (x.double().cpu() for x in (q, k, v, g))
    n, t, kv, dk = q.shape
    heads, dv = v.shape[2:]
    q, k = (x.repeat_interleave(heads // kv, 2) for x in (q, k))
    scale = dk ** -0.5 if scale is None else scale
    cut = torch.isneginf(g)
    if reset is not None:
        cut = cut | (reset.cpu() != 0)[..., None]
    S = torch.zeros(n, heads, dk, dv, dtype=torch.float64) if h0 is None else h0.double().cpu()
    out, states = [], [S]
    for i in range(t):
        f = torch.where(cut[:, i], 0.0, g[:, i].exp())[..., None, None]
        S = torch.where(cut[:, i][..., None, None], 0.0, f * S) + k[:, i, :, :, None] * v[:, i, :, None]
        states.append(S)
        out.append(scale * (S * q[:, i, :, :, None]).sum(2))
    return torch.stack(out, 1), S, states, cut


def gated_recurrence_backward(do, q, k, v, g, reset=None, h0=None, dhT=None, scale=None):
    _, _, states, cut = gated_recurrence(q, k, v, g, reset, h0, scale)
    do, q, k, v, g = (x.double().cpu() for x in (do, q, k, v, g))
    n, t, kv, dk_ = q.shape
    heads = v.shape[2]
    rep = heads // kv
    q, k = (x.repeat_interleave(rep, 2) for x in (q, k))
    scale = dk_ ** -0.5 if scale is None else scale
    R = torch.zeros_like(states[0]) if dhT is None else dhT.double().cpu()
    dq, dk, dv, dg = (torch.zeros_like(x) for x in (q, k, v, g))
    for i in range(t - 1, -1, -1):
        R = R + scale * q[:, i, :, :, None] * do[:, i, :, None]
        dq[:, i] = scale * (states[i + 1] * do[:, i, :, None]).sum(-1)
        dk[:, i] = (R * v[:, i, :, None]).sum(-1)
        dv[:, i] = (R * k[:, i, :, :, None]).sum(2)
        f = torch.where(cut[:, i], 0.0, g[:, i].exp())[..., None, None]
        R = f * R
        dg[:, i] = (R * states[i]).sum((-1, -2))
    shared = lambda x: x.unflatten(2, (kv, rep)).sum(3)  # noqa: E731
    return shared(dq), shared(dk), dv, dg, R


def norm_rotation(x, w, table, positions, eps, interleaved):
    """Positions outside the table give NaN."""
    x, w = x.double().cpu(), w.double().cpu()
    z = x / (x.square().mean(-1, keepdim=True) + eps).sqrt() * w
    if table is None or table.shape[1] == 0:
        return z
    rot = table.shape[1]
    pos = positions.cpu().long()
    bad = (pos < 0) | (pos >= table.shape[0])
    rows = table.double().cpu()[pos.clamp(0, table.shape[0] - 1)][..., None, :]
    cos, sin = rows[..., :rot // 2], rows[..., rot // 2:]
    y = z.clone()
    one = slice(0, rot, 2) if interleaved else slice(0, rot // 2)
    two = slice(1, rot, 2) if interleaved else slice(rot // 2, rot)
    a, b = z[..., one], z[..., two]
    y[..., one] = a * cos - b * sin
    y[..., two] = b * cos + a * sin
    y[bad] = float("nan")
    return y
