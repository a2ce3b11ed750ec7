"""The windowed attention and the policy loss from their definitions, in 64 bits on
the CPU, with bounds of what float32 sums and one rounding to the type leave.
Inputs are torch tensors of any float type, [N, T, heads, dim]."""
import math

import torch

F32 = 2.0 ** -24


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def seen(t, tk, window, sinks, reset=None):
    """[N or 1, T, TK]: which keys each query sees, step by step."""
    past = tk - t
    n = 1 if reset is None else reset.shape[0]
    ok = torch.zeros(n, t, tk, dtype=torch.bool)
    for b in range(n):
        e = 0
        for j in range(tk):
            if reset is not None and reset[b, j]:
                e = j
            if j >= past:
                ok[b, j - past, max(e, j - window + 1):j + 1] = True
                ok[b, j - past, e:min(e + sinks, j + 1)] = True
    return ok


def attention(q, k, v, window, sinks=0, reset=None, scale=None, do=None):
    """Results, gradients where do is given, and how far each may be off: a dict
    of (value, bound)."""
    dt = q.dtype
    u = half_step(dt)
    uw = u if dt != torch.float32 else 0.0  # weights are rounded to 16-bit types
    # and float16 has steps of 2^-24 below 2^-14, so that a rounding there is off by 2^-25 whatever the
    # value: of a result, of a weight beside a largest one of 1, of ds, and of a weight of dv times 2^10
    low = 2.0 ** -25 if dt == torch.float16 else 0.0
    reset = None if reset is None else reset.cpu()
    q, k, v = (x.double().cpu() for x in (q, k, v))
    n, t, heads, dk = q.shape
    tk, kv = k.shape[1:3]
    g = heads // kv
    scale = dk ** -0.5 if scale is None else scale
    ok = seen(t, tk, window, sinks, reset)[:, None]
    Q = q.transpose(1, 2)
    K, V = (x.transpose(1, 2).repeat_interleave(g, 1) for x in (k, v))
    zero = torch.zeros((), dtype=torch.float64)
    # what is not seen does not count, whatever it is
    s = torch.where(ok, scale * torch.einsum("nhid,nhjd->nhij", Q, K), -math.inf)
    lse = torch.logsumexp(s, -1)
    p = torch.where(ok, torch.exp(s - lse[..., None]), zero)
    fin = lambda x: torch.nan_to_num(x, 0.0, 0.0, 0.0)  # noqa: E731
    out = _rows(p, V, ok)
    # float32 score sums, scaled; exponents up to 64 in size rounded to float32
    absqk = (fin(Q).abs().amax((-1, -2)) * fin(K).abs().amax((-1, -2)))[..., None, None] * abs(scale) * dk
    ds = min(1.0, float((dk + 8) * F32 * absqk.max()))
    rel = uw + 2 * ds + 2.0 ** -18
    tol = u * out.abs() + rel * (fin(p) @ fin(V).abs()) + low * (1 + ok.double() @ fin(V).abs())
    res = {"out": (out.transpose(1, 2), tol.transpose(1, 2)),
           "lse": (lse.transpose(1, 2), ds + 2.0 ** -21 * (1 + fin(lse).abs().transpose(1, 2)))}
    if do is None:
        return res
    DO = do.double().cpu().transpose(1, 2)
    dp = torch.einsum("nhid,nhjd->nhij", DO, V)
    delta = (DO * out).sum(-1, keepdim=True)
    dS = torch.where(ok, scale * p * (dp - delta), zero)
    e_dp = (k.shape[-1] + V.shape[-1]) * F32 * (fin(DO).abs() @ fin(V).abs().transpose(-1, -2))
    e_delta = (fin(DO).abs() * fin(tol)).sum(-1, keepdim=True) + 2 * 128 * F32 * (fin(DO).abs() * fin(out).abs()).sum(-1, keepdim=True)
    e_ds = abs(scale) * fin(p) * (rel * fin(dp - delta).abs() + e_dp + e_delta) + uw * fin(dS).abs() + abs(scale) * low * ok
    share = lambda x: x.unflatten(1, (kv, g)).sum(2)  # noqa: E731
    turn = lambda x: x.transpose(-1, -2)  # noqa: E731
    dq = _rows(dS, K, ok)
    dkk, dvv = share(_rows(turn(dS), Q, turn(ok))), share(_rows(turn(p), DO, turn(ok)))
    sums = 2.0 ** -18  # float32 sums over up to 64 tiles
    tq = low + u * dq.abs() + (e_ds + sums * fin(dS).abs()) @ fin(K).abs()
    tkk = low + u * dkk.abs() + share(turn(e_ds + sums * fin(dS).abs()) @ fin(Q).abs())
    tv = low + u * dvv.abs() + share(turn((rel + sums) * fin(p) + low * 2.0 ** -10 * ok) @ fin(DO).abs())
    for name, val, bound in (("dq", dq, tq), ("dk", dkk, tkk), ("dv", dvv, tv)):
        res[name] = (val.transpose(1, 2), bound.transpose(1, 2))
    return res


def _rows(w, x, ok):
    """w @ x over the pairs that are seen only: 0 where they are not, even if x is not finite."""
    if torch.isfinite(x).all():
        return w @ x
    out = torch.zeros(*torch.broadcast_shapes(w.shape[:-2], x.shape[:-2]), w.shape[-2], x.shape[-1],
                      dtype=torch.float64)
    ok = ok.expand(w.shape)
    for i in range(w.shape[-2]):
        term = torch.where(ok[..., i, :, None], w[..., i, :, None] * x, 0.0)
        out[..., i, :] = term.sum(-2)
    return out


def step(q, k, v, key_cache, value_cache, positions, sinks, scale=None):
    """(out, bound) and the caches after it."""
    kc, vc = key_cache.cpu().clone(), value_cache.cpu().clone()
    n, heads, dk = q.shape
    kv, window = kc.shape[2], kc.shape[1] - sinks
    dt = q.dtype
    scale = dk ** -0.5 if scale is None else scale
    out = torch.zeros(n, heads, vc.shape[-1], dtype=torch.float64)
    tol = torch.zeros_like(out)
    for b, p in enumerate(positions.tolist()):
        if p < 0:
            continue
        at = p if p < sinks else sinks + (p - sinks) % window
        kc[b, at], vc[b, at] = k[b].cpu(), v[b].cpu()
        m = min(p + 1, sinks + window)
        K, V = (x[b, :m].double().transpose(0, 1).repeat_interleave(heads // kv, 0) for x in (kc, vc))
        Q = q[b].double().cpu()
        s = scale * (K * Q[:, None]).sum(-1)
        w = torch.softmax(s, -1)
        out[b] = (w[..., None] * V).sum(1)
        ds = (dk + 8) * F32 * abs(scale) * (K.abs() * Q[:, None].abs()).sum(-1).amax(-1)
        tol[b] = half_step(dt) * out[b].abs() + (2 * ds + 2.0 ** -17)[:, None] * (w[..., None] * V.abs()).sum(1)
    return out, tol, kc, vc


def policy(logits, actions, old=None, adv=None, ref=None, mask=None, weights=None, clip=0.2, clip_high=None,
           kl=0.0, ent=0.0, temperature=1.0, c_lp=None, c_ent=None):
    """(value, bound) of log_probs, entropy, lse, loss and grad: the gradient of sum(weights * loss), or of
    sum(c_lp * log_probs + c_ent * entropy)."""
    dt = logits.dtype
    u = half_step(dt)
    clip_high = clip if clip_high is None else clip_high
    f = lambda x: None if x is None else x.double().cpu()  # noqa: E731
    z, old, adv, ref, weights, c_lp, c_ent = map(f, (logits, old, adv, ref, weights, c_lp, c_ent))
    actions = actions.cpu().long()
    V = z.shape[-1]
    z = z / temperature
    lse = torch.logsumexp(z, -1)
    logp = z - lse[..., None]
    p = torch.exp(logp)
    plogp = torch.where(p > 0, p * logp, 0.0)
    H = -plogp.sum(-1)
    inside = (actions >= 0) & (actions < V)
    a = actions.clamp(0, V - 1)
    lp = torch.where(inside, logp.gather(-1, a[..., None])[..., 0], math.nan)
    big = torch.where(torch.isfinite(z), z.abs(), 0.0).amax(-1)
    # a lane sums up to 128 terms in order, and lanes are joined in 16 steps; logits are scaled once
    t = 144 * F32 + 2.0 ** -21 * (1 + big)
    tH = t * (2 + 2 * H.abs())
    tlp = t + 2.0 ** -22 * lp.abs()
    res = {"log_probs": (lp, tlp), "entropy": (H, tH), "lse": (lse, t + 2.0 ** -22 * lse.abs())}
    one = torch.zeros_like(z).scatter_(-1, a[..., None], 1.0)
    if old is not None:
        r = torch.exp(lp - old)
        most, least = 1 + clip_high, 1 - clip
        cut = torch.where(adv >= 0, r > most, r < least)
        bound = torch.where(cut, torch.where(adv >= 0, most, least), r)
        loss = -bound * adv - ent * H
        tr = r * (2 * tlp + 2.0 ** -21 * (1 + (lp - old).abs()))
        tol = adv.abs() * tr + abs(ent) * tH + 4 * F32 * (bound * adv).abs()
        c = torch.where(cut, 0.0, -adv * r)
        tc = adv.abs() * tr
        if kl:
            d = ref - lp
            e = torch.expm1(d)
            loss = loss + kl * (e - d)
            te = (e + 1) * (2 * tlp + 2.0 ** -21 * (1 + d.abs()))
            tol = tol + abs(kl) * (te + tlp + 2.0 ** -21 * d.abs())
            c = c - kl * e
            tc = tc + abs(kl) * te
        h = -ent * torch.ones_like(H)
        w = torch.ones_like(H) if weights is None else weights
        c, tc, h = c * w, tc * w.abs(), h * w
        res["loss"] = (loss, tol + 4 * F32 * loss.abs())
    else:
        c = torch.zeros_like(H) if c_lp is None else torch.where(inside, c_lp, math.nan)
        h = torch.zeros_like(H) if c_ent is None else c_ent
        tc = 2.0 ** -22 * c.abs()
    c, tc, h = (x[..., None] for x in (c, tc, h))
    down = torch.where(p > 0, p * (torch.where(p > 0, logp, 0.0) + H[..., None]), 0.0)
    # the derivative of H by a logit is -p (log p + H)
    grad = (c * (one - p) - h * down) / temperature
    # (a row that is NaN is so in every column)
    grad = grad + 0 * (c + lse[..., None])
    t3, tH3 = t[..., None], tH[..., None]
    g_tol = (2 * t3 * p * c.abs() + tc * (p + one) + h.abs() * p * (2 * t3 * (logp.clamp(min=-200) + H[..., None]).abs()
             + tH3 + 2 * t3) + 4 * F32 * ((c * one).abs())) / temperature
    tiny = torch.finfo(dt).smallest_normal * torch.finfo(dt).eps
    res["grad"] = (grad, u * grad.abs() + g_tol + tiny)
    if mask is not None:
        on = mask.cpu() != 0
        for name, (val, tol) in res.items():
            o = on[..., None] if name == "grad" else on
            res[name] = (torch.where(o, val, 0.0), torch.where(o, tol, 0.0))
    return res


def check(got, want, what=""):
    """got within want = (value, bound); NaN and infinities where they are."""
    val, tol = want
    got = got.double().cpu()
    assert got.shape == val.shape, (what, got.shape, val.shape)
    fin = torch.isfinite(val)
    assert torch.equal(torch.isfinite(got), fin), f"{what}: not finite at {int((torch.isfinite(got) != fin).sum())} places"
    over = ((got - val).abs() - tol)[fin]
    if over.numel() and over.max() > 0:
        i = over.argmax()
        raise AssertionError(f"{what}: {int((over > 0).sum())} of {over.numel()} beyond the bound; at worst "
                             f"{got[fin][i]:.9g} for {val[fin][i]:.9g} +- {tol[fin][i]:.3g}")
