"""Python binding of the windowed attention of liblrs.so: attention over a window
of steps and the first steps of each episode (whole sequences, their gradients,
single steps over caches and the filling of those), on float32, bfloat16 or
float16 tensors of one dtype per call.

Tensors are [num_envs, seq_len, heads, dim], or [seq_len, num_envs, heads, dim]
with time_major=True, of any strides over environments, steps and heads, like
those of the gated recurrence; queries and keys usually come from
qk_norm_rotation.  Every call runs on the current stream and allocates its
workspace from torch there.

compute_* functions are plain calls; windowed_attention is the same operator for
autograd.
"""
from __future__ import annotations

import functools

import torch

from . import api as _api
from .sequence import (_F32, _call, _described, _gpu, _in_place, _need_tensor, _ptr, _seq_in, _seq_mask,
                       _seq_out, _strides, _workspace)


class _Att:
    """The checked sizes and inputs of a call over whole sequences."""

    def __init__(self, q, k, v, window, sinks, reset, time_major):
        for x, name in ((q, "q"), (k, "k"), (v, "v")):
            _need_tensor(x, name, 4)
        env, step = (1, 0) if time_major else (0, 1)
        self.axes, self.axes2 = (env, step, 2), (env, step, None)
        self.sfx, self.dt, self.dev = _api._suffix(q, "q"), q.dtype, _gpu(q, "q")
        n, t, self.tk = q.shape[env], q.shape[step], k.shape[step]
        h, dk, kv, dv = q.shape[2], q.shape[3], k.shape[2], v.shape[3]
        if self.tk < t:
            raise ValueError(f"k must have at least the {t} steps of q, got {self.tk}")
        lead = tuple(q.shape[:2])
        key_lead = (self.tk, n) if time_major else (n, self.tk)
        self.sizes = (n, t, self.tk, h, kv, dk, dv, int(window), int(sinks))
        self.q_shape, self.o_shape, self.lse_shape = (*lead, h, dk), (*lead, h, dv), (*lead, h)
        self.k_shape, self.v_shape = (*key_lead, kv, dk), (*key_lead, kv, dv)
        self.q = _seq_in(q, "q", self.dt, self.q_shape, None, self.axes)
        self.k = _seq_in(k, "k", self.dt, self.k_shape, self.dev, self.axes)
        self.v = _seq_in(v, "v", self.dt, self.v_shape, self.dev, self.axes)
        self.reset = _seq_mask(reset, "reset", key_lead, self.dev, self.axes2)

    def out(self, x, name, shape):
        return _seq_out(x, name, self.dt, shape, self.dev, self.axes)

    def scale(self, scale):
        return float(self.sizes[5]) ** -0.5 if scale is None else float(scale)

    def workspace(self, backward):
        need = _api.load().lrs_windowed_attention_workspace_bytes(*self.sizes, int(self.reset is not None),
                                                                  backward)
        return _workspace(need, self.dev)


def compute_windowed_attention(q, k, v, *, window, sinks=0, reset=None, scale=None, time_major=False,
                               out=None, want_lse=True):
    """Attention of every step over the last `window` steps (its own among them)
    and the first `sinks` steps of its episode: returns (out, lse).

    q, out [num_envs, seq_len, heads, key_dim and value_dim]; k, v [num_envs,
    key_steps, kv_heads, ...], key_steps >= seq_len: the queries are the keys'
    last steps, those before are what went before them (head h reads key head
    h // (heads // kv_heads)).  reset [num_envs, key_steps]: set at the first step
    of an episode; no step sees one of another episode.  A row whose first step
    is not set counts as an episode that begins there.  scale: key_dim ** -0.5
    if None.  lse float32 [num_envs, seq_len, heads]: the log of the sum of
    exp(scale * q . k), which the gradients need (None with want_lse=False)."""
    a = _Att(q, k, v, window, sinks, reset, time_major)
    o = a.out(out, "out", a.o_shape)
    lse = _seq_out(None, "lse", _F32, a.lse_shape, a.dev, a.axes) if want_lse else None
    ws = a.workspace(0)
    _call("windowed_attention", a.sfx, a.dev, "compute_windowed_attention", *a.sizes, _ptr(a.q), _ptr(a.k),
          _ptr(a.v), _ptr(a.reset), a.scale(scale), _ptr(o), _ptr(lse),
          _strides(a.q, a.k, a.v, a.reset, o, lse), _ptr(ws), 0 if ws is None else ws.numel())
    return o.t, None if lse is None else lse.t


def compute_windowed_attention_backward(grad_out, q, k, v, out, lse, *, window, sinks=0, reset=None,
                                        scale=None, time_major=False):
    """Gradients of compute_windowed_attention with these inputs and results:
    returns (grad_q, grad_k, grad_v)."""
    a = _Att(q, k, v, window, sinks, reset, time_major)
    do = _seq_in(grad_out, "grad_out", a.dt, a.o_shape, a.dev, a.axes)
    o = _seq_in(out, "out", a.dt, a.o_shape, a.dev, a.axes)
    if lse is None:
        raise ValueError("lse is required")
    ls = _seq_in(lse, "lse", _F32, a.lse_shape, a.dev, a.axes)
    dq, dk, dv = a.out(None, "grad_q", a.q_shape), a.out(None, "grad_k", a.k_shape), a.out(None, "grad_v", a.v_shape)
    ws = a.workspace(1)
    _call("windowed_attention_backward", a.sfx, a.dev, "compute_windowed_attention_backward", *a.sizes,
          _ptr(do), _ptr(a.q), _ptr(a.k), _ptr(a.v), _ptr(a.reset), _ptr(o), _ptr(ls), a.scale(scale),
          _ptr(dq), _ptr(dk), _ptr(dv), _strides(do, a.q, a.k, a.v, a.reset, o, ls, dq, dk, dv), _ptr(ws),
          0 if ws is None else ws.numel())
    return dq.t, dk.t, dv.t


@functools.lru_cache(maxsize=256)
def _step_workspace(*sizes):
    """Bytes of a step's workspace, which go by its sizes alone."""
    return _api.load().lrs_windowed_attention_step_workspace_bytes(*sizes)


def _cache(x, name, dtype, shape, device):
    x = _api._checked(x, name, dtype, shape, device)
    if not _in_place(x, (0, 1, 2)):
        raise ValueError(f"{name} must have consecutive rows and no expanded axis")
    return _described(x, (0, 1, 2))


def _positions(x, shape, device):
    x = _api._checked(x, "positions", torch.int32, shape, device)
    return x if x.is_contiguous() else x.contiguous()


def compute_windowed_attention_step(q, k, v, key_cache, value_cache, positions, *, sinks=0, scale=None,
                                    out=None):
    """One step of the windowed attention for every environment, over caches that
    it updates in place: returns out [num_envs, heads, value_dim].

    q [num_envs, heads, key_dim]; k, v [num_envs, kv_heads, ...]; key_cache,
    value_cache [num_envs, sinks + window, kv_heads, ...]; positions int32
    [num_envs]: which step of its episode each environment is at, from 0, when
    nothing of its caches is left to see.  The step's key and value go into slot
    position, or sinks + (position - sinks) % window from position sinks on.  An
    environment with a negative position waits: its caches stay as they are and
    its output is 0."""
    _need_tensor(q, "q", 3)
    _need_tensor(key_cache, "key_cache", 4)
    _need_tensor(value_cache, "value_cache", 4)
    sfx, dt, dev = _api._suffix(q, "q"), q.dtype, _gpu(q, "q")
    n, h, dk = q.shape
    slots, kv, dv = key_cache.shape[1], key_cache.shape[2], value_cache.shape[3]
    axes = (0, None, 1)
    qs = _seq_in(q, "q", dt, (n, h, dk), None, axes)
    ks = _seq_in(k, "k", dt, (n, kv, dk), dev, axes)
    vs = _seq_in(v, "v", dt, (n, kv, dv), dev, axes)
    kc = _cache(key_cache, "key_cache", dt, (n, slots, kv, dk), dev)
    vc = _cache(value_cache, "value_cache", dt, (n, slots, kv, dv), dev)
    pos = _positions(positions, (n,), dev)
    o = _seq_out(out, "out", dt, (n, h, dv), dev, axes)
    ws = _workspace(_step_workspace(n, h, kv, slots, int(sinks), dk, dv), dev)
    _call("windowed_attention_step", sfx, dev, "compute_windowed_attention_step", n, h, kv, slots, int(sinks),
          dk, dv, _ptr(qs), _ptr(ks), _ptr(vs), _ptr(kc), _ptr(vc), _ptr(pos),
          float(dk) ** -0.5 if scale is None else float(scale), _ptr(o), _strides(qs, ks, vs, kc, vc, None, o),
          _ptr(ws), 0 if ws is None else ws.numel())
    return o.t


def compute_windowed_attention_fill(k, v, key_cache, value_cache, positions, *, sinks=0, time_major=False):
    """Puts the steps of whole sequences into the caches of
    compute_windowed_attention_step, as their single steps would have: returns
    (key_cache, value_cache), updated in place.

    k [num_envs, seq_len, kv_heads, key_dim] and v as in
    compute_windowed_attention; positions int32 [num_envs, seq_len]: each step's
    place in its episode, from 0.  Of each row its last episode counts, which the
    last step's position says: that step and those before it, as many as there
    are, go into their slots.  Slots whose steps lie before the row stay as they
    are, and so do all of a row whose last position is negative."""
    for x, name in ((k, "k"), (v, "v"), (key_cache, "key_cache"), (value_cache, "value_cache")):
        _need_tensor(x, name, 4)
    env, step = (1, 0) if time_major else (0, 1)
    sfx, dt, dev = _api._suffix(k, "k"), k.dtype, _gpu(k, "k")
    lead, n, t = tuple(k.shape[:2]), k.shape[env], k.shape[step]
    kv, dk, dv, slots = k.shape[2], k.shape[3], v.shape[3], key_cache.shape[1]
    axes = (env, step, 2)
    ks = _seq_in(k, "k", dt, (*lead, kv, dk), None, axes)
    vs = _seq_in(v, "v", dt, (*lead, kv, dv), dev, axes)
    kc = _cache(key_cache, "key_cache", dt, (n, slots, kv, dk), dev)
    vc = _cache(value_cache, "value_cache", dt, (n, slots, kv, dv), dev)
    pos = _seq_in(positions, "positions", torch.int32, lead, dev, (env, step, None))
    _call("windowed_attention_fill", sfx, dev, "compute_windowed_attention_fill", n, t, kv, slots, int(sinks),
          dk, dv, _ptr(ks), _ptr(vs), _ptr(pos), _ptr(kc), _ptr(vc), _strides(ks, vs, pos, kc, vc))
    return key_cache, value_cache


# ----------------------------------------------------------------- autograd

class _WindowedAttention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, reset, opts):
        out, lse = compute_windowed_attention(q, k, v, reset=reset, **opts)
        ctx.save_for_backward(q, k, v, out, lse, reset)
        ctx.opts = opts
        return out

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad_out):
        q, k, v, out, lse, reset = ctx.saved_tensors
        grads = compute_windowed_attention_backward(grad_out, q, k, v, out, lse, reset=reset, **ctx.opts)
        return (*grads, None, None)


def windowed_attention(q, k, v, *, window, sinks=0, reset=None, scale=None, time_major=False):
    """compute_windowed_attention for autograd: differentiable in q, k and v;
    returns out.  To capture both directions into a graph, call the compute_
    functions, or first drop every eager result of the same leaves: torch does
    not capture a backward pass beside those."""
    return _WindowedAttention.apply(q, k, v, reset, dict(window=window, sinks=sinks, scale=scale,
                                                         time_major=time_major))
