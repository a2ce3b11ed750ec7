"""Python binding of the sequence operators of liblrs.so: the gated recurrence
with a matrix state (whole sequences, their gradients, single steps) and the
norm of queries and keys with the position rotation (and its gradients), on
float32, bfloat16 or float16 tensors of one dtype per call.

Tensors are [num_envs, seq_len, heads, dim]; with time_major=True
[seq_len, num_envs, heads, dim].  Any strides over environments, steps and
heads are read in place (q, k and v may be views of one projection); rows of
dim must be consecutive, and tensors expanded over an axis, or with another
inner stride, are first copied with .contiguous().  Every call runs on the
current stream and allocates its workspace from torch there.

compute_* functions are plain calls; gated_recurrence and qk_norm_rotation are
the same operators for autograd.
"""
from __future__ import annotations

import ctypes

import torch

from . import api as _api

_F32 = torch.float32


class _Seq:
    """A tensor as passed to a call, with its (environment, step, head) strides;
    None where it is contiguous in that order."""
    __slots__ = ("t", "strides")

    def __init__(self, t, strides):
        self.t, self.strides = t, strides


def _need_tensor(x, name, dims):
    if not isinstance(x, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if x.dim() != dims:
        raise ValueError(f"{name} must have {dims} dimensions, got {x.dim()}")


def _inner(shape, axes):
    """Whether the tensor has an axis within a row, besides environment, step and head."""
    return len(shape) + axes.count(None) > len(axes)


def _in_place(x, axes):
    """Whether the kernels can address x: consecutive inner elements, no axis expanded."""
    sizes, strides = x.shape, x.stride()
    if _inner(sizes, axes) and sizes[-1] > 1 and strides[-1] != 1:
        return False
    return all(st > 0 or n <= 1 for n, st in zip(sizes, strides))


def _described(x, axes):
    """axes: the positions of (environment, step, head) in x, None where it has none."""
    if x.is_contiguous() and axes[0] == 0:
        return _Seq(x, None)
    st, n = x.stride(), x.shape
    return _Seq(x, tuple(0 if a is None or n[a] <= 1 else st[a] for a in axes))


def _seq_in(x, name, dtype, shape, device, axes):
    x = _api._checked(x, name, dtype, shape, device)
    if not x.is_contiguous() and not _in_place(x, axes):
        x = x.contiguous()
    return _described(x, axes)


def _seq_mask(x, name, shape, device, axes):
    if x is None:
        return None
    if not isinstance(x, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if x.dtype == torch.bool:
        x = x.view(torch.uint8)
    elif x.dtype != torch.uint8:
        x = (x != 0).view(torch.uint8)
    return _seq_in(x, name, torch.uint8, shape, device, axes)


def _seq_out(out, name, dtype, shape, device, axes):
    if out is None:
        return _described(torch.empty(shape, dtype=dtype, device=device), axes)
    o = _api._checked(out, name, dtype, shape, device)
    if not _in_place(o, axes):
        raise ValueError(f"{name} must have consecutive rows and no expanded axis")
    return _described(o, axes)


def _state(x, name, shape, device):
    return None if x is None else _api._checked(x, name, _F32, shape, device).contiguous()


def _state_out(x, name, shape, device):
    if x is None:
        return torch.empty(shape, dtype=_F32, device=device)
    if not _api._checked(x, name, _F32, shape, device).is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return x


def _strides(*arrays):
    """The strides argument of a call: None where every array is contiguous."""
    if all(a is None or a.strides is None for a in arrays):
        return None
    vals = [s for a in arrays for s in ((0, 0, 0) if a is None or a.strides is None else a.strides)]
    return (ctypes.c_int64 * len(vals))(*vals)


def _ptr(x):
    if x is None:
        return None
    return x.t.data_ptr() if isinstance(x, _Seq) else x.data_ptr()


_entries = {}


def _call(stem, sfx, device, what, *args):
    """Calls an entry point on a tensor's device, whichever is current, and its current stream."""
    fn = _entries.get((stem, sfx))
    if fn is None:
        fn = _entries[stem, sfx] = getattr(_api.load(), f"lrs_{stem}_{sfx}")
    stream = torch.cuda.current_stream(device).cuda_stream
    if device.index == torch.cuda.current_device():
        status = fn(*args, stream)
    else:
        with torch.cuda.device(device):
            status = fn(*args, stream)
    if status:
        _api._check(status, what)


def _workspace(bytes_, device):
    return torch.empty(bytes_, dtype=torch.uint8, device=device) if bytes_ else None


def _gpu(x, name):
    if x.device.type != "cuda":
        raise ValueError(f"{name} must be on a GPU (there is no CPU path)")
    return x.device


class _Rec:
    """The checked sizes and inputs of a gated recurrence call."""

    def __init__(self, q, k, v, log_decay, reset, time_major):
        _need_tensor(q, "q", 4)
        _need_tensor(v, "v", 4)
        self.env, self.step = (1, 0) if time_major else (0, 1)
        self.axes, self.axes2 = (self.env, self.step, 2), (self.env, self.step, None)
        self.sfx, self.dt, self.dev = _api._suffix(q, "q"), q.dtype, _gpu(q, "q")
        self.lead = tuple(q.shape[:2])
        self.n, self.t = self.lead[self.env], self.lead[self.step]
        self.kv, self.dk, self.h, self.dv = q.shape[2], q.shape[3], v.shape[2], v.shape[3]
        self.sizes = (self.n, self.t, self.h, self.kv, self.dk, self.dv)
        self.qk_shape, self.v_shape = (*self.lead, self.kv, self.dk), (*self.lead, self.h, self.dv)
        self.g_shape = (*self.lead, self.h)
        self.state_shape = (self.n, self.h, self.dk, self.dv)
        self.q = _seq_in(q, "q", self.dt, self.qk_shape, None, self.axes)
        self.k = _seq_in(k, "k", self.dt, self.qk_shape, self.dev, self.axes)
        self.v = _seq_in(v, "v", self.dt, self.v_shape, self.dev, self.axes)
        self.g = _seq_in(log_decay, "log_decay", self.dt, self.g_shape, self.dev, self.axes)
        self.reset = _seq_mask(reset, "reset", self.lead, self.dev, self.axes2)

    def out(self, x, name, shape):
        return _seq_out(x, name, self.dt, shape, self.dev, self.axes)

    def scale(self, scale):
        return float(self.dk) ** -0.5 if scale is None else float(scale)


def compute_gated_recurrence(q, k, v, log_decay, *, reset=None, initial_state=None, scale=None,
                             time_major=False, out=None, final_state=None, want_final_state=True):
    """The gated recurrence over whole sequences: returns (out, final_state).

    Per environment and head, S_t = exp(log_decay_t) S_{t-1} + k_t v_t^T and
    out_t = scale * S_t^T q_t, the old state dropped where reset_t is set (the
    first step of an episode) or log_decay_t is below -87.33654 (a decay under the
    smallest normal float32 is 0; -inf and torch.finfo's lowest values alike).  q, k
    [num_envs, seq_len, kv_heads, key_dim]; v, out [..., heads, value_dim]
    (value head h reads key head h // (heads // kv_heads)); log_decay
    [num_envs, seq_len, heads]; reset [num_envs, seq_len]; states float32
    [num_envs, heads, key_dim, value_dim].  scale: key_dim ** -0.5 if None.
    With want_final_state=False the second value is None and is not computed."""
    r = _Rec(q, k, v, log_decay, reset, time_major)
    init = _state(initial_state, "initial_state", r.state_shape, r.dev)
    y = r.out(out, "out", r.v_shape)
    last = None
    if want_final_state:
        last = _state_out(final_state, "final_state", r.state_shape, r.dev)
    ws = _workspace(_api.load().lrs_gated_recurrence_workspace_bytes(*r.sizes, 0), r.dev)
    _call("gated_recurrence", r.sfx, r.dev, "compute_gated_recurrence",
          *r.sizes, _ptr(r.q), _ptr(r.k), _ptr(r.v), _ptr(r.g), _ptr(r.reset), _ptr(init),
          r.scale(scale), _ptr(y), _ptr(last), _strides(r.q, r.k, r.v, r.g, r.reset, y), _ptr(ws),
          0 if ws is None else ws.numel())
    return y.t, last


def compute_gated_recurrence_backward(grad_out, q, k, v, log_decay, *, reset=None,
                                      initial_state=None, grad_final_state=None, scale=None,
                                      time_major=False, want_initial_state=True):
    """Gradients of compute_gated_recurrence with these inputs: returns
    (grad_q, grad_k, grad_v, grad_log_decay, grad_initial_state), the last one
    float32 (None with want_initial_state=False).  grad_final_state: 0 if None."""
    r = _Rec(q, k, v, log_decay, reset, time_major)
    do = _seq_in(grad_out, "grad_out", r.dt, r.v_shape, r.dev, r.axes)
    init = _state(initial_state, "initial_state", r.state_shape, r.dev)
    dlast = _state(grad_final_state, "grad_final_state", r.state_shape, r.dev)
    dq, dk = r.out(None, "grad_q", r.qk_shape), r.out(None, "grad_k", r.qk_shape)
    dv, dg = r.out(None, "grad_v", r.v_shape), r.out(None, "grad_log_decay", r.g_shape)
    dinit = _state_out(None, "", r.state_shape, r.dev) if want_initial_state else None
    ws = _workspace(_api.load().lrs_gated_recurrence_workspace_bytes(*r.sizes, 1), r.dev)
    _call("gated_recurrence_backward", r.sfx, r.dev, "compute_gated_recurrence_backward",
          *r.sizes, _ptr(do), _ptr(r.q), _ptr(r.k), _ptr(r.v), _ptr(r.g), _ptr(r.reset), _ptr(init),
          _ptr(dlast), r.scale(scale), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dg), _ptr(dinit),
          _strides(do, r.q, r.k, r.v, r.g, r.reset, dq, dk, dv, dg), _ptr(ws),
          0 if ws is None else ws.numel())
    return dq.t, dk.t, dv.t, dg.t, dinit


def compute_gated_recurrence_step(q, k, v, log_decay, state, *, reset=None, scale=None, out=None,
                                  out_state=None):
    """One step of the gated recurrence for every environment: returns
    (out, next state).  q, k [num_envs, kv_heads, key_dim]; v, out [num_envs,
    heads, value_dim]; log_decay [num_envs, heads]; reset [num_envs]; state
    float32 [num_envs, heads, key_dim, value_dim].  out_state=state updates
    the state in place."""
    _need_tensor(q, "q", 3)
    _need_tensor(v, "v", 3)
    sfx, dt, dev = _api._suffix(q, "q"), q.dtype, _gpu(q, "q")
    n, kv, dk = q.shape
    h, dv = v.shape[1:]
    axes = (0, None, 1)
    qs = _seq_in(q, "q", dt, (n, kv, dk), None, axes)
    ks = _seq_in(k, "k", dt, (n, kv, dk), dev, axes)
    vs = _seq_in(v, "v", dt, (n, h, dv), dev, axes)
    gs = _seq_in(log_decay, "log_decay", dt, (n, h), dev, axes)
    rs = _seq_mask(reset, "reset", (n,), dev, (0, None, None))
    if state is None:
        raise ValueError("state is required")
    old = _state(state, "state", (n, h, dk, dv), dev)
    y = _seq_out(out, "out", dt, (n, h, dv), dev, axes)
    new = _state_out(out_state, "out_state", (n, h, dk, dv), dev)
    _call("gated_recurrence_step", sfx, dev, "compute_gated_recurrence_step",
          n, h, kv, dk, dv, _ptr(qs), _ptr(ks), _ptr(vs), _ptr(gs), _ptr(rs), _ptr(old),
          float(dk) ** -0.5 if scale is None else float(scale), _ptr(y), _ptr(new),
          _strides(qs, ks, vs, gs, rs, y))
    return y.t, new


def rotary_table(max_positions, rotary_dim, *, base=10000.0, position_scale=1.0, device="cuda"):
    """The table of compute_qk_norm_rotation, float32 [max_positions, rotary_dim]:
    the cosines, then the sines, of position * position_scale * base ** (-2j /
    rotary_dim), from angles in 64 bits.  position_scale < 1 interpolates
    positions beyond those trained on."""
    max_positions, rotary_dim = int(max_positions), int(rotary_dim)
    if max_positions < 1 or rotary_dim < 0 or rotary_dim % 2:
        raise ValueError("rotary_table: max_positions must be >= 1 and rotary_dim even and >= 0, "
                         f"got {max_positions} and {rotary_dim}")
    j = torch.arange(0, rotary_dim, 2, dtype=torch.float64, device=device)
    p = torch.arange(max_positions, dtype=torch.float64, device=device) * float(position_scale)
    angles = p[:, None] * float(base) ** (-j / max(1, rotary_dim))
    return torch.cat([angles.cos(), angles.sin()], 1).float()


class _Rot:
    """The checked sizes and inputs of a norm and rotation call."""

    def __init__(self, q, k, q_weight, k_weight, table, positions):
        _need_tensor(q, "q", 4)
        _need_tensor(k, "k", 4)
        self.axes = (0, 1, 2)
        self.sfx, self.dt, self.dev = _api._suffix(q, "q"), q.dtype, _gpu(q, "q")
        self.lead, self.dim = tuple(q.shape[:2]), q.shape[3]
        self.q_shape = (*self.lead, q.shape[2], self.dim)
        self.k_shape = (*self.lead, k.shape[2], self.dim)
        self.q = _seq_in(q, "q", self.dt, self.q_shape, None, self.axes)
        self.k = _seq_in(k, "k", self.dt, self.k_shape, self.dev, self.axes)
        self.qw = _api._dev_tensor(q_weight, "q_weight", self.dt, (self.dim,), self.dev)
        self.kw = _api._dev_tensor(k_weight, "k_weight", self.dt, (self.dim,), self.dev)
        self.rot, self.max, self.table, self.positions = 0, 0, None, None
        if table is not None:
            _need_tensor(table, "table", 2)
            self.max, self.rot = table.shape
            self.table = _api._dev_tensor(table, "table", _F32, (self.max, self.rot), self.dev)
            if positions is None:
                raise ValueError("table given without positions")
            self.positions = _seq_in(positions, "positions", torch.int32, self.lead, self.dev,
                                     (0, 1, None))
        self.sizes = (*self.lead, q.shape[2], k.shape[2], self.dim, self.rot)

    def out(self, x, name, shape):
        return _seq_out(x, name, self.dt, shape, self.dev, self.axes)


def compute_qk_norm_rotation(q, k, q_weight, k_weight, table=None, positions=None, *, eps=1e-6,
                             interleaved=False, out=None):
    """Each head of q and k divided by its root mean square and multiplied by
    its weight, then rotated by the token's position: returns (q_out, k_out).

    q [rows, columns, q_heads, dim] and k [rows, columns, k_heads, dim] (either
    layout of environments and steps); weights [dim]; table float32
    [max_positions, rotary_dim] (see rotary_table; None: no rotation);
    positions int32 [rows, columns].  The first rotary_dim elements of a head
    are rotated, in pairs (j, j + rotary_dim / 2), or (2j, 2j + 1) where
    interleaved.  Positions outside the table give NaN."""
    r = _Rot(q, k, q_weight, k_weight, table, positions)
    yq = r.out(None if out is None else out[0], "out[0]", r.q_shape)
    yk = r.out(None if out is None else out[1], "out[1]", r.k_shape)
    _call("qk_norm_rotation", r.sfx, r.dev, "compute_qk_norm_rotation",
          *r.sizes, _ptr(r.q), _ptr(r.k), _ptr(r.qw), _ptr(r.kw), _ptr(r.table), r.max,
          _ptr(r.positions), float(eps), int(bool(interleaved)), _ptr(yq), _ptr(yk),
          _strides(r.q, r.k, r.positions, yq, yk))
    return yq.t, yk.t


def compute_qk_norm_rotation_backward(grad_q_out, grad_k_out, q, k, q_weight, k_weight, table=None,
                                      positions=None, *, eps=1e-6, interleaved=False):
    """Gradients of compute_qk_norm_rotation with these inputs: returns
    (grad_q, grad_k, grad_q_weight, grad_k_weight)."""
    r = _Rot(q, k, q_weight, k_weight, table, positions)
    gq = _seq_in(grad_q_out, "grad_q_out", r.dt, r.q_shape, r.dev, r.axes)
    gk = _seq_in(grad_k_out, "grad_k_out", r.dt, r.k_shape, r.dev, r.axes)
    dq, dk = r.out(None, "grad_q", r.q_shape), r.out(None, "grad_k", r.k_shape)
    dqw, dkw = torch.empty_like(r.qw), torch.empty_like(r.kw)
    ws = _workspace(_api.load().lrs_qk_norm_rotation_workspace_bytes(*r.sizes[:5]), r.dev)
    _call("qk_norm_rotation_backward", r.sfx, r.dev, "compute_qk_norm_rotation_backward",
          *r.sizes, _ptr(gq), _ptr(gk), _ptr(r.q), _ptr(r.k), _ptr(r.qw), _ptr(r.kw), _ptr(r.table),
          r.max, _ptr(r.positions), float(eps), int(bool(interleaved)), _ptr(dq), _ptr(dk),
          _ptr(dqw), _ptr(dkw), _strides(gq, gk, r.q, r.k, r.positions, dq, dk), _ptr(ws),
          0 if ws is None else ws.numel())
    return dq.t, dk.t, dqw, dkw


# ----------------------------------------------------------------- autograd

class _GatedRecurrence(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, log_decay, initial_state, reset, scale, time_major):
        out, last = compute_gated_recurrence(q, k, v, log_decay, reset=reset,
                                             initial_state=initial_state, scale=scale,
                                             time_major=time_major)
        ctx.save_for_backward(q, k, v, log_decay, initial_state, reset)
        ctx.scale, ctx.time_major, ctx.out_shape = scale, time_major, out.shape
        ctx.set_materialize_grads(False)
        return out, last

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad_out, grad_last):
        q, k, v, log_decay, initial_state, reset = ctx.saved_tensors
        if grad_out is None:
            grad_out = q.new_zeros(ctx.out_shape)
        grads = compute_gated_recurrence_backward(
            grad_out, q, k, v, log_decay, reset=reset, initial_state=initial_state,
            grad_final_state=grad_last, scale=ctx.scale, time_major=ctx.time_major,
            want_initial_state=ctx.needs_input_grad[4])
        return (*grads, None, None, None)


def gated_recurrence(q, k, v, log_decay, *, reset=None, initial_state=None, scale=None,
                     time_major=False):
    """compute_gated_recurrence for autograd: differentiable in q, k, v,
    log_decay and initial_state; returns (out, final_state).  To capture both
    directions into a graph, call the compute_ functions, or first drop every
    eager result of the same leaves: torch does not capture a backward pass
    beside those."""
    return _GatedRecurrence.apply(q, k, v, log_decay, initial_state, reset, scale, time_major)


class _QkNormRotation(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, q_weight, k_weight, table, positions, eps, interleaved):
        ctx.save_for_backward(q, k, q_weight, k_weight, table, positions)
        ctx.eps, ctx.interleaved = eps, interleaved
        return compute_qk_norm_rotation(q, k, q_weight, k_weight, table, positions, eps=eps,
                                        interleaved=interleaved)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad_q, grad_k):
        grads = compute_qk_norm_rotation_backward(grad_q, grad_k, *ctx.saved_tensors, eps=ctx.eps,
                                                  interleaved=ctx.interleaved)
        return (*grads, None, None, None, None)


def qk_norm_rotation(q, k, q_weight, k_weight, table=None, positions=None, *, eps=1e-6,
                     interleaved=False):
    """compute_qk_norm_rotation for autograd: differentiable in q, k and the weights."""
    return _QkNormRotation.apply(q, k, q_weight, k_weight, table, positions, eps, interleaved)
