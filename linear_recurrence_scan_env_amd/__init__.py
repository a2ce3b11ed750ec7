"""MI355X (gfx950) linear-recurrence scans for RL credit assignment.

Seven estimators and the generic segmented affine scan, one C-ABI call each
(include/lrs.h), backed by hand-written HIP kernels in csrc/.  The Python functions here only marshal torch tensors
into those calls; nothing runs on the CPU.  Beside them, sequence operators
for the policies trained on these targets: a gated recurrence with a matrix
state and the norm of queries and keys with the position rotation, each with
its gradients.
"""
from .api import (  # noqa: F401
    LrsError,
    compute_affine_scan,
    compute_discounted_returns,
    compute_eligibility_traces,
    compute_episodic_prefix_sum,
    compute_gae,
    compute_lambda_returns,
    compute_retrace,
    compute_vtrace,
    lib_path,
    load,
    set_schedule,
    set_time_major_waves,
    workspace_state,
)
from .sequence import (  # noqa: F401
    compute_gated_recurrence,
    compute_gated_recurrence_backward,
    compute_gated_recurrence_step,
    compute_qk_norm_rotation,
    compute_qk_norm_rotation_backward,
    gated_recurrence,
    qk_norm_rotation,
    rotary_table,
)

__all__ = [
    "compute_gae", "compute_vtrace", "compute_retrace", "compute_lambda_returns",
    "compute_discounted_returns", "compute_eligibility_traces", "compute_episodic_prefix_sum",
    "compute_affine_scan",
    "compute_gated_recurrence", "compute_gated_recurrence_backward",
    "compute_gated_recurrence_step", "compute_qk_norm_rotation",
    "compute_qk_norm_rotation_backward", "gated_recurrence", "qk_norm_rotation", "rotary_table",
    "LrsError", "load", "lib_path", "set_schedule", "set_time_major_waves", "workspace_state",
]
