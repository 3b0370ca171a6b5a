"""Diagonal linear-recurrence scan for AMD MI355X (gfx950).

h_t = a_t * h_{t-1} + b_t, element-wise over channels, evaluated as a parallel
prefix scan by hand-written HIP kernels behind the C ABI declared in
include/lrs.h.  The functions exported here come from ``binding`` (a thin
ctypes layer: argument marshalling only, no compute and no fallback).
"""
# DEER stop rule defaults: eps = 1e-5 and K_max = 5, the example values of the
# DEER page ("cuda-parallel-rnn-training-logt-optimization", engineering section).
DEER_DEFAULT_EPS = 1e-5
DEER_DEFAULT_KMAX = 5

_BINDING_NAMES = ("scan_fwd", "scan_bwd", "scan_fwd_bwd", "sru_fwd", "sru_bwd", "deer_solve", "deer_stats",
                  "deer_bwd", "deer_solve_seq", "deer_eps_schedule", "lstm_fwd", "lstm_bwd",
                  "sru_deer_fwd", "rnn_seq", "scan_workspace_bytes", "plan_options",
                  "LrsError")

# operators of recurrent language models (include/lrs_lm.h)
_LM_NAMES = ("glr_checkpoints", "glr_fwd", "glr_bwd", "glr_step", "layernorm_fwd", "layernorm_bwd",
             "linear_ce_fwd", "linear_ce_bwd", "linear_ce_fwd_bwd")

# operators of delta-rule language models (include/lrs_block.h); load sets the prototypes
# of all headers
_BLOCK_NAMES = ("gdr_checkpoints", "gdr_fwd", "gdr_bwd", "gdr_step", "rmsnorm_fwd",
                "rmsnorm_fwd_fp8", "rmsnorm_bwd", "logprobs_fwd", "logprobs_bwd", "load")

__all__ = ["DEER_DEFAULT_EPS", "DEER_DEFAULT_KMAX", *_BINDING_NAMES, *_LM_NAMES, *_BLOCK_NAMES]


def __getattr__(name):
    # the bindings import torch; load them only when a device entry point is used,
    # and look each name up once
    if name in _BINDING_NAMES:
        from . import binding as module
    elif name in _LM_NAMES:
        from . import lm as module
    elif name in _BLOCK_NAMES:
        from . import block as module
    else:
        raise AttributeError(name)
    globals()[name] = value = getattr(module, name)
    return value
