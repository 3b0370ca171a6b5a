"""ctypes binding of the operators of delta-rule language models (include/lrs_block.h).

Argument marshalling only, in the manner of ``binding`` and ``lm``: shapes, dtypes and devices
are checked, outputs and workspaces are torch device tensors, and raw pointers plus the
current HIP stream go to the C ABI.
"""
from __future__ import annotations

import ctypes

import torch

from . import lm
from .binding import DTYPES, _i64, _int, _sz, _vp
from .binding import _check_dev as _refuse
from .lm import _call, _ptr, _stream

EXPORTS = ("lrs_gdr_checkpoint_rows", "lrs_gdr_workspace_bytes", "lrs_gdr_fwd",
           "lrs_gdr_bwd_workspace_bytes", "lrs_gdr_bwd", "lrs_gdr_step", "lrs_rmsnorm_fwd",
           "lrs_rmsnorm_fwd_fp8", "lrs_rmsnorm_bwd_workspace_bytes", "lrs_rmsnorm_bwd",
           "lrs_logprobs_fwd", "lrs_logprobs_bwd")

_lib = None


def load():
    """liblrs.so with the prototypes of lrs.h, lrs_lm.h and lrs_block.h set."""
    global _lib, _several
    lib = lm.load()
    if _lib is lib:
        return lib
    f = ctypes.c_float
    lib.lrs_gdr_checkpoint_rows.argtypes = [_i64]
    lib.lrs_gdr_checkpoint_rows.restype = _i64
    for name in ("lrs_gdr_workspace_bytes", "lrs_gdr_bwd_workspace_bytes"):
        getattr(lib, name).argtypes = [_i64] * 6 + [_int]
        getattr(lib, name).restype = _sz
    qkv = [_vp, _i64] * 3
    lib.lrs_gdr_fwd.argtypes = qkv + [_vp] * 7 + [_i64] * 6 + [f, _int, _vp, _sz, _vp]
    lib.lrs_gdr_bwd.argtypes = qkv + [_vp] * 6 + qkv + [_vp] * 3 + [_i64] * 6 + [f, _int, _vp, _sz, _vp]
    lib.lrs_gdr_step.argtypes = qkv + [_vp] * 5 + [_i64] * 6 + [f, _int, _vp]
    lib.lrs_rmsnorm_fwd.argtypes = [_vp] * 6 + [_i64] * 2 + [f, _int, _vp]
    lib.lrs_rmsnorm_fwd_fp8.argtypes = [_vp] * 6 + [_i64] * 3 + [f, _int, _vp]
    lib.lrs_rmsnorm_bwd_workspace_bytes.argtypes = [_i64] * 2
    lib.lrs_rmsnorm_bwd_workspace_bytes.restype = _sz
    lib.lrs_rmsnorm_bwd.argtypes = [_vp] * 7 + [_i64] * 2 + [_int, _vp, _sz, _vp]
    lib.lrs_logprobs_fwd.argtypes = [_vp, _i64] + [_vp] * 6 + [_i64] * 3 + [_int, _vp]
    lib.lrs_logprobs_bwd.argtypes = [_vp, _i64] + [_vp] * 6 + [_i64] * 3 + [_int, _vp]
    for name in EXPORTS:
        if name.endswith(("_fwd", "_bwd", "_step", "_fp8")):
            getattr(lib, name).restype = _int
    _several = torch.cuda.device_count() > 1
    _lib = lib
    return lib


_current = torch._C._cuda_getDevice
_several = True  # whether the process sees more devices than one (asked by load: a call's
                 # check takes 0.4 us)


def _elsewhere(t):
    """Whether t is on a device that is not the current one, which launches on the default
    stream go to: such a call is made again with t's device as the current one."""
    return isinstance(t, torch.Tensor) and t.is_cuda and t.get_device() != _current()


def _same_device(name, t, dev):
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on cuda:{dev} like the other tensors, got {t.device}")


def _check_dev(name, t, dtype, shape, dev):
    """A contiguous tensor of this type and shape on device number dev, or None."""
    if t is None:
        return
    try:
        if t.get_device() == dev and t.dtype is dtype and t.shape == shape and t.is_contiguous():
            return
    except AttributeError:
        pass
    _refuse(name, t, dtype, shape)
    _same_device(name, t, dev)


def _workspace(nbytes, dev, workspace):
    ws = lm._workspace(nbytes, dev, workspace)
    if workspace is not None and ws is not None:
        _same_device("workspace", ws, dev.index)
    return ws


def _reset(reset, T, B, dev):
    reset = lm._reset(reset, T, B)
    if reset is not None:
        _same_device("reset", reset, dev)
    return reset


def _heads(name, t, lead, like=None):
    """(heads, features, row pitch) of a tensor [*lead, heads, features] whose rows of
    heads * features are contiguous and evenly spaced (contiguous, or one slice of a
    wider array's last axis, unflattened)."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a device tensor")
    if t.dtype not in DTYPES:
        raise TypeError(f"{name} must be float32 or bfloat16, got {t.dtype}")
    if like is not None and (t.dtype is not like.dtype or t.get_device() != like.get_device()):
        if t.dtype is not like.dtype:
            raise TypeError(f"{name} must be {like.dtype}, got {t.dtype}")
        _same_device(name, t, like.get_device())
    shape, stride = t.shape, t.stride()
    n = len(lead)
    if len(shape) != n + 2 or shape[:n] != lead:
        raise ValueError(f"{name} must be [{', '.join(str(v) for v in lead)}, heads, features], "
                         f"got {tuple(shape)}")
    H, D = shape[n], shape[n + 1]
    width = H * D
    if not t.numel():
        return H, D, width
    if (stride[n + 1] != 1 and D > 1) or (stride[n] != D and H > 1):
        raise ValueError(f"{name}: heads and features must be contiguous")
    ld = expect = None
    for axis in range(n - 1, -1, -1):
        if shape[axis] == 1:
            continue
        if ld is None:
            ld = expect = stride[axis]
        elif stride[axis] != expect:
            raise ValueError(f"{name}: rows must be evenly spaced")
        expect *= shape[axis]
    if ld is None:
        ld = width
    elif ld < width:
        raise ValueError(f"{name}: rows must not overlap")
    return H, D, ld


def _gdr_inputs(q, k, v, log_decay, beta, dims):
    if not isinstance(v, torch.Tensor) or v.dim() != dims + 2:
        raise ValueError("v must be [T,B,H,V]" if dims == 2 else "v must be [B,H,V]")
    lead = v.shape[:dims]
    H, V, ld_v = _heads("v", v, lead)
    Hk, K, ld_k = _heads("k", k, lead, v)
    Hq, Kq, ld_q = _heads("q", q, lead, v)
    if (Hq, Kq) != (Hk, K):
        raise ValueError(f"q must have the shape of k, {tuple(k.shape)}, got {tuple(q.shape)}")
    if not Hk or not H or H % Hk:
        raise ValueError(f"v's heads ({H}) must be a multiple of k's ({Hk})")
    gates, index = torch.Size((*lead, H)), v.get_device()
    for name, t in (("log_decay", log_decay), ("beta", beta)):
        if t is None:
            raise TypeError(f"{name} must be a device tensor")
        _check_dev(name, t, torch.float32, gates, index)
    return lead, H, Hk, K, V, (q.data_ptr(), ld_q, k.data_ptr(), ld_k, v.data_ptr(), ld_v,
                               log_decay.data_ptr(), beta.data_ptr())


def gdr_checkpoints(k, v):
    """The tensor that gdr_fwd fills for gdr_bwd: fp32, for each chunk of 64 time steps,
    sequence and head the state [K,V] that enters it and [64,V] of its steps (V rounded
    up to a multiple of 4).  k: [T,B,Hk,K], v: [T,B,H,V]."""
    T, B, H, V = (int(n) for n in v.shape)
    return torch.empty(_saved(T, B, H, int(k.shape[-1]), V), dtype=torch.float32, device=v.device)


def _saved(T, B, H, K, V):
    return torch.Size((load().lrs_gdr_checkpoint_rows(T), B, H, K + 64, (V + 3) // 4 * 4))


def gdr_fwd(q, k, v, log_decay, beta, scale=None, reset=None, state0=None,
            want_state: bool = False, checkpoints=None, out=None, workspace=None):
    """Gated delta rule: a state S [K,V] a head, S <- exp(log_decay) S,
    u = beta (v - S^T k), S <- S + k u^T, o = scale S^T q.

    q, k: [T,B,Hk,K], v: [T,B,H,V], bf16 or fp32, contiguous or slices of one
    projection, H a multiple of Hk (head h reads q and k of head h // (H // Hk)).
    log_decay, beta: [T,B,H] fp32.  scale: K**-0.5 if None.  reset: [T,B] uint8 or
    bool, nonzero where a document starts.  state0: [B,H,K,V] fp32.  checkpoints: a
    tensor of gdr_checkpoints, filled for gdr_bwd.  Returns o [T,B,H,V], or (o, state)."""
    lib = load()
    if _several and _elsewhere(v):
        with torch.cuda.device(v.device):
            return gdr_fwd(q, k, v, log_decay, beta, scale, reset, state0, want_state,
                           checkpoints, out, workspace)
    (T, B), H, Hk, K, V, args = _gdr_inputs(q, k, v, log_decay, beta, 2)
    dev = v.device
    index = dev.index
    reset = _reset(reset, T, B, index)
    shape = torch.Size((B, H, K, V))
    _check_dev("state0", state0, torch.float32, shape, index)
    if checkpoints is not None:
        _check_dev("checkpoints", checkpoints, torch.float32, _saved(T, B, H, K, V), index)
    o = torch.empty((T, B, H, V), dtype=v.dtype, device=dev) if out is None else out
    _check_dev("out", o, v.dtype, v.shape, index)
    state = torch.empty(shape, dtype=torch.float32, device=dev) if want_state else None
    io = DTYPES[v.dtype]
    nbytes = lib.lrs_gdr_workspace_bytes(T, B, H, Hk, K, V, io)
    ws = _workspace(nbytes, dev, workspace)
    _call(lib.lrs_gdr_fwd(*args, _ptr(reset), _ptr(state0), o.data_ptr(), _ptr(state),
                          _ptr(checkpoints), T, B, H, Hk, K, V,
                          K ** -0.5 if scale is None else float(scale), io, _ptr(ws), nbytes,
                          _stream(dev)), "lrs_gdr_fwd")
    return (o, state) if want_state else o


def gdr_bwd(q, k, v, log_decay, beta, checkpoints, grad_o, scale=None, reset=None,
            grad_state=None, grad_qkv=None, workspace=None):
    """Backward of gdr_fwd for the same inputs.  grad_o: [T,B,H,V], grad_state:
    [B,H,K,V] fp32 (the last state's gradient) or None.  grad_qkv: optional (grad_q,
    grad_k, grad_v) tensors to fill, e.g. the three slices of one projection's
    gradient.  Returns (grad_q, grad_k, grad_v, grad_log_decay, grad_beta,
    grad_state0)."""
    lib = load()
    if _several and _elsewhere(v):
        with torch.cuda.device(v.device):
            return gdr_bwd(q, k, v, log_decay, beta, checkpoints, grad_o, scale, reset,
                           grad_state, grad_qkv, workspace)
    (T, B), H, Hk, K, V, args = _gdr_inputs(q, k, v, log_decay, beta, 2)
    dev = v.device
    index = dev.index
    reset = _reset(reset, T, B, index)
    shape = torch.Size((B, H, K, V))
    if checkpoints is None:
        raise TypeError("checkpoints must be the tensor that gdr_fwd filled")
    _check_dev("checkpoints", checkpoints, torch.float32, _saved(T, B, H, K, V), index)
    if grad_o is None:
        raise TypeError("grad_o must be a device tensor")
    _check_dev("grad_o", grad_o, v.dtype, v.shape, index)
    _check_dev("grad_state", grad_state, torch.float32, shape, index)
    if grad_qkv is None:
        grad_qkv = tuple(torch.empty(t.shape, dtype=v.dtype, device=dev) for t in (q, k, v))
    grads = []
    for name, t, like in zip(("grad_q", "grad_k", "grad_v"), grad_qkv, (q, k, v)):
        h, d, ld = _heads(name, t, v.shape[:2], v)
        if (h, d) != tuple(like.shape[2:]):
            raise ValueError(f"{name} must have shape {tuple(like.shape)}, got {tuple(t.shape)}")
        grads += [t.data_ptr(), ld]
    gg, gb = (torch.empty((T, B, H), dtype=torch.float32, device=dev) for _ in range(2))
    gs = torch.empty(shape, dtype=torch.float32, device=dev)
    io = DTYPES[v.dtype]
    nbytes = lib.lrs_gdr_bwd_workspace_bytes(T, B, H, Hk, K, V, io)
    ws = _workspace(nbytes, dev, workspace)
    _call(lib.lrs_gdr_bwd(*args, _ptr(reset), checkpoints.data_ptr(), grad_o.data_ptr(),
                          _ptr(grad_state), *grads, gg.data_ptr(), gb.data_ptr(), gs.data_ptr(),
                          T, B, H, Hk, K, V, K ** -0.5 if scale is None else float(scale), io,
                          _ptr(ws), nbytes, _stream(dev)), "lrs_gdr_bwd")
    return (*grad_qkv, gg, gb, gs)


def gdr_step(q, k, v, log_decay, beta, state, slots=None, scale=None, out=None):
    """One token of gdr_fwd for each of B sequences: q, k [B,Hk,K], v [B,H,V],
    log_decay, beta [B,H] fp32; state [S,H,K,V] fp32, updated in place; slots [B]
    int32, each sequence's row of state (outside [0, S): idle, o = 0), or None for
    row b.  Returns o [B,H,V]."""
    lib = load()
    if _several and _elsewhere(v):
        with torch.cuda.device(v.device):
            return gdr_step(q, k, v, log_decay, beta, state, slots, scale, out)
    (B,), H, Hk, K, V, args = _gdr_inputs(q, k, v, log_decay, beta, 1)
    if not isinstance(state, torch.Tensor) or state.dim() != 4 or state.shape[1:] != (H, K, V):
        raise ValueError(f"state must be [S,{H},{K},{V}]")
    index = v.get_device()
    _check_dev("state", state, torch.float32, state.shape, index)
    _check_dev("slots", slots, torch.int32, (B,), index)
    if slots is None and state.shape[0] < B:
        raise ValueError("state needs a row for every sequence")
    o = torch.empty((B, H, V), dtype=v.dtype, device=v.device) if out is None else out
    _check_dev("out", o, v.dtype, v.shape, index)
    _call(lib.lrs_gdr_step(*args, _ptr(slots), state.data_ptr(), o.data_ptr(), B, H, Hk, K, V,
                           state.shape[0], K ** -0.5 if scale is None else float(scale),
                           DTYPES[v.dtype], _stream(v.device)), "lrs_gdr_step")
    return o


def _rms_inputs(x, gamma, residual, out_sum):
    if not isinstance(x, torch.Tensor) or x.dim() < 1:
        raise TypeError("x must be a device tensor")
    index = x.get_device()
    if index < 0:
        raise TypeError("x must be a device tensor")
    _check_dev("x", x, x.dtype, x.shape, index)
    if x.dtype not in DTYPES:
        raise TypeError(f"x must be float32 or bfloat16, got {x.dtype}")
    D = int(x.shape[-1])
    if gamma is None:
        raise TypeError("gamma must be a device tensor")
    _check_dev("gamma", gamma, torch.float32, (D,), index)
    _check_dev("residual", residual, x.dtype, x.shape, index)
    s = None
    if residual is not None:
        s = torch.empty_like(x) if out_sum is None else out_sum
        if out_sum is not None:
            _check_dev("out_sum", s, x.dtype, x.shape, index)
    return x.numel() // D if D else 0, D, s


def rmsnorm_fwd(x, gamma, residual=None, eps: float = 1e-6, save: bool = False, out=None,
                out_sum=None):
    """Root-mean-square norm over the last axis of x [..., D] (bf16 or fp32), of
    s = x + residual where a residual is given.  gamma: [D] fp32.  Returns (y, s or
    None, rstd); rstd ([rows] fp32) is None unless save, and is what rmsnorm_bwd
    takes.  out_sum may be x or residual (the residual stream in place)."""
    lib = load()
    if _several and _elsewhere(x):
        with torch.cuda.device(x.device):
            return rmsnorm_fwd(x, gamma, residual, eps, save, out, out_sum)
    R, D, s = _rms_inputs(x, gamma, residual, out_sum)
    y = torch.empty_like(x) if out is None else out
    if out is not None:
        _check_dev("out", y, x.dtype, x.shape, x.get_device())
    rstd = torch.empty(R, dtype=torch.float32, device=x.device) if save else None
    _call(lib.lrs_rmsnorm_fwd(_ptr(x), _ptr(residual), _ptr(gamma), _ptr(y), _ptr(s), _ptr(rstd),
                              R, D, float(eps), DTYPES[x.dtype], _stream(x.device)),
          "lrs_rmsnorm_fwd")
    return y, s, rstd


def rmsnorm_fwd_fp8(x, gamma, residual=None, eps: float = 1e-6, group: int = 128, out=None,
                    out_sum=None):
    """rmsnorm_fwd with y in 8 bits: q (torch.float8_e4m3fn, the shape of x) and
    scales [rows, groups] fp32, one for every `group` = 128 features of a row, or for
    the whole row with group = 0; q * scale is y.  Returns (q, scales, s or None)."""
    lib = load()
    if _several and _elsewhere(x):
        with torch.cuda.device(x.device):
            return rmsnorm_fwd_fp8(x, gamma, residual, eps, group, out, out_sum)
    R, D, s = _rms_inputs(x, gamma, residual, out_sum)
    if group not in (0, 128):
        raise ValueError("group must be 128, or 0 for the whole row")
    if out is None:
        q = torch.empty_like(x, dtype=torch.float8_e4m3fn)
    else:
        q = out
        _check_dev("out", q, torch.float8_e4m3fn, x.shape, x.get_device())
    scales = gamma.new_empty((R, -(-D // group) if group else 1))
    _call(lib.lrs_rmsnorm_fwd_fp8(_ptr(x), _ptr(residual), _ptr(gamma), _ptr(q), _ptr(scales),
                                  _ptr(s), R, D, group, float(eps), DTYPES[x.dtype],
                                  _stream(x.device)), "lrs_rmsnorm_fwd_fp8")
    return q, scales, s


def rmsnorm_bwd(s, gamma, rstd, grad_y, grad_sum=None, out=None, workspace=None):
    """Backward of rmsnorm_fwd.  s: what was normalised (x, or the sum); grad_sum:
    gradient that reaches s from elsewhere, or None.  out may be grad_y or grad_sum.
    Returns (grad_x, grad_gamma); grad_x is also the residual's gradient."""
    lib = load()
    if _several and _elsewhere(s):
        with torch.cuda.device(s.device):
            return rmsnorm_bwd(s, gamma, rstd, grad_y, grad_sum, out, workspace)
    R, D, _ = _rms_inputs(s, gamma, None, None)
    index = s.get_device()
    for name, t, dtype, shape in (("rstd", rstd, torch.float32, (R,)),
                                  ("grad_y", grad_y, s.dtype, s.shape)):
        if t is None:
            raise TypeError(f"{name} must be a device tensor")
        _check_dev(name, t, dtype, shape, index)
    _check_dev("grad_sum", grad_sum, s.dtype, s.shape, index)
    gx = torch.empty_like(s) if out is None else out
    _check_dev("out", gx, s.dtype, s.shape, index)
    gg = torch.empty(D, dtype=torch.float32, device=s.device)
    nbytes = lib.lrs_rmsnorm_bwd_workspace_bytes(R, D)
    ws = _workspace(nbytes, s.device, workspace)
    _call(lib.lrs_rmsnorm_bwd(_ptr(s), _ptr(gamma), _ptr(rstd), _ptr(grad_y), _ptr(grad_sum),
                              _ptr(gx), _ptr(gg), R, D, DTYPES[s.dtype], _ptr(ws), nbytes,
                              _stream(s.device)), "lrs_rmsnorm_bwd")
    return gx, gg


def _logit_rows(name, t, like=None):
    """(N, V, row pitch) of a matrix whose rows are contiguous."""
    if not isinstance(t, torch.Tensor) or t.dim() != 2:
        raise ValueError(f"{name} must be [N,V]")
    return (*t.shape, lm._pitch(name, t, like) or t.shape[1])


def logprobs_fwd(logits, target, top: int = 0):
    """Of logits [N,V] (bf16 or fp32, rows may be a slice of wider ones): the log
    probability of target [N] int64 (outside [0, V): ignored, 0), the entropy, and the
    `top` (up to 64) likeliest tokens with their log probabilities, in falling order,
    the lower index first where they are equal.  Returns (logprob, entropy, lse,
    top_ids, top_logprobs): [N] fp32 three times, [N,top] int64 and fp32 (None
    without)."""
    lib = load()
    if _several and _elsewhere(logits):
        with torch.cuda.device(logits.device):
            return logprobs_fwd(logits, target, top)
    N, V, ld = _logit_rows("logits", logits)
    dev = logits.device
    if target is None:
        raise TypeError("target must be a device tensor")
    _check_dev("target", target, torch.int64, (N,), dev.index)
    if not 0 <= top <= min(64, V):
        raise ValueError("top must be between 0 and 64 and at most the number of logits")
    logprob, entropy, lse = (torch.empty(N, dtype=torch.float32, device=dev) for _ in range(3))
    ids = tops = None
    if top:
        ids = torch.empty((N, top), dtype=torch.int64, device=dev)
        tops = torch.empty((N, top), dtype=torch.float32, device=dev)
    _call(lib.lrs_logprobs_fwd(logits.data_ptr(), ld, target.data_ptr(), logprob.data_ptr(),
                               entropy.data_ptr(), lse.data_ptr(), _ptr(ids), _ptr(tops), N, V,
                               top, DTYPES[logits.dtype], _stream(dev)), "lrs_logprobs_fwd")
    return logprob, entropy, lse, ids, tops


def logprobs_bwd(logits, target, lse, entropy, grad_logprob, grad_entropy=None, out=None):
    """Gradient of logprobs_fwd's logprob and entropy for grad_logprob and
    grad_entropy ([N] fp32; the latter None for 0, entropy is then not read).  out may
    be the logits.  Returns grad_logits [N,V]."""
    lib = load()
    if _several and _elsewhere(logits):
        with torch.cuda.device(logits.device):
            return logprobs_bwd(logits, target, lse, entropy, grad_logprob, grad_entropy, out)
    N, V, ld = _logit_rows("logits", logits)
    index = logits.get_device()
    for name, t, dtype in (("target", target, torch.int64), ("lse", lse, torch.float32),
                           ("grad_logprob", grad_logprob, torch.float32)):
        if t is None:
            raise TypeError(f"{name} must be a device tensor")
        _check_dev(name, t, dtype, (N,), index)
    _check_dev("grad_entropy", grad_entropy, torch.float32, (N,), index)
    _check_dev("entropy", entropy, torch.float32, (N,), index)
    if grad_entropy is not None and entropy is None:
        raise TypeError("entropy must be the tensor that logprobs_fwd returned")
    g = torch.empty((N, V), dtype=logits.dtype, device=logits.device) if out is None else out
    _, _, ld_grad = _logit_rows("out", g, logits)
    _same_device("out", g, index)
    _call(lib.lrs_logprobs_bwd(logits.data_ptr(), ld, target.data_ptr(), lse.data_ptr(),
                               _ptr(entropy), grad_logprob.data_ptr(), _ptr(grad_entropy),
                               g.data_ptr(), ld_grad, N, V, DTYPES[logits.dtype],
                               _stream(logits.device)), "lrs_logprobs_bwd")
    return g
