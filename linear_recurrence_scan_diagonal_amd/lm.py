"""ctypes binding of the language-model operators (include/lrs_lm.h).

Argument marshalling only, in the manner of ``binding``: shapes and dtypes are
checked, outputs and workspaces are torch device tensors, and raw pointers plus
the current HIP stream go to the C ABI.
"""
from __future__ import annotations

import ctypes

import torch

from . import binding
from .binding import DTYPES, LrsError, _i64, _int, _sz, _vp
from .binding import _check_dev as _refuse

EXPORTS = ("lrs_glr_checkpoint_rows", "lrs_glr_workspace_bytes", "lrs_glr_fwd",
           "lrs_glr_bwd_workspace_bytes", "lrs_glr_bwd", "lrs_glr_step", "lrs_layernorm_fwd",
           "lrs_layernorm_bwd_workspace_bytes", "lrs_layernorm_bwd",
           "lrs_linear_ce_workspace_bytes", "lrs_linear_ce_fwd", "lrs_linear_ce_bwd",
           "lrs_linear_ce_fwd_bwd")

_lib = None


def load():
    """liblrs.so with the prototypes of lrs_lm.h set."""
    global _lib
    lib = binding.load()
    if _lib is lib:
        return lib
    f = ctypes.c_float
    lib.lrs_glr_checkpoint_rows.argtypes = [_i64]
    lib.lrs_glr_checkpoint_rows.restype = _i64
    for name in ("lrs_glr_workspace_bytes", "lrs_glr_bwd_workspace_bytes"):
        getattr(lib, name).argtypes = [_i64] * 3
        getattr(lib, name).restype = _sz
    lib.lrs_glr_fwd.argtypes = [_vp] * 3 + [_i64] + [_vp] * 8 + [_i64] * 3 + [f, _int, _vp, _sz, _vp]
    lib.lrs_glr_bwd.argtypes = ([_vp] * 3 + [_i64] + [_vp] * 10 + [_i64] + [_vp] * 4 + [_i64] * 3 +
                                [f, _int, _vp, _sz, _vp])
    lib.lrs_glr_step.argtypes = [_vp] * 3 + [_i64] + [_vp] * 6 + [_i64] * 3 + [f, _int, _vp]
    lib.lrs_layernorm_fwd.argtypes = [_vp] * 8 + [_i64] * 2 + [f, _int, _vp]
    lib.lrs_layernorm_bwd_workspace_bytes.argtypes = [_i64] * 2
    lib.lrs_layernorm_bwd_workspace_bytes.restype = _sz
    lib.lrs_layernorm_bwd.argtypes = [_vp] * 9 + [_i64] * 2 + [_int, _vp, _sz, _vp]
    lib.lrs_linear_ce_workspace_bytes.argtypes = [_i64] * 3 + [_int, _int]
    lib.lrs_linear_ce_workspace_bytes.restype = _sz
    lib.lrs_linear_ce_fwd.argtypes = [_vp] * 5 + [_i64] * 3 + [_int, _vp, _sz, _vp]
    lib.lrs_linear_ce_bwd.argtypes = [_vp] * 7 + [_i64] * 3 + [_int, _vp, _sz, _vp]
    lib.lrs_linear_ce_fwd_bwd.argtypes = [_vp] * 8 + [_i64] * 3 + [_int, _vp, _sz, _vp]
    for name in EXPORTS:
        if name.endswith(("_fwd", "_bwd", "_step")):
            getattr(lib, name).restype = _int
    _lib = lib
    return lib


# The smallest calls take a few microseconds on the device, so the checks below
# first ask one cheap question and look for the reason only if the answer is no;
# pointers go to ctypes as plain integers.

_raw_stream = torch._C._cuda_getCurrentRawStream


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(dev):
    return _raw_stream(dev.index)


def _call(rc, where):
    if rc:
        raise LrsError(rc, where)


def _check_dev(name, t, dtype, shape):
    """A contiguous device tensor of this type and shape, or None."""
    if t is None:
        return
    try:
        if t.is_cuda and t.dtype is dtype and t.shape == shape and t.is_contiguous():
            return
    except AttributeError:
        pass
    _refuse(name, t, dtype, shape)


def _workspace(nbytes, dev, workspace):
    if nbytes == 0:
        return None
    if workspace is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=dev)
    if not isinstance(workspace, torch.Tensor) or not workspace.is_cuda:
        raise TypeError("workspace must be a device tensor")
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    if workspace.numel() * workspace.element_size() < nbytes:
        raise ValueError(f"workspace needs {nbytes} bytes")
    return workspace


def _pitch(name, t, like=None):
    """Row pitch of a tensor [..., D] whose last axis is contiguous and whose
    leading axes are evenly spaced rows (contiguous, or one slice of a wider
    array's last axis); None if it has at most one row."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a device tensor")
    if t.dtype not in DTYPES:
        raise TypeError(f"{name} must be float32 or bfloat16, got {t.dtype}")
    if like is not None:
        if t.dtype is not like.dtype:
            raise TypeError(f"{name} must be {like.dtype}, got {t.dtype}")
        if t.shape != like.shape:
            raise ValueError(f"{name} must have shape {tuple(like.shape)}, got {tuple(t.shape)}")
    shape, stride = t.shape, t.stride()
    D = shape[-1]
    if stride[-1] != 1 and D > 1 and t.numel():
        raise ValueError(f"{name}: the last axis must be contiguous")
    ld = expect = None  # pitch of a row, stride that the next axis must have
    for axis in range(len(shape) - 2, -1, -1):
        if shape[axis] == 1:
            continue
        if ld is None:
            ld = expect = stride[axis]
        elif stride[axis] != expect and t.numel():
            raise ValueError(f"{name}: rows must be evenly spaced")
        expect *= shape[axis]
    if ld is not None and ld < D and t.numel():
        raise ValueError(f"{name}: rows must not overlap")
    return ld


def _same_pitch(n0, t0, n1, t1, n2, t2, like=None):
    """The common row pitch of three tensors of one shape and type."""
    ld = _pitch(n0, t0, like)
    alike = False
    try:
        st = t0.stride()
        alike = (t1.stride() == st and t2.stride() == st and t1.shape == t0.shape and
                 t2.shape == t0.shape and t1.dtype is t0.dtype and t2.dtype is t0.dtype and
                 t1.is_cuda and t2.is_cuda)
    except AttributeError:
        pass
    if not alike and (_pitch(n1, t1, t0) != ld or _pitch(n2, t2, t0) != ld):
        if t0.numel():
            raise ValueError(f"{n0}, {n1} and {n2} must have the same row pitch")
    return int(t0.shape[-1]) if ld is None or not t0.numel() else ld


def _glr_params(D, bias_r, bias_i, decay):
    shape = (D,)
    for name, t in (("bias_r", bias_r), ("bias_i", bias_i), ("decay", decay)):
        if t is None:
            raise TypeError(f"{name} must be a device tensor")
        _check_dev(name, t, torch.float32, shape)


def glr_checkpoints(z_r):
    """The tensor that glr_fwd fills for glr_bwd: fp32, one [B,D] state a stretch
    of time steps of z_r's [T,B,D]."""
    T, B, D = (int(v) for v in z_r.shape)
    return torch.empty((load().lrs_glr_checkpoint_rows(T), B, D), dtype=torch.float32,
                       device=z_r.device)


def glr_fwd(z_r, z_i, x, bias_r, bias_i, decay, c: float = 8.0, reset=None, h0=None,
            want_h_last: bool = False, checkpoints=None, out=None, workspace=None):
    """Gated linear recurrence h_t = a_t h_{t-1} + sqrt(1 - a_t^2) i_t x_t with
    a = exp(-c softplus(decay) sigmoid(z_r + bias_r)), i = sigmoid(z_i + bias_i).

    z_r, z_i, x: [T,B,D] bf16 or fp32, contiguous or slices of one [T,B,3D]
    projection.  bias_r, bias_i, decay: [D] fp32.  reset: [T,B] uint8 or bool,
    nonzero where a document starts.  h0: [B,D] fp32.  checkpoints: a tensor of
    glr_checkpoints, filled for glr_bwd.  Returns h or (h, h_last)."""
    lib = load()
    if z_r.dim() != 3:
        raise ValueError("z_r must be [T,B,D]")
    T, B, D = (int(v) for v in z_r.shape)
    ld = _same_pitch("z_r", z_r, "z_i", z_i, "x", x)
    _glr_params(D, bias_r, bias_i, decay)
    reset = _reset(reset, T, B)
    _check_dev("h0", h0, torch.float32, (B, D))
    _check_dev("checkpoints", checkpoints, torch.float32, (lib.lrs_glr_checkpoint_rows(T), B, D))
    h = torch.empty((T, B, D), dtype=z_r.dtype, device=z_r.device) if out is None else out
    _check_dev("out", h, z_r.dtype, z_r.shape)
    h_last = torch.empty((B, D), dtype=torch.float32, device=z_r.device) if want_h_last else None
    nbytes = lib.lrs_glr_workspace_bytes(T, B, D)
    ws = _workspace(nbytes, z_r.device, workspace)
    _call(lib.lrs_glr_fwd(_ptr(z_r), _ptr(z_i), _ptr(x), ld, _ptr(bias_r), _ptr(bias_i),
                          _ptr(decay), _ptr(reset), _ptr(h0), _ptr(h), _ptr(h_last),
                          _ptr(checkpoints), T, B, D, float(c), DTYPES[z_r.dtype], _ptr(ws), nbytes,
                          _stream(z_r.device)), "lrs_glr_fwd")
    return (h, h_last) if want_h_last else h


def _reset(reset, T, B):
    if reset is None:
        return None
    if isinstance(reset, torch.Tensor) and reset.dtype == torch.bool:
        reset = reset.view(torch.uint8)
    _check_dev("reset", reset, torch.uint8, (T, B))
    return reset


def glr_bwd(z_r, z_i, x, bias_r, bias_i, decay, checkpoints, grad_h, c: float = 8.0, reset=None,
            grad_h_last=None, grad_z=None, workspace=None):
    """Backward of glr_fwd for the same inputs.  grad_h: [T,B,D], grad_h_last:
    [B,D] fp32 or None.  grad_z: optional (grad_zr, grad_zi, grad_x) tensors to
    fill, e.g. the three slices of one [T,B,3D] gradient.  Returns (grad_zr,
    grad_zi, grad_x, grad_bias_r, grad_bias_i, grad_decay, grad_h0)."""
    lib = load()
    if z_r.dim() != 3:
        raise ValueError("z_r must be [T,B,D]")
    T, B, D = (int(v) for v in z_r.shape)
    ld = _same_pitch("z_r", z_r, "z_i", z_i, "x", x)
    _glr_params(D, bias_r, bias_i, decay)
    reset = _reset(reset, T, B)
    _check_dev("checkpoints", checkpoints, torch.float32, (lib.lrs_glr_checkpoint_rows(T), B, D))
    if checkpoints is None:
        raise TypeError("checkpoints must be the tensor that glr_fwd filled")
    _check_dev("grad_h", grad_h, z_r.dtype, z_r.shape)
    _check_dev("grad_h_last", grad_h_last, torch.float32, (B, D))
    dev = z_r.device
    if grad_z is None:
        grad_z = tuple(torch.empty((T, B, D), dtype=z_r.dtype, device=dev) for _ in range(3))
    gr, gi, gx = grad_z
    ldg = _same_pitch("grad_zr", gr, "grad_zi", gi, "grad_x", gx, like=z_r)
    gbr, gbi, gd = (torch.empty(D, dtype=torch.float32, device=dev) for _ in range(3))
    gh0 = torch.empty((B, D), dtype=torch.float32, device=dev)
    nbytes = lib.lrs_glr_bwd_workspace_bytes(T, B, D)
    ws = _workspace(nbytes, dev, workspace)
    _call(lib.lrs_glr_bwd(_ptr(z_r), _ptr(z_i), _ptr(x), ld, _ptr(bias_r), _ptr(bias_i),
                          _ptr(decay), _ptr(reset), _ptr(checkpoints), _ptr(grad_h),
                          _ptr(grad_h_last), _ptr(gr), _ptr(gi), _ptr(gx), ldg, _ptr(gbr),
                          _ptr(gbi), _ptr(gd), _ptr(gh0), T, B, D, float(c), DTYPES[z_r.dtype],
                          _ptr(ws), nbytes, _stream(dev)), "lrs_glr_bwd")
    return gr, gi, gx, gbr, gbi, gd, gh0


def glr_step(z_r, z_i, x, bias_r, bias_i, decay, state, slots=None, c: float = 8.0, out=None):
    """One token of glr_fwd for each of B sequences: z_r, z_i, x [B,D]; state
    [S,D] fp32, updated in place; slots [B] int32, each sequence's row of state
    (outside [0, S): idle, h = 0), or None for row b.  Returns h [B,D]."""
    lib = load()
    if z_r.dim() != 2:
        raise ValueError("z_r must be [B,D]")
    B, D = (int(v) for v in z_r.shape)
    ld = _same_pitch("z_r", z_r, "z_i", z_i, "x", x)
    _glr_params(D, bias_r, bias_i, decay)
    if not isinstance(state, torch.Tensor) or state.dim() != 2 or state.shape[1] != D:
        raise ValueError(f"state must be [S,{D}]")
    _check_dev("state", state, torch.float32, state.shape)
    _check_dev("slots", slots, torch.int32, (B,))
    if slots is None and state.shape[0] < B:
        raise ValueError("state needs a row for every sequence")
    h = torch.empty((B, D), dtype=z_r.dtype, device=z_r.device) if out is None else out
    _check_dev("out", h, z_r.dtype, (B, D))
    _call(lib.lrs_glr_step(_ptr(z_r), _ptr(z_i), _ptr(x), ld, _ptr(bias_r), _ptr(bias_i),
                           _ptr(decay), _ptr(slots), _ptr(state), _ptr(h), B, D,
                           int(state.shape[0]), float(c), DTYPES[z_r.dtype], _stream(z_r.device)),
          "lrs_glr_step")
    return h


def layernorm_fwd(x, gamma, beta=None, residual=None, eps: float = 1e-5, save: bool = False,
                  out=None, out_sum=None):
    """Layer norm over the last axis of x [..., D] (bf16 or fp32), of
    s = x + residual where a residual is given.  gamma, beta: [D] fp32.
    Returns (y, s or None, mean, rstd); mean and rstd ([rows] fp32) are None
    unless save, and are what layernorm_bwd takes.  out_sum may be x or residual
    (the residual stream in place)."""
    lib = load()
    if not isinstance(x, torch.Tensor) or x.dim() < 1:
        raise TypeError("x must be a device tensor")
    _check_dev("x", x, x.dtype, x.shape)
    if x.dtype not in DTYPES:
        raise TypeError(f"x must be float32 or bfloat16, got {x.dtype}")
    D = int(x.shape[-1])
    R = x.numel() // D if D else 0
    _check_dev("gamma", gamma, torch.float32, (D,))
    _check_dev("beta", beta, torch.float32, (D,))
    _check_dev("residual", residual, x.dtype, x.shape)
    y = torch.empty_like(x) if out is None else out
    _check_dev("out", y, x.dtype, x.shape)
    s = None
    if residual is not None:
        s = torch.empty_like(x) if out_sum is None else out_sum
        _check_dev("out_sum", s, x.dtype, x.shape)
    mean = rstd = None
    if save:
        mean, rstd = (torch.empty(R, dtype=torch.float32, device=x.device) for _ in range(2))
    _call(lib.lrs_layernorm_fwd(_ptr(x), _ptr(residual), _ptr(gamma), _ptr(beta), _ptr(y), _ptr(s),
                                _ptr(mean), _ptr(rstd), R, D, float(eps), DTYPES[x.dtype],
                                _stream(x.device)), "lrs_layernorm_fwd")
    return y, s, mean, rstd


def layernorm_bwd(s, gamma, mean, rstd, grad_y, grad_sum=None, want_grad_beta: bool = True,
                  out=None, workspace=None):
    """Backward of layernorm_fwd.  s: what was normalised (x, or the sum);
    grad_sum: gradient that reaches s from elsewhere, or None.  out may be
    grad_y or grad_sum.  Returns (grad_x, grad_gamma, grad_beta or None);
    grad_x is also the residual's gradient."""
    lib = load()
    _check_dev("s", s, s.dtype, s.shape)
    if s.dtype not in DTYPES:
        raise TypeError(f"s must be float32 or bfloat16, got {s.dtype}")
    D = int(s.shape[-1])
    R = s.numel() // D if D else 0
    _check_dev("gamma", gamma, torch.float32, (D,))
    for name, t in (("mean", mean), ("rstd", rstd)):
        _check_dev(name, t, torch.float32, (R,))
    _check_dev("grad_y", grad_y, s.dtype, s.shape)
    _check_dev("grad_sum", grad_sum, s.dtype, s.shape)
    gx = torch.empty_like(s) if out is None else out
    _check_dev("out", gx, s.dtype, s.shape)
    gg = torch.empty(D, dtype=torch.float32, device=s.device)
    gb = torch.empty(D, dtype=torch.float32, device=s.device) if want_grad_beta else None
    nbytes = lib.lrs_layernorm_bwd_workspace_bytes(R, D)
    ws = _workspace(nbytes, s.device, workspace)
    _call(lib.lrs_layernorm_bwd(_ptr(s), _ptr(gamma), _ptr(mean), _ptr(rstd), _ptr(grad_y),
                                _ptr(grad_sum), _ptr(gx), _ptr(gg), _ptr(gb), R, D,
                                DTYPES[s.dtype], _ptr(ws), nbytes, _stream(s.device)),
          "lrs_layernorm_bwd")
    return gx, gg, gb


def _ce_args(x, w, target, backward):
    if not isinstance(x, torch.Tensor) or x.dim() != 2 or not isinstance(w, torch.Tensor) \
            or w.dim() != 2:
        raise ValueError("x must be [N,D] and w [V,D]")
    if x.dtype not in DTYPES:
        raise TypeError(f"x must be float32 or bfloat16, got {x.dtype}")
    N, D = (int(v) for v in x.shape)
    V = int(w.shape[0])
    _check_dev("x", x, x.dtype, (N, D))
    _check_dev("w", w, x.dtype, (V, D))
    _check_dev("target", target, torch.int64, (N,))
    return N, V, D, load().lrs_linear_ce_workspace_bytes(N, V, D, DTYPES[x.dtype],
                                                                int(backward))


def linear_ce_fwd(x, w, target, workspace=None):
    """Cross entropy of the logits x w^T (x [N,D], w [V,D], bf16 or fp32) against
    target [N] int64; a target outside [0, V) is ignored.  Returns (loss, lse),
    [N] fp32 each."""
    lib = load()
    N, V, D, nbytes = _ce_args(x, w, target, False)
    loss, lse = (torch.empty(N, dtype=torch.float32, device=x.device) for _ in range(2))
    ws = _workspace(nbytes, x.device, workspace)
    _call(lib.lrs_linear_ce_fwd(_ptr(x), _ptr(w), _ptr(target), _ptr(loss), _ptr(lse), N, V, D,
                                DTYPES[x.dtype], _ptr(ws), nbytes, _stream(x.device)),
          "lrs_linear_ce_fwd")
    return loss, lse


def linear_ce_bwd(x, w, target, lse, grad_loss, out=None, workspace=None):
    """Gradient of linear_ce_fwd for dL/dloss = grad_loss [N] fp32, with the lse
    it returned.  Returns (grad_x, grad_w)."""
    lib = load()
    N, V, D, nbytes = _ce_args(x, w, target, True)
    _check_dev("lse", lse, torch.float32, (N,))
    _check_dev("grad_loss", grad_loss, torch.float32, (N,))
    gx, gw = (torch.empty_like(x), torch.empty_like(w)) if out is None else out
    _check_dev("grad_x", gx, x.dtype, x.shape)
    _check_dev("grad_w", gw, x.dtype, w.shape)
    ws = _workspace(nbytes, x.device, workspace)
    _call(lib.lrs_linear_ce_bwd(_ptr(x), _ptr(w), _ptr(target), _ptr(lse), _ptr(grad_loss),
                                _ptr(gx), _ptr(gw), N, V, D, DTYPES[x.dtype], _ptr(ws), nbytes,
                                _stream(x.device)), "lrs_linear_ce_bwd")
    return gx, gw


def linear_ce_fwd_bwd(x, w, target, grad_loss, out=None, workspace=None):
    """linear_ce_fwd and linear_ce_bwd in one call, for a grad_loss known before
    the loss.  Returns (loss, lse, grad_x, grad_w)."""
    lib = load()
    N, V, D, nbytes = _ce_args(x, w, target, True)
    _check_dev("grad_loss", grad_loss, torch.float32, (N,))
    loss, lse = (torch.empty(N, dtype=torch.float32, device=x.device) for _ in range(2))
    gx, gw = (torch.empty_like(x), torch.empty_like(w)) if out is None else out
    _check_dev("grad_x", gx, x.dtype, x.shape)
    _check_dev("grad_w", gw, x.dtype, w.shape)
    ws = _workspace(nbytes, x.device, workspace)
    _call(lib.lrs_linear_ce_fwd_bwd(_ptr(x), _ptr(w), _ptr(target), _ptr(grad_loss), _ptr(loss),
                                    _ptr(lse), _ptr(gx), _ptr(gw), N, V, D, DTYPES[x.dtype],
                                    _ptr(ws), nbytes, _stream(x.device)), "lrs_linear_ce_fwd_bwd")
    return loss, lse, gx, gw
