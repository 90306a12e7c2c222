"""Norms and the linear layer with an epilogue, forward and backward.

What stands before and beside the SwiGLU block in the same models. Op level, as in
the package's other wrappers (every arithmetic step runs in the HIP kernels
behind the C ABI of include/swiglu_mlp.h; no fallback):

* ``norm_fwd``, ``norm_bwd``      layer norm and RMS norm over the last axis
* ``linear_fwd``, ``linear_bwd``  y = act(x W^T + b) + residual

with autograd: ``layer_norm``, ``rms_norm``, ``linear`` and, of all three, the
ungated feed-forward layer x + fc2(act(fc1(norm(x)))): ``feed_forward`` and the
module ``FeedForward``. Their nodes are in C++ (csrc/nodes.cpp), since small training
steps are bound by host code; they call the same library.
All tensors of a call share dtype (bf16, fp16 or fp32) and device.

Second derivatives, forward-mode derivatives and tracers (torch.jit.trace, make_fx) are
refused. The backward may run more than once
(``retain_graph``): it changes nothing that the forward kept.

Calls can be captured in a graph, with their backward. While an autograd graph of
the same leaves that was built on the default stream is alive, a captured call that
needs gradients is refused: the leaves' accumulation would leave the capture. A forward
without a backward is captured under torch.no_grad.
"""

import ctypes
import functools
import math

import torch

from . import _lib as _L
from .serve import _DT, _bytes, _check, _code, _device, _no_transforms, _on_gpu, _ptr, _stream, _workspace

ACTIVATIONS = tuple(_L.ACTS)


@functools.lru_cache(maxsize=None)
def _nodes():
    """The autograd nodes (csrc/nodes.cpp), which call the library."""
    _L.lib()
    try:
        from . import _nodes as nodes
    except ImportError as e:
        raise ImportError("backward_gate_up_amd/_nodes.so is missing or does not load: build it with "
                          "`python -m backward_gate_up_amd.build` (there is no fallback)") from e
    return nodes


@functools.lru_cache(maxsize=None)
def _c(name):
    return getattr(_L.lib(), "swiglu_mlp_" + name)


def _on(device, call, *args):
    """call(*args) with ``device`` current: the library launches on the current one."""
    if device.index == _device():
        return call(*args)
    with torch.cuda.device(device):
        return call(*args)


def _act(activation):
    try:
        return _L.ACTS[activation]
    except (KeyError, TypeError):
        raise ValueError(f"unknown activation {activation!r}; use one of {ACTIVATIONS}") from None


def _same(x, *others):
    """(dtype's code, device) of tensors that share them."""
    dtype, device = x.dtype, x.device
    for t in others:
        if t is not None and (t.dtype != dtype or t.device != device):
            raise ValueError("all tensors must share dtype and device")
    if not x.is_cuda:
        _on_gpu(x)
    dt = _DT.get(dtype)
    return (_code(x) if dt is None else dt), device


def _opt(t):
    return None if t is None else _ptr(t)


def _flat(t):
    """Contiguous, and without a negation that torch has put off."""
    if t is None or (t.is_contiguous() and not t.is_neg()):
        return t
    return t.resolve_neg().contiguous()


def _flat16(t):
    """As ``_flat``, and at an address that the matrix kernels take (a gradient may
    be a view that starts anywhere)."""
    t = _flat(t)
    return t.clone() if t is not None and t.data_ptr() & 15 else t


# ---- norms ------------------------------------------------------------------


def _norm_args(x, weight, bias, eps, rms):
    """(dtype's code, device), after checking the arguments."""
    shape = x.shape
    if len(shape) != 2 or weight.shape != shape[1:] or shape[1] == 0:
        raise ValueError(f"expected X[T,D] and weight[D]: X{tuple(shape)} weight{tuple(weight.shape)}")
    if bias is not None and (rms or bias.shape != weight.shape):
        raise ValueError("RMS norm has no bias" if rms else f"bias must be [D]: {tuple(bias.shape)}")
    if not 0 <= eps < math.inf:
        raise ValueError(f"eps must be a number from 0 up: got {eps}")
    return _same(x, weight, bias)


def _norm_fwd(x, weight, bias, eps, rms, stats, dt, device):
    T, D = x.shape
    y = torch.empty_like(x)
    st = torch.empty((1 if rms else 2, T), dtype=torch.float32, device=device) if stats else None
    rc = _c("norm_fwd")(x.data_ptr(), weight.data_ptr(), None if bias is None else bias.data_ptr(), y.data_ptr(),
                        st.data_ptr() if stats else None, T, D, eps, rms, dt, _stream(device))
    if rc:
        _check(rc, "swiglu_mlp_norm_fwd")
    return y, st


def norm_fwd(x, weight, bias=None, eps=1e-5, rms=False, stats=True):
    """Y = (x - mean) rstd weight + bias over the last axis of x[T, D], rstd = 1 /
    sqrt(mean((x - mean)^2) + eps); with ``rms`` the mean is 0 and there is no
    bias. Returns (Y, stats): fp32 [2, T] (mean, rstd), with ``rms`` [1, T]
    (rstd), for ``norm_bwd``; None without ``stats``."""
    _no_transforms(x, weight, bias)
    dt, device = _norm_args(x, weight, bias, eps, rms)
    return _on(device, _norm_fwd, _flat(x), _flat(weight), _flat(bias), eps, bool(rms), stats, dt, device)


def _norm_bwd(dy, x, weight, st, rms, bias, dt, device, dres=None, workspace=None):
    T, D = x.shape
    dx, dw = torch.empty_like(x), torch.empty_like(weight)
    db = torch.empty_like(weight) if bias else None
    need = _bytes("swiglu_mlp_norm_bwd_workspace_bytes", T, D, rms, dt)
    ws, nbytes, keep = _workspace(workspace, need, device) if need else (None, 0, None)
    rc = _c("norm_bwd")(dy.data_ptr(), x.data_ptr(), weight.data_ptr(), st.data_ptr(), None if dres is None else dres.data_ptr(),
                        dx.data_ptr(), dw.data_ptr(), db.data_ptr() if bias else None, ws, nbytes, T, D, rms, dt,
                        _stream(device))
    if rc:
        _check(rc, "swiglu_mlp_norm_bwd")
    return dx, dw, db


def norm_bwd(dy, x, weight, stats, rms=False, bias=False, dres=None, workspace=None):
    """(dX, dweight, dbias) of ``norm_fwd``; dbias is None unless ``bias``. ``dres``
    [T, D] is added to dX (the gradient that reaches x past the norm)."""
    _no_transforms(dy, x, weight, dres)
    if dy.shape != x.shape or (dres is not None and dres.shape != x.shape):
        raise ValueError("dY and dres must match X in shape")
    _norm_args(x, weight, None, 0.0, rms)
    dt, device = _same(x, dy, dres)
    if tuple(stats.shape) != (1 if rms else 2, x.shape[0]) or stats.dtype != torch.float32 or stats.device != device:
        raise ValueError("stats must be the fp32 tensor returned by norm_fwd")
    if bias and rms:
        raise ValueError("RMS norm has no bias")
    return _on(device, _norm_bwd, _flat(dy), _flat(x), _flat(weight), _flat(stats), bool(rms), bool(bias), dt, device,
               _flat(dres), workspace)


def layer_norm(x, weight, bias=None, eps=1e-5):
    """Layer norm over the last axis of x[..., D]: (x - mean) / sqrt(var + eps) *
    weight + bias."""
    return _nodes().norm(x, weight, bias, eps, False)


def rms_norm(x, weight, eps=1e-6):
    """RMS norm over the last axis of x[..., D]: x / sqrt(mean(x^2) + eps) *
    weight."""
    return _nodes().norm(x, weight, None, eps, True)


# ---- linear layer -------------------------------------------------------------


def _linear_args(x, w, bias, residual):
    """(dtype's code, device), after checking the arguments."""
    shape, (N, K) = x.shape, w.shape if w.dim() == 2 else (None, None)
    if len(shape) != 2 or shape[1] != K:
        raise ValueError(f"shape mismatch (expected X[T,K], W[N,K]): X{tuple(shape)} W{tuple(w.shape)}")
    if bias is not None and bias.shape != (N,):
        raise ValueError(f"bias must be [N] = [{N}]: {tuple(bias.shape)}")
    if residual is not None and residual.shape != (shape[0], N):
        raise ValueError(f"residual must be [T, N] = {[shape[0], N]}: {tuple(residual.shape)}")
    return _same(x, w, bias, residual)


def _linear_fwd(x, w, bias, act, residual, keep, dt, device, workspace=None):
    T, K = x.shape
    N = w.shape[0]
    y = torch.empty((T, N), dtype=x.dtype, device=device)
    z = torch.empty_like(y) if keep and act else None
    need = _bytes("swiglu_mlp_linear_workspace_bytes", T, N, K, dt)
    ws, nbytes, held = _workspace(workspace, need, device) if need else (None, 0, None)
    rc = _c("linear_fwd")(x.data_ptr(), w.data_ptr(), None if bias is None else bias.data_ptr(), _opt(residual), y.data_ptr(),
                          _opt(z), ws, nbytes, T, N, K, act, dt, _stream(device))
    if rc:
        _check(rc, "swiglu_mlp_linear_fwd")
    return y, z


def linear_fwd(x, w, bias=None, activation=None, residual=None, keep=True, workspace=None):
    """Y = act(x W^T + bias) + residual: x[T, K], w[N, K], bias[N], residual[T, N];
    ``activation`` None, "relu", "gelu", "gelu_tanh" or "silu". K and N are
    multiples of 8. Returns (Y, Z): Z[T, N] is the activation's argument in the
    inputs' dtype, for ``linear_bwd``; None without an activation or ``keep``."""
    _no_transforms(x, w, bias, residual)
    act = _act(activation)
    dt, device = _linear_args(x, w, bias, residual)
    return _on(device, _linear_fwd, _flat16(x), _flat16(w), _flat16(bias), act, _flat16(residual), keep, dt, device, workspace)


def _linear_bwd(dy, x, w, z, act, needs, dt, device, workspace=None):
    T, K = x.shape
    N = w.shape[0]
    dx = torch.empty_like(x) if needs[0] else None
    dw = torch.empty_like(w) if needs[1] else None
    db = torch.empty(N, dtype=x.dtype, device=device) if needs[2] else None
    need = _bytes("swiglu_mlp_linear_bwd_workspace_bytes", T, N, K, act, dt)
    ws, nbytes, held = _workspace(workspace, need, device) if need else (None, 0, None)
    rc = _c("linear_bwd")(dy.data_ptr(), x.data_ptr(), w.data_ptr(), z.data_ptr() if act else None, _opt(dx), _opt(dw), _opt(db),
                          ws, nbytes, T, N, K, act, dt, _stream(device))
    if rc:
        _check(rc, "swiglu_mlp_linear_bwd")
    return dx, dw, db


def linear_bwd(dy, x, w, z=None, activation=None, needs=(True, True, True), workspace=None):
    """(dX, dW, dbias) of ``linear_fwd``; ``needs`` says which are wanted, the
    others are None. ``z``: what ``linear_fwd`` kept, where there is an
    activation. The residual's gradient is dY."""
    _no_transforms(dy, x, w)
    act = _act(activation)
    if dy.dim() != 2 or tuple(dy.shape) != (x.shape[0], w.shape[0]):
        raise ValueError(f"dY must be [T, N]: {tuple(dy.shape)}")
    if act and (z is None or z.shape != dy.shape):
        raise ValueError("z must be the [T, N] tensor returned by linear_fwd")
    z = z if act else None
    dt, device = _linear_args(x, w, None, dy)
    _same(x, z)
    return _on(device, _linear_bwd, _flat16(dy), _flat16(x), _flat16(w), _flat16(z), act, needs, dt, device, workspace)


def linear_plan(T, N, K, dtype, dw=False, dx=False):
    """How a linear layer of these sizes runs on the current device, for profiles and
    tests: {"fwd": (engine, parts of K)}, or with ``dw`` or ``dx`` what the backward
    does for them, {"dw": ..., "dx": ..., "together": both in one launch}. Engines are
    "stream" (of the weight), tiles "64x64", "64x128", "128x128", and "ring" (of 256 x
    256 tiles)."""
    if dtype not in _DT:
        raise TypeError(f"unsupported dtype {dtype}; use bfloat16, float16, float32")
    p = _L.LinearPlan()
    _check(_c("linear_plan")(T, N, K, _DT[dtype], dw, dx, ctypes.byref(p)), "swiglu_mlp_linear_plan")
    if not (dw or dx):
        return {"fwd": (_L.ENGINES[p.fwd_engine], p.fwd_parts)}
    plan = {"together": bool(p.together)}
    if dw:
        plan["dw"] = (_L.ENGINES[p.dw_engine], p.dw_parts)
    if dx:
        plan["dx"] = (_L.ENGINES[p.dx_engine], p.dx_parts)
    return plan


def linear(x, w, bias=None, activation=None, residual=None):
    """Y = act(x W^T + bias) + residual for x[..., K]: the product with bias,
    activation and residual in its epilogue. w[N, K] (nn.Linear layout), bias[N],
    residual[..., N] or None; ``activation`` None, "relu", "gelu", "gelu_tanh"
    or "silu"."""
    return _nodes().linear(x, w, bias, residual, _act(activation))


# ---- the layer of them ----------------------------------------------------------


def feed_forward(x, norm_weight, norm_bias, w1, b1, w2, b2, activation="gelu", eps=1e-5, rms=False):
    """Y = x + act(norm(x) w1^T + b1) w2^T + b2 for x[..., D]: the ungated feed-forward
    layer with its norm in front and the stream added. norm_weight[D], w1[H, D],
    w2[D, H]; norm_bias, b1 and b2 or None; ``activation`` as in ``linear``; with
    ``rms`` an RMS norm (no norm_bias)."""
    act = _act(activation)
    if not act:
        raise ValueError(f"a feed-forward layer needs an activation: one of {ACTIVATIONS[1:]}")
    return _nodes().feed_forward(x, norm_weight, norm_bias, w1, b1, w2, b2, act, eps, rms)


_CONFIG_ACTS = {"relu": "relu", "gelu": "gelu", "gelu_new": "gelu_tanh", "gelu_pytorch_tanh": "gelu_tanh",
                "gelu_tanh": "gelu_tanh", "silu": "silu", "swish": "silu"}


_HOOKS = ("_forward_pre_hooks", "_forward_hooks", "_backward_pre_hooks", "_backward_hooks")


def _own(name, layer, *kinds):
    """``layer``, of which only the weights are read: one of torch's ``kinds`` (or a
    parametrized one), as it is. A layer of another kind in its place and hooks on it
    would not run, so they are refused."""
    if not any(type(layer).forward is k.forward for k in kinds) or "forward" in layer.__dict__:
        raise TypeError(f"FeedForward reads the weights of {name} and does not call it: it has to be a "
                        f"{' or '.join('torch.nn.' + k.__name__ for k in kinds)}, got {type(layer).__name__}")
    if any(layer.__dict__[h] for h in _HOOKS):
        raise RuntimeError(f"FeedForward reads the weights of {name} and does not call it: hooks on it would not run "
                           f"(hook the FeedForward itself)")
    return layer


class FeedForward(torch.nn.Module):
    """The ungated feed-forward layer with its norm in front and the stream added:
    y = x + fc2(act(fc1(norm(x)))). ``config`` has hidden_size, intermediate_size
    and optionally hidden_act (default "gelu"), mlp_bias (default true) and the
    norm's epsilon, as layer_norm_eps (default 1e-5) or, for an RMS norm in front,
    rms_norm_eps. Submodules ``norm``, ``fc1`` and ``fc2`` are torch's, whose
    weights the kernels read in place: they are never called, so layers of another kind
    in their place (adapters, quantised ones) and hooks on them are refused;
    parametrizations of their weights work."""

    def __init__(self, config):
        super().__init__()
        act = getattr(config, "hidden_act", "gelu")
        if act not in _CONFIG_ACTS:
            raise ValueError(f"FeedForward has no activation {act!r}; use one of {tuple(_CONFIG_ACTS)}")
        self.activation = _CONFIG_ACTS[act]
        D, H = int(config.hidden_size), int(config.intermediate_size)
        bias = bool(getattr(config, "mlp_bias", True))
        rms = getattr(config, "rms_norm_eps", None)
        if rms is not None:
            self.norm = torch.nn.RMSNorm(D, eps=float(rms))
        else:
            self.norm = torch.nn.LayerNorm(D, eps=float(getattr(config, "layer_norm_eps", 1e-5)))
        self.fc1 = torch.nn.Linear(D, H, bias=bias)
        self.fc2 = torch.nn.Linear(H, D, bias=bias)

    def forward(self, x):
        norm = _own("norm", self.norm, torch.nn.LayerNorm, torch.nn.RMSNorm)
        fc1, fc2 = _own("fc1", self.fc1, torch.nn.Linear), _own("fc2", self.fc2, torch.nn.Linear)
        rms = isinstance(norm, torch.nn.RMSNorm)
        return feed_forward(x, norm.weight, None if rms else norm.bias, fc1.weight, fc1.bias, fc2.weight, fc2.bias,
                            self.activation, norm.eps, rms)

    def extra_repr(self):
        return f"activation={self.activation!r}"
