"""Norms and the linear layer with an epilogue, forward and backward.

What stands before and beside the SwiGLU block in the same models. Op level, as in
the package's other wrappers (every arithmetic step runs in the HIP kernels
behind the C ABI of include/swiglu_mlp.h; no fallback):

* ``norm_fwd``, ``norm_bwd``      layer norm and RMS norm over the last axis
* ``linear_fwd``, ``linear_bwd``  y = act(x W^T + b) + residual

with autograd: ``layer_norm``, ``rms_norm``, ``linear`` and, of all three, the
ungated feed-forward layer x + fc2(act(fc1(norm(x)))): ``feed_forward`` and the
module ``FeedForward``.
All tensors of a call share dtype (bf16, fp16 or fp32) and device.

Second derivatives are refused. The backward may run more than once
(``retain_graph``): it changes nothing that the forward kept.
"""

import functools
import math

import torch

from . import _lib as _L
from .serve import _DT, _bytes, _check, _code, _on_gpu, _ptr, _stream, _workspace

ACTIVATIONS = tuple(_L.ACTS)

# A small training step is bound by the host: an autograd engine's thread runs the
# backward on a core whose caches are cold, where every Python call counts double.
# So arguments are checked once, in the forward; what the backward gets from
# autograd (shape, dtype, device) the engine has checked.


@functools.lru_cache(maxsize=None)
def _c(name):
    return getattr(_L.lib(), "swiglu_mlp_" + name)


_device = torch._C._cuda_getDevice if hasattr(torch._C, "_cuda_getDevice") else torch.cuda.current_device


def _on(fn):
    """The library launches on the current device: makes it that of the first
    tensor."""

    @functools.wraps(fn)
    def call(x, *args, **kw):
        device = x.device
        if device.type != "cuda" or device.index == _device():  # (other tensors are refused further in)
            return fn(x, *args, **kw)
        with torch.cuda.device(device):
            return fn(x, *args, **kw)

    return call


def _act(activation):
    try:
        return _L.ACTS[activation]
    except (KeyError, TypeError):
        raise ValueError(f"unknown activation {activation!r}; use one of {ACTIVATIONS}") from None


def _same(x, *others):
    for t in others:
        if t is not None and (t.dtype != x.dtype or t.device != x.device):
            raise ValueError("all tensors must share dtype and device")
    _on_gpu(x)


def _opt(t):
    return None if t is None else _ptr(t)


def _flat(t):
    return t if t is None or t.is_contiguous() else t.contiguous()


def _flat16(t):
    """Contiguous and at an address that the matrix kernels take (a gradient may
    be a view that starts anywhere)."""
    if t is None:
        return t
    if not t.is_contiguous():
        t = t.contiguous()
    return t.clone() if t.data_ptr() & 15 else t


# ---- norms ------------------------------------------------------------------


def _norm_shapes(x, weight, bias, eps, rms):
    if x.dim() != 2 or weight.dim() != 1 or weight.shape[0] != x.shape[1] or x.shape[1] == 0:
        raise ValueError(f"expected X[T,D] and weight[D]: X{tuple(x.shape)} weight{tuple(weight.shape)}")
    if bias is not None and (rms or bias.shape != weight.shape):
        raise ValueError("RMS norm has no bias" if rms else f"bias must be [D]: {tuple(bias.shape)}")
    if not 0 <= eps < math.inf:
        raise ValueError(f"eps must be a number from 0 up: got {eps}")
    _same(x, weight, bias)


@_on
def norm_fwd(x, weight, bias=None, eps=1e-5, rms=False, stats=True):
    """Y = (x - mean) rstd weight + bias over the last axis of x[T, D], rstd = 1 /
    sqrt(mean((x - mean)^2) + eps); with ``rms`` the mean is 0 and there is no
    bias. Returns (Y, stats): fp32 [2, T] (mean, rstd), with ``rms`` [1, T]
    (rstd), for ``norm_bwd``; None without ``stats``."""
    _norm_shapes(x, weight, bias, eps, rms)
    x, weight, bias = _flat(x), _flat(weight), _flat(bias)
    T, D = x.shape
    y = torch.empty_like(x)
    st = torch.empty((1 if rms else 2, T), dtype=torch.float32, device=x.device) if stats else None
    rc = _c("norm_fwd")(_ptr(x), weight.data_ptr(), _opt(bias), _ptr(y), _opt(st), T, D, eps, rms, _code(x), _stream(x.device))
    _check(rc, "swiglu_mlp_norm_fwd")
    return y, st


def _norm_bwd(dy, x, weight, st, rms, bias, dres=None, workspace=None):
    T, D = x.shape
    dt, device = _DT[x.dtype], x.device
    dx, dw = torch.empty_like(x), torch.empty_like(weight)
    db = torch.empty_like(weight) if bias else None
    need = _bytes("swiglu_mlp_norm_bwd_workspace_bytes", T, D, rms, dt)
    ws, nbytes, keep = _workspace(workspace, need, device) if need else (None, 0, None)
    rc = _c("norm_bwd")(_ptr(dy), _ptr(x), weight.data_ptr(), _ptr(st), _opt(dres), _ptr(dx), dw.data_ptr(),
                        db.data_ptr() if bias else None, ws, nbytes, T, D, rms, dt, _stream(device))
    _check(rc, "swiglu_mlp_norm_bwd")
    return dx, dw, db


@_on
def norm_bwd(dy, x, weight, stats, rms=False, bias=False, dres=None, workspace=None):
    """(dX, dweight, dbias) of ``norm_fwd``; dbias is None unless ``bias``. ``dres``
    [T, D] is added to dX (the gradient that reaches x past the norm)."""
    if dy.shape != x.shape or (dres is not None and dres.shape != x.shape):
        raise ValueError("dY and dres must match X in shape")
    _norm_shapes(x, weight, None, 0.0, rms)
    _same(x, dy, dres)
    _code(x)
    if tuple(stats.shape) != (1 if rms else 2, x.shape[0]) or stats.dtype != torch.float32 or stats.device != x.device:
        raise ValueError("stats must be the fp32 tensor returned by norm_fwd")
    if bias and rms:
        raise ValueError("RMS norm has no bias")
    return _norm_bwd(_flat(dy), _flat(x), _flat(weight), _flat(stats), bool(rms), bool(bias), _flat(dres), workspace)


def _no_second():
    if torch.is_grad_enabled():
        raise RuntimeError("create_graph=True (double backward) is not supported")


class NormFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, eps, rms):
        x, weight = _flat(x), _flat(weight)
        y, stats = norm_fwd(x, weight, bias, eps, rms)
        ctx.save_for_backward(x, weight, stats)
        ctx.form = rms, bias is not None
        return y

    @staticmethod
    def backward(ctx, dy):
        _no_second()
        x, weight, stats = ctx.saved_tensors
        dx, dw, db = _norm_bwd(_flat(dy), x, weight, stats, *ctx.form)
        return dx, dw, db, None, None


def _norm(x, weight, bias, eps, rms):
    if x.dim() == 0:
        raise ValueError("expected X[..., D]")
    x2 = x if x.dim() == 2 else x.reshape(-1, x.shape[-1])
    if torch.is_grad_enabled() and (x.requires_grad or weight.requires_grad or (bias is not None and bias.requires_grad)):
        y = NormFunction.apply(x2, weight, bias, eps, rms)
    else:
        y = norm_fwd(x2, weight, bias, eps, rms, False)[0]
    return y if x.dim() == 2 else y.reshape(x.shape)


def layer_norm(x, weight, bias=None, eps=1e-5):
    """Layer norm over the last axis of x[..., D]: (x - mean) / sqrt(var + eps) *
    weight + bias."""
    return _norm(x, weight, bias, eps, False)


def rms_norm(x, weight, eps=1e-6):
    """RMS norm over the last axis of x[..., D]: x / sqrt(mean(x^2) + eps) *
    weight."""
    return _norm(x, weight, None, eps, True)


# ---- linear layer -------------------------------------------------------------


def _linear_shapes(x, w, bias, residual):
    if x.dim() != 2 or w.dim() != 2 or x.shape[1] != w.shape[1]:
        raise ValueError(f"shape mismatch (expected X[T,K], W[N,K]): X{tuple(x.shape)} W{tuple(w.shape)}")
    T, (N, K) = x.shape[0], w.shape
    if bias is not None and bias.shape != (N,):
        raise ValueError(f"bias must be [N] = [{N}]: {tuple(bias.shape)}")
    if residual is not None and residual.shape != (T, N):
        raise ValueError(f"residual must be [T, N] = {[T, N]}: {tuple(residual.shape)}")
    _same(x, w, bias, residual)
    return T, N, K


@_on
def linear_fwd(x, w, bias=None, activation=None, residual=None, keep=True, workspace=None):
    """Y = act(x W^T + bias) + residual: x[T, K], w[N, K], bias[N], residual[T, N];
    ``activation`` None, "relu", "gelu", "gelu_tanh" or "silu". K and N are
    multiples of 8. Returns (Y, Z): Z[T, N] is the activation's argument in the
    inputs' dtype, for ``linear_bwd``; None without an activation or ``keep``."""
    act = _act(activation)
    T, N, K = _linear_shapes(x, w, bias, residual)
    x, w, bias, residual = _flat16(x), _flat16(w), _flat16(bias), _flat16(residual)
    dt, device = _code(x), x.device
    y = torch.empty((T, N), dtype=x.dtype, device=device)
    z = torch.empty_like(y) if keep and act else None
    need = _bytes("swiglu_mlp_linear_workspace_bytes", T, N, K, dt)
    ws, nbytes, held = _workspace(workspace, need, device) if need else (None, 0, None)
    rc = _c("linear_fwd")(_ptr(x), _ptr(w), _opt(bias), _opt(residual), _ptr(y), _opt(z), ws, nbytes, T, N, K, act, dt,
                          _stream(device))
    _check(rc, "swiglu_mlp_linear_fwd")
    return y, z


def _linear_bwd(dy, x, w, z, act, needs, workspace=None):
    T, K = x.shape
    N = w.shape[0]
    dt, device = _DT[x.dtype], x.device
    dx = torch.empty_like(x) if needs[0] else None
    dw = torch.empty_like(w) if needs[1] else None
    db = torch.empty(N, dtype=x.dtype, device=device) if needs[2] else None
    need = _bytes("swiglu_mlp_linear_bwd_workspace_bytes", T, N, K, act, dt)
    ws, nbytes, held = _workspace(workspace, need, device) if need else (None, 0, None)
    rc = _c("linear_bwd")(_ptr(dy), _ptr(x), w.data_ptr(), _opt(z), _opt(dx), _opt(dw), _opt(db), ws, nbytes, T, N, K, act, dt,
                          _stream(device))
    _check(rc, "swiglu_mlp_linear_bwd")
    return dx, dw, db


@_on
def linear_bwd(dy, x, w, z=None, activation=None, needs=(True, True, True), workspace=None):
    """(dX, dW, dbias) of ``linear_fwd``; ``needs`` says which are wanted, the
    others are None. ``z``: what ``linear_fwd`` kept, where there is an
    activation. The residual's gradient is dY."""
    act = _act(activation)
    if dy.dim() != 2 or tuple(dy.shape) != (x.shape[0], w.shape[0]):
        raise ValueError(f"dY must be [T, N]: {tuple(dy.shape)}")
    if act and (z is None or z.shape != dy.shape):
        raise ValueError("z must be the [T, N] tensor returned by linear_fwd")
    z = z if act else None
    _linear_shapes(x, w, None, dy)
    _same(x, z)
    _code(x)
    return _linear_bwd(_flat16(dy), _flat16(x), _flat16(w), _flat16(z), act, needs, workspace)


class LinearFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, bias, residual, activation):
        x, w = _flat16(x), _flat16(w)
        y, z = linear_fwd(x, w, bias, activation, residual)
        ctx.save_for_backward(x, w, z)
        ctx.act = _L.ACTS[activation]
        return y

    @staticmethod
    def backward(ctx, dy):
        _no_second()
        x, w, z = ctx.saved_tensors
        needs = ctx.needs_input_grad
        dx = dw = db = None
        if needs[0] or needs[1] or needs[2]:
            dx, dw, db = _linear_bwd(_flat16(dy), x, w, z, ctx.act, needs)
        return dx, dw, db, dy if needs[3] else None, None


def linear(x, w, bias=None, activation=None, residual=None):
    """Y = act(x W^T + bias) + residual for x[..., K]: the product with bias,
    activation and residual in its epilogue. w[N, K] (nn.Linear layout), bias[N],
    residual[..., N] or None; ``activation`` None, "relu", "gelu", "gelu_tanh"
    or "silu"."""
    if x.dim() == 0 or w.dim() != 2:
        raise ValueError("expected X[..., K] and W[N, K]")
    shape = (*x.shape[:-1], w.shape[0])
    if residual is not None and residual.shape != shape:
        raise ValueError(f"residual must be {list(shape)}: {tuple(residual.shape)}")
    if len(shape) != 2:
        x = x.reshape(-1, x.shape[-1])
        residual = None if residual is None else residual.reshape(-1, shape[-1])
    if torch.is_grad_enabled() and (x.requires_grad or w.requires_grad or (bias is not None and bias.requires_grad)
                                    or (residual is not None and residual.requires_grad)):
        y = LinearFunction.apply(x, w, bias, residual, activation)
    else:
        y = linear_fwd(x, w, bias, activation, residual, False)[0]
    return y if len(shape) == 2 else y.reshape(shape)


# ---- the layer of them ----------------------------------------------------------


class FeedForwardFunction(torch.autograd.Function):
    """The layer as one node: its backward hands the stream's gradient to the norm's
    backward, which adds it to its own, instead of leaving a sum of two tensors."""

    @staticmethod
    def forward(ctx, x, nw, nb, w1, b1, w2, b2, activation, eps, rms):
        x, nw, w1, w2 = _flat16(x), _flat(nw), _flat16(w1), _flat16(w2)
        n, stats = norm_fwd(x, nw, nb, eps, rms)
        a, z = linear_fwd(n, w1, b1, activation)
        y = linear_fwd(a, w2, b2, None, x)[0]
        ctx.save_for_backward(x, nw, w1, w2, n, stats, a, z)
        ctx.form = _L.ACTS[activation], rms, nb is not None
        return y

    @staticmethod
    def backward(ctx, dy):
        _no_second()
        x, nw, w1, w2, n, stats, a, z = ctx.saved_tensors
        act, rms, norm_bias = ctx.form
        need = ctx.needs_input_grad
        dy = _flat16(dy)
        norm = need[0] or need[1] or need[2]
        inner = norm or need[3] or need[4]
        da, dw2, db2 = _linear_bwd(dy, a, w2, None, 0, (inner, need[5], need[6]))
        dx = dnw = dnb = dw1 = db1 = None
        if inner:
            dn, dw1, db1 = _linear_bwd(da, n, w1, z, act, (norm, need[3], need[4]))
            del da
            if norm:
                dx, dnw, dnb = _norm_bwd(dn, x, nw, stats, rms, norm_bias, dy)
        return dx, dnw, dnb, dw1, db1, dw2, db2, None, None, None


def feed_forward(x, norm_weight, norm_bias, w1, b1, w2, b2, activation="gelu", eps=1e-5, rms=False):
    """Y = x + act(norm(x) w1^T + b1) w2^T + b2 for x[..., D]: the ungated feed-forward
    layer with its norm in front and the stream added. norm_weight[D], w1[H, D],
    w2[D, H]; norm_bias, b1 and b2 or None; ``activation`` as in ``linear``; with
    ``rms`` an RMS norm (no norm_bias)."""
    if x.dim() == 0:
        raise ValueError("expected X[..., D]")
    if not activation:
        raise ValueError(f"a feed-forward layer needs an activation: one of {ACTIVATIONS[1:]}")
    x2 = x if x.dim() == 2 else x.reshape(-1, x.shape[-1])
    if torch.is_grad_enabled() and any(t is not None and t.requires_grad
                                       for t in (x, norm_weight, norm_bias, w1, b1, w2, b2)):
        y = FeedForwardFunction.apply(x2, norm_weight, norm_bias, w1, b1, w2, b2, activation, eps, rms)
    else:
        n = norm_fwd(x2, norm_weight, norm_bias, eps, rms, False)[0]
        a = linear_fwd(n, w1, b1, activation, None, False)[0]
        y = linear_fwd(a, w2, b2, None, x2, False)[0]
    return y if x.dim() == 2 else y.reshape(x.shape)


_CONFIG_ACTS = {"relu": "relu", "gelu": "gelu", "gelu_new": "gelu_tanh", "gelu_pytorch_tanh": "gelu_tanh",
                "gelu_tanh": "gelu_tanh", "silu": "silu", "swish": "silu"}


class FeedForward(torch.nn.Module):
    """The ungated feed-forward layer with its norm in front and the stream added:
    y = x + fc2(act(fc1(norm(x)))). ``config`` has hidden_size, intermediate_size
    and optionally hidden_act (default "gelu"), mlp_bias (default true) and the
    norm's epsilon, as layer_norm_eps (default 1e-5) or, for an RMS norm in front,
    rms_norm_eps. Submodules ``norm``, ``fc1`` and ``fc2`` are torch's, whose
    weights the kernels read in place."""

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
        rms = isinstance(self.norm, torch.nn.RMSNorm)
        return feed_forward(x, self.norm.weight, None if rms else self.norm.bias, self.fc1.weight, self.fc1.bias,
                            self.fc2.weight, self.fc2.bias, self.activation, self.norm.eps, rms)

    def extra_repr(self):
        return f"activation={self.activation!r}"
