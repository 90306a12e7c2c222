"""Serving with few tokens: a mixture of SwiGLU experts and 4-bit weights.

Op level, as in the package's other wrappers (every arithmetic step runs in the
HIP kernels behind the C ABI of include/swiglu_mlp.h; no fallback):

* ``moe_route``   top-k experts of each token and their weights
* ``moe_experts`` the chosen experts' SwiGLU blocks, weighted and summed
* ``moe_infer``   both in one call
* ``w4_quantize``, ``w4_pack``, ``W4Weight``  4-bit weights with group scales
* ``w4_linear``   y = x W^T with a 4-bit weight
* ``infer_w4``    the dense SwiGLU block with 4-bit weights

and the modules ``SwiGLUMoE`` and ``SwiGLUMLPW4``. Weights are in the nn.Linear
layout. The operators have no backward: inputs that need gradients are refused
while autograd is on.
"""

import ctypes
import functools

import torch

from . import _lib as _L
from ._lib import SwiGLUError

_DT = {torch.bfloat16: _L.BF16, torch.float16: _L.FP16, torch.float32: _L.FP32}
_DT16 = {torch.bfloat16: _L.BF16, torch.float16: _L.FP16}


def _check(rc, where):
    if rc != 0:
        raise SwiGLUError(rc, where)


# A decoding step is a few calls of about 20 us, so what Python adds to each counts:
# the raw stream costs 0.1 us where a Stream object costs 2, size queries are kept.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(device):
    if _raw_stream is not None:
        return _raw_stream(device.index)
    return torch.cuda.current_stream(device).cuda_stream


def _ptr(t):
    return t.data_ptr() if t.numel() else None


@functools.lru_cache(maxsize=4096)
def _bytes(query, *sizes):
    return getattr(_L.lib(), query)(*sizes)


def _code(t, table=_DT):
    try:
        return table[t.dtype]
    except KeyError:
        names = ", ".join(str(d)[6:] for d in table)
        raise TypeError(f"unsupported dtype {t.dtype}; use {names}") from None


def _no_grad(*tensors):
    if not torch.is_grad_enabled():
        return
    if any(t.requires_grad for t in tensors):
        raise RuntimeError("the few-token serving operators have no backward: call them under torch.no_grad()")


def _on_gpu(x):
    if x.device.type != "cuda":
        raise ValueError("tensors must be on a GPU (cuda/HIP device)")


def _buf(t, shape, dtype, device, name):
    if t is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if t.device != device or t.dtype != dtype or not t.is_contiguous() or tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on {device}")
    return t


def _like(y, x):
    return torch.empty_like(x) if y is None else _buf(y, x.shape, x.dtype, x.device, "y")


def _workspace(ws, need, device):
    """(pointer, bytes, the tensor that holds them)"""
    if ws is None:
        ws = torch.empty(need, dtype=torch.uint8, device=device)
        return ws.data_ptr(), need, ws
    if ws.device != device or not ws.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {device}")
    return ws.data_ptr(), ws.numel() * ws.element_size(), ws


class W4Weight:
    """A weight [N, K], or a stack [E, N, K], in 4 bits with a scale (and a
    zero point) for each ``group`` of K, in the kernels' packed layout.
    ``dtype`` is the type of the scales and of the activations it multiplies.
    Made by ``w4_pack`` or ``W4Weight.quantize``; ``dequantize`` writes it back
    as rows."""

    def __init__(self, data, shape, group, has_zeros, dtype):
        self.data, self.shape, self.group = data, tuple(shape), int(group)
        self.has_zeros, self.dtype = bool(has_zeros), dtype
        self.experts = self.shape[0] if len(self.shape) == 3 else 1
        self.device = data.device
        self._c = _L.W4(data.data_ptr(), self.experts, self.shape[-2], self.shape[-1], self.group, int(self.has_zeros))
        self._ref = ctypes.byref(self._c)

    requires_grad = False

    def __getstate__(self):  # the C structure holds an address: copies and loads make their own
        return self.data, self.shape, self.group, self.has_zeros, self.dtype

    def __setstate__(self, state):
        self.__init__(*state)

    @classmethod
    def quantize(cls, w, group=128, zeros=False):
        """The nearest 4-bit weight of ``w`` under ``w4_quantize``'s rule."""
        return w4_pack(*w4_quantize(w, group, zeros))

    def dequantize(self):
        """The weight as rows in ``dtype``, each value rounded once (for
        prompts long enough that ``infer(..., linear=True)`` is the faster)."""
        w = torch.empty(self.shape, dtype=self.dtype, device=self.device)
        _check(_L.lib().swiglu_mlp_w4_dequantize(self._ref, w.data_ptr(), _DT16[self.dtype], _stream(w.device)),
               "swiglu_mlp_w4_dequantize")
        return w

    def __repr__(self):
        z = ", zeros" if self.has_zeros else ""
        return f"W4Weight({list(self.shape)}, group={self.group}{z}, dtype={self.dtype}, device={self.device})"


def _w4_shape(shape, group):
    if len(shape) not in (2, 3):
        raise ValueError("a 4-bit weight is [N, K] or [E, N, K]")
    *lead, N, K = shape
    if group not in (32, 64, 128) or K <= 0 or K % group or N <= 0 or N % 8:
        raise ValueError(f"4-bit weights need group 32, 64 or 128 dividing K, and N a multiple of 8: "
                         f"got N={N}, K={K}, group={group}")
    return (lead[0] if lead else 1), N, K


def w4_quantize(w, group=128, zeros=False):
    """(codes, scales, zero points or None) of ``w`` [N, K] or [E, N, K]: codes
    [.., N, K/2] uint8, two to a byte (the even k in the low half), scales
    [.., N, K/group] in w's dtype, zero points [.., N, K/group] uint8. Without
    zero points scale = max|w| / 7.5 and code = round(w / scale) + 8, with
    them scale = (max(w, 0) - min(w, 0)) / 15 and code = round(w / scale) +
    round(-min / scale), all clamped to 0..15. A NaN in ``w`` makes its group's
    scale NaN."""
    w = w.detach().contiguous()
    _on_gpu(w)
    dt = _code(w, _DT16)
    E, N, K = _w4_shape(w.shape, group)
    lead, g = w.shape[:-1], (*w.shape[:-1], K // group)
    codes = torch.empty((*lead, K // 2), dtype=torch.uint8, device=w.device)
    scales = torch.empty(g, dtype=w.dtype, device=w.device)
    zp = torch.empty(g, dtype=torch.uint8, device=w.device) if zeros else None
    rc = _L.lib().swiglu_mlp_w4_quantize(w.data_ptr(), codes.data_ptr(), scales.data_ptr(),
                                         zp.data_ptr() if zeros else None, E, N, K, group, dt, _stream(w.device))
    _check(rc, "swiglu_mlp_w4_quantize")
    return codes, scales, zp


def w4_pack(codes, scales, zeros=None):
    """The ``W4Weight`` of codes, scales and zero points laid out as
    ``w4_quantize`` returns them (any quantiser's, with codes and zero points
    0..15). W = scale * (code - zero), zero = 8 where ``zeros`` is None."""
    codes, scales = codes.contiguous(), scales.contiguous()
    _on_gpu(codes)
    _code(scales, _DT16)
    if codes.dtype != torch.uint8 or codes.dim() not in (2, 3) or scales.dim() != codes.dim():
        raise ValueError("codes must be uint8 [.., N, K/2] and scales [.., N, K/group]")
    K = 2 * codes.shape[-1]
    if scales.shape[:-1] != codes.shape[:-1] or scales.shape[-1] == 0 or K % scales.shape[-1]:
        raise ValueError(f"scales {tuple(scales.shape)} do not divide codes {tuple(codes.shape)} into groups")
    group = K // scales.shape[-1]
    shape = (*codes.shape[:-1], K)
    E, N, K = _w4_shape(shape, group)
    if scales.device != codes.device:
        raise ValueError("all tensors must be on one device")
    if zeros is not None:
        zeros = zeros.contiguous()
        if zeros.dtype != torch.uint8 or zeros.shape != scales.shape or zeros.device != codes.device:
            raise ValueError("zeros must be uint8, shaped like scales, on the same device")
    L = _L.lib()
    data = torch.empty(L.swiglu_mlp_w4_bytes(E, N, K, group, zeros is not None), dtype=torch.uint8, device=codes.device)
    rc = L.swiglu_mlp_w4_pack(codes.data_ptr(), scales.data_ptr(), zeros.data_ptr() if zeros is not None else None,
                              data.data_ptr(), E, N, K, group, _stream(codes.device))
    _check(rc, "swiglu_mlp_w4_pack")
    return W4Weight(data, shape, group, zeros is not None, scales.dtype)


def moe_route(x, w_router, top_k, renormalize=True, weights=None, ids=None, workspace=None):
    """The router: (weights [T, k] fp32, ids [T, k] int32) of the ``top_k``
    largest logits of x[T, D] w_router[E, D]^T per token, in descending order
    (equal logits: the lower index first). Weights are the softmax over all
    experts, divided by the chosen ones' sum with ``renormalize``."""
    _no_grad(x, w_router)
    x, w_router = x.contiguous(), w_router.contiguous()
    T, D, E = _router_shapes(x, w_router, top_k)
    weights = _buf(weights, (T, top_k), torch.float32, x.device, "weights")
    ids = _buf(ids, (T, top_k), torch.int32, x.device, "ids")
    dt, L = _code(x), _L.lib()
    need = _bytes("swiglu_mlp_moe_route_workspace_bytes", T, D, E, dt)
    ws, nbytes, keep = _workspace(workspace, need, x.device)
    rc = L.swiglu_mlp_moe_route(_ptr(x), w_router.data_ptr(), _ptr(weights), _ptr(ids), ws, nbytes, T, D, E, top_k,
                                bool(renormalize), dt, _stream(x.device))
    _check(rc, "swiglu_mlp_moe_route")
    return weights, ids


def _router_shapes(x, w_router, top_k):
    if x.dim() != 2 or w_router.dim() != 2 or x.shape[1] != w_router.shape[1]:
        raise ValueError(f"expected X[T,D] and a router weight [E,D]: {tuple(x.shape)}, {tuple(w_router.shape)}")
    if w_router.dtype != x.dtype or w_router.device != x.device:
        raise ValueError("all tensors must share dtype and device")
    _on_gpu(x)
    E = w_router.shape[0]
    if not 1 <= top_k <= min(E, 32):
        raise ValueError(f"top_k must be between 1 and min(E, 32): got {top_k} of {E}")
    return x.shape[0], x.shape[1], E


def _expert_shapes(x, wg, wu, wd):
    """(E, H, 4-bit?) after checking the experts' weights against x."""
    w4 = isinstance(wg, W4Weight)
    if isinstance(wu, W4Weight) != w4 or isinstance(wd, W4Weight) != w4:
        raise TypeError("the experts' weights must be all tensors or all W4Weight")
    if x.dim() != 2 or len(wg.shape) != 3:
        raise ValueError("expected X[T,D] and weights [E,H,D], [E,H,D], [E,D,H]")
    E, H, D = wg.shape
    if x.shape[1] != D or wu.shape != wg.shape or wd.shape != (E, D, H):
        raise ValueError(f"shape mismatch (expected Wg[E,H,D], Wu[E,H,D], Wd[E,D,H]): X{tuple(x.shape)} "
                         f"Wg{tuple(wg.shape)} Wu{tuple(wu.shape)} Wd{tuple(wd.shape)}")
    dtype, device = x.dtype, x.device
    if not (wg.dtype == wu.dtype == wd.dtype == dtype and wg.device == wu.device == wd.device == device):
        raise ValueError("all tensors must share dtype and device")
    if w4:
        _same_form(wg, wu, wd)
    _on_gpu(x)
    return E, H, w4


def _same_form(wg, wu, wd):
    if not (wg.group, wg.has_zeros) == (wu.group, wu.has_zeros) == (wd.group, wd.has_zeros):
        raise ValueError("the three weights must share their group size and have zero points all or none")


def moe_experts(x, weights, ids, wg, wu, wd, y=None, workspace=None):
    """Y[t] = sum over j of weights[t, j] * SwiGLU block of expert ids[t, j] on
    x[t]. x [T, D]; weights fp32 and ids int32 [T, k]; wg, wu [E, H, D] and wd
    [E, D, H], tensors of x's dtype or three ``W4Weight``. An id outside
    [0, E) chooses nothing (dropped tokens, experts of another device)."""
    _no_grad(x, weights, *(() if isinstance(wg, W4Weight) else (wg, wu, wd)))
    x, weights, ids = x.contiguous(), weights.contiguous(), ids.contiguous()
    E, H, w4 = _expert_shapes(x, wg, wu, wd)
    T, D = x.shape
    if (ids.dim() != 2 or ids.shape[0] != T or ids.dtype != torch.int32 or weights.shape != ids.shape
            or weights.dtype != torch.float32 or ids.device != x.device or weights.device != x.device):
        raise ValueError("weights must be fp32 and ids int32, both [T, k] on x's device")
    k, dt, L = ids.shape[1], _code(x), _L.lib()
    y = _like(y, x)
    need = _bytes("swiglu_mlp_moe_workspace_bytes", T, D, H, E, k, dt)
    ws, nbytes, keep = _workspace(workspace, need, x.device)
    if w4:
        rc = L.swiglu_mlp_moe_experts_w4(_ptr(x), _ptr(weights), _ptr(ids), wg._ref, wu._ref, wd._ref, _ptr(y),
                                         ws, nbytes, T, k, dt, _stream(x.device))
    else:
        wg, wu, wd = wg.contiguous(), wu.contiguous(), wd.contiguous()
        rc = L.swiglu_mlp_moe_experts(_ptr(x), _ptr(weights), _ptr(ids), wg.data_ptr(), wu.data_ptr(), wd.data_ptr(),
                                      _ptr(y), ws, nbytes, T, D, H, E, k, dt, _stream(x.device))
    _check(rc, "swiglu_mlp_moe_experts")
    return y


def moe_infer(x, w_router, wg, wu, wd, top_k, renormalize=True, y=None, workspace=None):
    """A whole mixture-of-experts layer: ``moe_route`` then ``moe_experts``,
    four launches in one call. x [T, D], w_router [E, D]; wg, wu [E, H, D] and
    wd [E, D, H], tensors of x's dtype or three ``W4Weight``."""
    _no_grad(x, w_router, *(() if isinstance(wg, W4Weight) else (wg, wu, wd)))
    x, w_router = x.contiguous(), w_router.contiguous()
    T, D, E = _router_shapes(x, w_router, top_k)
    E2, H, w4 = _expert_shapes(x, wg, wu, wd)
    if E2 != E:
        raise ValueError(f"the router has {E} experts, the weights {E2}")
    dt, L = _code(x), _L.lib()
    y = _like(y, x)
    need = _bytes("swiglu_mlp_moe_workspace_bytes", T, D, H, E, top_k, dt)
    ws, nbytes, keep = _workspace(workspace, need, x.device)
    if w4:
        rc = L.swiglu_mlp_moe_infer_w4(_ptr(x), w_router.data_ptr(), wg._ref, wu._ref, wd._ref, _ptr(y), ws,
                                       nbytes, T, top_k, bool(renormalize), dt, _stream(x.device))
    else:
        wg, wu, wd = wg.contiguous(), wu.contiguous(), wd.contiguous()
        rc = L.swiglu_mlp_moe_infer(_ptr(x), w_router.data_ptr(), wg.data_ptr(), wu.data_ptr(), wd.data_ptr(), _ptr(y),
                                    ws, nbytes, T, D, H, E, top_k, bool(renormalize), dt, _stream(x.device))
    _check(rc, "swiglu_mlp_moe_infer")
    return y


def w4_linear(x, w, y=None, workspace=None):
    """Y[T, N] = x[T, K] W^T with a 4-bit weight [N, K]."""
    _no_grad(x)
    x = x.contiguous()
    if x.dim() != 2 or len(w.shape) != 2 or x.shape[1] != w.shape[1]:
        raise ValueError(f"shape mismatch (expected X[T,K], W[N,K]): X{tuple(x.shape)} W{tuple(w.shape)}")
    if w.dtype != x.dtype or w.device != x.device:
        raise ValueError("all tensors must share dtype and device")
    _on_gpu(x)
    T, (N, K), dt = x.shape[0], w.shape, _DT16[x.dtype]
    y = _buf(y, (T, N), x.dtype, x.device, "y")
    need = _bytes("swiglu_mlp_w4_linear_workspace_bytes", T, N, K, dt)
    ws, nbytes, keep = _workspace(workspace, need, x.device) if need else (None, 0, None)
    _check(_L.lib().swiglu_mlp_w4_linear(_ptr(x), w._ref, _ptr(y), ws, nbytes, T, dt, _stream(x.device)),
           "swiglu_mlp_w4_linear")
    return y


def infer_w4(x, wg, wu, wd, y=None, workspace=None):
    """The no-grad SwiGLU block Y = (SiLU(x Wg^T) * (x Wu^T)) Wd^T with 4-bit
    weights wg, wu [H, D] and wd [D, H]; two launches."""
    _no_grad(x)
    x = x.contiguous()
    if x.dim() != 2 or len(wg.shape) != 2:
        raise ValueError("expected X[T,D] and weights [H,D], [H,D], [D,H]")
    T, D = x.shape
    H = wg.shape[0]
    if tuple(wg.shape) != (H, D) or tuple(wu.shape) != (H, D) or tuple(wd.shape) != (D, H):
        raise ValueError(f"shape mismatch (expected Wg[H,D], Wu[H,D], Wd[D,H]): X{tuple(x.shape)} "
                         f"Wg{tuple(wg.shape)} Wu{tuple(wu.shape)} Wd{tuple(wd.shape)}")
    for t in (wg, wu, wd):
        if t.dtype != x.dtype or t.device != x.device:
            raise ValueError("all tensors must share dtype and device")
    _same_form(wg, wu, wd)
    _on_gpu(x)
    dt, L = _DT16[x.dtype], _L.lib()
    y = _like(y, x)
    need = _bytes("swiglu_mlp_w4_infer_workspace_bytes", T, D, H, dt)
    ws, nbytes, keep = _workspace(workspace, need, x.device)
    rc = L.swiglu_mlp_w4_infer(_ptr(x), wg._ref, wu._ref, wd._ref, _ptr(y), ws, nbytes, T, dt, _stream(x.device))
    _check(rc, "swiglu_mlp_w4_infer")
    return y


class _W4Module(torch.nn.Module):
    """Keeps 4-bit weights as byte buffers, so that they follow the module to
    another device and into its state dict, and hands them out as W4Weight. Their
    form (shape, group, zero points, type) stands in the state dict's metadata, and a
    module that loads it takes that form, whatever it held before; a state dict
    without metadata has to be of the module's own form."""

    def _keep(self, name, w):
        if name in self._parameters:
            del self._parameters[name]
        self.register_buffer(name, w.data)
        self._forms[name] = w

    def _save_to_state_dict(self, destination, prefix, keep_vars):
        super()._save_to_state_dict(destination, prefix, keep_vars)
        if self._forms and hasattr(destination, "_metadata"):
            destination._metadata[prefix[:-1]]["w4"] = {n: (w.shape, w.group, w.has_zeros, w.dtype)
                                                        for n, w in self._forms.items()}

    def _load_from_state_dict(self, state_dict, prefix, local_metadata, strict, missing_keys, unexpected_keys, error_msgs):
        forms = {n: f for n, f in (local_metadata.get("w4") or {}).items() if prefix + n in state_dict and hasattr(self, n)}
        for name, (shape, group, zeros, _) in forms.items():
            data, mine = state_dict[prefix + name], self._forms.get(name, getattr(self, name))
            if tuple(mine.shape) != shape or data.numel() != _L.lib().swiglu_mlp_w4_bytes(*_w4_shape(shape, group), group, zeros):
                error_msgs.append(f"4-bit weight {prefix + name} {list(shape)} of {data.numel()} bytes does not fit the "
                                  f"module's {list(mine.shape)}")
                return
        for name, (shape, group, zeros, dtype) in forms.items():
            room = torch.empty(state_dict[prefix + name].numel(), dtype=torch.uint8, device=getattr(self, name).device)
            self._keep(name, W4Weight(room, shape, group, zeros, dtype))
        super()._load_from_state_dict(state_dict, prefix, local_metadata, strict, missing_keys, unexpected_keys, error_msgs)

    def _weight(self, name):
        data, w = self._buffers[name], self._forms[name]
        if data.data_ptr() != w._c.data:
            w = self._forms[name] = W4Weight(data, w.shape, w.group, w.has_zeros, w.dtype)
        return w

    def _apply(self, fn, recurse=True):
        super()._apply(fn, recurse)
        for name in self._forms:  # a move: the old buffers go
            self._weight(name)
        return self


class SwiGLUMLPW4(_W4Module):
    """The dense SwiGLU block with 4-bit weights, made from a ``SwiGLUMLP`` (or any
    module with gate_proj, up_proj and down_proj layers without bias). No gradients. Above
    ``long_tokens`` tokens the weights are written back to rows and the no-grad
    path of 16-bit weights runs, which is bound by arithmetic then (D = 4096, H = 11008,
    4 bits against rows: 512 tokens 248 and 462 us, 768 400 and 459, 1024 475 and 479;
    D = 2048, H = 5632: 512 tokens 94 and 136, 1024 148 and 168)."""

    def __init__(self, mlp, group=128, zeros=False, long_tokens=1024):
        super().__init__()
        self._forms, self.long_tokens = {}, long_tokens
        layers = {name: getattr(mlp, name) for name in ("gate_proj", "up_proj", "down_proj")}
        if any(getattr(layer, "bias", None) is not None for layer in layers.values()):
            raise ValueError("SwiGLUMLPW4 has no bias terms")
        for name, layer in layers.items():
            self._keep(name, W4Weight.quantize(layer.weight, group, zeros))

    def forward(self, x):
        w = [self._weight(n) for n in ("gate_proj", "up_proj", "down_proj")]
        x2 = x.reshape(-1, x.shape[-1])
        if x2.shape[0] > self.long_tokens:
            from . import infer

            _no_grad(x)
            return infer(x2, *(t.dequantize() for t in w), linear=True).reshape(x.shape)
        return infer_w4(x2, *w).reshape(x.shape)


class SwiGLUMoE(_W4Module):
    """A mixture of SwiGLU experts for inference: ``gate`` (nn.Linear, hidden_size
    -> num_experts, no bias) and the experts' stacked weights ``gate_proj``,
    ``up_proj`` [E, H, D] and ``down_proj`` [E, D, H]. ``config`` has hidden_size,
    moe_intermediate_size (or intermediate_size), num_experts (or
    num_local_experts), num_experts_per_tok and optionally norm_topk_prob (default
    true). ``from_experts`` stacks existing blocks, ``quantize_`` puts the experts
    into 4 bits."""

    def __init__(self, config):
        super().__init__()
        pick = lambda *names: next(int(getattr(config, n)) for n in names if getattr(config, n, None) is not None)  # noqa: E731
        act = getattr(config, "hidden_act", "silu")
        if act not in ("silu", "swish"):
            raise ValueError(f"SwiGLUMoE computes SiLU gating; config.hidden_act is {act!r}")
        D, H = pick("hidden_size"), pick("moe_intermediate_size", "intermediate_size")
        E, self.top_k = pick("num_experts", "num_local_experts"), pick("num_experts_per_tok")
        self.renormalize = bool(getattr(config, "norm_topk_prob", True))
        self._forms = {}
        self.gate = torch.nn.Linear(D, E, bias=False)
        par = lambda *shape: torch.nn.Parameter(torch.randn(shape) / shape[-1] ** 0.5)  # noqa: E731
        self.gate_proj, self.up_proj, self.down_proj = par(E, H, D), par(E, H, D), par(E, D, H)

    @classmethod
    def from_experts(cls, gate, experts, top_k, renormalize=True):
        """From a router nn.Linear and a list of blocks with gate_proj, up_proj
        and down_proj layers (no bias)."""
        m = cls.__new__(cls)
        torch.nn.Module.__init__(m)
        m._forms, m.top_k, m.renormalize, m.gate = {}, int(top_k), bool(renormalize), gate
        if gate.bias is not None:
            raise ValueError("the router has no bias term")
        for name in ("gate_proj", "up_proj", "down_proj"):
            layers = [getattr(e, name) for e in experts]
            if any(layer.bias is not None for layer in layers):
                raise ValueError("SwiGLUMoE has no bias terms")
            setattr(m, name, torch.nn.Parameter(torch.stack([layer.weight.detach() for layer in layers])))
        if gate.weight.shape != (len(experts), m.gate_proj.shape[2]):
            raise ValueError("the router must map hidden_size to the number of experts")
        return m

    def quantize_(self, group=128, zeros=False):
        """Replaces the experts' weights by 4-bit ones (in place; not undone)."""
        if self._forms:
            raise RuntimeError("the experts' weights are in 4 bits already")
        names = ("gate_proj", "up_proj", "down_proj")
        for name, w in zip(names, [W4Weight.quantize(getattr(self, n), group, zeros) for n in names]):
            self._keep(name, w)
        return self

    def forward(self, x):
        if self._forms:
            w = [self._weight(n) for n in ("gate_proj", "up_proj", "down_proj")]
        else:
            w = [self.gate_proj, self.up_proj, self.down_proj]
        x2 = x.reshape(-1, x.shape[-1])
        return moe_infer(x2, self.gate.weight, *w, self.top_k, self.renormalize).reshape(x.shape)
