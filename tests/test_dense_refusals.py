"""What the operators keep between calls, and what they refuse rather than leave out
without a word (CPU where a refusal comes first, GPU where a call has to run)."""

import types

import pytest
import torch

import backward_gate_up_amd as mlp
from backward_gate_up_amd import dense, serve


def test_workspace_sizes_are_kept_by_device(monkeypatch):
    """Two devices with other numbers of compute units need other workspaces: a size
    that one was told is not handed to the other."""
    now = types.SimpleNamespace(device=0)
    asked = []

    def query(*sizes):
        asked.append((now.device, sizes))
        return 1000 * (now.device + 1) + sum(sizes)

    monkeypatch.setattr(serve, "_device", lambda: now.device)
    monkeypatch.setattr(serve, "_L", types.SimpleNamespace(lib=lambda: types.SimpleNamespace(some_workspace_bytes=query)))
    got = []
    for now.device in (0, 1, 0, 1):
        got.append(dense._bytes("some_workspace_bytes", 3, 4))
    assert got == [1007, 2007, 1007, 2007]
    assert asked == [(0, (3, 4)), (1, (3, 4))]  # each asked once


# ---- forward mode and tracers -----------------------------------------------------


def entries(device, dtype=torch.bfloat16):
    """name -> (call of its first input, that input) of every operator, the rest at hand."""
    z = lambda *s: torch.randn(s, device=device, generator=torch.Generator(device).manual_seed(len(s))).to(dtype)  # noqa: E731
    x, w, v, b, r = z(4, 64), z(72, 64), z(64), z(72), z(4, 72)
    wl, wd, e = z(72, 64), z(64, 72), z(2, 72, 64)
    ids, weights = torch.zeros(4, 1, dtype=torch.int32, device=device), torch.ones(4, 1, device=device)
    stats = torch.ones(2, 4, device=device)
    return {
        "layer_norm": (lambda t: mlp.layer_norm(t, v, v), x), "layer_norm weight": (lambda t: mlp.layer_norm(x, t), v),
        "rms_norm": (lambda t: mlp.rms_norm(t, v), x),
        "linear": (lambda t: mlp.linear(t, w, b, "gelu", r), x), "linear w": (lambda t: mlp.linear(x, t), w),
        "linear bias": (lambda t: mlp.linear(x, w, t), b), "linear residual": (lambda t: mlp.linear(x, w, None, None, t), r),
        "feed_forward": (lambda t: mlp.feed_forward(t, v, None, wl, None, wd, None), x),
        "feed_forward w2": (lambda t: mlp.feed_forward(x, v, None, wl, None, t, None), wd),
        "norm_fwd": (lambda t: mlp.norm_fwd(t, v)[0], x), "norm_bwd": (lambda t: mlp.norm_bwd(t, x, v, stats)[0], x),
        "linear_fwd": (lambda t: mlp.linear_fwd(t, w)[0], x), "linear_bwd": (lambda t: mlp.linear_bwd(t, x, w)[0], r),
        "swiglu_mlp": (lambda t: mlp.swiglu_mlp(t, wl, wl, wd, linear=True), x),
        "fwd": (lambda t: mlp.fwd(t, wl, wl, wd, linear=True)[0], x), "infer": (lambda t: mlp.infer(t, wl, wl, wd, linear=True), x),
        "infer_noalloc": (lambda t: mlp.infer_noalloc(t, wl, wl, wd, linear=True), x),
        "moe_route": (lambda t: mlp.moe_route(t, w, 2)[0], x),
        "moe_experts": (lambda t: mlp.moe_experts(t, weights, ids, e, e, e.mT.contiguous()), x),
        "moe_infer": (lambda t: mlp.moe_infer(t, w[:2], e, e, e.mT.contiguous(), 1), x),
        "w4_quantize": (lambda t: mlp.w4_quantize(t, 32)[1], w),
    }


ENTRIES = list(entries("cpu"))


@pytest.mark.parametrize("name", ENTRIES)
def test_tangents_are_refused(name):
    """An input with a tangent, with and without reverse-mode gradients: no operator
    has a forward-mode derivative, and none returns an output without one."""
    f, t = entries("cpu")[name]
    with torch.autograd.forward_ad.dual_level():
        dual = torch.autograd.forward_ad.make_dual(t, torch.ones_like(t))
        for grad in (torch.no_grad(), torch.enable_grad()):
            with grad, pytest.raises(RuntimeError, match="no forward-mode derivative"):
                f(dual)
        # where forward mode is off, and for inputs without a tangent, the call goes on
        with torch.autograd.forward_ad._set_fwd_grad_enabled(False), pytest.raises(ValueError, match="on a GPU"):
            f(dual)
        with pytest.raises(ValueError, match="on a GPU"):
            f(t)


@pytest.mark.parametrize("name", ENTRIES)
def test_tracers_are_refused(name):
    from torch.fx.experimental.proxy_tensor import make_fx

    f, t = entries("cpu")[name]
    with torch.no_grad():
        with pytest.raises(RuntimeError, match="cannot be traced"):
            torch.jit.trace(f, (t,), check_trace=False)
        with pytest.raises(RuntimeError, match="cannot be traced"):
            make_fx(f)(t)
    if name in ("layer_norm", "rms_norm", "linear", "feed_forward", "swiglu_mlp"):
        t = t.clone().requires_grad_()
        with pytest.raises(RuntimeError, match="cannot be traced"):
            make_fx(f)(t)
        if name != "swiglu_mlp":
            with pytest.raises(RuntimeError, match="cannot be traced"):
                torch.jit.trace(f, (t,), check_trace=False)
    with pytest.raises(ValueError, match="on a GPU"):
        f(t)


@pytest.mark.gpu
@pytest.mark.parametrize("name", [n for n in ENTRIES if n != "w4_quantize"])
def test_function_transforms_are_refused(name):
    """torch.func's transforms and vmap wrap the inputs, which have no memory of their own."""
    f, t = entries("cuda")[name]
    with torch.no_grad():
        f(t)
        for transform in (lambda: torch.func.jvp(f, (t,), (torch.ones_like(t),)), lambda: torch.vmap(f)(torch.stack([t, t])),
                          lambda: torch.func.vjp(f, t)):
            with pytest.raises(RuntimeError):
                transform()


@pytest.mark.gpu
def test_a_forward_is_captured_beside_a_live_graph_without_gradients():
    x, w = (torch.randn(s, device="cuda").bfloat16() for s in ((5, 64), (72, 64)))
    w.requires_grad_()
    eager = mlp.linear(x, w, None, "gelu")  # alive, on the default stream
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.no_grad(), torch.cuda.graph(graph):
        y = mlp.linear(x, w, None, "gelu")
    for i in range(3):
        x.copy_(torch.randn_like(x))
        graph.replay()
        torch.cuda.synchronize()
        with torch.no_grad():
            assert torch.equal(y, mlp.linear(x, w, None, "gelu"))
    assert eager.requires_grad


@pytest.mark.gpu
def test_what_is_recorded_still_is():
    """swiglu_mlp with gradients under torch.jit.trace, as before; the dense operators under
    torch.compile, which leaves them to be run as they are; a dispatch mode that only looks."""
    x = torch.randn(5, 64, device="cuda").bfloat16()
    wl, wd = (torch.randn(s, device="cuda").bfloat16().requires_grad_() for s in ((72, 64), (64, 72)))
    block = lambda t: mlp.swiglu_mlp(t, wl, wl, wd, linear=True)  # noqa: E731
    # (weights as inputs: torch takes none that need gradients as constants of a trace)
    traced = torch.jit.trace(lambda t, w, d: mlp.swiglu_mlp(t, w, w, d, linear=True), (x, wl, wd), check_trace=False)
    assert torch.equal(traced(x + 1, wl, wd), block(x + 1))
    dense_chain = lambda t: mlp.linear(mlp.rms_norm(t, wd[:, 0]), wl, None, "gelu") * 2  # noqa: E731
    layer = lambda t: mlp.feed_forward(t * 2, wd[:, 0], None, wl, None, wd, None)  # noqa: E731
    for f in (dense_chain, layer):
        compiled = torch.compile(f, backend="eager")
        for grad in (False, True):
            with torch.set_grad_enabled(grad):
                y, want = compiled(x), f(x)
                assert torch.equal(y, want)
            if grad:
                dy = torch.randn_like(y)
                got, ref = (torch.autograd.grad(t, (wl, wd), dy) for t in (y, want))
                assert all(torch.equal(a, c) for a, c in zip(got, ref))
    from torch.utils._python_dispatch import TorchDispatchMode

    class Sees(TorchDispatchMode):
        def __torch_dispatch__(self, func, types, args=(), kwargs=None):
            return func(*args, **(kwargs or {}))

    with Sees():
        assert torch.equal(layer(x), layer(x))


# ---- the layer's submodules -------------------------------------------------------


class Config:
    hidden_size, intermediate_size, hidden_act = 64, 72, "silu"


class Adapted(torch.nn.Linear):
    """A linear layer with something of its own beside its weight."""

    def forward(self, x):
        return super().forward(x) + 1


@pytest.mark.parametrize("name", ["norm", "fc1", "fc2"])
def test_layers_that_would_not_run_are_refused(name):
    x = torch.zeros(3, 64)
    block = mlp.FeedForward(Config())
    layer = getattr(block, name)
    with pytest.raises(ValueError, match="on a GPU"):  # nothing to refuse but the host's tensors
        block(x)
    for add in ("register_forward_pre_hook", "register_forward_hook", "register_full_backward_hook",
                "register_full_backward_pre_hook"):
        handle = getattr(layer, add)(lambda *a: None)
        with pytest.raises(RuntimeError, match=f"of {name} and does not call it: hooks"):
            block(x)
        handle.remove()
    with pytest.raises(ValueError, match="on a GPU"):
        block(x)
    layer.forward = layer.forward
    with pytest.raises(TypeError, match=f"of {name} and does not call it: it has to be a torch.nn"):
        block(x)
    del layer.forward
    for other in (Adapted(64, 72), torch.nn.Identity(), torch.nn.Sequential(layer)):
        setattr(block, name, other)
        with pytest.raises(TypeError, match=f"of {name} and does not call it: it has to be a torch.nn"):
            block(x)
    setattr(block, name, layer)
    with pytest.raises(ValueError, match="on a GPU"):
        block(x)


@pytest.mark.gpu
def test_parametrized_layers_and_hooks_on_the_layer_run():
    """A parametrization's weight is the layer's weight, its gradient reaches what it
    is made of; hooks on the FeedForward itself run; so do copies."""
    import copy

    torch.manual_seed(1)
    block = mlp.FeedForward(Config()).to("cuda")
    torch.nn.utils.parametrizations.weight_norm(block.fc1)
    block.fc1.parametrizations.weight.original0.data.mul_(1.5)
    x = torch.randn(5, 64, device="cuda")
    want = mlp.feed_forward(x, block.norm.weight, block.norm.bias, block.fc1.weight, block.fc1.bias, block.fc2.weight,
                            block.fc2.bias, "silu")
    seen = []
    block.register_forward_hook(lambda m, args, out: seen.append(out))
    for m in (block, copy.deepcopy(block)):
        y = m(x)
        assert torch.equal(y, want) and seen.pop() is y
        y.sum().backward()
        assert m.fc1.parametrizations.weight.original0.grad.abs().sum() > 0
