"""What the autograd nodes keep: only what a wanted gradient reads, so that the rest
may be freed or changed in place (GPU); what the C entry takes without (CPU, GPU)."""

import ctypes

import pytest
import torch

import backward_gate_up_amd as mlp
from backward_gate_up_amd import _lib
from tests._util import banner
from tests.test_dense import DEV, gen, normal

BF = torch.bfloat16


def kept(call):
    """(output, addresses of what its node keeps)"""
    at = []

    def pack(t):
        at.append(t.data_ptr())
        return t

    with torch.autograd.graph.saved_tensors_hooks(pack, lambda t: t):
        y = call()
    return y, at


@pytest.mark.gpu
@pytest.mark.parametrize("act", [None, "silu"])
@pytest.mark.parametrize("T", [5, 90])
def test_linear_keeps_what_it_reads(T, act):
    banner(f"kept by linear T={T} {act}")
    x, w, b, r = (normal(gen(i), s, BF) for i, s in enumerate(((T, 136), (264, 136), (264,), (T, 264))))
    dy = normal(gen(9), (T, 264), BF)
    z = mlp.linear_fwd(x, w, b, act, r)[1]
    want = dict(zip("xwb", mlp.linear_bwd(dy, x, w, z, act)), r=dy)
    for wanted in ("x", "w", "b", "r", "xw", "xb", "wr", "br", "xwbr"):
        t = {k: v.clone().requires_grad_(k in wanted) for k, v in zip("xwbr", (x, w, b, r))}
        y, at = kept(lambda: mlp.linear(t["x"], t["w"], t["b"], act, t["r"]))
        assert (t["x"].data_ptr() in at) == ("w" in wanted), wanted
        assert (t["w"].data_ptr() in at) == ("x" in wanted), wanted
        assert len(at) == ("w" in wanted) + ("x" in wanted) + (act is not None and wanted != "r"), wanted
        with torch.no_grad():  # what is not kept may change
            for k, other in (("x", "w"), ("w", "x")):
                if other not in wanted:
                    t[k].zero_()
            t["b"].zero_()
            t["r"].zero_()
        for k, g in zip(wanted, torch.autograd.grad(y, [t[k] for k in wanted], dy)):
            assert torch.equal(g, want[k]), (wanted, k)


@pytest.mark.gpu
def test_a_frozen_layers_input_may_be_added_to():
    """x = x + f(x) in place after a frozen projection, as torch's own layer allows."""
    banner("in place after a frozen layer")
    w = normal(gen(1), (136, 136), BF, 0.1)
    x0, dy = normal(gen(2), (30, 136), BF).requires_grad_(), normal(gen(3), (30, 136), BF)

    def chain(linear):
        x = x0 * 2
        h = linear(x)
        x += h
        return torch.autograd.grad(x, x0, dy)[0]

    got = chain(lambda x: mlp.linear(x, w))
    assert torch.equal(got, 2 * (dy + mlp.linear_bwd(dy, x0.detach() * 2, w)[0]))
    x = normal(gen(4), (30, 136), BF).requires_grad_()
    z = x * 2
    y = mlp.linear(z, w.clone().requires_grad_())
    z += 1
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        torch.autograd.grad(y, x, dy)


@pytest.mark.gpu
def test_feed_forward_keeps_what_it_reads():
    banner("kept by feed_forward")
    sh = {"x": (90, 136), "nw": (136,), "nb": (136,), "w1": (264, 136), "b1": (264,), "w2": (136, 264), "b2": (136,)}
    # which inputs a wanted gradient reads, and how many tensors of the forward's own (statistics, norm's output, z, hidden values)
    needs = {"x": ({"x", "nw", "w1", "w2"}, 2), "nb": ({"x", "nw", "w1", "w2"}, 2), "w1": ({"w2"}, 2), "b1": ({"w2"}, 1),
             "w2": (set(), 1), "b2": (set(), 0)}
    dy = normal(gen(50), (90, 136), BF)
    for wanted, (inputs, own) in needs.items():
        t = {k: normal(gen(i), s, BF, 0.1 if k[0] == "w" else 1.0).requires_grad_(k == wanted) for i, (k, s) in enumerate(sh.items())}
        y, at = kept(lambda: mlp.feed_forward(*t.values(), activation="silu"))
        assert {k for k in t if t[k].data_ptr() in at} == inputs, wanted
        assert len(at) == len(inputs) + own, wanted
        g, = torch.autograd.grad(y, t[wanted], dy)
        full = {k: v.detach().clone().requires_grad_() for k, v in t.items()}
        ref, = torch.autograd.grad(mlp.feed_forward(*full.values(), activation="silu"), full[wanted], dy)
        assert torch.equal(g, ref), wanted


@pytest.mark.gpu
@pytest.mark.parametrize("T,N,K", [(5, 264, 136), (700, 264, 136), (2100, 4104, 2056)])
def test_operands_that_are_not_read_may_be_absent(T, N, K):
    banner(f"absent operands T={T}")
    L = _lib.lib()
    x, w, dy = (normal(gen(i), s, BF) for i, s in enumerate(((T, K), (N, K), (T, N))))
    need = L.swiglu_mlp_linear_bwd_workspace_bytes(T, N, K, 0, 0)
    ws = torch.empty(max(need, 16), dtype=torch.uint8, device=DEV)
    p = lambda t: None if t is None else t.data_ptr()  # noqa: E731
    for needs in ((True, False, True), (False, True, False), (False, False, True)):
        out = [torch.empty(s, dtype=BF, device=DEV) if n else None for s, n in zip(((T, K), (N, K), (N,)), needs)]
        rc = L.swiglu_mlp_linear_bwd(p(dy), p(x) if needs[1] else None, p(w) if needs[0] else None, None, *map(p, out), p(ws), need,
                                     T, N, K, 0, 0, 0)
        assert rc == 0
        torch.cuda.synchronize()
        for got, want in zip(out, mlp.linear_bwd(dy, x, w, needs=needs)):
            assert got is None or torch.equal(got, want)


def test_operands_that_are_read_may_not():
    L, S = _lib.lib(), {v: k for k, v in _lib.STATUS.items()}
    a = [ctypes.c_void_p(0x10000000 * (i + 1)) for i in range(8)]  # nothing reads them
    call = lambda x, w, dx, dw: L.swiglu_mlp_linear_bwd(a[0], x, w, None, dx, dw, None, a[6], 1 << 30, 4, 32, 64, 0, 0, None)  # noqa: E731
    assert call(None, a[2], a[3], a[4]) == call(a[1], None, a[3], a[4]) == S["SWIGLU_ERR_NULL"]
    assert call(None, a[2], None, a[4]) == call(a[1], None, a[3], None) == S["SWIGLU_ERR_NULL"]
    if not torch.cuda.is_available():  # past every check but the device's
        assert call(None, a[2], a[3], None) == call(a[1], None, None, a[4]) == call(None, None, None, None) == S["SWIGLU_ERR_DEVICE"]
