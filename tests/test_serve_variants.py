"""The few-token serving operators: each launch variant at the sizes that select
it, with the other dimensions small. Formulas and bounds are those of
tests/test_serve.py: a result of one product carries one rounding of half a step,
one of two products two, and 1e-5 for the fp32 sums.
"""

import copy
import gc
import io
import os
import pickle
import subprocess
import sys
import weakref

import numpy as np
import pytest
import torch

import backward_gate_up_amd as m
from backward_gate_up_amd import _lib
from tests._util import assert_local, banner, f64
from tests.test_serve import (DT, _moe_config, bound, cuda, expert_weights, gen, make_w4, randn, ref_block, ref_experts,
                              ref_route, ref_w4)

gpu = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def check_linear(T, N, K, group, zeros, dt):
    g = gen(N + K + T)
    raw = make_w4(g, (N, K), group, zeros, DT[dt])
    x = randn(g, (T, K), 1, DT[dt])
    y = m.w4_linear(x.cuda(), m.w4_pack(*cuda(raw)))
    assert_local(f64(y), f64(x) @ ref_w4(*raw).T, bound(DT[dt], 1), ("w4", dt, T, N, K))


@gpu
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("T", [1, 4, 5, 16])
@pytest.mark.parametrize("N,K,group", [(24544, 128, 128), (24552, 128, 128), (24584, 96, 32), (32000, 192, 64),
                                       (24576, 1024, 128)])
def test_w4_linear_many_columns(T, N, K, group, dt):
    """Tiles of 32 columns (more than 24544 on 256 CUs), N that ends in either half."""
    banner(f"w4_linear {dt} T={T} N={N} K={K} g={group}")
    check_linear(T, N, K, group, T % 2 == 0, dt)


# ---- calls without a token ----------------------------------------------------------

EMPTY_CALLS = {
    "moe_experts": "L.swiglu_mlp_moe_experts(*at[:8], 1 << 30, 0, 64, 128, 8, 2, 0, None)",
    "moe_infer": "L.swiglu_mlp_moe_infer(at[0], at[8], *at[3:8], 1 << 30, 0, 64, 128, 8, 2, 1, 0, None)",
    "moe_experts, NULL": "L.swiglu_mlp_moe_experts(None, None, None, *at[3:6], None, None, 0, 0, 64, 128, 8, 2, 0, None)",
    "moe_experts_w4": "L.swiglu_mlp_moe_experts_w4(*at[:3], *w(8), at[6], at[7], 1 << 30, 0, 2, 0, None)",
    "moe_infer_w4": "L.swiglu_mlp_moe_infer_w4(at[0], at[8], *w(8), at[6], at[7], 1 << 30, 0, 2, 1, 0, None)",
    "w4_infer": "L.swiglu_mlp_w4_infer(at[0], *w(1), at[6], at[7], 1 << 30, 0, 0, None)",
    "w4_infer, NULL": "L.swiglu_mlp_w4_infer(None, *w(1), None, None, 0, 0, 0, None)",
    "w4_linear": "L.swiglu_mlp_w4_linear(at[0], w(1)[0], at[6], None, 0, 0, 0, None)",
    "moe_route": "L.swiglu_mlp_moe_route(at[0], at[8], at[1], at[2], None, 0, 0, 64, 8, 2, 1, 0, None)",
}


@pytest.mark.parametrize("call", EMPTY_CALLS)
def test_no_tokens_at_the_c_entries(call):
    """T = 0 passes the argument checks and does nothing (a process of its own:
    addresses are made up, and nothing may end the process)."""
    code = ("import ctypes\nfrom backward_gate_up_amd import _lib\nL = _lib.lib()\n"
            "at = [(1 << 40) + (i << 34) for i in range(9)]\n"
            "w4 = lambda i, E, N, K: ctypes.byref(_lib.W4(at[i], E, N, K, 32, 0))\n"
            "w = lambda E: [w4(3, E, 64, 128), w4(4, E, 64, 128), w4(5, E, 128, 64)]\n"
            f"print('status', {EMPTY_CALLS[call]})\n")
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=120, cwd=ROOT)
    assert r.returncode == 0, (r.returncode, r.stderr[-500:])
    assert int(r.stdout.split("status")[1]) in (0, 7), r.stdout  # 7: no gfx950 here


@gpu
@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_no_tokens(dt):
    banner(f"no tokens {dt}")
    g, E, D, H, k = gen(1), 4, 64, 96, 2
    x, wr = torch.empty((0, D), dtype=DT[dt], device="cuda"), randn(g, (E, D), 1, DT[dt]).cuda()
    w = cuda(expert_weights(g, E, D, H, DT[dt]))
    p, ids = m.moe_route(x, wr, k)
    assert p.shape == ids.shape == (0, k)
    assert m.moe_experts(x, p, ids, *w).shape == m.moe_infer(x, wr, *w, k).shape == (0, D)
    if dt == "fp32":
        return
    w4 = [m.W4Weight.quantize(t, 32) for t in w]
    assert m.moe_experts(x, p, ids, *w4).shape == m.moe_infer(x, wr, *w4, k).shape == (0, D)
    dense = [m.W4Weight.quantize(t[0], 32) for t in w]
    assert m.infer_w4(x, *dense).shape == (0, D) and m.w4_linear(x, dense[0]).shape == (0, H)


# ---- values past the storage type's range -------------------------------------------


def large_block(D, H, dt, a):
    """Weights of one expert and a token for which every A = SiLU(g) u is about
    `a` or -a: g = u's magnitude = sqrt(a), and down weights of both signs."""
    g = gen(D + H)
    x = torch.ones(1, D)
    wg = torch.full((1, H, D), a ** 0.5 / D)
    wu = wg * torch.where(torch.rand((1, H, 1), generator=g) < 0.5, -1.0, 1.0)
    wd = torch.randn((1, D, H), generator=g) / 64
    return tuple(t.to(dt) for t in (x, wg, wu, wd))


@gpu
@pytest.mark.parametrize("T", [1, 5, 8])
@pytest.mark.parametrize("a", [4e4, 6.55e4, 9e4, 1.3e5])
def test_hidden_values_past_the_range_of_fp16(T, a):
    """With 8 or fewer token rows A is held in two parts: values to twice the
    type's largest come out as the finite results they are."""
    banner(f"large A T={T} a={a}")
    D, H, dt = 128, 200, torch.float16
    x, wg, wu, wd = large_block(D, H, dt, a)
    x = x.repeat(T, 1)
    p, ids = torch.ones(T, 1), torch.zeros((T, 1), dtype=torch.int32)
    y = m.moe_experts(x.cuda(), p.cuda(), ids.cuda(), *cuda((wg, wu, wd)))
    ref, got = ref_block(f64(x), *(f64(t[0]) for t in (wg, wu, wd))), f64(y)
    past = np.abs(ref) >= 65520  # results that are past the range themselves round to infinities
    assert np.array_equal(got[past], np.sign(ref[past]) * np.inf)
    got[past] = ref[past] = 0
    assert_local(got, ref, bound(dt, 2), ("large", T, a))


@gpu
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("T", [1, 8, 20, 40])
def test_infinite_hidden_values(T, dt):
    """A token with an infinity, whose every A is infinite: y is the infinity of
    the definition's sign in each column of one sign, NaN where both meet, at
    every number of tokens."""
    banner(f"infinite A {dt} T={T}")
    D, H = 128, 200
    x, wg, wu, wd = large_block(D, H, DT[dt], 100)
    x = x.repeat(T, 1)
    x[0, 3] = float("inf")
    wu, wd = wu.abs(), wd.abs() + 2.0 ** -6
    wd[0, 1::3] *= -1
    wd[0, 2::3, ::2] *= -1
    p, ids = torch.ones(T, 1), torch.zeros((T, 1), dtype=torch.int32)
    y = m.moe_experts(x.cuda(), p.cuda(), ids.cuda(), *cuda((wg, wu, wd))).float().cpu()
    assert (y[0, 0::3] == float("inf")).all() and (y[0, 1::3] == -float("inf")).all() and y[0, 2::3].isnan().all()
    ref = ref_block(f64(x)[1:], *(f64(t[0]) for t in (wg, wu, wd)))
    if T > 1:
        assert_local(f64(y)[1:], ref, bound(DT[dt], 2), ("rest", T))


def same_values(got, ref, tol):
    """NaN and infinities in the same places with the same signs, the rest within tol of the largest."""
    fin = np.isfinite(ref)
    assert np.array_equal(np.isnan(got), np.isnan(ref))
    assert np.array_equal(got[~fin & ~np.isnan(ref)], ref[~fin & ~np.isnan(ref)])
    if fin.any():
        assert np.abs(got[fin] - ref[fin]).max() <= tol * np.abs(ref[fin]).max()


@gpu
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("T", [1, 4, 5, 16, 17, 40, 70])
@pytest.mark.parametrize("N,K,group,zeros", [(72, 416, 32, True), (264, 1152, 128, False), (136, 6272, 64, True)])
def test_w4_linear_infinite_and_large_tokens(T, N, K, group, zeros, dt):
    """An infinity in x gives s (q - z) times it, NaN where q = z, and large values
    the finite results they have, at every number of tokens; other tokens keep
    their bits."""
    banner(f"w4 inf {dt} T={T} N={N} K={K}")
    g = gen(N + K)
    raw = make_w4(g, (N, K), group, zeros, DT[dt])
    w = m.w4_pack(*cuda(raw))
    x = randn(g, (T, K), 1, DT[dt])
    clean = m.w4_linear(x.cuda(), w)
    big = 3e37 if dt == "bf16" else 6e4
    for t, what in ((0, "inf"), (T // 2, "large"), (T - 1, "-inf")):
        z = x.clone()
        if what == "large":
            z[t, 5], z[t, K - 3] = big, -big
        else:
            z[t, K // 2 + 1] = float(what)
        y = m.w4_linear(z.cuda(), w)
        with np.errstate(invalid="ignore"):
            ref = (f64(z)[t] * ref_w4(*raw)).sum(1)
        same_values(f64(y)[t], ref, bound(DT[dt], 1))
        rest = [i for i in range(T) if i != t]
        assert torch.equal(y[rest], clean[rest])


@gpu
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("T,D,H,group", [(1, 256, 128, 64), (4, 6272, 64, 64), (16, 160, 96, 32), (20, 64, 128, 32),
                                         (40, 64, 128, 64)])
def test_infer_w4_infinite_tokens(T, D, H, group, dt):
    """Infinite gate and up values, and infinite A, through the 4-bit block: no zero
    weights, signs such that nothing cancels."""
    banner(f"infer_w4 inf {dt} T={T} D={D} H={H}")
    g = gen(D)
    raw = [make_w4(g, s, group, False, DT[dt]) for s in ((H, D), (H, D), (D, H))]
    for i, (codes, _, _) in enumerate(raw):  # gate above zero, up too; down rows of one sign
        high, low = codes | 0x99, codes & 0x77  # q >= 9, q <= 7: weights above and below zero
        codes[:] = high
        if i == 2:
            codes[1::2] = low[1::2]
    w = [m.w4_pack(*cuda(r)) for r in raw]
    x = randn(g, (T, D), 1, DT[dt])
    clean = m.infer_w4(x.cuda(), *w)
    z = x.clone()
    z[T // 2, 7] = float("inf")
    y = m.infer_w4(z.cuda(), *w).float().cpu()
    assert (y[T // 2, 0::2] == float("inf")).all() and (y[T // 2, 1::2] == -float("inf")).all()
    rest = [i for i in range(T) if i != T // 2]
    assert torch.equal(y[rest], clean.float().cpu()[rest])
    z[T // 2, 7] = -float("inf")  # SiLU(-inf) = -inf / inf
    assert m.infer_w4(z.cuda(), *w)[T // 2].isnan().all()


@gpu
@pytest.mark.parametrize("T,E,k", [(1, 4, 2), (24, 4, 2), (64, 6, 3), (60, 48, 12)])
def test_moe_w4_infinite_tokens(T, E, k):
    banner(f"moe_w4 inf T={T} E={E} k={k}")
    D, H, group, dt = 128, 256, 64, torch.bfloat16
    g = gen(T + E)
    raw = [make_w4(g, s, group, False, dt) for s in ((E, H, D), (E, H, D), (E, D, H))]
    for i, (codes, _, _) in enumerate(raw):
        high, low = codes | 0x99, codes & 0x77
        codes[:] = high
        if i == 2:
            codes[:, 1::2] = low[:, 1::2]
    w = [m.w4_pack(*cuda(r)) for r in raw]
    x = randn(g, (T, D), 1, dt)
    ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).int()
    p = torch.rand((T, k), generator=g) + 0.1
    clean = m.moe_experts(x.cuda(), p.cuda(), ids.cuda(), *w)
    z = x.clone()
    z[T // 3, 90] = float("inf")
    y = m.moe_experts(z.cuda(), p.cuda(), ids.cuda(), *w).float().cpu()
    assert (y[T // 3, 0::2] == float("inf")).all() and (y[T // 3, 1::2] == -float("inf")).all()
    rest = [i for i in range(T) if i != T // 3]
    assert torch.equal(y[rest], clean.float().cpu()[rest])


# ---- the router's order for very small numbers ----------------------------------------


@gpu
@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("T", [3, 12, 600])
@pytest.mark.parametrize("sx,sw", [(-80, 0), (0, -80), (-60, -60), (-78, -40), (-100, 20)])
def test_route_order_of_small_numbers(T, sx, sw, dt):
    """Experts that differ in the last digits of a long sum, with tokens or weights
    whose squares are below fp32's range: the order is the exact logits'."""
    banner(f"route small T={T} 2^{sx} 2^{sw} {dt}")
    D, E, k = 1024, 12, 5
    g = gen(T)
    x, base = torch.randn((T, D), generator=g), torch.randn((1, D), generator=g).repeat(E, 1)
    base[:, 17] *= 1 + torch.arange(E).float()[torch.randperm(E, generator=g)] * 2.0 ** -6
    x[:, 17] *= 2.0 ** -12
    # powers of two change no digit (none falls below the smallest normal number)
    x, wr = x.to(DT[dt]) * 2.0 ** sx, base.to(DT[dt]) * 2.0 ** sw
    _, ids = m.moe_route(x.cuda(), wr.cuda(), k)
    assert np.array_equal(ids.cpu().numpy(), ref_route(f64(x), f64(wr), k, True)[0])


@gpu
@pytest.mark.parametrize("dt", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("T", [3, 12, 600])
def test_route_of_zeros(T, dt):
    banner(f"route zeros T={T} {dt}")
    D, E, k = 1000, 100, 6
    g = gen(T)
    x, wr = randn(g, (T, D), 1, DT[dt]), randn(g, (E, D), D ** -0.5, DT[dt])
    x[1] = 0
    x[2] = -0.0
    p, ids = m.moe_route(x.cuda(), wr.cuda(), k, False)
    assert (ids[1:3].cpu() == torch.arange(k)).all() and (p[1:3].cpu() - 0.01).abs().max() < 1e-8
    assert np.array_equal(ids.cpu().numpy(), ref_route(f64(x), f64(wr), k, False)[0])
    p, ids = m.moe_route(x.cuda(), torch.zeros_like(wr).cuda(), k, True)
    assert (ids.cpu() == torch.arange(k)).all() and (p.cpu() - 1 / k).abs().max() < 1e-7


# ---- 4-bit weights and modules as objects (host) ---------------------------------------


def host_w4(g, shape, group, zeros, dtype=torch.bfloat16):
    """A 4-bit weight of random bytes in host memory, which no kernel reads."""
    *lead, N, K = shape
    n = _lib.lib().swiglu_mlp_w4_bytes(lead[0] if lead else 1, N, K, group, zeros)
    return m.W4Weight(torch.randint(0, 256, (n,), generator=g, dtype=torch.uint8), shape, group, zeros, dtype)


def host_moe(seed, group=32, zeros=False):
    """SwiGLUMoE with 4-bit experts in host memory."""
    mod = m.SwiGLUMoE(_moe_config())
    for name in ("gate_proj", "up_proj", "down_proj"):
        w = host_w4(gen(seed), getattr(mod, name).shape, group, zeros)
        delattr(mod, name)
        mod._keep(name, w)
    return mod


def same_w4(a, b):
    form = lambda w: (w.shape, w.group, w.has_zeros, w.dtype, w.experts, w.device)  # noqa: E731
    return form(a) == form(b) and torch.equal(a.data, b.data) and a._c.data == a.data.data_ptr()


def test_w4_weights_can_be_copied_and_saved():
    w = host_w4(gen(1), (3, 16, 128), 64, True, torch.float16)
    for c in (copy.copy(w), copy.deepcopy(w), pickle.loads(pickle.dumps(w))):
        assert same_w4(c, w) and (c._c.N, c._c.K, c._c.group, c._c.has_zeros) == (16, 128, 64, 1)
    assert copy.deepcopy(w).data.data_ptr() != w.data.data_ptr()


def test_modules_with_4_bit_weights_can_be_copied_and_saved():
    mod = host_moe(2)
    buf = io.BytesIO()
    torch.save(mod, buf)
    buf.seek(0)
    for c in (copy.deepcopy(mod), torch.load(buf, weights_only=False)):  # our own file
        assert set(c.state_dict()) == set(mod.state_dict())
        for name in ("gate_proj", "up_proj", "down_proj"):
            assert same_w4(c._weight(name), mod._weight(name))
            assert c._weight(name).data is getattr(c, name)


def test_modules_let_go_of_the_weights_they_replace():
    """After a move the module holds no copy of the old buffers."""
    mod = host_moe(3)
    old = [weakref.ref(getattr(mod, n)) for n in ("gate_proj", "up_proj", "down_proj")]
    mod._apply(lambda t: t.clone())
    gc.collect()
    assert all(r() is None for r in old)
    assert mod._weight("up_proj").data is mod.up_proj


def saved(state):
    buf = io.BytesIO()
    torch.save(state, buf)
    buf.seek(0)
    return torch.load(buf, weights_only=True)


@pytest.mark.parametrize("assign", [False, True])
def test_state_dicts_carry_the_form_of_4_bit_weights(assign):
    """Group size, zero points and type travel in the state dict's metadata: a saved
    module of 4-bit experts loads into a fresh one, inside a larger model too, and
    over weights of another form of equally many bytes."""
    src = host_moe(4, 32, True)
    names = ("gate_proj", "up_proj", "down_proj")
    assert set(src.state_dict()) == {"gate.weight", *names}
    fresh = m.SwiGLUMoE(_moe_config())
    fresh.load_state_dict(saved(src.state_dict()), assign=assign)
    assert all(same_w4(fresh._weight(n), src._weight(n)) for n in names) and not list(fresh.named_parameters())[1:]
    assert torch.equal(fresh.gate.weight, src.gate.weight)
    model = torch.nn.ModuleDict({"layer": m.SwiGLUMoE(_moe_config())})
    model.load_state_dict(saved(torch.nn.ModuleDict({"layer": src}).state_dict()), assign=assign)
    assert all(same_w4(model["layer"]._weight(n), src._weight(n)) for n in names)
    # 64 without and 128 with zero points take the same bytes
    cfg = dict(hidden_size=128, moe_intermediate_size=256)
    a, b = m.SwiGLUMoE(_moe_config(**cfg)), m.SwiGLUMoE(_moe_config(**cfg))
    for mod, group, zeros in ((a, 64, False), (b, 128, True)):
        for n in names:
            w = host_w4(gen(group), getattr(mod, n).shape, group, zeros)
            delattr(mod, n)
            mod._keep(n, w)
    assert a.up_proj.numel() == b.up_proj.numel()
    b.load_state_dict(saved(a.state_dict()), assign=assign)
    assert all(same_w4(b._weight(n), a._weight(n)) for n in names)


def test_state_dicts_that_do_not_fit_are_refused():
    src = host_moe(5)
    other = m.SwiGLUMoE(_moe_config(moe_intermediate_size=128))
    with pytest.raises(RuntimeError, match="4-bit weight"):
        other.load_state_dict(src.state_dict())
    assert other.gate_proj.shape == (6, 128, 64)  # as it was
    with pytest.raises(RuntimeError, match="size mismatch"):
        src.load_state_dict(m.SwiGLUMoE(_moe_config()).state_dict())
    # without metadata (another file format) the module's own form is taken
    again = host_moe(6)
    again.load_state_dict(dict(src.state_dict()))
    assert same_w4(again._weight("up_proj"), src._weight("up_proj"))
    with pytest.raises(RuntimeError, match="size mismatch"):
        m.SwiGLUMoE(_moe_config()).load_state_dict(dict(src.state_dict()))


@pytest.mark.parametrize("biased", ["gate_proj", "up_proj", "down_proj", None])
def test_biases_are_refused_in_the_4_bit_block(biased):
    block = torch.nn.Module()
    for name, (n_in, n_out) in (("gate_proj", (64, 96)), ("up_proj", (64, 96)), ("down_proj", (96, 64))):
        setattr(block, name, torch.nn.Linear(n_in, n_out, bias=name == biased))
    with pytest.raises(ValueError, match="bias" if biased else "GPU"):  # without one, as far as the device
        m.SwiGLUMLPW4(block, 32)


def test_quantize_leaves_the_module_whole_when_it_is_refused(monkeypatch):
    """A group that divides one weight's K and not another's: nothing is replaced."""
    mod = m.SwiGLUMoE(_moe_config())  # K 64, 64 and 96
    before = {n: p for n, p in mod.named_parameters()}

    def quantize(w, group=128, zeros=False):
        m.serve._w4_shape(tuple(w.shape), group)
        return host_w4(gen(1), tuple(w.shape), group, zeros)

    monkeypatch.setattr(m.W4Weight, "quantize", quantize)
    with pytest.raises(ValueError, match="group"):
        mod.quantize_(64)
    assert not mod._forms and all(p is before[n] for n, p in mod.named_parameters()) and len(before) == 4
    mod.quantize_(32)
    assert set(mod._forms) == {"gate_proj", "up_proj", "down_proj"} and [n for n, _ in mod.named_parameters()] == ["gate.weight"]
    with pytest.raises(RuntimeError, match="4 bits"):
        mod.quantize_(32)


@gpu
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_w4_quantize_keeps_nan(group, zeros, dt):
    """A group with a NaN or an infinity does not become finite numbers; others are not touched."""
    banner(f"quantize NaN {dt} g={group} zeros={zeros}")
    w = randn(gen(9), (16, 384), 0.05, DT[dt])
    bad = w.clone()
    bad[3, 5], bad[8, 383], bad[11, 2 * group] = float("nan"), float("nan"), float("inf")
    clean, got = (m.W4Weight.quantize(t.cuda(), group, zeros).dequantize().cpu().view(16, -1, group) for t in (w, bad))
    hit = [(3, 0), (8, 384 // group - 1), (11, 2)]
    assert all(got[r, c].isnan().all() for r, c in hit[:2]) and not got[hit[2]].isfinite().any()
    for r, c in hit:
        got[r, c] = clean[r, c]
    assert torch.equal(got, clean)


# ---- variants chosen by length and width ------------------------------------------------


def check_moe(T, E, k, D, H, dt):
    g = gen(T * E + D)
    x, w = randn(g, (T, D), 1, DT[dt]), expert_weights(g, E, D, H, DT[dt])
    ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).int()
    p = torch.rand((T, k), generator=g) + 0.1
    y = m.moe_experts(x.cuda(), p.cuda(), ids.cuda(), *cuda(w))
    assert_local(f64(y), ref_experts(f64(x), f64(p), ids.numpy(), *map(f64, w)), bound(DT[dt], 2), (T, D, H))


def check_block_w4(T, D, H, group, zeros, dt):
    g = gen(D + H)
    raw = [make_w4(g, s, group, zeros, DT[dt]) for s in ((H, D), (H, D), (D, H))]
    x = randn(g, (T, D), 1, DT[dt])
    y = m.infer_w4(x.cuda(), *(m.w4_pack(*cuda(r)) for r in raw))
    assert_local(f64(y), ref_block(f64(x), *(ref_w4(*r) for r in raw)), bound(DT[dt], 2), ("w4", T, D, H))


@gpu
@pytest.mark.parametrize("dt", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("T", [1, 5, 12])
@pytest.mark.parametrize("D", [3136, 3144, 4360])
def test_long_rows_few_tiles(T, D, dt):
    """48 stages of K or more and fewer tiles than CUs: 8 waves split K."""
    banner(f"8 waves {dt} T={T} D={D}")
    check_moe(T, 4, 2, D // 16 * 8 if dt == "fp32" else D, 40, dt)


@gpu
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("T", [1, 4, 16])
@pytest.mark.parametrize("D,group,zeros", [(6144, 128, False), (6176, 32, True), (8256, 64, False)])
def test_long_rows_few_tiles_w4(T, D, group, zeros, dt):
    banner(f"8 waves in 4 bits {dt} T={T} D={D}")
    check_block_w4(T, D, 2 * group, group, zeros, dt)
    check_linear(T, 72, D, group, zeros, dt)


@gpu
@pytest.mark.parametrize("dt", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("T", [1, 8, 12, 16])
@pytest.mark.parametrize("D", [2552, 2560, 6136, 6152, 8192, 16392])
def test_wide_down_projections(T, D, dt):
    """160, 384 and 1024 tiles of 16 columns: 16, 8 and 4 waves, no split."""
    banner(f"down {dt} T={T} D={D}")
    check_moe(T, 3, 2, D, 72, dt)


@gpu
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("T", [1, 4, 9, 16])
@pytest.mark.parametrize("D,group,zeros", [(2560, 64, False), (6176, 32, True), (8192, 128, False), (16416, 32, False)])
def test_wide_down_projections_w4(T, D, group, zeros, dt):
    banner(f"down in 4 bits {dt} T={T} D={D}")
    check_block_w4(T, D, 128, group, zeros, dt)


@gpu
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("T", [17, 20, 32, 33, 64])
@pytest.mark.parametrize("D,H,group,zeros", [(64, 12224, 32, True), (128, 12416, 64, False), (320, 12288, 64, True)])
def test_wide_gate_up_w4_shared_rows(T, D, H, group, zeros, dt):
    """96 tiles of 128 hidden columns: 32 and 64 token rows shared by 8 waves."""
    banner(f"shared rows in 4 bits {dt} T={T} D={D} H={H}")
    check_block_w4(T, D, H, group, zeros, dt)


@gpu
@pytest.mark.parametrize("T,E,k", [(64, 48, 12), (64, 48, 16), (40, 64, 32)])
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_moe_w4_shared_rows(T, E, k, dt):
    """An average of more than 12 pairs per expert in 4 bits, and 96 tiles."""
    banner(f"experts' shared rows in 4 bits {dt} T={T} E={E} k={k}")
    D, H, group = 160, 256, 32
    g = gen(T + E)
    raw = [make_w4(g, s, group, True, DT[dt]) for s in ((E, H, D), (E, H, D), (E, D, H))]
    x = randn(g, (T, D), 1, DT[dt])
    ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).int()
    ids[:, 0] = 1  # one expert that takes every token: several passes
    p = torch.rand((T, k), generator=g) + 0.1
    y = m.moe_experts(x.cuda(), p.cuda(), ids.cuda(), *(m.w4_pack(*cuda(r)) for r in raw))
    assert_local(f64(y), ref_experts(f64(x), f64(p), ids.numpy(), *(ref_w4(*r) for r in raw)), bound(DT[dt], 2), (T, E, k))


@gpu
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("T,D,H", [(1, 256, 128), (1, 2688, 128), (16, 256, 256), (16, 2688, 128), (20, 128, 12288), (20, 256, 128),
                                   (40, 128, 12288), (40, 256, 128)])
def test_every_group_size(T, D, H, group, dt):
    banner(f"group {group} {dt} T={T} D={D} H={H}")
    check_block_w4(T, D, H, group, T % 16 == 4, dt)
    check_linear(T, 72, 2 * D, group, T % 16 == 4, dt)


@gpu
@pytest.mark.parametrize("fmt", [("bf16", 0), ("fp16", 0), ("fp32", 0)] + [(t, n) for t in ("bf16", "fp16") for n in (32, 64, 128)])
@pytest.mark.parametrize("T,E,k", [(40, 64, 1), (40, 20, 2), (70, 64, 1), (70, 30, 3)])
def test_lightly_loaded_experts(T, E, k, fmt):
    """More than 16 tokens with few pairs per expert: 4, 8 or 16 token rows, whole chunks' sums."""
    dt, group = fmt
    banner(f"light experts {dt} g={group} T={T} E={E} k={k}")
    D, H = 256, 128
    if not group:
        check_moe(T, E, k, D, H, dt)
        return
    g = gen(T + E)
    raw = [make_w4(g, s, group, False, DT[dt]) for s in ((E, H, D), (E, H, D), (E, D, H))]
    x = randn(g, (T, D), 1, DT[dt])
    ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).int()
    p = torch.rand((T, k), generator=g) + 0.1
    y = m.moe_experts(x.cuda(), p.cuda(), ids.cuda(), *(m.w4_pack(*cuda(r)) for r in raw))
    assert_local(f64(y), ref_experts(f64(x), f64(p), ids.numpy(), *(ref_w4(*r) for r in raw)), bound(DT[dt], 2), (T, E, k))


@gpu
@pytest.mark.parametrize("dt", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("T,E,k,D", [(1023, 60, 4, 520), (1024, 64, 8, 264), (2047, 33, 2, 136), (2048, 129, 3, 72), (2085, 256, 8, 1000)])
def test_route_around_many_tokens(T, E, k, D, dt):
    """The logits come from another kernel from 1024 tokens on, in fp32 from 2048."""
    banner(f"route {dt} T={T} E={E} k={k} D={D}")
    g = gen(T + E)
    x, wr = randn(g, (T, D), 1, DT[dt]), randn(g, (E, D), D ** -0.5, DT[dt])
    for renorm in (True, False):
        p, ids = m.moe_route(x.cuda(), wr.cuda(), k, renorm)
        ri, rp = ref_route(f64(x), f64(wr), k, renorm)
        assert np.array_equal(ids.cpu().numpy(), ri)
        assert np.all(np.abs(f64(p) - rp) <= 3e-5 * rp)  # as in tests/test_serve.py


@gpu
@pytest.mark.parametrize("dt", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("lane", [0, 3, 7])
@pytest.mark.parametrize("small", [0, -80])
def test_route_order_of_many_tokens(lane, small, dt):
    """Orders below fp32's steps at 2050 tokens, at ordinary and (bf16, fp32) very small sizes."""
    banner(f"route order 2050 lane={lane} {dt}")
    T, D, E, k = 2050, 1024, 12, 5
    g = gen(lane)
    at = torch.arange(lane, D, 8)
    x, base = torch.zeros(T, D), torch.zeros(E, D)
    x[:, at] = torch.randn((T, at.numel()), generator=g)
    base[:, at] = torch.randn(at.numel(), generator=g)
    base[:, at[-1]] *= 1 + torch.arange(E).float()[torch.randperm(E, generator=g)] * 2.0 ** -6
    x[:, at[-1]] *= 2.0 ** -12
    x, wr = x.to(DT[dt]) * (1.0 if dt == "fp16" else 2.0 ** small), base.to(DT[dt])
    _, ids = m.moe_route(x.cuda(), wr.cuda(), k)
    assert np.array_equal(ids.cpu().numpy(), ref_route(f64(x), f64(wr), k, True)[0])
