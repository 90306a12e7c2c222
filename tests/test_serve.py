"""The few-token serving operators: router, mixture of experts, 4-bit weights.

References are plain fp64 on the CPU from the operators' definitions. Bounds,
fixed before the first run: a 16-bit result carries at most two roundings of half
a step each (A between the two products, the result), so its normalized L2 error over
the tensor, each row, each 32 x 32 block and each tile is at most eps =
2 * (eps / 2) of the type; one product alone (w4_linear) has one. fp32 sums add
less than 1e-5 of the operands' scale, the framework's bound in that mode.
"""

import numpy as np
import pytest
import torch

import backward_gate_up_amd as m
from backward_gate_up_amd import _lib
from tests._util import assert_local, banner, f64

gpu = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def bound(dtype, roundings):
    e = torch.finfo(dtype).eps / 2
    return 1e-5 if dtype == torch.float32 else roundings * e + 1e-5


def gen(seed):
    return torch.Generator().manual_seed(seed)


def randn(g, shape, std, dtype):
    return (torch.randn(shape, generator=g) * std).to(dtype)


# ---- definitions in fp64 --------------------------------------------------------


def ref_block(x, wg, wu, wd):
    g, u = x @ wg.T, x @ wu.T
    return (g / (1 + np.exp(-g)) * u) @ wd.T


def ref_route(x, wr, k, renorm):
    """ids and weights by a stable sort of the exact logits; also the logits."""
    with np.errstate(invalid="ignore"):
        l = x @ wr.T
        ids = np.argsort(-l, axis=1, kind="stable")[:, :k]
        p = np.exp(l - l.max(1, keepdims=True))
        p /= p.sum(1, keepdims=True)
        p = np.take_along_axis(p, ids, 1)
    return ids, p / p.sum(1, keepdims=True) if renorm else p


def ref_experts(x, p, ids, wg, wu, wd):
    y = np.zeros_like(x)
    E = wg.shape[0]
    for t in range(x.shape[0]):
        for j in range(ids.shape[1]):
            e = int(ids[t, j])
            if 0 <= e < E:
                y[t] += p[t, j] * ref_block(x[t:t + 1], wg[e], wu[e], wd[e])[0]
    return y


def ref_w4(codes, scales, zeros):
    c = codes.numpy().astype(np.int64)
    q = np.stack((c & 15, c >> 4), -1).reshape(*c.shape[:-1], -1).astype(np.float64)
    g = q.shape[-1] // scales.shape[-1]
    z = 8.0 if zeros is None else np.repeat(zeros.numpy().astype(np.float64), g, -1)
    return (q - z) * np.repeat(f64(scales), g, -1)


def make_w4(g, shape, group, zeros, dtype):
    """Random codes, scales and zero points, extremes among them."""
    *lead, K = shape
    codes = torch.randint(0, 256, (*lead, K // 2), generator=g, dtype=torch.uint8)
    codes[..., 0], codes[..., -1] = 0x0F, 0xF0
    scales = ((torch.rand((*lead, K // group), generator=g) + 0.5) / (4.6 * K ** 0.5)).to(dtype)
    z = torch.randint(0, 16, scales.shape, generator=g, dtype=torch.uint8) if zeros else None
    return codes, scales, z


def cuda(t):
    return tuple(cuda(v) for v in t) if isinstance(t, tuple) else t.cuda() if t is not None else None


# ---- CPU: refusals --------------------------------------------------------------


def test_host_tensors_and_bad_arguments_refused():
    bf = torch.bfloat16
    x, wr = torch.zeros(3, 64, dtype=bf), torch.zeros(4, 64, dtype=bf)
    wg, wd = torch.zeros(4, 32, 64, dtype=bf), torch.zeros(4, 64, 32, dtype=bf)
    p, ids = torch.zeros(3, 2), torch.zeros(3, 2, dtype=torch.int32)
    for call in (lambda: m.moe_route(x, wr, 2), lambda: m.moe_infer(x, wr, wg, wg, wd, 2),
                 lambda: m.moe_experts(x, p, ids, wg, wg, wd), lambda: m.w4_quantize(wr, 32),
                 lambda: m.w4_pack(torch.zeros(8, 32, dtype=torch.uint8), torch.zeros(8, 1, dtype=bf))):
        with pytest.raises(ValueError, match="GPU"):
            call()
    with pytest.raises(ValueError, match="router weight"):
        m.moe_route(x, wr[:, :32], 2)
    with pytest.raises(ValueError, match="share dtype"):
        m.moe_route(x, wr.float(), 2)
    with pytest.raises(ValueError, match="shape mismatch"):
        m.moe_experts(x, p, ids, wg, wg, wg)
    with pytest.raises(ValueError, match="Wg|weights"):
        m.moe_experts(x, p, ids, wg[0], wg, wd)
    with pytest.raises(RuntimeError, match="no backward"):
        m.moe_route(x.float().requires_grad_(), wr.float(), 2)
    with pytest.raises(RuntimeError, match="no backward"):
        m.moe_experts(x, p, ids, wg.requires_grad_(), wg, wd)


def test_w4_shapes_refused():
    for shape, group in (((8, 64), 16), ((8, 96), 64), ((12, 64), 32), ((64,), 32), ((8, 0), 32)):
        with pytest.raises(ValueError):
            m.serve._w4_shape(shape, group)
    assert m.serve._w4_shape((3, 8, 96), 32) == (3, 8, 96)


B = 1 << 40  # fake device addresses: validation fails before any use


def _w4(n, N=64, K=128, experts=1, group=32, zeros=0, data=None):
    return _lib.W4(B + (n << 34) if data is None else data, experts, N, K, group, zeros)


def _codes(L):
    import ctypes
    r = ctypes.byref
    at = [B + (i << 34) for i in range(10)]

    def route(X=at[0], W=at[1], P=at[2], I=at[3], T=4, D=64, E=8, k=2, dt=0, ws=at[9], n=1 << 30):
        return L.swiglu_mlp_moe_route(X, W, P, I, ws, n, T, D, E, k, 1, dt, None)

    def experts(X=at[0], P=at[1], I=at[2], Wg=at[3], Wu=at[4], Wd=at[5], Y=at[6], ws=at[7], n=1 << 30, T=4, D=64, H=128,
                E=8, k=2, dt=0):
        return L.swiglu_mlp_moe_experts(X, P, I, Wg, Wu, Wd, Y, ws, n, T, D, H, E, k, dt, None)

    def infer(Wr=at[8], **kw):
        a = dict(X=at[0], Wg=at[3], Wu=at[4], Wd=at[5], Y=at[6], ws=at[7], n=1 << 30, T=4, D=64, H=128, E=8, k=2, dt=0)
        a.update(kw)
        return L.swiglu_mlp_moe_infer(a["X"], Wr, a["Wg"], a["Wu"], a["Wd"], a["Y"], a["ws"], a["n"], a["T"], a["D"],
                                      a["H"], a["E"], a["k"], 1, a["dt"], None)

    def linear(w=None, X=at[0], Y=at[1], ws=None, n=0, T=4, dt=0):
        return L.swiglu_mlp_w4_linear(X, r(w or _w4(2)), Y, ws, n, T, dt, None)

    def block(wg=None, wu=None, wd=None, X=at[0], Y=at[1], ws=at[2], n=1 << 30, T=4, dt=0):
        return L.swiglu_mlp_w4_infer(X, r(wg or _w4(3)), r(wu or _w4(4)), r(wd or _w4(5, 128, 64)), Y, ws, n, T, dt, None)

    return at, route, experts, infer, linear, block


def test_host_validation_codes():
    L = _lib.lib()
    at, route, experts, infer, linear, block = _codes(L)
    for f in (route, experts, infer, linear, block):
        assert f(dt=7) == 3 and f(T=-1) == 2 and f(T=_lib.FEW_MAX_T + 1) == 2 and f(X=None) == 1 and f(X=at[0] + 8) == 4
        assert f() in (7, 8, 0) if not torch.cuda.is_available() else True
    for f in (route, experts, infer):
        assert f(D=60) == 2 and f(E=0) == 2 and f(E=1025) == 2 and f(k=0) == 2 and f(k=9) == 2 and f(E=64, k=33) == 2
    assert route(P=None) == 1 and route(P=at[2] + 2) == 4 and route(P=at[0] + 64) == 5 and route(I=at[2] + 4) == 5
    assert experts(H=4) == 2 and experts(I=None) == 1 and experts(P=at[1] + 1) == 4
    assert experts(ws=None, n=0) == 6 and experts(n=100) == 6 and experts(ws=at[7] + 8) == 4
    assert experts(Y=at[3] + 128) == 5 and experts(ws=at[6]) == 5 and experts(Y=at[2]) == 5 and infer(Y=at[8]) == 5
    assert infer(Wr=None) == 1
    assert linear(dt=2) == 3 and block(dt=2) == 3
    for bad in (_w4(2, group=48), _w4(2, K=100), _w4(2, N=12), _w4(2, experts=2), _w4(2, K=0)):
        assert linear(bad) == 2
    need = L.swiglu_mlp_w4_linear_workspace_bytes(32, 64, 4096, 0)
    assert need % (32 * 64 * 4) == 0 and need > 0 and L.swiglu_mlp_w4_linear_workspace_bytes(4, 64, 4096, 0) == 0
    long = _w4(2, 64, 4096)
    assert linear(long, T=32) == 6 and linear(long, T=32, ws=at[3], n=need - 1) == 6
    assert linear(long, T=32, ws=at[3] + 8, n=need) == 4 and linear(long, T=32, ws=at[1], n=need) == 5
    assert linear(_w4(2, data=0)) == 1 and linear(_w4(2, data=at[2] + 8)) == 4 and linear(Y=at[2] + 256) == 5
    assert block(wu=_w4(4, 128, 64)) == 2 and block(wd=_w4(5)) == 2 and block(wu=_w4(4, group=64)) == 2
    assert block(ws=None, n=0) == 6 and block(n=4 * 64 * 2 - 1) == 6
    # the queries
    ws = L.swiglu_mlp_moe_workspace_bytes
    assert ws(4, 64, 128, 8, 2, 0) >= 8 * 128 * 2 + 256 + 256 and ws(200, 65536, 128, 8, 2, 0) == 400 * 128 * 2 + 2 * 1792
    assert ws(0, 64, 128, 8, 2, 0) == 0 and ws(4, 64, 128, 64, 33, 0) == 0 and ws(4, 60, 128, 8, 2, 0) == 0
    rw = L.swiglu_mlp_moe_route_workspace_bytes
    assert rw(4, 64, 8, 0) == 4 * (4 * 8 + 8 + 4) and rw(1 << 14, 64, 8, 0) == 4 * ((1 << 14) * 9 + 8)
    assert rw(4, 60, 8, 0) == 0 and rw(0, 64, 8, 0) == 0
    assert route(ws=None, n=0) == 6 and route(n=100) == 6 and route(ws=at[9] + 4) == 4 and route(ws=at[2]) == 5
    assert L.swiglu_mlp_w4_bytes(1, 64, 128, 32, 0) == 4 * (1024 + 16 * 4 * 2)
    assert L.swiglu_mlp_w4_bytes(1, 64, 128, 32, 1) == 4 * (1024 + 16 * 4 * 2 + 32)
    assert L.swiglu_mlp_w4_bytes(1, 64, 100, 32, 0) == 0


# ---- router ---------------------------------------------------------------------


@gpu
@pytest.mark.parametrize("dt", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("T,E,k,D", [(1, 8, 2, 1024), (1, 64, 8, 2048), (5, 3, 3, 8), (16, 130, 7, 136), (17, 1, 1, 64),
                                     (33, 128, 8, 1000), (100, 1024, 32, 256), (1000, 60, 4, 520), (0, 8, 2, 64),
                                     (1030, 64, 8, 264), (1100, 129, 3, 72), (1025, 256, 2, 1000)])
@pytest.mark.parametrize("renorm", [True, False])
def test_route(T, E, k, D, dt, renorm):
    banner(f"route {dt} T={T} E={E} k={k} D={D} renorm={renorm}")
    g = gen(T + E)
    x, wr = randn(g, (T, D), 1, DT[dt]), randn(g, (E, D), D ** -0.5, DT[dt])
    p, ids = m.moe_route(x.cuda(), wr.cuda(), k, renorm)
    ri, rp = ref_route(f64(x), f64(wr), k, renorm)
    assert np.array_equal(ids.cpu().numpy(), ri)
    # a logit is off by at most about D 2^-24 of sum |x w| < 1e-5 here; a weight by twice that, relatively
    assert np.all(np.abs(f64(p) - rp) <= 3e-5 * rp)


@gpu
@pytest.mark.parametrize("dt", ["bf16", "fp16", "fp32"])
def test_route_ties_and_near_ties(dt):
    banner(f"route ties {dt}")
    D, E, k = 512, 40, 6
    g = gen(3)
    x = randn(g, (24, D), 1, DT[dt])
    x[5] = 0                                  # every logit equal
    wr = randn(g, (E, D), D ** -0.5, DT[dt])
    wr[7] = wr[3]                             # exact ties
    wr[31] = wr[3]
    for e in (11, 12, 13, 14):                # differ in one element by one step: below fp32 sums
        wr[e] = wr[10]
        j = 17 * e % D
        wr[e, j] = torch.nextafter(wr[e, j].float(), torch.tensor(2.0)).to(DT[dt]) if dt == "fp32" else \
            wr[e, j] * (1 + torch.finfo(DT[dt]).eps)
    x[:, :8] *= 30                            # large cancelling parts
    wr[:, 4:8] = -wr[:, :4]
    x[:, 4:8] = x[:, :4]
    p, ids = m.moe_route(x.cuda(), wr.cuda(), k)
    ri, rp = ref_route(f64(x), f64(wr), k, True)
    # the fp64 sums are exact to about 1e-13; order by index inside that
    l = f64(x) @ f64(wr).T
    for t in range(x.shape[0]):
        got = ids[t].tolist()
        assert len(set(got)) == k
        for a, b in zip(got, ri[t]):
            assert a == b or abs(l[t, a] - l[t, b]) < 1e-12, (t, got, ri[t])
    assert ids[5].tolist() == list(range(k))
    assert np.allclose(f64(p).sum(1), 1, atol=1e-6)


@gpu
@pytest.mark.parametrize("dt", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("lane", [0, 1, 2, 5, 7])
@pytest.mark.parametrize("T", [12, 600])
def test_route_order_below_fp32(T, lane, dt):
    """Experts that differ in the last digits of a long sum: only exact logits
    give their order. The data sits in one element of every eight, so that each
    part of a 16-byte chunk has to count in the bound that asks for them."""
    banner(f"route order T={T} lane={lane} {dt}")
    D, E, k = 4096, 12, 5
    g = gen(lane)
    at = torch.arange(lane, D, 8)
    x, base = torch.zeros(T, D), torch.zeros(E, D)
    x[:, at] = torch.randn((T, at.numel()), generator=g)
    base[:, at] = torch.randn(at.numel(), generator=g)
    base[:, at[-1]] *= 1 + torch.arange(E).float()[torch.randperm(E, generator=g)] * 2.0 ** -6
    x[:, at[-1]] *= 2.0 ** -12
    x, wr = x.to(DT[dt]), base.to(DT[dt])
    _, ids = m.moe_route(x.cuda(), wr.cuda(), k)
    assert np.array_equal(ids.cpu().numpy(), ref_route(f64(x), f64(wr), k, True)[0])


@gpu
def test_route_nonfinite_tokens_stay_in_range():
    banner("route NaN / Inf")
    g = gen(4)
    x, wr = randn(g, (20, 256), 1, torch.bfloat16), randn(g, (16, 256), 1 / 16, torch.bfloat16)
    clean = m.moe_route(x.cuda(), wr.cuda(), 4)
    y = x.clone()
    y[3, 7], y[9, 0], y[10] = float("nan"), float("inf"), float("nan")
    p, ids = m.moe_route(y.cuda(), wr.cuda(), 4)
    ids = ids.cpu()
    assert ((ids >= 0) & (ids < 16)).all() and all(len(set(r.tolist())) == 4 for r in ids)
    rest = [t for t in range(20) if t not in (3, 9, 10)]
    assert torch.equal(p.cpu()[rest], clean[0].cpu()[rest]) and torch.equal(ids[rest], clean[1].cpu()[rest])
    assert p[10].isnan().all() and p[3].isnan().all()


# ---- experts --------------------------------------------------------------------


def expert_weights(g, E, D, H, dtype):
    return (randn(g, (E, H, D), D ** -0.5, dtype), randn(g, (E, H, D), D ** -0.5, dtype),
            randn(g, (E, D, H), H ** -0.5, dtype))


SHAPES = [(40, 2, 1, 1000, 328), (64, 4, 2, 64, 6200), (1, 8, 2, 128, 256), (1, 6, 6, 1000, 712), (2, 4, 1, 8, 8), (16, 16, 4, 264, 40), (17, 5, 3, 96, 72),
          (64, 4, 2, 256, 136), (65, 9, 2, 64, 200), (130, 3, 2, 72, 64), (9, 1, 1, 512, 1024), (3, 200, 8, 64, 64)]


@gpu
@pytest.mark.parametrize("dt", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("T,E,k,D,H", SHAPES)
def test_moe(T, E, k, D, H, dt):
    banner(f"moe {dt} T={T} E={E} k={k} D={D} H={H}")
    g = gen(T * E + D)
    x, wr = randn(g, (T, D), 1, DT[dt]), randn(g, (E, D), D ** -0.5, DT[dt])
    w = expert_weights(g, E, D, H, DT[dt])
    ri, rp = ref_route(f64(x), f64(wr), k, True)
    ref = ref_experts(f64(x), rp, ri, *map(f64, w))
    y = m.moe_infer(x.cuda(), wr.cuda(), *cuda(w), k)
    assert_local(f64(y), ref, bound(DT[dt], 2), ("moe", dt, T))
    p, ids = m.moe_route(x.cuda(), wr.cuda(), k)
    assert torch.equal(m.moe_experts(x.cuda(), p, ids, *cuda(w)), y)


@gpu
@pytest.mark.parametrize("T,k,E", [(40, 3, 8), (64, 1, 4), (70, 2, 2), (16, 4, 6), (30, 2, 80), (64, 2, 24), (40, 1, 30),
                                   (64, 8, 100)])
def test_experts_choices(T, k, E):
    """One expert taking every token, dropped ids, a token without a choice,
    one expert chosen twice by a token, zero weights."""
    banner(f"choices T={T} k={k} E={E}")
    D, H, dt = 160, 96, torch.bfloat16
    g = gen(T)
    x, w = randn(g, (T, D), 1, dt), expert_weights(g, E, D, H, dt)
    raw = [make_w4(g, s, 32, False, dt) for s in ((E, H, D), (E, H, D), (E, D, H))]
    w4 = [ref_w4(*r) for r in raw]
    p = torch.rand((T, k), generator=g)
    for kind in ("one", "drop", "twice", "none"):
        ids = torch.randint(0, E, (T, k), generator=g, dtype=torch.int32)
        q = p.clone()
        if kind == "one":
            ids[:, 0] = 1
        elif kind == "drop":
            ids[torch.rand((T, k), generator=g) < 0.5] = -1
            ids[0], ids[1], ids[2] = -1, E, 1 << 30
        elif kind == "twice":
            ids[:] = ids[:, :1]
            q[3] = 0
        else:
            ids[:] = -1
        y = m.moe_experts(x.cuda(), q.cuda(), ids.cuda(), *cuda(w))
        ref = ref_experts(f64(x), f64(q), ids.numpy(), *map(f64, w))
        assert_local(f64(y), ref, bound(dt, 2), (kind, T, k))
        y4 = m.moe_experts(x.cuda(), q.cuda(), ids.cuda(), *(m.w4_pack(*cuda(r)) for r in raw))
        assert_local(f64(y4), ref_experts(f64(x), f64(q), ids.numpy(), *w4), bound(dt, 2), (kind, "4 bits", T, k))
        empty = ((ids < 0) | (ids >= E)).all(1)
        assert not f64(y)[empty.numpy()].any()
        assert torch.equal(y, m.moe_experts(x.cuda(), q.cuda(), ids.cuda(), *cuda(w)))  # fixed order of sums


@gpu
@pytest.mark.parametrize("w4", [False, True])
def test_nonfinite_values_stay_where_they_belong(w4):
    """NaN in one token reaches only that token, NaN and Inf in an expert only
    the tokens that chose it, also across the padding of rows and of K."""
    banner(f"non-finite w4={w4}")
    T, E, k, D, H, dt = 24, 5, 2, 160, 96, torch.bfloat16
    g = gen(8)
    x = randn(g, (T, D), 1, dt)
    ids = torch.stack([torch.randperm(E - 1, generator=g)[:k] for _ in range(T)]).int()
    ids[4, 1] = E - 1
    p = torch.rand((T, k), generator=g) + 0.1
    if w4:
        raw = [make_w4(g, s, 32, True, dt) for s in ((E, H, D), (E, H, D), (E, D, H))]
        bad = [tuple(t.clone() if t is not None else None for t in r) for r in raw]
        bad[0][1][E - 1], bad[2][1][E - 1] = float("nan"), float("inf")
        w, b = [m.w4_pack(*cuda(r)) for r in raw], [m.w4_pack(*cuda(r)) for r in bad]
    else:
        w = cuda(expert_weights(g, E, D, H, dt))
        b = tuple(t.clone() for t in w)
        b[0][E - 1], b[2][E - 1] = float("nan"), float("inf")
    y = m.moe_experts(x.cuda(), p.cuda(), ids.cuda(), *w)
    yb = m.moe_experts(x.cuda(), p.cuda(), ids.cuda(), *b)
    rest = [t for t in range(T) if t != 4]
    assert torch.equal(y[rest], yb[rest]) and not yb[4].isfinite().all()
    x2 = x.clone()
    x2[9] = float("nan")
    x2[11, 0] = float("inf")
    y2 = m.moe_experts(x2.cuda(), p.cuda(), ids.cuda(), *w)
    rest = [t for t in range(T) if t not in (9, 11)]
    assert torch.equal(y[rest], y2[rest]) and y2[9].isnan().all()


# ---- 4-bit weights ----------------------------------------------------------------


@gpu
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("shape,group", [((8, 32), 32), ((40, 160), 32), ((24, 192), 64), ((3, 16, 128), 128),
                                         ((2, 1000, 384), 128)])
def test_w4_pack_round_trip(shape, group, zeros, dt):
    banner(f"pack {dt} {shape} g={group} zeros={zeros}")
    raw = make_w4(gen(1), shape, group, zeros, DT[dt])
    w = m.w4_pack(*cuda(raw))
    assert w.shape == shape and w.group == group and w.has_zeros == zeros
    # scale * integer is rounded once: the correctly rounded value
    ref = torch.from_numpy(ref_w4(*raw)).float().to(DT[dt])
    assert torch.equal(w.dequantize().cpu(), ref)


@gpu
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_w4_quantize(group, zeros, dt):
    banner(f"quantize {dt} g={group} zeros={zeros}")
    w = randn(gen(2), (3, 24, 384), 0.05, DT[dt])
    w[1, 3] = 0
    w[2, 5, :group] = w[2, 5, :group].abs()
    codes, scales, zp = m.w4_quantize(w.cuda(), group, zeros)
    v = f64(w).reshape(3, 24, -1, group)
    lo, hi = np.minimum(v.min(-1), 0), np.maximum(v.max(-1), 0)
    want = (hi - lo) / 15 if zeros else np.maximum(hi, -lo) / 7.5
    # one fp32 division and one rounding to the type
    assert np.all(np.abs(f64(scales) - want) <= want * (torch.finfo(DT[dt]).eps / 2 + 1e-6))
    back = ref_w4(codes.cpu(), scales.cpu(), zp.cpu() if zeros else None).reshape(v.shape)
    # nearest code: half a step, plus the clamp's excess where the rounded scale or zero falls short
    s = f64(scales)[..., None]
    assert np.all(np.abs(back - v) <= s * (1.0 if zeros else 0.55) + 1e-12)
    assert np.abs(back - v).mean() <= 0.3 * s.mean()
    assert not back[1, 3].any()


@gpu
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("T,N,K,group", [(1, 8, 32, 32), (1, 4096, 512, 128), (2, 40, 160, 32), (16, 1000, 192, 64),
                                         (17, 264, 1152, 128), (33, 128, 2816, 64), (64, 72, 416, 32), (65, 16, 128, 128),
                                         (200, 24, 96, 32), (0, 16, 64, 32), (20, 104, 2112, 32), (48, 320, 4992, 64),
                                         (70, 136, 1536, 128)])
def test_w4_linear(T, N, K, group, zeros, dt):
    banner(f"w4_linear {dt} T={T} N={N} K={K} g={group} zeros={zeros}")
    g = gen(N + K)
    raw = make_w4(g, (N, K), group, zeros, DT[dt])
    x = randn(g, (T, K), 1, DT[dt])
    y = m.w4_linear(x.cuda(), m.w4_pack(*cuda(raw)))
    assert_local(f64(y), f64(x) @ ref_w4(*raw).T, bound(DT[dt], 1), ("w4", dt, T, N, K))


@gpu
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_w4_offset_sums_keep_their_digits(dt):
    """Tokens with a large common part: the codes' offset must cancel in fp32
    (bound: the result's half step, and OFF + 15 < 144 fp32 roundings of the
    sum of |x| per group of 128 for the offset, at most 128 * 2^-24 each)."""
    banner(f"offset {dt}")
    g = gen(6)
    raw = make_w4(g, (64, 1024), 128, False, DT[dt])
    x = (torch.randn((4, 1024), generator=g) + 20).to(DT[dt])
    y = m.w4_linear(x.cuda(), m.w4_pack(*cuda(raw)))
    w = ref_w4(*raw)
    ref = f64(x) @ w.T
    slack = 144 * 128 * 2.0 ** -24 * (np.abs(f64(x)) @ np.repeat(f64(raw[1]), 128, 1).T)
    assert np.all(np.abs(f64(y) - ref) <= torch.finfo(DT[dt]).eps / 2 * np.abs(ref) + slack)


@gpu
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("T,D,H,group,zeros", [(1, 256, 512, 128, False), (5, 160, 96, 32, True), (16, 1024, 704, 64, False),
                                               (40, 128, 1408, 128, True), (70, 64, 64, 64, False),
                                               (20, 256, 1088, 32, True), (40, 64, 12416, 64, False)])
def test_infer_w4(T, D, H, group, zeros, dt):
    banner(f"infer_w4 {dt} T={T} D={D} H={H} g={group} zeros={zeros}")
    g = gen(D + H)
    raw = [make_w4(g, s, group, zeros, DT[dt]) for s in ((H, D), (H, D), (D, H))]
    x = randn(g, (T, D), 1, DT[dt])
    w = [m.w4_pack(*cuda(r)) for r in raw]
    y = m.infer_w4(x.cuda(), *w)
    assert_local(f64(y), ref_block(f64(x), *(ref_w4(*r) for r in raw)), bound(DT[dt], 2), ("w4 mlp", dt, T))


@gpu
@pytest.mark.parametrize("T,E,k,D,H,group,zeros", [(1, 8, 2, 128, 256, 128, False), (7, 12, 4, 96, 160, 32, True),
                                                   (40, 3, 2, 320, 64, 64, False), (64, 2, 2, 128, 128, 128, True),
                                                   (40, 64, 1, 128, 96, 32, False), (60, 20, 2, 256, 128, 64, True),
                                                   (60, 12, 2, 128, 384, 128, False)])
def test_moe_w4(T, E, k, D, H, group, zeros):
    banner(f"moe_w4 T={T} E={E} k={k} D={D} H={H} g={group} zeros={zeros}")
    g = gen(D * E)
    dt = torch.bfloat16
    raw = [make_w4(g, s, group, zeros, dt) for s in ((E, H, D), (E, H, D), (E, D, H))]
    x, wr = randn(g, (T, D), 1, dt), randn(g, (E, D), D ** -0.5, dt)
    y = m.moe_infer(x.cuda(), wr.cuda(), *(m.w4_pack(*cuda(r)) for r in raw), k, False)
    ri, rp = ref_route(f64(x), f64(wr), k, False)
    assert_local(f64(y), ref_experts(f64(x), rp, ri, *(ref_w4(*r) for r in raw)), bound(dt, 2), ("moe w4", T))


# ---- how they are called ------------------------------------------------------------


@gpu
def test_strides_streams_buffers_and_graph():
    banner("strides, streams, graph")
    T, E, k, D, H, dt = 20, 8, 2, 256, 128, torch.bfloat16
    g = gen(12)
    x, wr, w = randn(g, (T, D), 1, dt).cuda(), randn(g, (E, D), 1 / 16, dt).cuda(), cuda(expert_weights(g, E, D, H, dt))
    y = m.moe_infer(x, wr, *w, k)
    # strided and offset inputs
    xs = torch.empty((T, 2 * D), dtype=dt, device="cuda")[:, ::2].copy_(x)
    ws = tuple(t.transpose(1, 2).contiguous().transpose(1, 2) for t in w)
    assert torch.equal(m.moe_infer(xs, wr, *ws, k), y)
    assert torch.equal(m.moe_infer(torch.cat([x[:1], x])[1:], wr, *w, k), y)
    p, ids = m.moe_route(x, wr, k)
    assert torch.equal(m.moe_experts(x[3:], p[3:], ids[3:], *w), y[3:])
    # another stream, with the caller's own buffers
    out = torch.empty_like(y)
    need = _lib.lib().swiglu_mlp_moe_workspace_bytes(T, D, H, E, k, 0)
    buf = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        m.moe_infer(x, wr, *w, k, y=out, workspace=buf)
    s.synchronize()
    assert torch.equal(out, y)
    with pytest.raises(ValueError, match="shape"):
        m.moe_infer(x, wr, *w, k, y=out[:3])
    with pytest.raises(m.SwiGLUError, match="WORKSPACE"):
        m.moe_infer(x, wr, *w, k, workspace=buf[:256])
    # captured, replayed with other inputs
    w4 = [m.W4Weight.quantize(t, 64, True) for t in w]
    graph = torch.cuda.CUDAGraph()
    out4, buf4 = torch.empty_like(y), buf.clone()
    m.moe_infer(x, wr, *w4, k, y=out4, workspace=buf4)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        m.moe_infer(x, wr, *w, k, y=out, workspace=buf)
        m.moe_infer(x, wr, *w4, k, y=out4, workspace=buf4)
    for seed in range(4):
        x.copy_(randn(gen(seed), (T, D), 1, dt))
        graph.replay()
        float(torch.randn(1 << 18, device="cuda").square().sum())
        torch.cuda.synchronize()
        assert torch.equal(out, m.moe_infer(x, wr, *w, k)) and torch.equal(out4, m.moe_infer(x, wr, *w4, k))


# ---- modules and the example --------------------------------------------------------


def _moe_config(**kw):
    from types import SimpleNamespace

    return SimpleNamespace(**{**dict(hidden_size=64, moe_intermediate_size=96, num_experts=6, num_experts_per_tok=2), **kw})


def test_modules_on_the_host():
    mod = m.SwiGLUMoE(_moe_config(norm_topk_prob=False))
    assert mod.gate.weight.shape == (6, 64) and mod.gate_proj.shape == (6, 96, 64) and mod.down_proj.shape == (6, 64, 96)
    assert mod.top_k == 2 and not mod.renormalize
    assert set(mod.state_dict()) == {"gate.weight", "gate_proj", "up_proj", "down_proj"}
    with pytest.raises(ValueError, match="hidden_act"):
        m.SwiGLUMoE(_moe_config(hidden_act="gelu"))
    from types import SimpleNamespace

    blocks = [m.SwiGLUMLP(SimpleNamespace(hidden_size=64, intermediate_size=96)) for _ in range(6)]
    stacked = m.SwiGLUMoE.from_experts(torch.nn.Linear(64, 6, bias=False), blocks, 2)
    assert torch.equal(stacked.up_proj[3], blocks[3].up_proj.weight) and stacked.down_proj.shape == (6, 64, 96)
    with pytest.raises(ValueError, match="bias"):
        m.SwiGLUMoE.from_experts(torch.nn.Linear(64, 6), blocks, 2)
    with pytest.raises(ValueError, match="experts"):
        m.SwiGLUMoE.from_experts(torch.nn.Linear(64, 5, bias=False), blocks, 2)
    with torch.no_grad(), pytest.raises(ValueError, match="GPU"):
        mod(torch.zeros(2, 3, 64))
    with pytest.raises(RuntimeError, match="no backward"):
        mod(torch.zeros(2, 3, 64))


@gpu
def test_modules():
    banner("modules")
    dt = torch.bfloat16
    torch.manual_seed(1)
    mod = m.SwiGLUMoE(_moe_config(hidden_size=128, moe_intermediate_size=160)).to("cuda", dt)
    x = randn(gen(5), (3, 5, 128), 1, dt).cuda()
    with torch.no_grad():
        y = mod(x)
        assert y.shape == x.shape
        args = [mod.gate.weight, mod.gate_proj, mod.up_proj, mod.down_proj]
        assert torch.equal(y.view(15, 128), m.moe_infer(x.view(15, 128), *args, 2))
        w = [m.W4Weight.quantize(t, 32, True) for t in args[1:]]
        y4 = mod.quantize_(32, True)(x)
        assert torch.equal(y4.view(15, 128), m.moe_infer(x.view(15, 128), args[0], *w, 2))
        assert set(mod.state_dict()) == {"gate.weight", "gate_proj", "up_proj", "down_proj"}
        # the buffers may be replaced (a load, another device): the next call takes the new ones
        old = mod.gate_proj
        mod.gate_proj = old.clone()
        old.zero_()
        assert torch.equal(mod(x), y4)
        # the dense block: few tokens on the 4-bit kernels, many on rows
        from types import SimpleNamespace

        mlp = m.SwiGLUMLP(SimpleNamespace(hidden_size=128, intermediate_size=256)).to("cuda", dt)
        q = m.SwiGLUMLPW4(mlp, 64, long_tokens=40)
        rows = [q._weight(n).dequantize() for n in ("gate_proj", "up_proj", "down_proj")]
        ref = ref_block(f64(x.view(15, 128)), *map(f64, rows))
        # the rows are the 4-bit weights rounded once more: half a step of each of two products' weights
        assert_local(f64(q(x).view(15, 128)), ref, bound(dt, 4), "dense 4 bits")
        long = randn(gen(6), (50, 128), 1, dt).cuda()
        assert torch.equal(q(long), m.infer(long, *rows, linear=True))


@gpu
def test_example(monkeypatch, capsys):
    banner("example")
    import importlib.util
    import os
    import sys

    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "serve_moe.py")
    spec = importlib.util.spec_from_file_location("serve_moe", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    monkeypatch.setattr(sys, "argv", ["serve_moe.py", "--experts", "12", "--top-k", "3", "--dim", "256", "--hidden", "128",
                                      "--steps", "3"])
    # a code's step is max|w| / 7.5, about 0.36 of the weights' deviation in groups of 128, its rounding
    # 0.10 of it; the three weights' together about 0.18 of the output's norm
    assert 0.1 < mod.main() < 0.25
