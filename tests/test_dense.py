"""Norms, the linear layer and FeedForward against plain formulas in 64 bits (GPU),
and their refusals (CPU).

Tolerances, derived before the first run. h = finfo.eps / 2 is a rounding to the
storage type, u = 2^-24 one in fp32.

Norms: a sum over a row passes through at most 32 terms per lane, D / 1024 more in
the widest rows, 6 steps of the wave and 16 of the waves: G = 72 + D / 1024
roundings. So the mean is off by G u mean|x|, n by en = rstd G u mean|x| + (G +
16) u |n|, and y by its own rounding and |w| en. dx = rstd (g - level - n along)
collects the errors of level (G u mean|g|) and of along; a column sum over rows
passes through at most T / 256 + 64 terms.

Products: a 16x16x32 (32x32x16) matrix instruction counts as 8 fp32 roundings of
its sum of magnitudes, the fp32 ones as one per term: C u sum|x||w| with C = K / 4 +
64 or K + 64. Activations have slopes below 1.2 and are evaluated to 2e-5 (16
bits) or 1e-5 of their value, their slopes to 3e-5 or 1e-5. dz is rounded to the
storage type before the products: at worst h sum|dz||w|. Besides these worst
cases, normalized L2 of every output, row and block within the package's bounds
(1e-2 and 1e-5).
"""

import copy
import ctypes
import math

import pytest
import torch

import backward_gate_up_amd as mlp
from backward_gate_up_amd import _lib, dense
from tests._util import FMT, TOL, banner

U = 2.0 ** -24
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
ACTS = [None, "relu", "gelu", "gelu_tanh", "silu"]
DEV = "cuda:0"


def gen(seed):
    return torch.Generator().manual_seed(seed)


def normal(g, shape, dtype, scale=1.0, shift=0.0):
    return (torch.randn(shape, generator=g) * scale + shift).to(dtype).to(DEV)


def half(dtype):
    return torch.finfo(dtype).eps / 2


def tiny(dtype):
    """Half of the smallest step: what a rounding may be off near zero."""
    return torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps / 2


def inside(got, ref, tol, what):
    off = (got.double() - ref).abs()
    bad = ~(off <= tol + tiny(got.dtype))
    assert not bad.any(), (what, int(bad.sum()), float((off / (tol + 1e-300)).max()), bad.nonzero()[:4].tolist())


def near(got, ref, what):
    """Normalized L2 of the whole, of every row, 32 x 32 block and 256 x 256 tile, as
    tests/_util.py's assert_local has them, on the GPU."""
    if ref.numel() == 0:
        return
    tol = TOL[FMT[got.dtype]]
    diff, ref = (got.double() - ref) ** 2, ref ** 2
    floor = ref.mean()
    assert (diff.sum() / ref.sum()).sqrt() <= tol, (what, "whole")
    for m, n in ((1, ref.shape[1]), (32, 32), (256, 256)):
        pad = lambda t: torch.nn.functional.pad(t, (0, -t.shape[1] % n, 0, -t.shape[0] % m))  # noqa: E731
        total = lambda t: pad(t).unflatten(1, (-1, n)).unflatten(0, (-1, m)).sum((1, 3))  # noqa: E731
        count = total(torch.ones_like(ref))
        err = (total(diff) / count).sqrt() / torch.maximum(total(ref) / count, floor).sqrt()
        assert (err <= tol).all(), (what, (m, n), float(err.max()), (err == err.max()).nonzero()[0].tolist())


# ---- norms ----------------------------------------------------------------------


def norm_reference(x, w, b, eps, rms, dy=None, dres=None):
    """(y, tolerance) and, with dy, the same of dx, dw, db."""
    dt, T, D = x.dtype, *x.shape
    h, G = half(dt), 72 + D / 1024
    x, w = x.double(), w.double()
    b = torch.zeros_like(w) if b is None else b.double()
    mean = torch.zeros_like(x[:, :1]) if rms else x.mean(1, keepdim=True)
    rstd = 1 / torch.sqrt(((x - mean) ** 2).mean(1, keepdim=True) + eps)
    n = (x - mean) * rstd
    en = rstd * G * U * x.abs().mean(1, keepdim=True) + (G + 16) * U * n.abs()
    y = n * w + b
    out = [(y, h * y.abs() + w.abs() * en + 4 * U * ((n * w).abs() + b.abs()))]
    if dy is None:
        return out
    dy = dy.double()
    g = dy * w
    along = (g * n).mean(1, keepdim=True)
    level = torch.zeros_like(along) if rms else g.mean(1, keepdim=True)
    dx = rstd * (g - level - n * along)
    e_level = (G + 4) * U * g.abs().mean(1, keepdim=True)
    e_along = (G + 4) * U * (g * n).abs().mean(1, keepdim=True) + (g.abs() * en).mean(1, keepdim=True)
    tol = rstd * (e_level + n.abs() * e_along + en * along.abs() + 8 * U * (g.abs() + level.abs() + (n * along).abs()))
    tol = tol + (G + 16) * U * dx.abs()
    if dres is not None:
        dx = dx + dres.double()
    out.append((dx, h * dx.abs() + tol + U * dx.abs()))
    C = T / 256 + 64
    dw, db = (dy * n).sum(0), dy.sum(0)
    out.append((dw, h * dw.abs() + (C * U * dy.abs() * n.abs() + dy.abs() * en).sum(0)))
    out.append((db, h * db.abs() + C * U * dy.abs().sum(0)))
    return out


NORM_SHAPES = [
    (1, 1), (5, 3), (1, 8), (3, 64), (130, 100), (777, 256), (2, 511), (64, 512), (5, 1000), (700, 1001), (1, 2048), (9, 2047),
    (33, 2056), (7, 4095), (300, 4096), (1, 4100), (3, 8192), (5, 8191), (2, 11008), (33, 12345), (4, 16384), (2, 16392),
    (3, 40001), (0, 64),
]


@pytest.mark.gpu
@pytest.mark.parametrize("rms", [False, True], ids=["layer", "rms"])
@pytest.mark.parametrize("dtype", list(DTYPES))
def test_norm(dtype, rms):
    dt = DTYPES[dtype]
    for i, (T, D) in enumerate(NORM_SHAPES):
        banner(f"norm {dtype} rms={rms} T={T} D={D}")
        g = gen(100 + i)
        x = normal(g, (T, D), dt, 1.0, 3.0 if i % 2 else 0.3)
        w, b = normal(g, (D,), dt, 0.2, 1.0), normal(g, (D,), dt, 0.3)
        dy, dres = normal(g, (T, D), dt), normal(g, (T, D), dt) if i % 3 == 0 else None
        bias = b if not rms and i % 4 else None
        eps = (1e-5, 1e-6, 1e-2)[i % 3]
        y, stats = mlp.norm_fwd(x, w, bias, eps, rms)
        assert torch.equal(y, mlp.norm_fwd(x, w, bias, eps, rms, stats=False)[0])
        dx, dw, db = mlp.norm_bwd(dy, x, w, stats, rms, bias is not None, dres)
        ref = norm_reference(x, w, bias, eps, rms, dy, dres)
        for name, got, (r, tol) in zip(("y", "dx", "dw", "db"), (y, dx, dw, db), ref):
            if got is not None:
                inside(got, r, tol, (name, T, D))
        assert (db is None) == (bias is None)
        again = mlp.norm_bwd(dy, x, w, stats, rms, bias is not None, dres)
        assert all(a is None or torch.equal(a, c) for a, c in zip(again, (dx, dw, db)))


@pytest.mark.gpu
@pytest.mark.parametrize("T,D,rms", [(257, 100, False), (300, 511, True), (300, 1000, False), (260, 1001, True), (400, 2047, False),
                                     (300, 4100, False), (290, 8191, True), (270, 8192, False), (280, 11008, False),
                                     (300, 12345, True), (261, 16392, False), (258, 40001, False), (70000, 64, True), (20000, 300, False), (5000, 2048, False), (3000, 4096, True),
                                     (2500, 9000, False)])
def test_norm_of_many_rows(T, D, rms):
    """Every workgroup walks several rows, the last of them fewer."""
    banner(f"norm many rows T={T} D={D}")
    g = gen(T)
    x, w, b, dy = normal(g, (T, D), torch.bfloat16, 1.0, 0.5), normal(g, (D,), torch.bfloat16), normal(g, (D,), torch.bfloat16), \
        normal(g, (T, D), torch.bfloat16)
    b = None if rms else b
    y, stats = mlp.norm_fwd(x, w, b, 1e-5, rms)
    got = (y, *mlp.norm_bwd(dy, x, w, stats, rms, not rms))
    for name, a, (r, tol) in zip(("y", "dx", "dw", "db"), got, norm_reference(x, w, b, 1e-5, rms, dy)):
        if a is not None:
            inside(a, r, tol, name)


@pytest.mark.gpu
@pytest.mark.parametrize("rms", [False, True], ids=["layer", "rms"])
@pytest.mark.parametrize("dtype", list(DTYPES))
def test_norm_every_width(dtype, rms):
    """More rows than one launch's gradient takes, at widths for each number of waves
    and pieces, whole and odd."""
    dt = DTYPES[dtype]
    for i, D in enumerate((512, 1000, 2048, 4096, 8192, 16384, 16392, 511, 701, 1001, 2047, 4095, 8191, 12345, 40001)):
        D = D if dt != torch.float32 else D // 2
        T = 257 + 13 * i % 50
        banner(f"norm width {dtype} rms={rms} T={T} D={D}")
        g = gen(300 + i)
        x, w, dy = normal(g, (T, D), dt, 1.0, 0.5), normal(g, (D,), dt, 0.2, 1.0), normal(g, (T, D), dt)
        b, dres = None if rms else normal(g, (D,), dt), normal(g, (T, D), dt) if i % 2 else None
        y, stats = mlp.norm_fwd(x, w, b, 1e-5, rms)
        got = (y, *mlp.norm_bwd(dy, x, w, stats, rms, not rms, dres))
        for name, a, (r, tol) in zip(("y", "dx", "dw", "db"), got, norm_reference(x, w, b, 1e-5, rms, dy, dres)):
            if a is not None:
                inside(a, r, tol, (name, T, D))


@pytest.mark.gpu
def test_norm_large_offset_and_constant_rows():
    """The variance is that of the differences: a mean a thousand times the spread
    costs only its own rounding. A constant row is the bias."""
    banner("norm large offset")
    x = normal(gen(1), (40, 1024), torch.float32, 1.0, 1000.0)
    w, b = normal(gen(2), (1024,), torch.float32), normal(gen(3), (1024,), torch.float32)
    (ref, tol), = norm_reference(x, w, b, 1e-5, False)
    inside(mlp.layer_norm(x, w, b), ref, tol, "offset")
    c = torch.full((3, 1024), 2.5, device=DEV)
    assert torch.equal(mlp.layer_norm(c, w, b), b.expand(3, -1))
    assert torch.equal(mlp.rms_norm(torch.zeros_like(c), w), torch.zeros_like(c))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(DTYPES))
def test_norm_nan_and_infinity_stay_in_their_row(dtype):
    banner(f"norm nan {dtype}")
    dt = DTYPES[dtype]
    for D in (100, 4096, 20000):
        x = normal(gen(D), (5, D), dt)
        w, b = normal(gen(4), (D,), dt), normal(gen(5), (D,), dt)
        dy = normal(gen(6), (5, D), dt)
        clean, stats = mlp.norm_fwd(x, w, b)
        cdx = mlp.norm_bwd(dy, x, w, stats)[0]
        x[1, D // 2], x[3, 0] = math.nan, math.inf
        y, stats = mlp.norm_fwd(x, w, b)
        dx = mlp.norm_bwd(dy, x, w, stats)[0]
        for r in (0, 2, 4):
            assert torch.equal(y[r], clean[r]) and torch.equal(dx[r], cdx[r])
        assert y[1].isnan().all() and dx[1].isnan().all() and y[3, 0].isnan()


@pytest.mark.gpu
def test_norm_reads_and_writes_nothing_beyond_its_rows():
    """Rows that start at any element, in the middle of a larger buffer."""
    banner("norm unaligned")
    for dt in DTYPES.values():
        for T, D, off in ((3, 1001, 1), (2, 8, 3), (5, 250, 1), (1, 4099, 5), (300, 77, 3)):
            room = torch.full((T * D + 64,), 7.0, dtype=dt, device=DEV)
            x = room[off:off + T * D].view(T, D)
            x.copy_(normal(gen(D), (T, D), dt))
            w, b, dy = normal(gen(1), (D,), dt), normal(gen(2), (D,), dt), normal(gen(3), (T, D), dt)
            out = torch.full((T * D + 64,), 7.0, dtype=dt, device=DEV)
            y = out[off:off + T * D].view(T, D)
            p = lambda t: t.data_ptr()  # noqa: E731
            stats = torch.empty((2, T), device=DEV)
            assert _lib.lib().swiglu_mlp_norm_fwd(p(x), p(w), p(b), p(y), p(stats), T, D, 1e-5, 0, _lib_code(dt), 0) == 0
            (ref, tol), *rest = norm_reference(x, w, b, 1e-5, False, dy)
            inside(y, ref, tol, "y")
            dx = torch.full_like(out, 7.0)[off:off + T * D].view(T, D)
            grads = torch.full((2 * D + 64,), 7.0, dtype=dt, device=DEV)
            dw, db = grads[1:1 + D], grads[33 + D:33 + 2 * D]
            need = _lib.lib().swiglu_mlp_norm_bwd_workspace_bytes(T, D, 0, _lib_code(dt))
            ws = torch.empty(need + 16, dtype=torch.uint8, device=DEV)
            assert _lib.lib().swiglu_mlp_norm_bwd(p(dy), p(x), p(w), p(stats), None, p(dx), p(dw), p(db), p(ws), ws.numel(), T, D, 0,
                                                  _lib_code(dt), 0) == 0
            torch.cuda.synchronize()
            for got, (r, t) in zip((dx, dw, db), rest):
                inside(got, r, t, "gradient")
            for whole, a, n in ((out, off, T * D), (room, off, T * D)):
                assert (whole[:a] == 7).all() and (whole[a + n:] == 7).all()
            assert grads[0] == 7 and (grads[1 + D:33 + D] == 7).all() and (grads[33 + 2 * D:] == 7).all()


def _lib_code(dt):
    return {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}[dt]


@pytest.mark.gpu
@pytest.mark.parametrize("rms", [False, True], ids=["layer", "rms"])
def test_norm_gradients_against_differences(rms):
    """Central differences in 64 bits of the formula along random directions."""
    banner("norm differences")
    T, D = 6, 37
    x, w, b = (normal(gen(s), sh, torch.float32) for s, sh in ((1, (T, D)), (2, (D,)), (3, (D,))))
    dy = normal(gen(4), (T, D), torch.float32)
    _, stats = mlp.norm_fwd(x, w, None if rms else b, 1e-3, rms)
    grads = mlp.norm_bwd(dy, x, w, stats, rms, not rms)
    x, w, b = x.double(), w.double(), b.double()
    for i, g in enumerate(grads):
        if g is None:
            continue
        step = [torch.zeros_like(t) for t in (x, w, b)]
        step[i] = normal(gen(9 + i), g.shape, torch.float64) * 1e-5
        use_b = lambda s: None if rms else b + s * step[2]  # noqa: E731
        num = (_loss(x + step[0], w + step[1], use_b(1), dy, rms) - _loss(x - step[0], w - step[1], use_b(-1), dy, rms)) / 2
        want = (g.double() * step[i]).sum()
        assert abs(num - want) <= 1e-5 * (g.double().abs() * step[i].abs()).sum(), i


def _loss(x, w, b, dy, rms):
    mean = 0.0 if rms else x.mean(1, keepdim=True)
    n = (x - mean) / torch.sqrt(((x - mean) ** 2).mean(1, keepdim=True) + 1e-3)
    return ((n * w + (0 if b is None else b)) * dy.double()).sum()


# ---- linear -----------------------------------------------------------------------


def act64(z, act):
    if act is None:
        return z, torch.ones_like(z)
    if act == "relu":
        return z.clamp(min=0), (z > 0).double()
    if act == "silu":
        s = torch.sigmoid(z)
        return z * s, s * (1 + z * (1 - s))
    if act == "gelu":
        c = 0.5 * torch.special.erfc(-z / math.sqrt(2))
        return z * c, c + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    k = math.sqrt(2 / math.pi)
    t = torch.tanh(k * (z + 0.044715 * z ** 3))
    s = torch.sigmoid(2 * k * (z + 0.044715 * z ** 3))
    return z * s, s + 0.5 * z * (1 - t * t) * k * (1 + 3 * 0.044715 * z * z)


def product_error(a, b, dt):
    """The sums' error of a @ b (64-bit operands), term by term."""
    K = a.shape[1]
    C = K + 64 if dt == torch.float32 else K / 4 + 64
    return C * U * (a.abs() @ b.abs())


ALL = (True, True, True)


def check_linear(T, N, K, dt, act, bias, res, seed, needs=(ALL,)):
    g = gen(seed)
    x, w = normal(g, (T, K), dt), normal(g, (N, K), dt, 1.5 / math.sqrt(K))
    b = normal(g, (N,), dt, 0.5) if bias else None
    r = normal(g, (T, N), dt) if res else None
    dy = normal(g, (T, N), dt)
    y, z = mlp.linear_fwd(x, w, b, act, r)
    assert (z is None) == (act is None)
    assert torch.equal(y, mlp.linear_fwd(x, w, b, act, r, keep=False)[0])
    h, ea, es = half(dt), *((1e-5, 1e-5) if dt == torch.float32 else (2e-5, 3e-5))
    zr = x.double() @ w.double().t() + (0 if b is None else b.double())
    ez = product_error(x.double(), w.double().t(), dt) + 2 * U * zr.abs()
    yr, _ = act64(zr, act)
    tol = 1.2 * ez + ea * yr.abs()
    if r is not None:
        yr = yr + r.double()
    inside(y, yr, h * yr.abs() + tol + 2 * U * yr.abs(), ("y", T, N, K))
    near(y, yr, ("y", T, N, K))
    if z is not None:
        inside(z, zr, h * zr.abs() + ez, ("z", T, N, K))
    # the backward differentiates at the values kept
    slope = act64(z.double(), act)[1] if act else torch.ones_like(zr)
    dz = dy.double() * slope
    ed = 0 if act is None else es * dy.double().abs()
    r_dz = (h if act else 0) * dz.abs() + ed + tiny(dt) * (1 if act else 0) + 0 * dz
    refs = {"dx": (dz @ w.double(), product_error(dz, w.double(), dt) + r_dz @ w.double().abs()),
            "dw": (dz.t() @ x.double(), product_error(dz.t(), x.double(), dt) + r_dz.t() @ x.double().abs()),
            "db": (dz.sum(0), ((T / 4 + 64) * U * dz.abs() + ed).sum(0))}
    for wanted in needs:
        grads = mlp.linear_bwd(dy, x, w, z, act, wanted)
        for name, got, want in zip(("dx", "dw", "db"), grads, wanted):
            assert (got is not None) == want
            if want:
                ref, tol = refs[name]
                inside(got, ref, h * ref.abs() + 1.01 * tol, (name, T, N, K, wanted))
                if name != "db":
                    near(got, ref, (name, T, N, K, wanted))
        again = mlp.linear_bwd(dy, x, w, z, act, wanted)
        assert all(a is None or torch.equal(a, c) for a, c in zip(again, grads))


# (T, N, K): each launch variant, with partial tiles and stages
LINEAR_SHAPES = [
    (1, 8, 8), (1, 16, 72), (3, 264, 1000), (8, 712, 136), (9, 264, 1000), (16, 4104, 264), (1, 4112, 200), (7, 9000, 64),
    (13, 5000, 520),                                            # streams of 8 and 16 rows, both numbers of waves
    (17, 8, 8), (33, 264, 4096), (64, 712, 1000), (40, 8264, 136), (64, 72, 11008),  # 64 rows, split and whole
    (65, 264, 136), (130, 1000, 712), (300, 712, 1000), (512, 2056, 72), (257, 9000, 200), (500, 5000, 64),  # 64-row tiles
    (513, 264, 264), (600, 520, 2056),                          # a ring for dW only
    (2100, 2056, 328), (1100, 4104, 136), (4500, 264, 4104), (1025, 16392, 64), (5000, 1000, 8),  # rings
]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("T,N,K", LINEAR_SHAPES)
def test_linear_16_bits(T, N, K, dtype):
    banner(f"linear {dtype} T={T} N={N} K={K}")
    i = LINEAR_SHAPES.index((T, N, K)) + (dtype == "fp16")
    check_linear(T, N, K, DTYPES[dtype], ACTS[i % 5], i % 3 != 0, i % 2 == 0, 1000 + i)


@pytest.mark.gpu
@pytest.mark.parametrize("T,N,K", [s for s in LINEAR_SHAPES if s[0] * s[1] * s[2] < 4e9])
def test_linear_fp32(T, N, K):
    banner(f"linear fp32 T={T} N={N} K={K}")
    i = LINEAR_SHAPES.index((T, N, K))
    check_linear(T, N, K, torch.float32, ACTS[(i + 2) % 5], i % 3 != 1, i % 2 == 1, 2000 + i)


@pytest.mark.gpu
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("T,N,K", [(5, 264, 200), (33, 520, 1000), (200, 264, 136), (2200, 2072, 200)])
def test_linear_every_epilogue(T, N, K, act):
    """Each activation with each of bias and residual on each kind of launch."""
    for k, (bias, res) in enumerate(((True, True), (False, True), (True, False), (False, False))):
        banner(f"linear epilogue T={T} {act} bias={bias} res={res}")
        check_linear(T, N, K, torch.bfloat16 if k % 2 else torch.float16, act, bias, res, 3000 + k)


# (T, N, K) that the plan gives other launches, 16 bits: what each is there for
VARIANTS = {
    (1183, 3296, 240): "64 x 128 tiles", (313, 1672, 3856): "64 x 128 in parts", (471, 4664, 880): "dW on 64 x 128",
    (1677, 208, 4672): "dx on 64 x 128", (136, 2848, 1288): "dW on 128 x 128", (892, 176, 3944): "dx on 128 x 128",
    (1048, 3648, 464): "dx on 128 x 128 in parts", (2987, 80, 4232): "dW on 128 x 128 in parts", (548, 208, 176): "dx on 64 x 64",
    (1106, 288, 200): "dW on 64 x 64 in parts", (2100, 4104, 72): "both gradients together in parts",
    (2100, 2056, 4104): "ring, all tiles in parts; both gradients on the ring", (4200, 4104, 2056): "more than a round of ring tiles",
    (2100, 4104, 2056): "dW on the ring, dx there in parts", (2056, 4200, 4104): "both on the ring, dx's tiles the longer",
    (4096, 2048, 5632): "ring tiles in two parts",
}


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("T,N,K", list(VARIANTS))
def test_linear_launch_variants(T, N, K, dtype):
    banner(f"linear variants {dtype} T={T} N={N} K={K}")
    i = list(VARIANTS).index((T, N, K)) + (dtype == "fp16")
    check_linear(T, N, K, DTYPES[dtype], ACTS[i % 5], True, i % 2 == 0, 4000 + i,
                 (ALL, (False, True, False), (True, False, False)))


@pytest.mark.gpu
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_linear_epilogues_on_the_ring(dtype, act):
    """Whole ring tiles with partial edges in every direction."""
    banner(f"ring epilogue {dtype} {act}")
    for k, (bias, res) in enumerate(((True, True), (False, False))):
        check_linear(4100, 2056, 1032, DTYPES[dtype], act, bias, res, 5000 + k, ())


@pytest.mark.gpu
def test_linear_gradients_that_are_not_wanted():
    banner("linear needs")
    every = [(bool(k & 1), bool(k & 2), bool(k & 4)) for k in range(8)]
    for T, act in ((6, "gelu"), (300, None), (700, None), (700, "relu")):
        check_linear(T, 264, 136, torch.bfloat16, act, True, False, 77, every)
        check_linear(T, 264, 136, torch.float32, act, True, False, 78, every)


@pytest.mark.gpu
@pytest.mark.parametrize("act", ACTS[1:])
@pytest.mark.parametrize("dtype", list(DTYPES))
def test_activation_values(act, dtype):
    """The activation of every size of argument: x = identity, so z is a weight."""
    banner(f"activation {act} {dtype}")
    dt = DTYPES[dtype]
    v = torch.cat([torch.linspace(-12, 12, 4001), torch.logspace(-6, 2, 97), -torch.logspace(-6, 2, 97), torch.zeros(5)])
    v = v[:4192].to(dt)
    w = torch.zeros(4192, 8, dtype=dt)
    w[:v.numel(), 0] = v
    x = torch.zeros(3, 8, dtype=dt)
    x[:, 0] = 1
    x, w = x.to(DEV), w.to(DEV)
    y, z = mlp.linear_fwd(x, w, None, act)
    assert torch.equal(z[0], w[:, 0])
    ref, slope = act64(w[:, 0].double(), act)
    rel = 2e-5 if dt != torch.float32 else 1e-5
    tail = 2.0 ** -120  # where the exponential leaves fp32's range
    inside(y[1], ref, half(dt) * ref.abs() + rel * ref.abs() + tail, act)
    dy = torch.ones_like(y)
    db = mlp.linear_bwd(dy, x, w, z, act, (False, False, True))[2]
    es = 1e-5 if dt == torch.float32 else 3e-5
    inside(db, 3 * slope, 3 * es + half(dt) * 3 * slope.abs() + 4 * U, act)


@pytest.mark.gpu
def test_linear_nan_and_infinity_keep_their_place():
    banner("linear nan")
    for T, N, K in ((3, 264, 200), (12, 264, 200), (40, 264, 1000), (130, 264, 136), (2200, 2056, 136)):
        x, w = normal(gen(1), (T, K), torch.bfloat16), normal(gen(2), (N, K), torch.bfloat16)
        clean = mlp.linear(x, w, activation="gelu")
        x[1, K - 1], w[5, 0] = math.nan, math.inf
        y = mlp.linear(x, w, activation="relu" if T == 3 else "gelu")
        # x W^T is an infinity of x's sign there: relu keeps inf and makes -inf 0, gelu(-inf) is -inf * 0
        up = x[:, 0] > 0
        up[1] = False
        assert y[1].isnan().all() and (y[up, 5] == math.inf).all() and (y[~up, 5].isnan() | (y[~up, 5] == 0)).all()
        rows = [t for t in range(T) if t != 1][:50]
        if T != 3:
            cols = [n for n in range(N) if n != 5]
            assert torch.equal(y[rows][:, cols], clean[rows][:, cols])


@pytest.mark.gpu
@pytest.mark.parametrize("act", ACTS[1:])
@pytest.mark.parametrize("dtype", list(DTYPES))
def test_slopes_at_infinity_are_their_limits(act, dtype):
    """A sum past the storage type's range is kept as an infinity, y of a negative one
    is 0: its gradient is 0, that of a positive one dY; NaN stays NaN."""
    banner(f"slopes at infinity {act} {dtype}")
    dt, N, K = DTYPES[dtype], 64, 72
    for T in (5, 700):
        g = gen(T)
        x, w, dy = normal(g, (T, K), dt), normal(g, (N, K), dt), normal(g, (T, N), dt)
        z = torch.full((T, N), math.inf, dtype=dt, device=DEV)
        z[:, 1::2] = -math.inf
        z[2, 4] = math.nan
        dx, dw, db = mlp.linear_bwd(dy, x, w, z, act)
        dz = dy.double()
        dz[:, 1::2] = 0
        dz[2, 4] = 0 if act == "relu" else math.nan
        ref = (dz @ w.double(), dz.mT.contiguous() @ x.double(), dz.sum(0))
        bad = [torch.isnan(t) for t in ref]
        size = (dz.nan_to_num().abs() @ w.double().abs(), dz.nan_to_num().abs().mT.contiguous() @ x.double().abs(),
                dz.nan_to_num().abs().sum(0))
        for got, want, nan, s, n in zip((dx, dw, db), ref, bad, size, (N, T, T)):
            assert torch.equal(got.isnan(), nan), (act, T)
            # dz is exact; n fp32 additions and the rounding of the output
            bound = n * 2.0 ** -24 * s + half(dt) * want.abs() + tiny(dt)
            assert ((got.double() - want).abs() <= bound)[~nan].all(), (act, T)


@pytest.mark.gpu
def test_rows_behind_the_last_token_are_left():
    banner("linear rows behind")
    L = _lib.lib()
    for T in (3, 11, 50, 100, 1030):
        N, K = 4104, 136
        x, w = normal(gen(1), (T, K), torch.bfloat16), normal(gen(2), (N, K), torch.bfloat16)
        y = torch.full((T + 40, N), 7.0, dtype=torch.bfloat16, device=DEV)
        z = torch.full_like(y, 7.0)
        need = L.swiglu_mlp_linear_workspace_bytes(T, N, K, 0)
        ws = torch.empty(max(16, need), dtype=torch.uint8, device=DEV)
        p = lambda t: t.data_ptr()  # noqa: E731
        assert L.swiglu_mlp_linear_fwd(p(x), p(w), None, None, p(y), p(z), p(ws), need, T, N, K, 2, 0, 0) == 0
        torch.cuda.synchronize()
        assert (y[T:] == 7).all() and (z[T:] == 7).all()
        dx = torch.full((T + 40, K), 7.0, dtype=torch.bfloat16, device=DEV)
        dw = torch.full((N + 8, K), 7.0, dtype=torch.bfloat16, device=DEV)
        db = torch.full((N + 8,), 7.0, dtype=torch.bfloat16, device=DEV)
        need = L.swiglu_mlp_linear_bwd_workspace_bytes(T, N, K, 2, 0)
        ws = torch.full((need + 256,), 9, dtype=torch.uint8, device=DEV)
        assert L.swiglu_mlp_linear_bwd(p(y), p(x), p(w), p(z), p(dx), p(dw), p(db), p(ws), need, T, N, K, 2, 0, 0) == 0
        torch.cuda.synchronize()
        assert (dx[T:] == 7).all() and (dw[N:] == 7).all() and (db[N:] == 7).all() and (ws[need:] == 9).all()


@pytest.mark.gpu
def test_no_tokens():
    banner("no tokens")
    x, w, b = (torch.zeros(s, dtype=torch.bfloat16, device=DEV) for s in ((0, 64), (136, 64), (136,)))
    y, z = mlp.linear_fwd(x, w, b, "silu")
    assert y.shape == (0, 136)
    dx, dw, db = mlp.linear_bwd(y, x, w, z, "silu")
    assert dx.shape == (0, 64) and (dw == 0).all() and (db == 0).all()
    dx, dw, db = mlp.linear_bwd(y, x, w)
    assert (dw == 0).all() and (db == 0).all()
    s = mlp.norm_fwd(x, w[0], w[1])
    dx, dw, db = mlp.norm_bwd(x, x, w[0], s[1], bias=True)
    assert s[0].shape == (0, 64) and (dw == 0).all() and (db == 0).all()


def long(T, N, seed):
    """[T, N] in bf16 with rows that differ, made on the GPU."""
    g = torch.Generator(DEV).manual_seed(seed)
    t = torch.empty((T, N), dtype=torch.bfloat16, device=DEV)
    for i in range(0, T, 65536):
        t[i : i + 65536].normal_(generator=g)
    return t


@pytest.mark.gpu
def test_widest_rows():
    """Rows of SWIGLU_NORM_MAX_D elements, few of them and as many as leave partial sums."""
    D = 1 << 20
    for T, rms in ((2, False), (300, True)):
        banner(f"widest rows {T}")
        g = gen(T)
        x, w, dy = long(T, D, T), normal(g, (D,), torch.bfloat16), long(T, D, T + 1)
        b = None if rms else normal(g, (D,), torch.bfloat16)
        y, st = mlp.norm_fwd(x, w, b, 1e-6, rms)
        dx, dw, db = mlp.norm_bwd(dy, x, w, st, rms, not rms)
        rows = [0, T // 2, T - 1]
        ref = norm_reference(x[rows], w, b, 1e-6, rms, dy[rows])
        inside(y[rows], *ref[0], ("y", T))
        inside(dx[rows], *ref[1], ("dx", T))
        # the weight's gradient at a piece of the columns, from the statistics of all rows
        cols = torch.cat([torch.arange(0, 64), torch.arange(D - 64, D)]).to(DEV)
        mean = torch.zeros(T, 1, device=DEV, dtype=torch.float64) if rms else torch.stack([r.double().mean() for r in x])[:, None]
        rstd = torch.stack([1 / (((r.double() - m) ** 2).mean() + 1e-6).sqrt() for r, m in zip(x, mean)])[:, None]
        n, d = (x[:, cols].double() - mean) * rstd, dy[:, cols].double()
        # n's own error (G U, G = 72 + D / 1024, of rows whose mean is small beside their size) and T additions
        e = (72 + D / 1024) * U * (n.abs() + 1) * d.abs() + T * U * (n * d).abs()
        inside(dw[cols], (n * d).sum(0), half(torch.bfloat16) * (n * d).sum(0).abs() + e.sum(0), ("dw", T))
        if not rms:
            inside(db[cols], d.sum(0), half(torch.bfloat16) * d.sum(0).abs() + T * U * d.abs().sum(0), ("db", T))


@pytest.mark.gpu
def test_offsets_past_32_bits():
    """More than 2^31 elements per tensor: rows behind that are as the others."""
    U_bf16 = half(torch.bfloat16)
    banner("norm past 32 bits")
    T, D = 1060000, 2048
    x, dy = long(T, D, 1), long(T, D, 2)
    w, b = normal(gen(3), (D,), torch.bfloat16), normal(gen(4), (D,), torch.bfloat16)
    rows = [0, 1, T // 2 + 1, (1 << 31) // D - 1, (1 << 31) // D, T - 2, T - 1]
    y, st = mlp.norm_fwd(x, w, b)
    ref = norm_reference(x[rows], w, b, 1e-5, False, dy[rows])
    inside(y[rows], *ref[0], "y")
    del y
    dx, dw, db = mlp.norm_bwd(dy, x, w, st, bias=True)
    inside(dx[rows], *ref[1], "dx")
    cols = torch.tensor([0, 1, 1000, D - 1], device=DEV)
    d, n = dy[:, cols].double(), (x[:, cols].double() - st[0][:, None]) * st[1][:, None]
    # 2 rows' sums at a time per workgroup, T / 512 of them, then 256 parts
    C = T / 512 + 256 + 64
    for got, v in ((dw, n * d), (db, d)):
        want = v.sum(0)
        inside(got[cols], want, U_bf16 * want.abs() + (C + 8) * U * v.abs().sum(0), "dw, db")
    del x, dy, dx, st, d, n
    banner("linear past 32 bits")
    T, N, K = 264000, 8200, 72
    x, w = long(T, K, 5), normal(gen(6), (N, K), torch.bfloat16, 0.2)
    dy = long(T, N, 7)
    bias = normal(gen(8), (N,), torch.bfloat16)
    y, z = mlp.linear_fwd(x, w, bias, "silu", dy)
    rows = [0, 255, 256, T // 2, (1 << 31) // N - 1, (1 << 31) // N, T - 300, T - 2, T - 1]
    xr, wr = x[rows].double(), w.double()
    zr = xr @ wr.mT.contiguous() + bias.double()
    ez = (K / 4 + 64) * U * (xr.abs() @ wr.abs().mT.contiguous()) + 2 * U * zr.abs()
    inside(z[rows], zr, U_bf16 * zr.abs() + ez, "z")
    yr = act64(zr, "silu")[0]
    inside(y[rows], yr + dy[rows].double(), U_bf16 * (yr + dy[rows].double()).abs() + 1.2 * ez + 2e-5 * yr.abs()
           + 2 * U * (yr.abs() + dy[rows].double().abs()), "y")
    del y
    dx, dw, db = mlp.linear_bwd(dy, x, w, z, "silu")
    dz = dy[rows].double() * act64(z[rows].double(), "silu")[1]
    e = U_bf16 * dz.abs() + 3e-5 * dy[rows].double().abs()
    inside(dx[rows], dz @ wr, U_bf16 * (dz @ wr).abs() + 1.01 * (e @ wr.abs() + (N / 4 + 64) * U * (dz.abs() @ wr.abs())), "dx")
    cols = torch.tensor([0, 1, 4097, N - 1], device=DEV)
    dz = dy[:, cols].double() * act64(z[:, cols].double(), "silu")[1]
    e = U_bf16 * dz.abs() + 3e-5 * dy[:, cols].double().abs()
    want, size = (dz.mT.contiguous() @ x.double()), (dz.abs().mT.contiguous() @ x.double().abs())
    inside(dw[cols], want, U_bf16 * want.abs() + 1.01 * (e.mT.contiguous() @ x.double().abs() + (T / 4 + 64) * U * size), "dw")
    want = dz.sum(0)
    inside(db[cols], want, U_bf16 * want.abs() + ((T / 256 + 320) * U * dz.abs() + 3e-5 * dy[:, cols].double().abs()).sum(0), "db")


@pytest.mark.gpu
def test_strides_streams_and_leading_dimensions():
    banner("strides and streams")
    big = normal(gen(1), (4, 30, 400), torch.bfloat16)
    x = big[:, ::2, 100:300]  # not contiguous
    w = normal(gen(2), (400, 264), torch.bfloat16).t()[:, 100:300]
    b = normal(gen(3), (528,), torch.bfloat16)[::2]
    res = normal(gen(4), (264, 4, 15), torch.bfloat16).permute(1, 2, 0)
    y = mlp.linear(x, w, b, "gelu", res)
    want = mlp.linear(x.contiguous(), w.contiguous(), b.contiguous(), "gelu", res.contiguous())
    assert y.shape == (4, 15, 264) and torch.equal(y, want)
    n = mlp.layer_norm(x, b[:200], b[:200])
    assert torch.equal(n, mlp.layer_norm(x.contiguous(), b[:200].contiguous(), b[:200].contiguous()))
    assert mlp.rms_norm(x[0, 0], b[:200]).shape == (200,)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        y2 = mlp.linear(x, w, b, "gelu", res)
        n2 = mlp.layer_norm(x, b[:200], b[:200])
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(y2, y) and torch.equal(n2, n)


@pytest.mark.gpu
def test_autograd_matches_the_operators():
    banner("autograd")
    g = gen(5)
    x, w, b = normal(g, (2, 50, 136), torch.bfloat16), normal(g, (264, 136), torch.bfloat16, 0.1), normal(g, (264,), torch.bfloat16)
    res, dy = normal(g, (2, 50, 264), torch.bfloat16), normal(g, (2, 50, 264), torch.bfloat16)
    for t in (x, w, b, res):
        t.requires_grad_()
    y = mlp.linear(x, w, b, "silu", res)
    first = torch.autograd.grad(y, (x, w, b, res), dy, retain_graph=True)
    second = torch.autograd.grad(y, (x, w, b, res), dy)
    assert all(torch.equal(a, c) for a, c in zip(first, second))
    with torch.no_grad():
        y2, z = mlp.linear_fwd(x.view(100, 136), w, b, "silu", res.view(100, 264))
        want = mlp.linear_bwd(dy.view(100, 264), x.view(100, 136), w, z, "silu")
    assert torch.equal(y.view(100, 264), y2) and all(torch.equal(a.reshape(c.shape), c) for a, c in zip(first, want))
    assert torch.equal(first[3], dy)
    # a gradient that is a broadcast of one number
    (gx,) = torch.autograd.grad(mlp.linear(x, w).sum(), x)
    assert torch.equal(gx.view(100, 136), mlp.linear_bwd(torch.ones_like(dy).view(100, 264), x.detach().view(100, 136), w.detach())[0])
    for rms in (False, True):
        wn, bn = normal(gen(6), (136,), torch.bfloat16).requires_grad_(), normal(gen(7), (136,), torch.bfloat16).requires_grad_()
        n = mlp.rms_norm(x, wn, eps=1e-5) if rms else mlp.layer_norm(x, wn, bn)
        dn = normal(gen(8), n.shape, torch.bfloat16)
        got = torch.autograd.grad(n, (x, wn) if rms else (x, wn, bn), dn)
        with torch.no_grad():
            yn, st = mlp.norm_fwd(x.view(100, 136), wn, None if rms else bn, 1e-5, rms)
            want = mlp.norm_bwd(dn.view(100, 136), x.view(100, 136), wn, st, rms, not rms)
        assert torch.equal(n.view(100, 136), yn) and all(torch.equal(a.reshape(c.shape), c) for a, c in zip(got, want))
    y = mlp.linear(x, w, b, "silu")
    with pytest.raises(RuntimeError, match="double backward"):
        torch.autograd.grad(y, x, dy, create_graph=True)


@pytest.mark.gpu
def test_refusals_on_a_gpu():
    """What the library refuses comes back as the package's exception, also where
    gradients are wanted; nothing is launched for mixed types or devices."""
    x, w = torch.zeros(4, 60, device=DEV), torch.zeros(32, 60, device=DEV)
    for grad in (False, True):
        w.requires_grad_(grad)
        with pytest.raises(mlp.SwiGLUError) as e:
            mlp.linear(x, w)
        assert _lib.STATUS[e.value.status] == "SWIGLU_ERR_SHAPE"
        with pytest.raises(mlp.SwiGLUError) as e:
            mlp.feed_forward(x, x[0], None, w, None, w.mT, None)
        assert _lib.STATUS[e.value.status] == "SWIGLU_ERR_SHAPE"
        with pytest.raises(ValueError, match="share dtype and device"):
            mlp.linear(x, w.bfloat16())
        with pytest.raises(ValueError, match="share dtype and device"):
            mlp.layer_norm(x, w[0].cpu())
        with pytest.raises(TypeError, match="unsupported dtype"):
            mlp.linear(x.double(), w.double())
        with pytest.raises(ValueError, match="bias must be"):
            mlp.linear(x, w, x[0])
        with pytest.raises(ValueError, match="residual must be"):
            mlp.linear(x, w, None, None, x)
        with pytest.raises(ValueError, match="a number from 0 up"):
            mlp.rms_norm(x, x[0], eps=math.nan)


@pytest.mark.gpu
def test_graph_replays():
    """Operators captured and replayed between eager work on other values."""
    banner("graph")
    g = gen(11)
    shapes = [(3, 264, 200), (40, 264, 1000), (700, 520, 264)]
    for T, N, K in shapes:
        x, w, b = normal(g, (T, K), torch.bfloat16), normal(g, (N, K), torch.bfloat16, 0.1), normal(g, (N,), torch.bfloat16)
        wn, bn, dy = normal(g, (K,), torch.bfloat16), normal(g, (K,), torch.bfloat16), normal(g, (T, N), torch.bfloat16)

        def step():
            n, st = mlp.norm_fwd(x, wn, bn)
            y, z = mlp.linear_fwd(n, w, b, "gelu")
            dn, dw, db = mlp.linear_bwd(dy, n, w, z, "gelu")
            return (y, dw, db, *mlp.norm_bwd(dn, x, wn, st, bias=True, dres=x))

        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step()
        for i in range(4):
            x.copy_(normal(g, (T, K), torch.bfloat16))
            dy.copy_(normal(g, (T, N), torch.bfloat16))
            want = step()
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, c) for a, c in zip(out, want)), (T, i)


# ---- the layer -----------------------------------------------------------------------


class Config:
    def __init__(self, **kw):
        self.__dict__.update(kw)


@pytest.mark.gpu
@pytest.mark.parametrize("kw", [dict(), dict(hidden_act="gelu_new", rms_norm_eps=1e-6, mlp_bias=False), dict(hidden_act="relu")])
def test_feed_forward(kw):
    """The operators as they are used together, in fp32 and bf16 against torch's
    layers in 64 bits; a training step and a graph of a decoding step."""
    banner(f"FeedForward {kw}")
    torch.manual_seed(3)
    cfg = Config(hidden_size=200, intermediate_size=520, **kw)
    block = mlp.FeedForward(cfg).to(DEV)
    for dt, tol in ((torch.float32, 1e-5), (torch.bfloat16, 1e-2)):
        m = copy.deepcopy(block).to(dt)
        for T in ((1,), (3, 7), (2, 300)):
            x = normal(gen(sum(T)), (*T, 200), dt).requires_grad_()
            dy = normal(gen(1), (*T, 200), dt)
            y = m(x)
            grads = torch.autograd.grad(y, [x, *m.parameters()], dy)
            ref = copy.deepcopy(m).double()
            xr = x.detach().double().requires_grad_()
            z = ref.fc1(ref.norm(xr))
            yr = xr + ref.fc2(act64(z, m.activation)[0])
            want = torch.autograd.grad(yr, [xr, *ref.parameters()], dy.double())
            # relu's slope jumps: the norm's output is rounded before fc1, which moves z by at most
            # h of its spread s; with a density of at most 0.4 / s at zero a share of 0.4 h of all
            # signs turns, each with its whole dz, against the half that is not zero: sqrt(0.4 h /
            # 0.5) of the gradients' norm
            jump = math.sqrt(0.8 * half(dt)) if m.activation == "relu" and dt != torch.float32 else 0.0
            for k, (a, c) in enumerate(zip((y, *grads), (yr, *want))):
                # a chain of roundings of its own kind each: four times a single one's bound
                err = (a.double() - c).norm() / c.norm()
                assert err <= (4 * tol if dt == torch.float32 else 2 * tol) + (jump if k else 0), (T, k, float(err))
            with torch.no_grad():
                assert torch.equal(m(x), y)
    names = set(block.state_dict())
    assert {"norm.weight", "fc1.weight", "fc2.weight"} <= names and ("fc1.bias" in names) == kw.get("mlp_bias", True)


@pytest.mark.gpu
def test_feed_forward_is_its_operators():
    """The layer's one node gives what its operators give one after another, with
    any of its weights frozen."""
    banner("feed_forward")
    dt = torch.bfloat16
    sh = {"x": (90, 136), "nw": (136,), "nb": (136,), "w1": (264, 136), "b1": (264,), "w2": (136, 264), "b2": (136,)}
    t = {k: normal(gen(i), s, dt, 0.1 if k[0] == "w" else 1.0) for i, (k, s) in enumerate(sh.items())}
    dy = normal(gen(50), (90, 136), dt)
    n, st = mlp.norm_fwd(t["x"], t["nw"], t["nb"])
    a, z = mlp.linear_fwd(n, t["w1"], t["b1"], "silu")
    y = mlp.linear_fwd(a, t["w2"], t["b2"], None, t["x"])[0]
    da, dw2, db2 = mlp.linear_bwd(dy, a, t["w2"])
    dn, dw1, db1 = mlp.linear_bwd(da, n, t["w1"], z, "silu")
    dx, dnw, dnb = mlp.norm_bwd(dn, t["x"], t["nw"], st, bias=True, dres=dy)
    want = dict(x=dx, nw=dnw, nb=dnb, w1=dw1, b1=db1, w2=dw2, b2=db2)
    assert torch.equal(mlp.feed_forward(*t.values(), activation="silu"), y)
    for wanted in (list(sh), ["x"], ["w1"], ["b1", "w2"], ["b2"], ["nb"], ["w1", "w2"]):
        leaves = {k: v.detach().clone().requires_grad_(k in wanted) for k, v in t.items()}
        out = mlp.feed_forward(*leaves.values(), activation="silu")
        assert torch.equal(out, y)
        got = torch.autograd.grad(out, [leaves[k] for k in wanted], dy)
        for k, g in zip(wanted, got):
            assert torch.equal(g, want[k]), (wanted, k)


@pytest.mark.gpu
def test_gradients_without_some_inputs():
    """Inputs that are absent shift no other input's gradient, wanted or not."""
    banner("absent inputs")
    dt = torch.bfloat16
    sh = {"x": (90, 136), "nw": (136,), "nb": (136,), "w1": (264, 136), "b1": (264,), "w2": (136, 264), "b2": (136,)}
    t = {k: normal(gen(i), s, dt, 0.1 if k[0] == "w" else 1.0) for i, (k, s) in enumerate(sh.items())}
    dy = normal(gen(50), (90, 136), dt)
    zero = lambda k: torch.zeros_like(t[k])  # noqa: E731
    for absent in (("nb",), ("b1",), ("nb", "b2"), ("nb", "b1", "b2")):
        full = {k: (zero(k) if k in absent else v).clone().requires_grad_() for k, v in t.items()}
        want = dict(zip(sh, torch.autograd.grad(mlp.feed_forward(*full.values(), activation="gelu"), list(full.values()), dy)))
        for wanted in ([k for k in sh if k not in absent], ["w2"], ["w1", "x"], ["nw"]):
            leaves = {k: None if k in absent else v.clone().requires_grad_(k in wanted) for k, v in t.items()}
            out = mlp.feed_forward(*leaves.values(), activation="gelu")
            for k, g in zip(wanted, torch.autograd.grad(out, [leaves[k] for k in wanted], dy)):
                assert torch.equal(g, want[k]), (absent, wanted, k)
    x, w, b, r = t["x"], t["w1"], t["b1"], normal(gen(51), (90, 264), dt)
    dz = normal(gen(52), (90, 264), dt)
    for act in (None, "silu"):
        z = mlp.linear_fwd(x, w, None, act, r)[1]
        want = dict(zip("xwb", mlp.linear_bwd(dz, x, w, z, act)), r=dz)
        for wanted in ("xwr", "r", "wr", "x"):
            leaves = {k: v.clone().requires_grad_(k in wanted) for k, v in zip("xwr", (x, w, r))}
            out = mlp.linear(leaves["x"], leaves["w"], None, act, leaves["r"])
            for k, g in zip(wanted, torch.autograd.grad(out, [leaves[k] for k in wanted], dz)):
                assert torch.equal(g, want[k]), (act, wanted, k)
        z = mlp.linear_fwd(x, w, b, act)[1]
        gb, = torch.autograd.grad(mlp.linear(x, w, b.requires_grad_(), act), b, dz)
        assert torch.equal(gb, mlp.linear_bwd(dz, x, w, z, act)[2])
        b = b.detach()


@pytest.mark.gpu
def test_nodes_under_checkpoints_hooks_and_without_tokens():
    """The nodes keep what they need through autograd's own means: recomputed,
    moved to the host and back, for no tokens at all, after an in-place change."""
    banner("checkpoints")
    from torch.utils.checkpoint import checkpoint

    dt = torch.bfloat16
    block = mlp.FeedForward(Config(hidden_size=136, intermediate_size=264)).to(DEV, dt)
    x, dy = normal(gen(1), (3, 30, 136), dt).requires_grad_(), normal(gen(2), (3, 30, 136), dt)
    leaves = [x, *block.parameters()]

    def both(t):
        return mlp.linear(mlp.layer_norm(block(t), block.norm.weight, block.norm.bias), block.fc1.weight, None, "silu")

    dz = normal(gen(3), (3, 30, 264), dt)
    want = torch.autograd.grad(both(x), leaves, dz, allow_unused=True)
    for reentrant in (False, True):
        for p in leaves:
            p.grad = None
        checkpoint(both, x, use_reentrant=reentrant).backward(dz)
        assert all(torch.equal(p.grad, g) for p, g in zip(leaves, want) if g is not None)
    with torch.autograd.graph.save_on_cpu():
        y = both(x)
    got = torch.autograd.grad(y, leaves, dz, allow_unused=True)
    assert all(torch.equal(a, c) for a, c in zip(got, want) if c is not None)
    none = torch.zeros(0, 7, 136, dtype=dt, device=DEV, requires_grad=True)
    y = both(none)
    assert y.shape == (0, 7, 264)
    grads = torch.autograd.grad(y, [none, *leaves[1:]], torch.zeros_like(y), allow_unused=True)
    assert grads[0].shape == none.shape and all((g == 0).all() for g in grads if g is not None)
    y = block(x)
    with torch.no_grad():
        block.fc2.weight.mul_(2)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        torch.autograd.grad(y, x, dy)


@pytest.mark.gpu
def test_views_with_a_negation_put_off():
    banner("negations")
    c = torch.randn(20, 64, dtype=torch.complex64, device=DEV, generator=torch.Generator(DEV).manual_seed(1))
    x, w = c.conj().imag, normal(gen(2), (72, 64), torch.float32)
    assert x.is_neg()
    plain = (-c.imag).contiguous()
    assert torch.equal(mlp.linear(x, w, None, "gelu"), mlp.linear(plain, w, None, "gelu"))
    assert torch.equal(mlp.linear_fwd(x, w)[0], mlp.linear_fwd(plain, w)[0])
    assert torch.equal(mlp.layer_norm(x, w[0], x[1]), mlp.layer_norm(plain, w[0], plain[1]))
    assert torch.equal(mlp.norm_fwd(x, w[0], x[1])[0], mlp.norm_fwd(plain, w[0], plain[1])[0])


@pytest.mark.gpu
def test_backward_from_two_threads():
    """Nodes built on one stream and run backward from two threads at once give
    what one call gives."""
    banner("threads")
    import threading

    dt = torch.bfloat16
    x, w, b = (normal(gen(i), s, dt) for i, s in enumerate(((90, 136), (264, 136), (264,))))
    dy = normal(gen(9), (90, 264), dt)

    def one():
        xs, ws, bs = (t.clone().requires_grad_() for t in (x, w, b))
        n = mlp.rms_norm(xs, torch.ones_like(x[0]))
        return torch.autograd.grad(mlp.linear(n, ws, bs, "gelu"), (xs, ws, bs), dy)

    want, got = one(), {}

    def work(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(20):
                got[i] = one()
            torch.cuda.current_stream().synchronize()

    torch.cuda.synchronize()
    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for i in range(2):
        assert all(torch.equal(a, c) for a, c in zip(got[i], want))


@pytest.mark.gpu
def test_gradients_that_start_anywhere():
    """Views at odd addresses: of inputs, and as the gradient that a flattened
    concatenation hands back."""
    banner("odd addresses")
    dt = torch.bfloat16
    x, w = normal(gen(1), (20, 64), dt).requires_grad_(), normal(gen(2), (72, 64), dt).requires_grad_()
    room = normal(gen(3), (20 * 64 + 72 + 3,), dt)
    xo, bo = room[1:1 + 20 * 64].view(20, 64), room[1 + 20 * 64:1 + 20 * 64 + 72]
    assert torch.equal(mlp.linear(xo, w, bo, "relu"), mlp.linear(xo.clone(), w, bo.clone(), "relu"))
    y = mlp.linear(x, w, None, "gelu")
    weights = normal(gen(4), (1 + 20 * 72,), dt)
    out = (torch.cat([torch.ones(1, dtype=dt, device=DEV), y.flatten()]) * weights).sum()
    gx, gw = torch.autograd.grad(out, (x, w))
    _, z = mlp.linear_fwd(x.detach(), w.detach(), None, "gelu")
    want = mlp.linear_bwd(weights[1:].view(20, 72).clone(), x.detach(), w.detach(), z, "gelu")
    assert torch.equal(gx, want[0]) and torch.equal(gw, want[1])


@pytest.mark.gpu
def test_training_step_in_a_graph():
    """Forward and backward of the layer through autograd, captured; replayed
    between eager steps of other leaves on other values."""
    banner("training step in a graph")
    torch.manual_seed(1)
    block = mlp.FeedForward(Config(hidden_size=136, intermediate_size=264)).to(DEV, torch.bfloat16)
    eager = copy.deepcopy(block)
    for T in (5, 600):
        x, dy = normal(gen(T), (T, 136), torch.bfloat16), normal(gen(T + 1), (T, 136), torch.bfloat16)

        def step(m, x, dy):
            x = x.detach().requires_grad_()
            y = m(x)
            return (y.detach(), *torch.autograd.grad(y, [x, *m.parameters()], dy))

        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step(block, x, dy)
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step(block, x, dy)
        for i in range(4):
            x.copy_(normal(gen(100 + i), (T, 136), torch.bfloat16))
            dy.copy_(normal(gen(200 + i), (T, 136), torch.bfloat16))
            want = step(eager, x, dy)
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, c) for a, c in zip(out, want)), (T, i)


@pytest.mark.gpu
def test_capture_beside_a_live_eager_graph_is_refused():
    """A graph of the same leaves on the default stream keeps their accumulation
    nodes there; the captured forward says so. Without it the capture goes through."""
    banner("capture beside an eager graph")
    x, w = normal(gen(1), (5, 64), torch.bfloat16), normal(gen(2), (72, 64), torch.bfloat16).requires_grad_()
    n = normal(gen(3), (64,), torch.bfloat16).requires_grad_()
    dy = normal(gen(4), (5, 72), torch.bfloat16)
    step = lambda: mlp.linear(mlp.rms_norm(x, n), w, None, "gelu")  # noqa: E731
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.autograd.grad(step(), (n, w), dy)
    torch.cuda.current_stream().wait_stream(side)
    for alive in (lambda: mlp.linear(x, w), lambda: x * n):
        eager = alive()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with pytest.raises(RuntimeError, match="is alive"):
            with torch.cuda.graph(graph):
                dy + 0  # a graph of nothing would warn
                step()
        del eager, graph
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = step()
        grads = torch.autograd.grad(y, (n, w), dy)
    y = y.detach()
    for i in range(3):
        x.copy_(normal(gen(10 + i), (5, 64), torch.bfloat16))
        with torch.no_grad():
            want = step()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)
    m, v = n.detach().requires_grad_(), w.detach().requires_grad_()
    again = torch.autograd.grad(mlp.linear(mlp.rms_norm(x, m), v, None, "gelu"), (m, v), dy)
    assert all(torch.equal(a, c) for a, c in zip(grads, again))


# ---- refusals (CPU) ------------------------------------------------------------------


def cpu(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


def test_python_refusals():
    x, w = cpu(4, 64), cpu(32, 64)
    with pytest.raises(ValueError, match="on a GPU"):
        mlp.linear(x, w)
    with pytest.raises(ValueError, match="on a GPU"):
        mlp.layer_norm(x, cpu(64))
    with pytest.raises(ValueError, match="shape mismatch"):
        mlp.linear(x, cpu(32, 72))
    with pytest.raises(ValueError, match="unknown activation"):
        mlp.linear(x, w, activation="swiglu")
    with pytest.raises(ValueError, match="unknown activation"):
        mlp.linear(x, w, activation=["gelu"])
    with pytest.raises(ValueError, match="bias must be"):
        mlp.linear(x, w, cpu(64))
    for res in (cpu(32), cpu(1, 32), cpu(4, 64), cpu(2, 2, 32)):
        with pytest.raises(ValueError, match="residual must be"):
            mlp.linear(x, w, residual=res)
    with pytest.raises(ValueError, match="share dtype"):
        mlp.linear(x, cpu(32, 64, dtype=torch.float16))
    with pytest.raises(ValueError, match="share dtype"):
        mlp.layer_norm(x, cpu(64, dtype=torch.float32))
    for eps in (-1e-6, math.nan, math.inf):
        with pytest.raises(ValueError, match="eps"):
            mlp.rms_norm(x, cpu(64), eps)
    with pytest.raises(ValueError, match="expected X"):
        mlp.layer_norm(x, cpu(32))
    with pytest.raises(ValueError, match="bias must be"):
        mlp.layer_norm(x, cpu(64), cpu(32))
    with pytest.raises(ValueError, match="no bias"):
        mlp.norm_fwd(x, cpu(64), cpu(64), rms=True)
    with pytest.raises(ValueError, match="expected X"):
        mlp.layer_norm(torch.tensor(1.0), cpu(1))
    with pytest.raises(ValueError, match="expected X"):
        mlp.linear(torch.tensor(1.0), w)
    with pytest.raises(ValueError, match="z must be"):
        mlp.linear_bwd(cpu(4, 32), x, w, None, "gelu")
    with pytest.raises(ValueError, match="must match X"):
        mlp.norm_bwd(cpu(4, 32), x, cpu(64), torch.zeros(2, 4))
    with pytest.raises(ValueError, match="needs an activation"):
        mlp.feed_forward(x, cpu(64), None, w, None, cpu(64, 32), None, activation=None)
    with pytest.raises(ValueError, match="no activation"):
        mlp.FeedForward(Config(hidden_size=8, intermediate_size=8, hidden_act="tanh"))


# Addresses that nothing reads: every call here is refused before a launch.
A = [ctypes.c_void_p(0x10000000 * (i + 1)) for i in range(10)]


def test_c_refusals():
    L, S = _lib.lib(), {v: k for k, v in _lib.STATUS.items()}
    fwd = lambda T=4, N=32, K=64, act=0, dt=0, x=A[0], w=A[1], b=None, r=None, y=A[2], z=None, ws=A[3], n=1 << 30: \
        L.swiglu_mlp_linear_fwd(x, w, b, r, y, z, ws, n, T, N, K, act, dt, None)  # noqa: E731
    assert fwd(dt=3) == S["SWIGLU_ERR_DTYPE"]
    assert fwd(act=5) == fwd(act=-1) == S["SWIGLU_ERR_ARG"]
    for kw in (dict(T=-1), dict(N=0), dict(N=12), dict(K=4), dict(K=1 << 23), dict(T=1 << 31)):
        assert fwd(**kw) == S["SWIGLU_ERR_SHAPE"], kw
    assert fwd(x=None) == fwd(w=None) == fwd(y=None) == S["SWIGLU_ERR_NULL"]
    off = ctypes.c_void_p(A[4].value + 8)
    assert fwd(x=off) == fwd(b=off) == fwd(z=off) == fwd(r=off) == fwd(ws=off) == S["SWIGLU_ERR_ALIGN"]
    assert fwd(y=A[0]) == fwd(z=A[2]) == fwd(r=A[2]) == S["SWIGLU_ERR_ALIAS"]
    need = L.swiglu_mlp_linear_workspace_bytes(33, 64, 4096, 0)
    assert need > 0
    assert fwd(T=33, N=64, K=4096, n=need - 1) == fwd(T=33, N=64, K=4096, ws=None) == S["SWIGLU_ERR_WORKSPACE"]
    bwd = lambda T=4, N=32, K=64, act=0, dt=0, dy=A[0], x=A[1], w=A[2], z=None, dx=A[3], dw=A[4], db=A[5], ws=A[6], n=1 << 30: \
        L.swiglu_mlp_linear_bwd(dy, x, w, z, dx, dw, db, ws, n, T, N, K, act, dt, None)  # noqa: E731
    assert bwd(dt=9) == S["SWIGLU_ERR_DTYPE"] and bwd(act=7) == S["SWIGLU_ERR_ARG"] and bwd(K=65) == S["SWIGLU_ERR_SHAPE"]
    assert bwd(dy=None) == bwd(act=2) == S["SWIGLU_ERR_NULL"]
    assert bwd(dx=A[1]) == bwd(dw=A[3]) == bwd(db=A[0]) == bwd(act=2, z=A[3]) == S["SWIGLU_ERR_ALIAS"]
    assert bwd(act=2, z=A[7], ws=None) == bwd(act=2, z=A[7], n=0) == bwd(T=600, ws=None) == S["SWIGLU_ERR_WORKSPACE"]
    assert bwd(dx=ctypes.c_void_p(A[3].value + 4)) == S["SWIGLU_ERR_ALIGN"]
    nf = lambda T=4, D=64, eps=1e-5, rms=0, dt=0, x=A[0], w=A[1], b=None, y=A[2], st=None: \
        L.swiglu_mlp_norm_fwd(x, w, b, y, st, T, D, eps, rms, dt, None)  # noqa: E731
    assert nf(dt=-1) == S["SWIGLU_ERR_DTYPE"]
    assert nf(T=-1) == nf(D=0) == nf(D=(1 << 20) + 1) == nf(T=1 << 31) == S["SWIGLU_ERR_SHAPE"]
    assert nf(eps=-1.0) == nf(eps=math.nan) == nf(eps=math.inf) == nf(rms=2) == nf(rms=1, b=A[3]) == S["SWIGLU_ERR_ARG"]
    assert nf(x=None) == nf(w=None) == nf(y=None) == S["SWIGLU_ERR_NULL"]
    odd = ctypes.c_void_p(A[4].value + 1)
    assert nf(x=odd) == nf(b=odd) == nf(st=ctypes.c_void_p(A[4].value + 2)) == S["SWIGLU_ERR_ALIGN"]
    assert nf(y=A[0]) == nf(st=A[2]) == S["SWIGLU_ERR_ALIAS"]
    nb = lambda T=4, D=64, rms=0, dt=0, dy=A[0], x=A[1], w=A[2], st=A[3], dr=None, dx=A[4], dw=A[5], db=None, ws=A[6], n=1 << 30: \
        L.swiglu_mlp_norm_bwd(dy, x, w, st, dr, dx, dw, db, ws, n, T, D, rms, dt, None)  # noqa: E731
    assert nb(dy=None) == nb(st=None) == nb(dw=None) == S["SWIGLU_ERR_NULL"]
    assert nb(rms=1, db=A[7]) == S["SWIGLU_ERR_ARG"] and nb(D=-3) == S["SWIGLU_ERR_SHAPE"]
    assert nb(dx=A[0]) == nb(dr=A[4]) == nb(T=300, ws=A[5]) == S["SWIGLU_ERR_ALIAS"]
    assert nb(T=300, ws=None) == nb(T=300, n=8) == S["SWIGLU_ERR_WORKSPACE"]
    # no GPU here: a call without a fault reaches the device check
    if not torch.cuda.is_available():
        assert fwd() == bwd() == nf() == nb() == S["SWIGLU_ERR_DEVICE"]


def test_size_queries():
    L = _lib.lib()
    assert L.swiglu_mlp_norm_stats_bytes(10, 0) == 80 and L.swiglu_mlp_norm_stats_bytes(10, 1) == 40
    assert L.swiglu_mlp_norm_bwd_workspace_bytes(0, 64, 0, 0) == 0
    assert L.swiglu_mlp_norm_bwd_workspace_bytes(1, 64, 0, 0) == 0
    assert L.swiglu_mlp_norm_bwd_workspace_bytes(300, 64, 0, 0) == 2 * L.swiglu_mlp_norm_bwd_workspace_bytes(300, 64, 1, 0) > 0
    assert L.swiglu_mlp_norm_bwd_workspace_bytes(300, 64, 1, 7) == 0
    assert L.swiglu_mlp_linear_workspace_bytes(1, 64, 64, 0) == 0
    assert L.swiglu_mlp_linear_workspace_bytes(100, 64, 64, 0) == 0
    assert L.swiglu_mlp_linear_bwd_workspace_bytes(100, 64, 64, 0, 0) < L.swiglu_mlp_linear_bwd_workspace_bytes(100, 64, 64, 1, 0)
    assert L.swiglu_mlp_linear_bwd_workspace_bytes(100, 60, 64, 0, 0) == 0
    assert set(dense.ACTIVATIONS) == set(ACTS)
