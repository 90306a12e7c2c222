"""Layer norm where the mean's own error shows: rows without spread, and rows whose
mean is large beside it, at widths whose reciprocal is not exact (GPU).

Tolerances, derived before the first run. u = 2^-24, h a rounding to the storage type,
G = 72 + D / 1024 the roundings that a row's sum passes through.

The first mean m0 is off by d <= G u mean|x|. Of a constant row c every x - m0 is the
same number and exact, so its sum is off by G u of itself, and m0 plus its mean lies
within |d| (G + 2) u <= |c| G (G + 2) u^2, far less than half a step, of c: the kept
mean is c to the bit, n is 0 and y is the bias. Of other rows the kept mean is off by
its rounding and by the second sum's, u |mean| + (G + 2) u mean|x - m0|. The variance
loses the correction's square, whose own error is at most (2 G + 4) u d^2.
dx = rstd (g - level - n along) then counts as in tests/test_dense.py.
"""

import pytest
import torch

import backward_gate_up_amd as mlp
from tests._util import banner
from tests.test_dense import DTYPES, U, gen, half, inside, normal

# one, four and sixteen waves per row, walked rows; whole and odd pieces
WIDTHS = [3, 100, 1000, 1001, 1536, 6000, 11008, 12345, 40001]


def reference(x, w, b, eps, dy):
    """[(value, tolerance)] of y, dx, dw, db, in 64 bits."""
    dt, T, D = x.dtype, *x.shape
    h, G = half(dt), 72 + D / 1024
    x, w, b, dy = (t.double() for t in (x, w, b, dy))
    m = lambda t: t.mean(1, keepdim=True)  # noqa: E731
    mean = m(x)
    var = m((x - mean) ** 2)
    rstd = 1 / (var + eps).sqrt()
    n = (x - mean) * rstd
    d = G * U * m(x.abs())
    e_mean = torch.where(var == 0, torch.zeros_like(mean), U * mean.abs() + (G + 2) * U * (m((x - mean).abs()) + d))
    e_rstd = (G + 16) * U + (2 * G + 4) * U * d ** 2 / (2 * (var + eps))
    en = rstd * e_mean + e_rstd * n.abs()
    y = n * w + b
    out = [(y, h * y.abs() + w.abs() * en + 4 * U * ((n * w).abs() + b.abs()))]
    g = dy * w
    along, level = m(g * n), m(g)
    dx = rstd * (g - level - n * along)
    e_along = (G + 4) * U * m((g * n).abs()) + m(g.abs() * en)
    tol = rstd * ((G + 4) * U * m(g.abs()) + n.abs() * e_along + en * along.abs() + 8 * U * (g.abs() + level.abs() + (n * along).abs()))
    out.append((dx, h * dx.abs() + tol + e_rstd * dx.abs()))
    C = T / 256 + 64
    dw, db = (dy * n).sum(0), dy.sum(0)
    out.append((dw, h * dw.abs() + (C * U * dy.abs() * n.abs() + dy.abs() * en).sum(0)))
    out.append((db, h * db.abs() + C * U * dy.abs().sum(0)))
    return out


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("D", WIDTHS)
def test_constant_rows_are_the_bias(D, dtype):
    """Rows of one number each: the mean is it, y the bias, dw 0; so for few rows and
    for as many as leave partial sums."""
    banner(f"constant rows {dtype} D={D}")
    dt = DTYPES[dtype]
    w, b = normal(gen(1), (D,), dt), normal(gen(2), (D,), dt)
    c = torch.tensor([100.0, 1000.0, -3.7, 0.1, 1e4, 333.25, -1e-3], dtype=dt, device=w.device)
    for T in (7, 301):
        x = c.repeat(T // 7 + 1)[:T, None].expand(T, D).contiguous()
        dy = normal(gen(3), (T, D), dt)
        y, stats = mlp.norm_fwd(x, w, b, 1e-5)
        assert torch.equal(stats[0], x[:, 0].float())
        assert torch.equal(y, b.expand(T, -1)) and torch.equal(mlp.layer_norm(x, w, b), y)
        dx, dw, db = mlp.norm_bwd(dy, x, w, stats, bias=True)
        assert (dw == 0).all()
        for name, got, (ref, tol) in zip(("y", "dx", "dw", "db"), (y, dx, dw, db), reference(x, w, b, 1e-5, dy)):
            inside(got, ref, tol, (name, T, D))
        # a gradient that is the same everywhere goes nowhere
        one = torch.ones_like(w)
        assert (mlp.norm_bwd(torch.ones_like(x), x, one, stats, bias=True)[0] == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("D", WIDTHS)
def test_rows_of_a_large_mean(D, dtype):
    """Spread of 1 and of a few of the type's steps around means up to 1000."""
    banner(f"large means {dtype} D={D}")
    dt = DTYPES[dtype]
    for T in (6, 290):
        g = gen(D + T)
        scale = torch.tensor([1.0, 0.05, 3.0])[torch.arange(T) % 3, None]
        mean = torch.tensor([1000.0, -100.0, 7.0, 0.0])[torch.arange(T) % 4, None]
        x = (torch.randn((T, D), generator=g) * scale + mean).to(dt).cuda()
        w, b, dy = normal(g, (D,), dt, 0.2, 1.0), normal(g, (D,), dt, 0.3), normal(g, (T, D), dt)
        y, stats = mlp.norm_fwd(x, w, b, 1e-5)
        got = (y, *mlp.norm_bwd(dy, x, w, stats, bias=True))
        for name, a, (ref, tol) in zip(("y", "dx", "dw", "db"), got, reference(x, w, b, 1e-5, dy)):
            inside(a, ref, tol, (name, T, D))


@pytest.mark.gpu
def test_sums_past_the_range():
    """Squares past fp32's range make the variance an infinity and y the bias, as
    documented; a sum past it makes the row NaN; neither leaves its row."""
    banner("sums past the range")
    for D in (1000, 6000, 11008, 40001):
        w, b = normal(gen(1), (D,), torch.float32), normal(gen(2), (D,), torch.float32)
        x = normal(gen(3), (4, D), torch.float32)
        clean = mlp.layer_norm(x, w, b)
        x[1] *= 1e30
        x[2] = 3e38
        y = mlp.layer_norm(x, w, b)
        assert torch.equal(y[1], b) and y[2].isnan().all()
        assert torch.equal(y[0], clean[0]) and torch.equal(y[3], clean[3])
