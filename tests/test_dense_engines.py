"""The linear layer by engine: that the plan sends these sizes where they are meant to
run (CPU and GPU), every epilogue on each, and what tests/test_dense.py asks of the
small launches asked of the ring of 256 x 256 tiles (GPU).
Formulas and tolerances are those of tests/test_dense.py."""

import math

import pytest
import torch

import backward_gate_up_amd as mlp
from backward_gate_up_amd import _lib, dense
from tests._util import banner
from tests.test_dense import ACTS, ALL, DEV, DTYPES, U, act64, check_linear, gen, half, inside, long, normal

# (T, N, K) -> parts of K in the forward; no size is a whole number of tiles, K ends inside a stage
FORWARD = {(8293, 1456, 264): 1, (2100, 4104, 1032): 1, (513, 7224, 3544): 2, (2100, 2056, 4104): 3, (7941, 304, 7160): 4}
# -> parts of (dW, dx) on the ring, each asked for alone
DW = {(261, 9256, 1336): 1, (3713, 520, 8272): 2, (2716, 744, 5560): 3, (6343, 280, 8176): 4}
DX = {(2090, 264, 6488): 1, (856, 3176, 5560): 2, (990, 2656, 4264): 3, (388, 5328, 7952): 4}
# both in one launch; in the first two one of them sums over a few hundred only
TOGETHER = [(1139, 336, 9584), (334, 1168, 10208), (2100, 2056, 4104)]
# both apart, both there
APART = [(2100, 4104, 2056)]
LONG = (264000, 8200, 1032)  # more than 2^31 outputs


def plan(shape, **needs):
    return dense.linear_plan(*shape, torch.bfloat16, **needs)


def check_plans():
    for s, parts in FORWARD.items():
        assert plan(s) == {"fwd": ("ring", parts)}, s
    for s, parts in DW.items():
        assert plan(s, dw=True)["dw"] == ("ring", parts), s
    for s, parts in DX.items():
        assert plan(s, dx=True)["dx"] == ("ring", parts), s
    for s in TOGETHER:
        assert plan(s, dw=True, dx=True) == {"together": True, "dw": ("ring", 1), "dx": ("ring", 1)}, s
    for s in APART:
        p = plan(s, dw=True, dx=True)
        assert not p["together"] and p["dw"][0] == p["dx"][0] == "ring", s
    assert plan(LONG)["fwd"] == ("ring", 1) and plan(LONG, dw=True, dx=True) == {"together": True, "dw": ("ring", 1), "dx": ("ring", 1)}


def test_plans():
    check_plans()


def test_plans_of_other_engines():
    """One size of each of the other engines, and what the query refuses."""
    bf = torch.bfloat16
    assert dense.linear_plan(1, 4096, 4096, bf) == {"fwd": ("stream", 1)}
    assert dense.linear_plan(33, 264, 4096, bf) == {"fwd": ("stream", 5)}
    assert dense.linear_plan(300, 712, 1000, bf) == {"fwd": ("64x64", 1)}
    assert dense.linear_plan(1183, 3296, 240, bf) == {"fwd": ("64x128", 1)}
    assert dense.linear_plan(4500, 264, 4104, bf) == {"fwd": ("128x128", 4)}
    assert dense.linear_plan(8293, 1456, 264, torch.float32)["fwd"][0] == "64x64"
    assert dense.linear_plan(300, 712, 1000, bf, dw=True, dx=True) == {"together": True, "dw": ("64x64", 1), "dx": ("64x64", 1)}
    with pytest.raises(TypeError, match="unsupported dtype"):
        dense.linear_plan(1, 8, 8, torch.float64)
    with pytest.raises(mlp.SwiGLUError):
        dense.linear_plan(1, 12, 8, bf)
    assert _lib.lib().swiglu_mlp_linear_plan(1, 8, 8, 0, 0, 0, None) == 1


@pytest.mark.gpu
def test_plans_on_the_device():
    check_plans()


@pytest.mark.gpu
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("shape", list(FORWARD))
def test_every_epilogue(shape, act):
    """Each activation with each of bias and residual, whole tiles and parts."""
    for k, (bias, res) in enumerate(((True, True), (False, True), (True, False), (False, False))):
        dtype = ("bf16", "fp16")[(k + ACTS.index(act)) % 2]
        banner(f"ring forward {shape} {dtype} {act} bias={bias} res={res}")
        check_linear(*shape, DTYPES[dtype], act, bias, res, 7000 + k, ())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("shape,needs", [(s, (False, True, True)) for s in DW] + [(s, (True, False, False)) for s in DX]
                         + [(s, ALL) for s in TOGETHER + APART])
def test_gradients(shape, needs, dtype):
    banner(f"ring gradients {shape} {dtype} {needs}")
    check_linear(*shape, DTYPES[dtype], "silu" if shape[0] % 2 else None, True, False, 7100, (needs,))


@pytest.mark.gpu
@pytest.mark.parametrize("shape", list(FORWARD))
def test_nan_and_infinity_keep_their_place(shape):
    banner(f"ring nan {shape}")
    T, N, K = shape
    x, w, r = (normal(gen(i), s, torch.bfloat16) for i, s in enumerate(((T, K), (N, K), (T, N))))
    clean = mlp.linear(x, w, None, "silu", r)
    x[1, K - 1], w[5, 0], r[2, N - 1], r[T - 1, 0] = math.nan, math.inf, math.nan, math.inf
    y = mlp.linear(x, w, None, "silu", r)
    up = x[:, 0] > 0
    up[1] = False
    assert y[1].isnan().all() and (y[up, 5] == math.inf).all() and y[2, N - 1].isnan() and y[T - 1, 0] == math.inf
    same = torch.ones_like(y, dtype=torch.bool)
    same[1], same[:, 5], same[2, N - 1], same[T - 1, 0] = False, False, False, False
    assert torch.equal(y[same], clean[same])


@pytest.mark.gpu
@pytest.mark.parametrize("shape", list(DW) + list(DX) + TOGETHER + APART)
def test_nan_gradients_keep_their_place(shape):
    """A NaN of dY reaches its token's row of dx and its column's row of dW."""
    banner(f"ring nan gradients {shape}")
    T, N, K = shape
    needs = (shape not in DW, shape not in DX, False)
    x, w, dy = (normal(gen(i), s, torch.bfloat16) for i, s in enumerate(((T, K), (N, K), (T, N))))
    clean = mlp.linear_bwd(dy, x, w, needs=needs)
    for t, n in ((T - 1, 3), (7, N - 1)):
        bad = dy.clone()
        bad[t, n] = math.nan
        for got, want, row in zip(mlp.linear_bwd(bad, x, w, needs=needs), clean, (t, n)):
            if want is not None:
                assert got[row].isnan().all()
                rest = torch.arange(want.shape[0], device=DEV) != row
                assert torch.equal(got[rest], want[rest])


def guarded(rows, cols, before=16):
    room = torch.full((rows + 300 + before, cols), 7.0, dtype=torch.bfloat16, device=DEV)
    return room, room[before:before + rows]


def untouched(room, rows, before=16):
    return (room[:before] == 7).all() and (room[before + rows:] == 7).all()


@pytest.mark.gpu
@pytest.mark.parametrize("shape", list(FORWARD))
def test_rows_around_the_outputs_are_left(shape):
    """y and z in the middle of larger buffers, more than a tile of rows behind them."""
    banner(f"ring rows around {shape}")
    L, (T, N, K) = _lib.lib(), shape
    x, w = normal(gen(1), (T, K), torch.bfloat16), normal(gen(2), (N, K), torch.bfloat16)
    r = normal(gen(3), (T, N), torch.bfloat16)
    (yr, y), (zr, z) = guarded(T, N), guarded(T, N)
    need = L.swiglu_mlp_linear_workspace_bytes(T, N, K, 0)
    ws = torch.full((need + 4096,), 9, dtype=torch.uint8, device=DEV)
    p = lambda t: t.data_ptr()  # noqa: E731
    assert L.swiglu_mlp_linear_fwd(p(x), p(w), None, p(r), p(y), p(z), p(ws), need, T, N, K, 4, 0, 0) == 0
    torch.cuda.synchronize()
    assert untouched(yr, T) and untouched(zr, T) and (ws[need:] == 9).all()
    want = mlp.linear_fwd(x, w, None, "silu", r)
    assert torch.equal(y, want[0]) and torch.equal(z, want[1])


@pytest.mark.gpu
@pytest.mark.parametrize("shape", list(DW) + list(DX) + TOGETHER + APART)
def test_rows_around_the_gradients_are_left(shape):
    banner(f"ring rows around gradients {shape}")
    L, (T, N, K) = _lib.lib(), shape
    x, w, dy, z = (normal(gen(i), s, torch.bfloat16) for i, s in enumerate(((T, K), (N, K), (T, N), (T, N))))
    needs = (shape not in DW, shape not in DX, True)
    (xr, dx), (wr, dw), (br, db) = guarded(T, K), guarded(N, K), guarded(N, 1)
    need = L.swiglu_mlp_linear_bwd_workspace_bytes(T, N, K, 4, 0)
    ws = torch.full((need + 4096,), 9, dtype=torch.uint8, device=DEV)
    p = lambda t, on=True: t.data_ptr() if on else None  # noqa: E731
    assert L.swiglu_mlp_linear_bwd(p(dy), p(x), p(w), p(z), p(dx, needs[0]), p(dw, needs[1]), p(db), p(ws), need, T, N, K, 4, 0, 0) == 0
    torch.cuda.synchronize()
    assert untouched(xr, T) and untouched(wr, N) and untouched(br, N) and (ws[need:] == 9).all()
    for got, want in zip((dx, dw, db.view(-1)), mlp.linear_bwd(dy, x, w, z, "silu", needs)):
        assert want is None and (got == 7).all() or torch.equal(got, want)


@pytest.mark.gpu
def test_offsets_past_32_bits():
    """Residual, z, y, dY and dz of more than 2^31 elements."""
    banner("ring past 32 bits")
    h = half(torch.bfloat16)
    T, N, K = LONG
    x, w = long(T, K, 5), normal(gen(6), (N, K), torch.bfloat16, 0.2)
    dy, bias = long(T, N, 7), normal(gen(8), (N,), torch.bfloat16)
    y, z = mlp.linear_fwd(x, w, bias, "silu", dy)
    rows = [0, 255, 256, T // 2, (1 << 31) // N - 1, (1 << 31) // N, T - 300, T - 2, T - 1]
    xr, wr, dr = x[rows].double(), w.double(), dy[rows].double()
    zr = xr @ wr.mT.contiguous() + bias.double()
    ez = (K / 4 + 64) * U * (xr.abs() @ wr.abs().mT.contiguous()) + 2 * U * zr.abs()
    inside(z[rows], zr, h * zr.abs() + ez, "z")
    yr = act64(zr, "silu")[0]
    inside(y[rows], yr + dr, h * (yr + dr).abs() + 1.2 * ez + 2e-5 * yr.abs() + 2 * U * (yr.abs() + dr.abs()), "y")
    del y
    dx, dw, db = mlp.linear_bwd(dy, x, w, z, "silu")
    dz = dr * act64(z[rows].double(), "silu")[1]
    e = h * dz.abs() + 3e-5 * dr.abs()
    inside(dx[rows], dz @ wr, h * (dz @ wr).abs() + 1.01 * (e @ wr.abs() + (N / 4 + 64) * U * (dz.abs() @ wr.abs())), "dx")
    cols = torch.tensor([0, 1, 4097, N - 1], device=DEV)
    dz = dy[:, cols].double() * act64(z[:, cols].double(), "silu")[1]
    e = h * dz.abs() + 3e-5 * dy[:, cols].double().abs()
    want, size = dz.mT.contiguous() @ x.double(), dz.abs().mT.contiguous() @ x.double().abs()
    inside(dw[cols], want, h * want.abs() + 1.01 * (e.mT.contiguous() @ x.double().abs() + (T / 4 + 64) * U * size), "dw")
    want = dz.sum(0)
    inside(db[cols], want, h * want.abs() + ((T / 256 + 320) * U * dz.abs() + 3e-5 * dy[:, cols].double().abs()).sum(0), "db")


# Every other engine, whole and in parts, and the streams by rows and waves.
OTHERS = {(7, 264, 200): ("stream", 1), (3, 9000, 64): ("stream", 1), (12, 264, 200): ("stream", 1), (13, 5000, 72): ("stream", 1),
          (33, 264, 4096): ("stream", 5), (600, 520, 2056): ("64x64", 5), (1183, 3296, 240): ("64x128", 1),
          (313, 1672, 3856): ("64x128", 7), (4200, 4104, 328): ("128x128", 1), (4500, 264, 4104): ("128x128", 4)}
# What the sizes of tests/test_dense.py's VARIANTS are there for: (dW, dx) alone, or what "both" says of the two.
GRADS = {(471, 4664, 880): ("dw", "64x128", 1), (1677, 208, 4672): ("dx", "64x128", 1), (136, 2848, 1288): ("dw", "128x128", 1),
         (892, 176, 3944): ("dx", "128x128", 1), (1048, 3648, 464): ("dx", "128x128", 7), (2987, 80, 4232): ("dw", "128x128", 7),
         (548, 208, 176): ("dx", "64x64", 1), (1106, 288, 200): ("dw", "64x64", 4), (2100, 4104, 2056): ("dx", "ring", 3)}


def test_plans_of_the_other_sizes():
    """Sizes here and in tests/test_dense.py take the launches that they are there for."""
    from tests.test_dense import LINEAR_SHAPES, VARIANTS

    for s, want in OTHERS.items():
        assert plan(s) == {"fwd": want}, s
    for s, (which, *want) in GRADS.items():
        assert s in VARIANTS and plan(s, **{which: True})[which] == tuple(want), s
    assert {plan(s)["fwd"][0] for s in LINEAR_SHAPES} == {"stream", "64x64", "128x128"}
    assert plan((4100, 2056, 1032))["fwd"] == ("ring", 1) and plan((4096, 2048, 5632))["fwd"] == ("ring", 2)
    together = plan((2100, 4104, 72), dw=True, dx=True)
    assert together["together"] and together["dw"] == ("64x64", 3) and together["dx"] == ("64x64", 7)


@pytest.mark.gpu
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("shape", list(OTHERS))
def test_every_epilogue_of_the_other_engines(shape, act):
    for k, (bias, res) in enumerate(((True, True), (False, True), (True, False), (False, False))):
        dtype = ("bf16", "fp16", "fp32")[(k + ACTS.index(act)) % 3]
        banner(f"forward {shape} {dtype} {act} bias={bias} res={res}")
        check_linear(*shape, DTYPES[dtype], act, bias, res, 7200 + k, ())
