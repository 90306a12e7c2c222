"""The few-token serving operators: each launch variant at the sizes that select
it, with the other dimensions small. Formulas and bounds are those of
tests/test_serve.py: a result of one product carries one rounding of half a step,
one of two products two, and 1e-5 for the fp32 sums.
"""

import pytest

import backward_gate_up_amd as m
from tests._util import assert_local, banner, f64
from tests.test_serve import DT, bound, cuda, gen, make_w4, randn, ref_w4

gpu = pytest.mark.gpu


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
