"""Static checks of the compiled norm and linear kernels (CPU; compiled here): the
checks of tests/test_isa.py on the ring kernels with their epilogues, those of
tests/test_serve_isa.py on the streams of few tokens, and scratch only outside
of the ring's loops.
"""

import os
import re
import subprocess
import tempfile
from concurrent.futures import ThreadPoolExecutor

import pytest

from backward_gate_up_amd import build as B
from tests import test_isa as ring
from tests.test_serve_isa import hazards, matrix_hazards

UNITS = {name: defs for name, src, defs in B.UNITS if src == "dense_instantiate.hip"}


@pytest.fixture(scope="module")
def asm():
    def one(item):
        name, defs = item
        with tempfile.TemporaryDirectory() as d:
            out = os.path.join(d, "k.s")
            flags = [f for f in B.FLAGS if f != "-fPIC"]
            r = subprocess.run([B.HIPCC] + flags + defs + ["--cuda-device-only", "-S", "-o", out,
                                                           os.path.join(B.CSRC, "dense_instantiate.hip")],
                               capture_output=True, text=True)
            assert r.returncode == 0, r.stderr[-2000:]
            with open(out) as f:
                return name, f.read()

    if not os.path.exists(B.HIPCC):
        pytest.skip("hipcc not available")
    with ThreadPoolExecutor(min(8, len(UNITS))) as ex:
        return dict(ex.map(one, UNITS.items()))


def test_every_unit_is_checked():
    assert len(UNITS) == 16


def test_ring_loops_and_fences(asm):
    units = {u: t for u, t in asm.items() if "mfma_f32_16x16x32" in t}
    ring.test_mfma_loops_have_no_accumulator_copies_or_spills(units)
    assert sum(ring._check_valu_to_mfma_source(u, t) for u, t in units.items()) > 0
    for u, t in units.items():
        ring._check_fences(u, t)


def test_streams_keep_their_wait_states(asm):
    loads = products = kernels = 0
    for unit, text in asm.items():
        for name, body in ring._kernels(text):
            if "lin_few" not in name:
                continue
            kernels += 1
            bad, n = hazards(body)
            worse, k = matrix_hazards(body)
            assert not bad and not worse, (unit, name, bad[:3], worse[:3])
            loads, products = loads + n, products + k
    assert kernels >= 15 and loads >= 60 and products >= 60


def test_no_scratch(asm):
    for unit, text in asm.items():
        for m in re.finditer(r"^(_ZN6swiglu\w+):\s.*?ScratchSize: (\d+)", text, re.M | re.S):
            # a ring's last stages read their array pointers from scratch: none of it in a loop of matrix
            # instructions (above)
            limit = 64 if "ring" in m.group(1) else 0
            assert int(m.group(2)) <= limit, (unit, m.group(1), m.group(2))
