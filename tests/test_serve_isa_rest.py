"""The static checks of tests/test_serve_isa.py on the few-token units that its list
leaves out, so that every unit the build compiles is looked at: wait states
around the loads into LDS and the matrix instructions, and no scratch.
"""

import os
import re
import subprocess
import tempfile
from concurrent.futures import ThreadPoolExecutor

import pytest

from backward_gate_up_amd import build as B
from tests.test_serve_isa import COMBOS, hazards, matrix_hazards

UNITS = {tuple(int(d.split("=")[1]) for d in defs): defs for _, src, defs in B.UNITS if src == "few_instantiate.hip"}
REST = sorted(set(UNITS) - set(COMBOS))


@pytest.fixture(scope="module")
def kernels():
    def one(combo):
        with tempfile.TemporaryDirectory() as d:
            out = os.path.join(d, "k.s")
            cmd = [B.HIPCC] + B.FLAGS + UNITS[combo] + ["--cuda-device-only", "-S", "-o", out,
                                                        os.path.join(B.CSRC, "few_instantiate.hip")]
            r = subprocess.run(cmd, capture_output=True, text=True)
            assert r.returncode == 0, r.stderr[-2000:]
            with open(out) as f:
                text = f.read()
        return {k.group(1): (text[k.start():k.end(0)], int(k.group(3))) for k in
                re.finditer(r"^(_ZN6swiglu\w+):\s.*?^\s+s_endpgm(.*?)ScratchSize: (\d+)", text, re.M | re.S)}

    with ThreadPoolExecutor(len(REST)) as ex:
        return dict(zip(REST, ex.map(one, REST)))


def test_every_unit_is_checked():
    assert len(UNITS) == 9 and set(COMBOS) <= set(UNITS) and len(REST) == len(UNITS) - len(COMBOS)


@pytest.mark.parametrize("combo", REST)
def test_wait_states_and_scratch(kernels, combo):
    assert len(kernels[combo]) >= 4
    loads = products = 0
    for name, (asm, scratch) in kernels[combo].items():
        bad, n = hazards(asm)
        worse, k = matrix_hazards(asm)
        loads, products = loads + n, products + k
        assert not bad and not worse, (name, bad[:3], worse[:3])
        assert scratch == 0, name
    assert loads >= 20 and products >= 40
