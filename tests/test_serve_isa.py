"""Static checks of the few-token kernels' assembly (CPU; compiled here).

Their loads into LDS come from inline assembly, whose hazards the compiler does
not see: between a vector instruction that writes a scalar register and a memory
instruction that reads it, five wait states are needed, and one between a write
of M0 and a load into LDS. Likewise a matrix instruction reads what a vector
instruction wrote only two wait states later: the compiler sees to that for its
own instructions and not for assembly. Checked in program order, with self-tests
that a short distance is caught. And no kernel may use scratch.
"""

import os
import re
import subprocess
import tempfile
from concurrent.futures import ThreadPoolExecutor

import pytest

from backward_gate_up_amd import build as B

COMBOS = [(0, 0), (2, 0), (0, 128), (0, 32), (1, 32), (1, 64)]
LOAD = re.compile(r"^buffer_load_dword(?:x4)? v\d+, (s\[(\d+):(\d+)\]|v\S+), (\S+) offen.* lds")
DST = re.compile(r"^(v_\w+) (m0|vcc|s\d+|s\[\d+:\d+\])(?:,|$)")


def instructions(asm):
    """(mnemonic line, wait states it fills) of one kernel, in program order."""
    for ln in asm.splitlines():
        t = ln.split(";")[0].strip()
        if not t or t.startswith(".") or t.endswith(":"):
            continue
        m = re.match(r"s_nop (\d+)", t)
        yield t, (int(m.group(1)) + 1 if m else 1)


def scalars(t):
    if t.startswith("s["):
        a, b = map(int, t[2:-1].split(":"))
        return {f"s{i}" for i in range(a, b + 1)}
    return {t}


def hazards(asm):
    bad, at, written, m0 = [], 0, {}, -99
    n = 0
    for t, states in instructions(asm):
        m = LOAD.match(t)
        if m:
            n += 1
            if not m.group(1).startswith("s["):
                bad.append("descriptor in vector registers: " + t)
            need = scalars(m.group(1)) | ({m.group(4)} if m.group(4).startswith("s") else set()) | {"m0"}
            for r in need:
                if at - written.get(r, -99) < 6:
                    bad.append(f"{r} written {at - written[r] - 1} states before: {t}")
            if at - m0 < 2:
                bad.append("m0 written just before: " + t)
        d = DST.match(t)
        if d:
            for r in scalars(d.group(2)):
                written[r] = at + states - 1
        if re.match(r"^s_\w+ m0,", t):
            m0 = at
        at += states
    return bad, n


def vectors(t):
    m = re.match(r"v\[(\d+):(\d+)\]$", t)
    if m:
        return range(int(m.group(1)), int(m.group(2)) + 1)
    return [int(t[1:])] if re.match(r"v\d+$", t) else []


def matrix_hazards(asm):
    """Matrix instructions with fewer than 2 wait states after a vector
    instruction's write of one of their operands; and how many there are."""
    bad, at, written, n = [], 0, {}, 0
    for t, states in instructions(asm):
        op, _, rest = t.partition(" ")
        args = [a.strip() for a in rest.split(",")]
        if op.startswith("v_mfma"):
            n += 1
            for a in args[1:4]:
                bad += [f"v{r} written {at - written[r] - 1} states before: {t}" for r in vectors(a)
                        if at - written.get(r, -99) < 3]
        for r in vectors(args[0]):
            if op.startswith("v_") and not op.startswith("v_mfma"):
                written[r] = at
            elif op.startswith(("v_mfma", "ds_read", "buffer_load", "global_load")):
                written.pop(r, None)
        at += states
    return bad, n


@pytest.fixture(scope="module")
def kernels():
    def one(c):
        with tempfile.TemporaryDirectory() as d:
            out = os.path.join(d, "k.s")
            cmd = [B.HIPCC] + B.FLAGS + [f"-DSWIGLU_INST_DTYPE={c[0]}", f"-DSWIGLU_INST_FMT={c[1]}", "--cuda-device-only",
                                         "-S", "-o", out, os.path.join(B.CSRC, "few_instantiate.hip")]
            r = subprocess.run(cmd, capture_output=True, text=True)
            assert r.returncode == 0, r.stderr[-2000:]
            text = open(out).read()
        found = {}
        for m in re.finditer(r"^(_ZN6swiglu\w+):\s.*?^\s+s_endpgm(.*?)ScratchSize: (\d+)", text, re.M | re.S):
            found[m.group(1)] = (text[m.start():m.end(0)], int(m.group(3)))
        return found

    with ThreadPoolExecutor(len(COMBOS)) as ex:
        return dict(zip(COMBOS, ex.map(one, COMBOS)))


@pytest.mark.parametrize("combo", COMBOS)
def test_lds_loads_keep_their_wait_states(kernels, combo):
    loads = 0
    assert len(kernels[combo]) >= 4
    for name, (asm, scratch) in kernels[combo].items():
        bad, n = hazards(asm)
        loads += n
        assert not bad, (name, bad[:3])
        assert scratch == 0, name
    assert loads >= 20


@pytest.mark.parametrize("combo", COMBOS)
def test_matrix_operands_keep_their_wait_states(kernels, combo):
    count = 0
    for name, (asm, _) in kernels[combo].items():
        bad, n = matrix_hazards(asm)
        count += n
        assert not bad, (name, bad[:3])
    assert count >= 40


def test_matrix_checker_catches_short_distances():
    mfma = "v_mfma_f32_16x16x32_bf16 v[0:3], v[4:7], v[8:11], v[0:3]\n"
    assert matrix_hazards("v_and_or_b32 v9, v1, s0, v2\ns_nop 1\n" + mfma) == ([], 1)
    assert matrix_hazards("v_and_or_b32 v9, v1, s0, v2\ns_nop 0\n" + mfma)[0]
    assert not matrix_hazards("v_mov_b32 v9, v1\nds_read_b128 v[8:11], v20\n" + mfma)[0]


def test_checker_catches_short_distances():
    ok = "v_readfirstlane_b32 s4, v1\ns_nop 4\ns_mov_b32 m0, s9\ns_nop 0\nbuffer_load_dwordx4 v2, s[4:7], 0 offen lds\n"
    assert hazards(ok) == ([], 1)
    assert hazards(ok.replace("s_nop 4", "s_nop 1"))[0]
    assert hazards(ok.replace("s_nop 0\n", ""))[0]
    assert hazards(ok.replace("s[4:7]", "v[4:7]"))[0]
    assert hazards("v_readlane_b32 m0, v1, 3\ns_nop 3\nbuffer_load_dword v2, s[4:7], 0 offen lds\n")[0]
