"""Build the HIP library in-tree: backward_gate_up_amd/libswiglu_mlp.so (gfx950),
and the autograd nodes in C++ that call it: backward_gate_up_amd/_nodes.so.

The kernels are instantiated in eighteen translation units (csrc/instantiate.hip
compiled once per dtype, entry point and weight layout), the few-token serving
kernels in nine more (csrc/few_instantiate.hip, once per dtype and weight
format), the norms and the linear layer in sixteen (csrc/dense_instantiate.hip,
once per dtype and part), plus the C ABI (csrc/swiglu_mlp.hip, csrc/few.hip,
csrc/dense.hip); they compile in parallel and are linked into one shared library.
The nodes (csrc/nodes.cpp, host code) are compiled against torch's headers.
"""

import os
import subprocess
import sys
import tempfile
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
OUT = os.path.join(HERE, "libswiglu_mlp.so")
NODES = os.path.join(HERE, "_nodes.so")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")

FLAGS = [
    "--offload-arch=gfx950",
    "-O3",
    "-std=c++17",
    "-fPIC",
    # no packed-fp32 VALU instructions (v_pk_*_f32) anywhere
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wno-unused-result",
    "-I", os.path.join(ROOT, "include"),
]

# (object name, source, defines)
UNITS = [("abi", "swiglu_mlp.hip", [])] + [
    (f"{dt}_{op}_{lay}", "instantiate.hip",
     [f"-DSWIGLU_INST_DTYPE={i}", f"-DSWIGLU_INST_OP={j}", f"-DSWIGLU_INST_LIN={k}"])
    for i, dt in enumerate(("bf16", "fp16", "fp32")) for j, op in enumerate(("fwd", "bwd", "infer"))
    for k, lay in enumerate(("kernel", "linear"))
] + [("few", "few.hip", [])] + [
    (f"{dt}_few_{fmt}", "few_instantiate.hip", [f"-DSWIGLU_INST_DTYPE={i}", f"-DSWIGLU_INST_FMT={fmt}"])
    for i, dt in enumerate(("bf16", "fp16", "fp32")) for fmt in (0, 32, 64, 128) if fmt == 0 or dt != "fp32"
] + [("dense", "dense.hip", [])] + [
    (f"{dt}_dense_{part}", "dense_instantiate.hip", [f"-DSWIGLU_INST_DTYPE={i}", f"-DSWIGLU_INST_PART={part}"])
    for i, dt in enumerate(("bf16", "fp16", "fp32")) for part in range(7) if part < 2 or dt != "fp32"
]


def _node_commands(obj, tmp):
    """Compiling and linking csrc/nodes.cpp."""
    import sysconfig

    from torch.utils import cpp_extension as ext

    includes = [sysconfig.get_paths()["include"], os.path.join(ROOT, "include"), *ext.include_paths(),
                os.path.join(os.path.dirname(HIPCC), os.pardir, "include")]
    compile_ = ["g++", "-O2", "-std=c++17", "-fPIC", "-D__HIP_PLATFORM_AMD__", "-DUSE_ROCM", "-DTORCH_EXTENSION_NAME=_nodes"]
    compile_ += [f"-I{d}" for d in includes[:2]] + [a for d in includes[2:] for a in ("-isystem", d)]
    compile_ += ["-c", "-o", obj, os.path.join(CSRC, "nodes.cpp")]
    link = ["g++", "-shared", "-o", tmp, obj, f"-L{HERE}", "-lswiglu_mlp", "-Wl,-rpath,$ORIGIN"]
    link += [f"-L{d}" for d in ext.library_paths()] + ["-lc10", "-lc10_hip", "-ltorch_cpu", "-ltorch", "-ltorch_python"]
    return compile_, link


def _filter(text):
    return [ln for ln in text.splitlines() if "packed-fp32-ops' is not a recognized feature" not in ln]


def build(verbose=False, jobs=None):
    """Compile every unit and link the libraries (always). Raises on failure."""
    jobs = jobs or max(1, min(len(UNITS), len(os.sched_getaffinity(0))))
    with tempfile.TemporaryDirectory(prefix="swiglu_build_") as tmpdir:
        nodes = os.path.join(tmpdir, "nodes.o")
        compile_nodes, link_nodes = _node_commands(nodes, NODES + ".tmp")
        objs = [os.path.join(tmpdir, name + ".o") for name, _, _ in UNITS]
        work = [("nodes", compile_nodes)] + [
            (name, [HIPCC] + FLAGS + defs + ["-c", "-o", obj, os.path.join(CSRC, src)])
            for (name, src, defs), obj in zip(UNITS, objs)]
        with ThreadPoolExecutor(jobs) as ex:
            results = list(ex.map(lambda w: subprocess.run(w[1], capture_output=True, text=True), work))
        for (name, cmd), r in zip(work, results):
            msgs = _filter(r.stdout + r.stderr)
            if verbose:
                print(" ".join(cmd), flush=True)
                if msgs:
                    print("\n".join(msgs))
            if r.returncode != 0:
                raise RuntimeError(f"{os.path.basename(cmd[0])} failed on {name}:\n" + "\n".join(msgs))
        link = [HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", "-o", OUT + ".tmp"] + objs
        for cmd, tmp, out in ((link, OUT + ".tmp", OUT), (link_nodes, NODES + ".tmp", NODES)):
            r = subprocess.run(cmd, capture_output=True, text=True)
            if r.returncode != 0:
                raise RuntimeError("link failed:\n" + "\n".join(_filter(r.stdout + r.stderr)))
            os.replace(tmp, out)
    return OUT


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
