"""Build the HIP library ``libseacells_fw.so`` in-tree for gfx950."""
from __future__ import annotations

import os
import subprocess
import tempfile
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libseacells_fw.so")
SOURCES = ["abi.hip", "fw_a.hip", "fw_b.hip", "sparse_ops.hip", "abi_token.hip", "embed.hip",
           "layer_norm.hip", "logprobs.hip", "mm.hip", "ffn.hip", "ffn_d_pre.hip",
           "ffn_grad.hip", "linear_logprobs.hip", "few.hip"]
HEADERS = ["common.hpp", "token.hpp", "mm.hpp", "few.hpp", "ffn_grad.hpp"]

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC",
    # no packed-FP32 VALU forms anywhere in the device code
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-command-line-argument",
]


def sources():
    return [os.path.join(CSRC, s) for s in SOURCES]


def stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    deps = sources() + [os.path.join(CSRC, h) for h in HEADERS] + \
        [os.path.join(ROOT, "include", h) for h in ("seacells_fw.h", "seacells_sparse.h", "seacells_token.h",
                                                    "seacells_debug.h")]
    return any(os.path.getmtime(d) > t for d in deps)


def _run(cmd, verbose):
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("hipcc failed:\n" + res.stdout + res.stderr)


def build(verbose: bool = False) -> str:
    """Compile every HIP source into libseacells_fw.so (always recompiles),
    the sources side by side."""
    tmp = LIB + ".tmp%d" % os.getpid()
    with tempfile.TemporaryDirectory() as work:
        objects = [os.path.join(work, s.replace(".hip", ".o")) for s in SOURCES]

        def compile_one(pair):
            _run([HIPCC] + FLAGS + ["-I", os.path.join(ROOT, "include"), "-c", "-o", pair[1], pair[0]],
                 verbose)

        with ThreadPoolExecutor(min(len(SOURCES), os.cpu_count() or 1, 8)) as pool:
            list(pool.map(compile_one, zip(sources(), objects)))
        _run([HIPCC, "--offload-arch=gfx950", "-fPIC", "-shared", "-o", tmp] + objects, verbose)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
