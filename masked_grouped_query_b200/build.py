"""Build ``libgqa_attn.so`` in-tree with nvcc for sm_100a.

Run ``python -m masked_grouped_query_b200.build`` (or ``__graft_entry__.build()``).
The library has two translation units, ``csrc/gqa_attn.cu`` (forward pass and
KV cache) and ``csrc/gqa_train.cu`` (backward pass, rotary positions),
compiled side by side, with the C ABI of ``include/gqa_attn.h``; it links the
CUDA runtime statically and reaches the driver's tensor-map encoder through
``cudaGetDriverEntryPoint``.
"""
from __future__ import annotations

import os
import subprocess
import sys
import tempfile

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIBRARY = os.path.join(PKG, "libgqa_attn.so")

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC",
    "--expt-relaxed-constexpr",
]
UNITS = ("gqa_attn", "gqa_train")


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.sep not in cand or os.path.exists(cand)):
            return cand
    return "nvcc"


def sources() -> list[str]:
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC)
                  if f.endswith((".cu", ".cuh", ".h")))


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile the library unless it is newer than every source and header."""
    deps = sources() + [os.path.join(INCLUDE, "gqa_attn.h")]
    if (not force and os.path.exists(LIBRARY)
            and os.path.getmtime(LIBRARY) >= max(os.path.getmtime(d) for d in deps)):
        return LIBRARY
    flags = [*NVCC_FLAGS, *(["-Xptxas=-v"] if verbose else []), f"-I{INCLUDE}"]
    # Objects and library are made in a folder of this build alone and the
    # library is moved into place whole: two builds at once do not meet.
    with tempfile.TemporaryDirectory(prefix="building-", dir=PKG) as tmp:
        objects = [os.path.join(tmp, u + ".o") for u in UNITS]
        compiles = [subprocess.Popen([nvcc(), *flags, "-c", os.path.join(CSRC, u + ".cu"), "-o", o],
                                     stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
                    for u, o in zip(UNITS, objects)]
        # Every compiler has ended before any failure is reported.
        outputs = [proc.communicate()[0] for proc in compiles]
        for u, proc, out in zip(UNITS, compiles, outputs):
            if proc.returncode != 0:
                raise RuntimeError(f"nvcc failed on {u}.cu:\n{out}")
            if verbose:
                sys.stderr.write(out)
        made = os.path.join(tmp, os.path.basename(LIBRARY))
        res = subprocess.run([nvcc(), *NVCC_FLAGS, "-shared", *objects, "-o", made],
                             capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError("nvcc failed to link:\n" + res.stdout + res.stderr)
        os.replace(made, LIBRARY)
    return LIBRARY


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
