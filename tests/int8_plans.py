"""Which kernel the 8-bit integer operators take for a product, from the library's own header (csrc/int8_plan.h).

``tests/int8_plan_probe.cpp`` evaluates the functions that the library calls; this module compiles it once per process
(g++ and the CUDA headers), so that a test that means one kernel can say so and fails where another would run.
"""
from __future__ import annotations

import collections
import os
import shutil
import subprocess
import tempfile

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
DTYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
GB300 = 76, 38, 18          # clusters of one, two and four pairs of CTAs that run at once on the whole chip

Plan = collections.namedtuple("Plan", "ok small shape cols run splits join units run_taken tiles_r tiles_c")
_exe = None


def available():
    return shutil.which("g++") is not None


def _probe():
    global _exe
    if _exe is None:
        cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
        exe = os.path.join(tempfile.mkdtemp(prefix="int8_plan"), "probe")
        subprocess.run(["g++", "-std=c++17", "-O1", "-I", os.path.join(ROOT, "dense_fp32_gemm_03_gb300", "csrc"),
                        "-I", os.path.join(ROOT, "include"), "-I", os.path.join(cuda, "include"),
                        os.path.join(ROOT, "tests", "int8_plan_probe.cpp"), "-o", exe], check=True)
        _exe = exe
    return _exe


def plans(lines):
    """Plans of (kind, kept, dtype, in place, vectors, m, n, k, pairs, twos, fours) each."""
    out = subprocess.run([_probe()], input="".join(" ".join(str(int(v)) for v in line) + "\n" for line in lines), capture_output=True,
                         text=True, check=True).stdout
    return [Plan(*map(int, line.split())) for line in out.splitlines()]


def product(m, n, k, quantised=False, clusters=GB300):
    """int8_gemm's (quantised tokens) or int8_linear's plan."""
    return plans([(0, quantised, 0, 0, 0, m, n, k, *clusters)])[0]


def gradient(m, n, k, kept, dtype=None, aligned=True, clusters=GB300):
    """int8_weight_grad's plan for m tokens, n columns of dY and k channels; aligned: dY's rows are at multiples of 16 bytes."""
    dtype = kept if dtype is None else dtype
    return plans([(1, DTYPES[kept], DTYPES[dtype], aligned and kept != torch.float32, aligned and n % 8 == 0, m, n, k, *clusters)])[0]
