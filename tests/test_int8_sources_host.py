"""What the 8-bit integer operators' sources have to say for themselves (no GPU needed)."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "dense_fp32_gemm_03_gb300", "csrc")
BYTES = {"uint4": 16, "int4": 16, "float4": 16, "uint2": 8, "int2": 8, "float2": 8, "uint32_t": 4, "int32_t": 4, "float": 4, "__half2": 4, "int": 4,
         "uint64_t": 8, "uint16_t": 2, "int8_t": 1, "unsigned char": 1}


@pytest.mark.parametrize("path", sorted(glob.glob(os.path.join(CSRC, "int8_*.cu"))), ids=os.path.basename)
def test_shared_arrays_are_as_aligned_as_they_are_read(path):
    """An array in shared memory that is accessed as a wider type says its alignment; the compiler only knows its element's."""
    text = re.sub(r"//.*", "", open(path).read())
    kernels = re.split(r"(?=\n(?:template[^\n]*\n)?__global__ )", text)
    for kernel in kernels:
        for align, kind, name in re.findall(r"__shared__\s+(?:__align__\((\d+)\)\s+)?(unsigned char|\w+)\s+(\w+)\[", kernel):
            have = max(int(align or 1), BYTES[kind])
            # What points to it or to one of its rows counts as it (not what code aligned itself).
            names = {name} | set(re.findall(r"\*\s*(?:const\s+)?(\w+)\s*=\s*" + name + r"(?:\[[^;]*\])?;", kernel))
            for n in names:
                for wide in re.findall(r"reinterpret_cast<(?:const\s+)?([\w ]+?)\s*\*>\(&?" + n + r"\b", kernel):
                    assert have >= BYTES[wide], f"{os.path.basename(path)}: {name} is accessed as {wide}"
