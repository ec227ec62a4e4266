"""Shared arrays that the paged kernels access through vector types are declared with the vectors' alignment: the
compiler places others on 4 bytes, and where that happens to suffice a new variable beside them can undo it."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "sparse_dimension_attention_b200", "csrc")
WIDTH = {"float2": 8, "float4": 16, "double2": 16, "uint2": 8, "uint4": 16, "int4": 16}


@pytest.mark.parametrize("path", sorted(glob.glob(os.path.join(CSRC, "paged_*.cu"))), ids=os.path.basename)
def test_vector_accesses_of_shared_arrays_are_aligned(path):
    text = open(path).read()
    functions = re.split(r"\n(?=template|__global__|__device__|struct)", text)
    for body in functions:
        for align, names in re.findall(r"__shared__ (?:__align__\((\d+)\) )?(?:float|double|int|uint32_t|uint8_t) ([^;]+);", body):
            have = int(align or 4)
            for name in re.findall(r"(\w+)(?:\[[^\]]*\])+", names):
                for vector in re.findall(r"reinterpret_cast<(?:const )?(\w+)\*>\(&?%s\b" % name, body):
                    assert have >= WIDTH.get(vector, 1), f"{name} is accessed as {vector} with an alignment of {have}"
