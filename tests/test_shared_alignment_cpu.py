"""Static shared-memory arrays of the kernels that are read or written as
vectors have the vector's alignment by their declaration, not by where the
compiler happens to place them (CPU: read from the sources)."""
import os
import re

import pytest

from alibi_attention_block_gb300.build import CSRC

ALIGN = {"float": 4, "int": 4, "uint32_t": 4, "int32_t": 4, "unsigned": 4, "uint16_t": 2, "float2": 8, "uint2": 8,
         "int2": 8, "uint64_t": 8, "double": 8, "float4": 16, "uint4": 16, "int4": 16}
SHARED = re.compile(r"(?<!extern )__shared__\s+(?:__align__\((\d+)\)\s+|alignas\((\d+)\)\s+)?(\w+)\s+([^;]+);")
CAST = re.compile(r"reinterpret_cast<\s*(?:const\s+)?(\w+)\s*\*\s*>\(\s*&?(\w+)")


def misaligned(text):
    text = re.sub(r"//[^\n]*", "", text)
    declared = {}
    for a, b, kind, names in SHARED.findall(text):
        for name in re.findall(r"(\w+)\s*\[", names):
            declared[name] = max(int(a or 0), int(b or 0), ALIGN.get(kind, 0))
    return [(name, kind) for kind, name in CAST.findall(text)
            if name in declared and declared[name] < ALIGN.get(kind, 0)]


@pytest.mark.parametrize("file", sorted(f for f in os.listdir(CSRC) if f.endswith((".cu", ".cuh", ".h"))))
def test_vectors_in_static_shared_memory(file):
    with open(os.path.join(CSRC, file), encoding="utf-8") as f:
        assert misaligned(f.read()) == []


def test_the_check_sees_a_cast():
    body = "float4* p = reinterpret_cast<float4*>(&part[w][at]);"
    assert misaligned("__shared__ float part[16][64];" + body) == [("part", "float4")]
    assert misaligned("__shared__ __align__(16) float part[16][64];" + body) == []
    assert misaligned("__shared__ float4 part[16][16];" + body) == []
