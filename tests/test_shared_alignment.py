"""Shared arrays that kernels read or write as wider vectors are declared with that
alignment: where the compiler places the others is its own choice, and a vector
access at another address faults.  Read from the sources, on the CPU."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "linear_layers_b200", "csrc")
WIDTH = {"uint4": 16, "float4": 16, "int4": 16, "ulonglong2": 16, "longlong2": 16, "double2": 16,
         "uint2": 8, "float2": 8, "int2": 8, "uint64_t": 8, "int64_t": 8, "double": 8}
DECL = re.compile(r"^\s*(?:extern )?__shared__ (?:__align__\((\d+)\) )?(\w+) ([^;]+);", re.M)
CAST = re.compile(r"reinterpret_cast<(?:const )?(\w+)\*>\(&?(\w+)")


def misaligned(text):
    align = {}
    for m in DECL.finditer(text):
        own = max(int(m.group(1) or 1), WIDTH.get(m.group(2), 4))
        for name in re.findall(r"(\w+)(?=\[)", re.sub(r"\[[^\]]*\]", "[]", m.group(3))):
            align[name] = own
    for _ in range(2):                                 # pointers into them
        for new, old in re.findall(r"\b\w+\* (\w+) = &?(\w+)[\[;]", text):
            if old in align:
                align[new] = align[old]
    return [(name, t) for t, name in CAST.findall(text)
            if name in align and WIDTH.get(t, 1) > align[name]]


@pytest.mark.parametrize("path", sorted(glob.glob(os.path.join(CSRC, "*.cu*"))), ids=os.path.basename)
def test_vector_accesses_are_aligned(path):
    assert misaligned(open(path).read()) == []


def test_the_reading_finds_a_misaligned_array():
    text = """
  __shared__ uint32_t bits[4][64];
  __shared__ __align__(16) float fine[2][4], also[2][4];
  uint32_t* row = bits[warp];
  reinterpret_cast<uint4*>(row)[lane] = z;
  reinterpret_cast<const float4*>(also[k]);
"""
    assert misaligned(text) == [("row", "uint4")]
