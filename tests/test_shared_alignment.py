"""Shared arrays that a kernel accesses through a wider vector type carry that alignment in their declaration: a plain
array of 4-byte elements is 4-byte aligned, and whether it lands on a 16-byte boundary is the compiler's choice."""
import glob
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCES = sorted(glob.glob(os.path.join(ROOT, "hadamard_rotated_bit_kvq3_gb300", "csrc", "*.cu*")))
NATURAL = {"uint4": 16, "int4": 16, "float4": 16, "uint2": 8, "int2": 8, "float2": 8, "int64_t": 8, "uint64_t": 8,
           "long long": 8, "double": 8, "uint32_t": 4, "int32_t": 4, "int": 4, "float": 4, "__half": 2, "uint8_t": 1}
DECL = re.compile(r"(?:extern\s+)?__shared__\s+(?:__align__\((\d+)\)\s+)?(?:unsigned\s+)?(long long|\w+)\s+([^;]+);")
CAST = re.compile(r"reinterpret_cast<(?:const )?(?:volatile )?(u?int[24]|float[24])\s*\*>\(\s*&?(\w+)(?:\.\w+)?\b")


def violations(text):
    aligned = dict(NATURAL)
    for n, name in re.findall(r"struct __align__\((\d+)\) (\w+)", text):
        aligned[name] = int(n)
    arrays = {}
    for align, kind, names in DECL.findall(text):
        for name in re.findall(r"(\w+)\s*(?:\[|,|$)", names):
            arrays[name] = int(align) if align else aligned.get(kind, 1)
    return [(name, kind) for kind, name in CAST.findall(text) if name in arrays and arrays[name] < NATURAL[kind]]


def test_declared_alignment():
    assert SOURCES
    for path in SOURCES:
        assert violations(open(path).read()) == [], os.path.basename(path)


def test_the_check_finds_a_plain_array():
    use = "x = *reinterpret_cast<const uint4*>(&hist[4 * t]);"
    assert violations("__shared__ uint32_t hist[kBins];" + use) == [("hist", "uint4")]
    assert violations("__shared__ __align__(16) uint32_t hist[kBins];" + use) == []
    use = "x = *reinterpret_cast<const uint4*>(&hist.n[4 * t]);"
    assert violations("struct Bins { uint32_t n[8]; }; __shared__ Bins hist;" + use) == [("hist", "uint4")]
    assert violations("struct __align__(16) Bins { uint32_t n[8]; }; __shared__ Bins hist;" + use) == []
