"""Shared arrays that a kernel reads as vectors are declared with the vector's
alignment: nothing else guarantees it, wherever the compiler happens to place
them today (CPU only, by reading the sources)."""
import glob
import os
import re

from tests.conftest import ROOT

CSRC = os.path.join(ROOT, "mixed_precision_quantized_act_b200", "csrc")
BYTES = {"float2": 8, "uint2": 8, "int2": 8, "float4": 16, "uint4": 16, "int4": 16, "ulonglong2": 16, "double2": 16}
NATURAL = {"uint8_t": 1, "int8_t": 1, "int": 4, "uint32_t": 4, "float": 4, "unsigned int": 4, "uint64_t": 8,
           "int64_t": 8, "long long": 8, "unsigned long long": 8, **BYTES}
DECLARED = re.compile(r"__shared__\s+(?:__align__\((\d+)\)\s+)?(?:volatile\s+)?((?:unsigned |long )*\w+)\s+([^;]*);")
READ = re.compile(r"reinterpret_cast<(?:const )?(%s) \*>\(\s*&?(\w+)\s*(?:\[|\))" % "|".join(BYTES))


def _faults(text):
    align = {}
    for given, kind, names in DECLARED.findall(text):
        for name in re.findall(r"(\w+)\s*(?:\[[^\]]*\]\s*)+", names):
            align[name] = max(int(given or 0), NATURAL.get(kind, 1))
    return [(name, vec, align[name]) for vec, name in READ.findall(text)
            if name in align and align[name] < BYTES[vec]]


def test_vector_reads_of_shared_arrays_are_aligned():
    faults = {}
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu*"))):
        with open(path) as f:
            found = _faults(f.read())
        if found:
            faults[os.path.basename(path)] = found
    assert not faults


def test_the_search_finds_what_it_looks_for():
    bad = "__shared__ float top[4][4];\n x = *reinterpret_cast<const float4 *>(top[i]);"
    assert _faults(bad) == [("top", "float4", 4)]
    assert not _faults(bad.replace("float top", "__align__(16) float top"))
    assert _faults("__shared__ uint32_t a[2], b[8];\n reinterpret_cast<const uint2 *>(&b[at])") == [("b", "uint2", 4)]
