"""Rules that every kernel source keeps, checked in the text of csrc/."""
import glob
import os
import re

import pytest

import block_masked_token_gb300 as package

CSRC = os.path.join(os.path.dirname(package.__file__), "csrc")
SOURCES = sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh")))
BYTES = {"bool": 1, "uint8_t": 1, "uint16_t": 2, "int": 4, "int32_t": 4, "uint32_t": 4, "float": 4,
         "double": 8, "uint64_t": 8, "long long": 8, "int2": 8, "uint2": 8, "float2": 8, "int4": 16,
         "uint4": 16, "float4": 16}


def underaligned_casts(text):
    """Shared arrays cast to a type of a larger alignment than their declaration promises."""
    found = []
    for m in re.finditer(r"__shared__ (alignas\((\d+)\) )?([a-z_0-9]+(?: long)?) ([^;]*);", text):
        if m[3] not in BYTES:
            continue
        aligned = max(BYTES[m[3]], int(m[2] or 1))
        for name in re.findall(r"(\w+)\s*(?:\[[^,;]*\])", m[4]):
            for cast in re.findall(r"reinterpret_cast<(?:const )?(\w+(?: long)?)\s*\*>\(&?%s\b" % name, text):
                if BYTES.get(cast, 0) > aligned:
                    found.append((name, cast))
    return found


def test_the_rule_sees_a_cast():
    text = "__shared__ int a, b[3 * 4], c[2]; x = reinterpret_cast<const int2*>(b + 2);"
    assert underaligned_casts(text) == [("b", "int2")]
    assert not underaligned_casts(text.replace("__shared__ int a, b", "__shared__ alignas(8) int b"))


@pytest.mark.parametrize("path", SOURCES, ids=os.path.basename)
def test_shared_arrays_are_aligned_for_their_casts(path):
    assert not underaligned_casts(open(path).read())
