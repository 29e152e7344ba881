"""LDS arrays of the linear and block-scaled products that are accessed in
16-byte pieces are declared on 16-byte boundaries (CPU, from the sources): the
pieces need it, and where the compiler puts an array of 4-byte values is its own
choice otherwise."""
import os
import re

import pytest

from tests.conftest import ROOT

CSRC = os.path.join(ROOT, "fp4_expert_ffn_amd", "csrc")
FILES = ["linear.hip", "linear_tile.h", "linear_block.hip", "linear_block_big.hip", "linear_block_stream.hip"]
WIDE = r"reinterpret_cast<(?:const )?(?:uint4|int4|float4|lf32x4_t)\*>\(&?(\w+)"


def undeclared(text):
    """(LDS arrays, those accessed in 16-byte pieces whose declaration says nothing about their place)."""
    wide, arrays, bad = set(re.findall(WIDE, text)), {}, []
    for decl in re.findall(r"__shared__ ([^;]*);", text):
        for name in re.findall(r"(\w+)\[", re.sub(r"\[[^\]]*\]", "[", decl)):
            arrays[name] = decl
    for name, decl in arrays.items():
        kind = decl.split()[0]
        if name in wide and "__align__" not in decl and not re.search(r"struct __align__\(16\) " + kind + r"\b", text):
            bad.append(name)
    return set(arrays), wide, bad


@pytest.mark.parametrize("name", FILES)
def test_arrays_of_wide_accesses_say_where_they_lie(name):
    arrays, wide, bad = undeclared(open(os.path.join(CSRC, name)).read())
    assert arrays & wide, name  # the patterns find the accesses that are there
    assert not bad, bad


def test_the_check_sees_a_missing_declaration():
    read = "auto f = [&] { return *reinterpret_cast<const int4*>(&s_t[k]); };"
    assert undeclared("struct T {\n int a;\n};\n__shared__ T s_t[8], s_u[4];\n" + read)[2] == ["s_t"]
    assert undeclared("struct __align__(16) T {\n int a;\n};\n__shared__ T s_t[8];\n" + read)[2] == []
    assert undeclared("__shared__ __align__(16) int s_t[8][4];\n" + read)[2] == []
