"""Loads that a check guards stay behind it: an asm statement without volatile has no side effect for the compiler,
which may run it for every thread. cuda_bf16.h's and cuda_fp16.h's __ldg and its relatives are such statements."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mixture_experts_layer_tcgen05_b200", "csrc")
SIXTEEN = r"(__nv_bfloat16|__nv_bfloat162|__half|__half2|half|half2)"


def code(path):
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", open(path).read(), flags=re.S)


@pytest.mark.parametrize("path", sorted(glob.glob(os.path.join(CSRC, "*.cu*"))), ids=os.path.basename)
def test_no_load_that_the_compiler_may_move(path):
    text = code(path)
    assert not re.search(r"\basm\s*\(", text), "asm without volatile"
    # pointers to 16-bit floats, by names that are declared as nothing else
    declared = re.findall(r"\b(\w+)\s*\*\s*(?:const\s+)?(?:__restrict__\s+)?(\w+)\b", text)
    names = {n for t, n in declared if re.fullmatch(SIXTEEN, t)} - {n for t, n in declared if not re.fullmatch(SIXTEEN, t)}
    for arg in re.findall(r"\b__ld(?:g|cg|ca|cs|lu|cv)\s*\(((?:[^()]|\((?:[^()]|\([^()]*\))*\))*)\)", text):
        cast = re.match(r"\s*&?\s*(?:reinterpret|static)_cast<\s*(?:const\s+)?(\w+)", arg)
        if cast:
            assert not re.fullmatch(SIXTEEN, cast.group(1)), arg
        else:
            first = re.match(r"\s*&?\s*(\w+)", arg)
            assert not (first and first.group(1) in names), arg
