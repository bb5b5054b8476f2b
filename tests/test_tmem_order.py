"""Tensor memory and programmatic launches, from the sources.

A kernel's allocation of tensor memory blocks until another CTA gives some up,
without a limit.  A CTA of a dependent kernel that was launched early holds
what it allocated until the kernel in front has ended; so a kernel that lets
its dependents start has to have allocated before, in every CTA, or each can
come to wait for the other."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "grouped_gemm_glu_gb300", "csrc")


def _kernels(text):
    """(name, body) of the __global__ functions."""
    for m in re.finditer(r"__global__\s+void\s+(?:__launch_bounds__\s*\((?:[^()]|\([^()]*\))*\)\s*)?(\w+)\s*\(", text):
        i = text.index("{", m.end())
        depth, j = 0, i
        while True:
            depth += {"{": 1, "}": -1}.get(text[j], 0)
            j += 1
            if depth == 0:
                break
        yield m.group(1), text[i:j]


@pytest.mark.parametrize("name", sorted(f for f in os.listdir(CSRC) if f.endswith(".cu")))
def test_dependents_start_behind_the_allocation(name):
    with open(os.path.join(CSRC, name)) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    found = list(_kernels(text))
    assert len(found) == text.count("__global__"), name
    for kernel, body in found:
        alloc, launch = body.find("tmem_alloc"), body.find("launch_dependents")
        if alloc >= 0 and launch >= 0:
            assert alloc < launch, f"{kernel}: lets its dependents start before it has its tensor memory"
            assert "__syncthreads" in body[alloc:launch], f"{kernel}: any thread's signal counts for its CTA"


def test_the_kernels_that_the_rule_is_for_are_found():
    with open(os.path.join(CSRC, "lora.cu")) as f:
        names = [k for k, body in _kernels(re.sub(r"//[^\n]*", "", f.read())) if "tmem_alloc" in body]
    assert names == ["k_shrink", "k_wgrad", "k_expand"]
