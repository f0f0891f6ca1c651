"""The ncu summaries of the serving kernels, without a GPU: each names a kernel
that the sources have, with as many template arguments as it takes there, so
that a summary does not outlive the kernel that it shows."""
import os
import re

import pytest

import frequency_ranked_drafter_gb300 as vt

CSRC = os.path.join(os.path.dirname(vt.__file__), "csrc")
PROFILES = os.path.join(os.path.dirname(os.path.dirname(vt.__file__)), "profiles")


def kernels():
    """Name -> number of template arguments, of every __global__ function."""
    found = {}
    for name in os.listdir(CSRC):
        if name.endswith(".cu"):
            text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())
            for m in re.finditer(r"(?:template\s*<([^>]*)>\s*)?__global__\s+void\s+"
                                 r"(?:__launch_bounds__\([^)]*\)\s*)?(\w+)\s*\(", text):
                found[m[2]] = len(m[1].split(",")) if m[1] else 0
    return found


@pytest.mark.parametrize("name", ["matmul_i8.md", "quantize_sample_verify.md"])
def test_summaries_name_kernels_of_the_sources(name):
    have = kernels()
    named = re.findall(r"^Kernel: `(?:void )?(\w+)(?:<([^>]*)>)?\(",
                       open(os.path.join(PROFILES, name)).read(), flags=re.M)
    assert named
    for kernel, args in named:
        assert kernel in have, kernel
        assert (len(args.split(",")) if args else 0) == have[kernel], (kernel, args)
