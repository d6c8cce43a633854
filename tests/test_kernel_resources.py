"""What the compiler says of the kernels' registers: no norm kernel keeps a row in local memory.

A spilled row goes through memory twice more, which made rows off the vector
path slower than the same norm in separate torch operations.
"""
from __future__ import annotations

import os
import re
import subprocess

import pytest

from causal_depthwise_conv1d_fwd_gb300 import build


def resources(source: str, tmp_path):
    """{mangled kernel: (bytes spilled, registers)} of one source, from ptxas' report."""
    cmd = [build._nvcc(), *build.NVCC_FLAGS, "-Xptxas", "-v", "-c", os.path.join(build.CSRC, source), "-o",
           str(tmp_path / "x.o")]
    text = subprocess.run(cmd, capture_output=True, text=True, check=True).stderr
    found = re.findall(r"Compiling entry function '(\S+)'.*?(\d+) bytes spill stores, (\d+) bytes spill loads.*?Used (\d+) registers",
                       text, flags=re.S)
    return {name: (int(st) + int(ld), int(regs)) for name, st, ld, regs in found}


@pytest.fixture(scope="module")
def norms(tmp_path_factory):
    return resources("layer_norms.cu", tmp_path_factory.mktemp("norms"))


def test_norm_kernels_do_not_spill(norms):
    """No more than a few addresses of a thread: 16 bytes out and in.  What a thread has of a row is 64 bytes or more where
    registers are short."""
    assert len(norms) >= 2 * 13
    assert {name: r for name, r in norms.items() if r[0] > 32} == {}


def test_norm_blocks_fit_an_sm(norms):
    """Blocks of 1024 threads have 64 registers a thread."""
    for name, (_, regs) in norms.items():
        if "kernelILi1024E" in name:
            assert regs <= 64, name
