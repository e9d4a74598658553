"""The calls around a draft model start before the kernel ahead of them has ended
(programmatic dependent launch) and read what it, or one before it, writes.  The
read-only path (ld.global.nc, __ldg) is for memory that nobody writes while the
kernel runs: its lines may be older than the wait for that kernel.  None of their
kernels uses it, on the CPU by reading the sources."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "lossless_bit_weight_w12_gb300", "csrc")
READ_ONLY = re.compile(r"__ldg\(|\bldg_\w+\(|ld\.global\.nc|__restrict__")


@pytest.mark.parametrize("name", ["kernels_norm.cu", "kernels_fp4.cu", "kernels_fp4_tc.cu", "fp4_device.cuh", "kernels_cut.cu",
                                  "cut_device.cuh", "kernels_accept.cu", "step_device.cuh", "sample_device.cuh"])
def test_no_read_only_loads(name):
    for at, line in enumerate(open(os.path.join(CSRC, name)), 1):
        assert not READ_ONLY.search(line.split("//")[0]), (name, at, line.strip())
