"""What the dense training-side kernels' sources must not contain: read-only
loads.  Every one of these kernels may start while the launch before it still
runs and writes (programmatic dependent launch), and the read-only path assumes
memory that nobody writes for as long as the kernel lives."""

import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "bit_mixture_experts_route_b200", "csrc")
FILES = ["dense_gemm.cuh", "skinny_gemm.cuh", "ffn_gemv.cuh", "ffn.cu", "linear_ce.cu",
         "grad_clip.cu"]
# calls and instructions of that path, and what lets the compiler choose it
READ_ONLY = [r"__ldg\s*\(", r"ldg_stream_u\d\s*\(", r"\.global\.nc", r"const\s+\w+\s*\*\s*__restrict__"]


@pytest.mark.parametrize("name", FILES)
def test_no_read_only_loads(name):
    with open(os.path.join(CSRC, name)) as f:
        text = f.read()
    code = re.sub(r"//[^\n]*", "", text)
    found = [p for p in READ_ONLY if re.search(p, code)]
    assert not found, f"{name}: {found}"
