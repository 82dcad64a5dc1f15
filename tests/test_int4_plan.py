"""How the few-token kernel divides a call: the host's arithmetic, compiled by itself."""
import ctypes
import os
import subprocess

import pytest
import torch

from quantized_linear_layers_nf4_b200.build import CSRC, NVCC_FLAGS, build, nvcc

gpu = pytest.mark.gpu

# the widest rows that a pass of so many tokens takes, as nf4_int4_plan.h states them
BORDERS = [(16, 33792), (8, 64512), (4, 65536)]

SOURCE = r"""
#include "nf4_int4_plan.h"
using namespace nf4;
static Int4Args weight(int64_t n, int64_t k, int64_t group) { return Int4Args{n, k, group, nullptr, nullptr, nullptr, false}; }
extern "C" int64_t tokens_of_pass(int64_t m, int64_t k, int64_t group) { return nf4::int4::tokens_of_pass(m, weight(64, k, group)); }
"""


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    d = tmp_path_factory.mktemp("plan")
    (d / "plan.cu").write_text(SOURCE)
    subprocess.run([nvcc(), *NVCC_FLAGS, "-shared", "-cudart", "static", str(d / "plan.cu"), "-o", str(d / "plan.so")], check=True,
                   capture_output=True)
    lib = ctypes.CDLL(str(d / "plan.so"))
    lib.tokens_of_pass.restype = ctypes.c_int64
    lib.tokens_of_pass.argtypes = [ctypes.c_int64] * 3
    return lib


@pytest.mark.parametrize("unit", [32, 64])  # the two paddings of X
def test_tokens_of_a_pass(plan, unit):
    text = open(os.path.join(CSRC, "nf4_int4_plan.h")).read()
    stated = " ".join(text.replace("//", "").split())
    assert "all sixteen up to k = %d, eight to %d, then four" % (BORDERS[0][1], BORDERS[1][1]) in stated
    for (tokens, last), (fewer, _) in zip(BORDERS, BORDERS[1:]):
        assert plan.tokens_of_pass(16, last, unit) == tokens
        assert plan.tokens_of_pass(16, last + 64, unit) == fewer
    assert plan.tokens_of_pass(16, 64, unit) == 16 and plan.tokens_of_pass(16, 65536, unit) == 4


@gpu
@pytest.mark.parametrize("m,k", [(16, 33792), (16, 33856), (9, 33856), (8, 64512), (8, 64576), (16, 64576), (5, 64576), (4, 65536)])
@pytest.mark.parametrize("group", [32, 64])
def test_linear_at_the_borders(m, k, group):
    """Small integers and scales of a quarter: every sum is exact (below 2^24 quarters)."""
    build()
    import quantized_linear_layers_nf4_b200 as nf4
    n = 40
    g = torch.Generator(device="cuda").manual_seed(k + m)
    wq = torch.randint(0, 256, (n * k // 2,), dtype=torch.uint8, device="cuda", generator=g)
    zero = torch.randint(0, 16, (k // group, n), dtype=torch.uint8, device="cuda", generator=g)
    w = nf4.Int4Weight(n, k, group, wq, torch.full((k // group, n), 0.25, device="cuda"), zero)
    x = torch.randint(-4, 5, (m, k), device="cuda", generator=g).bfloat16()
    dense = nf4.nf4_int4_dequantize(w, torch.float32).double()
    assert torch.equal(nf4.nf4_int4_linear(x, w, torch.float32).double(), x.double() @ dense.t())
