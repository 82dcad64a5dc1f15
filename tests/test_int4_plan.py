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
// A device of `sms` SMs that runs clusters of up to `most` CTAs; with most = 0 the question fails.
struct Device {
    int sms, most;
    cudaError_t operator()(int splits, int* clusters) const {
        if (most == 0) return cudaErrorNoDevice;
        *clusters = splits > most ? 0 : sms / splits;
        return cudaSuccess;
    }
};
extern "C" int64_t tokens_of_pass(int64_t m, int64_t k, int64_t group, int widest) {
    return nf4::int4::tokens_of_pass(m, weight(64, k, group), widest);
}
extern "C" int widest_cluster(int sms, int most, int* out) { return nf4::int4::widest_cluster(Device{sms, most}, out); }
extern "C" int plan_pass(int64_t m, int64_t n, int64_t k, int64_t group, int sms, int most, int widest, int64_t* out) {
    nf4::int4::Pass p;
    const cudaError_t e = nf4::int4::plan_pass(m, weight(n, k, group), sms, widest, Device{sms, most}, &p);
    if (e == cudaSuccess) {
        const int64_t rows = (p.groups + p.clusters - 1) / p.clusters * 8;
        const int64_t v[6] = {p.splits, p.warps, p.clusters, few::kMaxSmem - p.at.left, p.splits > 1 ? rows * m * 4 : 0, few::kMaxSmem};
        for (int i = 0; i < 6; ++i) out[i] = v[i];
    }
    return e;
}
extern "C" int plan_gemm(int64_t m, int64_t n, int64_t k, int sms, int most, int64_t* out) {
    gemm::Plan p;
    const cudaError_t e = gemm::plan_int4(m, n, k, 1, Device{sms, most}, &p);
    const int64_t v[3] = {p.rows, p.splits, p.us < 1e29};
    for (int i = 0; i < 3; ++i) out[i] = v[i];
    return e;
}
"""


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    d = tmp_path_factory.mktemp("plan")
    (d / "plan.cu").write_text(SOURCE)
    subprocess.run([nvcc(), *NVCC_FLAGS, "-shared", "-cudart", "static", str(d / "plan.cu"), "-o", str(d / "plan.so")], check=True,
                   capture_output=True)
    lib = ctypes.CDLL(str(d / "plan.so"))
    i64, out = ctypes.c_int64, ctypes.POINTER(ctypes.c_int64)
    lib.tokens_of_pass.restype = i64
    lib.tokens_of_pass.argtypes = [i64] * 3 + [ctypes.c_int]
    lib.plan_pass.argtypes = [i64] * 4 + [ctypes.c_int] * 3 + [out]
    lib.plan_gemm.argtypes = [i64] * 3 + [ctypes.c_int] * 2 + [out]
    return lib


@pytest.mark.parametrize("unit", [32, 64])  # the two paddings of X
def test_tokens_of_a_pass(plan, unit):
    text = open(os.path.join(CSRC, "nf4_int4_plan.h")).read()
    stated = " ".join(text.replace("//", "").split())
    assert "all sixteen up to k = %d, eight to %d, then four" % (BORDERS[0][1], BORDERS[1][1]) in stated
    for (tokens, last), (fewer, _) in zip(BORDERS, BORDERS[1:]):
        assert plan.tokens_of_pass(16, last, unit, 8) == tokens
        assert plan.tokens_of_pass(16, last + 64, unit, 8) == fewer
    assert plan.tokens_of_pass(16, 64, unit, 8) == 16 and plan.tokens_of_pass(16, 65536, unit, 8) == 4


SIZES = [(1, 64, 64), (8, 65536, 65536), (40, 33792, 32), (4096, 4096, 128), (28672, 8192, 64), (1003, 1088, 32), (129, 64576, 64), (1 << 29, 64, 64)]


@pytest.mark.parametrize("sms", [148, 20, 7, 1])
@pytest.mark.parametrize("most", [8, 4, 2, 1])
def test_a_cluster_size_that_the_device_does_not_run_is_left_out(plan, sms, most):
    most = min(most, 1 << (sms.bit_length() - 1))
    widest = ctypes.c_int()
    assert plan.widest_cluster(sms, most, ctypes.byref(widest)) == 0 and widest.value == most
    for n, k, group in SIZES:
        for m in (1, 5, 8, 9, 16):
            tokens = plan.tokens_of_pass(m, k, group, most)
            assert 1 <= tokens <= 16
            for part in {min(m, tokens), m % tokens or tokens}:
                out = (ctypes.c_int64 * 6)()
                assert plan.plan_pass(part, n, k, group, sms, most, most, out) == 0, (n, k, part)
                splits, warps, clusters, used, sums, room = out
                assert splits <= most and part <= warps and clusters >= 1 and used + sums <= room
        for m in (17, 128, 129, 5000):
            out = (ctypes.c_int64 * 3)()
            assert plan.plan_gemm(m, n, k, sms, most, out) == 0
            assert out[1] <= most and 32 <= out[0] <= 256 and out[2] == 1


def test_other_errors_are_passed_on(plan):
    widest, six, three = ctypes.c_int(), (ctypes.c_int64 * 6)(), (ctypes.c_int64 * 3)()
    assert plan.widest_cluster(148, 0, ctypes.byref(widest)) == 100  # cudaErrorNoDevice
    assert plan.plan_pass(1, 64, 64, 64, 148, 0, 8, six) == 100
    assert plan.plan_gemm(64, 64, 64, 148, 0, three) == 100


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
