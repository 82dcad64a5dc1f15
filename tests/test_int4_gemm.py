"""The GEMM of integer 4-bit weights to the bit: every code's value, and every tile shape."""
import ctypes

import pytest
import torch

from quantized_linear_layers_nf4_b200.build import build
from tests.test_int4_plan import plan  # noqa: F401

gpu = pytest.mark.gpu


@pytest.fixture(scope="module")
def nf4():
    build()
    import quantized_linear_layers_nf4_b200 as m
    return m


def _weight(nf4, n, k, group, zero, scale, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    wq = torch.randint(0, 256, (n * k // 2,), dtype=torch.uint8, device="cuda", generator=g)
    z = torch.randint(0, 16, (k // group, n), dtype=torch.uint8, device="cuda", generator=g) if zero else None
    return nf4.Int4Weight(n, k, group, wq, scale(g, (k // group, n)), z)


def _any_scale(dtype):
    def make(g, shape):  # of both signs, over nine powers of two
        s = (torch.rand(shape, device="cuda", generator=g) + 0.5) * torch.exp2(torch.randint(-8, 1, shape, device="cuda", generator=g).float())
        return (s * (torch.randint(0, 2, shape, device="cuda", generator=g) * 2 - 1)).to(dtype)
    return make


def _power_of_two(dtype):
    return lambda g, shape: torch.exp2(torch.randint(-3, 1, shape, device="cuda", generator=g).float()).to(dtype)


@gpu
@pytest.mark.parametrize("group,k", [(32, 512), (64, 512), (128, 512), (512, 512), (192, 576), (320, 640)])
@pytest.mark.parametrize("scale", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("zero", [False, True])
@pytest.mark.parametrize("n", [1003, 4100])
def test_identity_gives_the_weight(nf4, group, k, scale, zero, n):
    """Row c of X picks column c of the weight: all of it comes back as nf4_int4_dequantize writes it."""
    w = _weight(nf4, n, k, group, zero, _any_scale(scale), group + n)
    want = nf4.nf4_int4_dequantize(w, torch.bfloat16).t()
    x = torch.eye(k, device="cuda").bfloat16()
    assert torch.equal(nf4.nf4_int4_linear(x, w), want)
    for c in range(0, k, 128):  # half a token tile
        assert torch.equal(nf4.nf4_int4_linear(x[c:c + 128], w), want[c:c + 128])


# (m, n, k) and the tile's weight rows and parts of k on 148 SMs
TILES = [((100, 40, 64), (32, 1)), ((130, 40, 1024), (32, 4)), ((100, 40, 2048), (32, 8)), ((100, 5000, 64), (64, 1)),
         ((100, 2048, 1024), (64, 4)), ((257, 333, 2048), (64, 8)), ((100, 11008, 64), (96, 1)), ((129, 6000, 1024), (96, 2)),
         ((100, 2500, 1024), (96, 4)), ((128, 14336, 64), (128, 1)), ((257, 4096, 1024), (128, 2)), ((100, 4096, 1024), (128, 4)),
         ((127, 2048, 2048), (128, 8)), ((100, 20000, 64), (160, 1)), ((100, 11008, 1024), (160, 2)), ((100, 5000, 1024), (160, 4)),
         ((100, 2500, 2048), (160, 8)), ((600, 9000, 64), (192, 1)), ((100, 6000, 1024), (192, 4)), ((100, 30000, 64), (224, 1)),
         ((100, 14336, 1024), (224, 2)), ((600, 11008, 64), (256, 1)), ((100, 9000, 1024), (256, 4)), ((100, 4096, 2048), (256, 8)),
         ((17, 1003, 1088), None), ((255, 1003, 1088), None), ((256, 1003, 1088), None), ((385, 1001, 1088), None)]


def test_the_tiles_are_all_there(plan):  # noqa: F811
    found = set()
    for size, tile in TILES:
        out = (ctypes.c_int64 * 3)()
        assert plan.plan_gemm(*size, 148, 8, out) == 0
        assert tile is None or (out[0], out[1]) == tile, (size, out[0], out[1])
        found.add(tile)
    assert {r for r, _ in found - {None}} == set(range(32, 257, 32)) and {s for _, s in found - {None}} == {1, 2, 4, 8}


@gpu
@pytest.mark.parametrize("size,tile", TILES)
@pytest.mark.parametrize("group,scale,zero", [(64, torch.bfloat16, True), (32, torch.float32, True), (64, torch.float32, False), (32, torch.bfloat16, False)])
def test_integers_are_exact(nf4, size, tile, group, scale, zero):
    """X of small integers, scales of powers of two: weights are exact in bf16, and sums (multiples of 1/8
    below 2^17 at most) in fp32, so that anything out of place shows."""
    m, n, k = size
    w = _weight(nf4, n, k, group, zero, _power_of_two(scale), n + k)
    x = torch.randint(-4, 5, (m, k), device="cuda", generator=torch.Generator(device="cuda").manual_seed(m)).bfloat16()
    want = x.double() @ nf4.nf4_int4_dequantize(w, torch.float32).double().t()
    assert torch.equal(nf4.nf4_int4_linear(x, w, torch.float32).double(), want)
    assert torch.equal(nf4.nf4_int4_linear(x, w), want.bfloat16())


@gpu
@pytest.mark.parametrize("group,k", [(32, 512), (64, 512), (128, 512), (512, 512), (192, 576), (320, 640)])
@pytest.mark.parametrize("scale", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("zero", [False, True])
@pytest.mark.parametrize("n", [1003, 4100])
def test_fp32_results_keep_the_weight(nf4, group, k, scale, zero, n):
    """With fp32 results a weight is two bf16 values.  The first is off by half a step of 2^-8 of the power
    of two below it at most; the rest has twelve bits less eight with a bf16 scale, which are kept,
    and is itself rounded with an fp32 one, by half a step of a value 2^-8 as large: 2^-17."""
    w = _weight(nf4, n, k, group, zero, _any_scale(scale), group + n)
    want = nf4.nf4_int4_dequantize(w, torch.float32).t()
    x = torch.eye(k, device="cuda").bfloat16()
    for y in (nf4.nf4_int4_linear(x, w, torch.float32), torch.cat([nf4.nf4_int4_linear(x[c:c + 100], w, torch.float32) for c in range(0, k, 100)])):
        if scale == torch.bfloat16:
            assert torch.equal(y, want)
        else:
            assert torch.all((y.double() - want.double()).abs() <= 2.0 ** -17 * want.double().abs())


@gpu
@pytest.mark.parametrize("m,n,k,group", [(300, 1003, 5184, 32), (130, 2048, 2048, 128), (40, 257, 8192, 64), (512, 4096, 4096, 128), (20, 96, 1024, 256)])
@pytest.mark.parametrize("scale", [torch.bfloat16, torch.float32])
def test_fp32_results_of_any_weight(nf4, m, n, k, group, scale):
    """Two products a weight, each sum off by 2^-23 of the magnitudes so far, and what the weight has lost."""
    w = _weight(nf4, n, k, group, True, _any_scale(scale), k)
    w64 = nf4.nf4_int4_dequantize(w, torch.float32).double()
    x = torch.randn(m, k, device="cuda", generator=torch.Generator(device="cuda").manual_seed(n)).bfloat16()
    ref, mag = x.double() @ w64.t(), x.double().abs() @ w64.abs().t()
    tol = 2 * k * 2.0 ** -23 * mag * (1 + 2.0 ** -7) + (2.0 ** -17 + 2.0 ** -24 if scale == torch.float32 else 0.0) * mag
    assert torch.all((nf4.nf4_int4_linear(x, w, torch.float32).double() - ref).abs() <= tol)


@gpu
@pytest.mark.parametrize("scale", [torch.bfloat16, torch.float32])
def test_scales_that_are_not_finite(nf4, scale):
    """An infinite or NaN scale: the rows that have it are infinite or NaN as a sum in 64 bits is, the others right."""
    n, k, group = 300, 512, 64
    w = _weight(nf4, n, k, group, False, _power_of_two(scale), 3)
    w.scale[2, 5], w.scale[0, 7], w.scale[7, 200] = float("inf"), float("nan"), float("-inf")
    x = torch.ones(512, k, device="cuda").bfloat16()
    x[:256, 128:192] = 0
    x[:, 129] = 1  # of group 2 the first half of the rows has one weight
    w64 = nf4.nf4_int4_dequantize(w, torch.float32).double()
    ref = (x.double().cpu() @ w64.t().cpu()).cuda()
    for dtype in (torch.float32, torch.bfloat16):
        y = nf4.nf4_int4_linear(x, w, dtype).double()
        fine = [r for r in range(n) if r not in (5, 7, 200)]
        assert torch.equal(y[:, fine], ref[:, fine].to(dtype).double())
        assert not torch.isfinite(y[:, [5, 7, 200]]).any() and torch.isnan(y[:, 7]).all()
