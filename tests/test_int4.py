"""Integer 4-bit weights with group scales: quantization, dequantization and the
fused linear against plain computations (quantization step by step in fp32 as it is
defined, everything else in 64 bits)."""
import copy
import ctypes
import io
import itertools

import numpy as np
import pytest
import torch

from quantized_linear_layers_nf4_b200 import _lib
from quantized_linear_layers_nf4_b200.build import build

gpu = pytest.mark.gpu
FAKE = 0x10000


@pytest.fixture(scope="module")
def nf4():
    build()
    import quantized_linear_layers_nf4_b200 as m
    return m


@pytest.fixture(scope="module")
def L():
    build()
    return _lib.lib()


# ------------------------------- plain forms -------------------------------
def _round_to(x, dtype):
    return torch.from_numpy(x).to(dtype).float().numpy()


def _quantize(W, group, symmetric, scale_dtype):
    """(q [n, k], scale [k/g, n], zero [k/g, n]) by the definition, in numpy fp32."""
    n, k = W.shape
    w = W.float().cpu().numpy().reshape(n, k // group, group)
    f = np.float32
    if symmetric:
        s = _round_to(np.abs(w).max(-1) / f(7), scale_dtype)
    else:
        lo, hi = np.minimum(w.min(-1), f(0)), np.maximum(w.max(-1), f(0))
        s = _round_to((hi - lo) / f(15), scale_dtype)
    d = np.where(s > 0, s, f(1))
    z = np.full_like(d, 8) if symmetric else np.clip(np.rint(-lo / d), 0, 15)
    q = np.clip(np.rint(w / d[..., None]) + z[..., None], 0, 15)
    return q.reshape(n, k).astype(np.uint8), s.T, z.T.astype(np.uint8)


def _unpack(wq, n, k):
    b = wq.cpu().numpy().reshape(n, k // 2)
    return np.stack((b >> 4, b & 15), -1).reshape(n, k)


def _dense64(w):
    """(q - z) s in 64 bits, on the host."""
    q = torch.from_numpy(_unpack(w.wq, w.n, w.k)).double().view(w.n, w.k // w.group, w.group)
    z = 8.0 if w.zero is None else (w.zero.cpu() & 15).t().double().unsqueeze(-1)
    return ((q - z) * w.scale.cpu().t().double().unsqueeze(-1)).view(w.n, w.k)


def _weight(nf4, n, k, group, zero, scale_dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    wq = torch.randint(0, 256, (n * k // 2,), dtype=torch.uint8, device="cuda", generator=g)
    s = (torch.rand(k // group, n, device="cuda", generator=g) * 0.02 + 0.001).to(scale_dtype)
    s *= torch.randint(0, 2, s.shape, device="cuda", generator=g) * 2 - 1  # a checkpoint may hold negative scales
    z = torch.randint(0, 16, (k // group, n), dtype=torch.uint8, device="cuda", generator=g) if zero else None
    return nf4.Int4Weight(n, k, group, wq, s, z)


def _check(y, x, w64, rounded_weight=False):
    """|y - ref| <= sums + roundings, element by element.  fp32 sums of k products in
    any order err by at most k steps of 2^-23 (an adder that truncates) of the sum of
    magnitudes; a weight rounded to bf16 is off by 2^-8 of itself, a bf16 result by
    2^-8 of it."""
    x64 = x.cpu().double()
    ref = x64 @ w64.t()
    mag = x64.abs() @ w64.abs().t()
    tol = w64.shape[1] * 2.0 ** -23 * mag + 1e-30
    if rounded_weight:
        tol = tol + 2.0 ** -8 * mag
    if y.dtype == torch.bfloat16:
        tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * ref.abs()
    bad = ((y.cpu().double() - ref).abs() > tol).nonzero()
    assert bad.numel() == 0, (bad.shape[0], bad[:4])


# ------------------------------ refusals (CPU) ------------------------------
def _struct(**kw):
    w = _lib.nf4_int4_weight_t(_lib.NF4_INT4_WEIGHT_MAGIC, _lib.NF4_WEIGHT_VERSION, 128, 256, 64, 1, 0, FAKE, FAKE, None)
    for k, v in kw.items():
        setattr(w, k, v)
    return ctypes.byref(w)


BAD_STRUCTS = [({"magic": 1}, -5), ({"version": 2}, -5), ({"scale_dtype": 2}, -5), ({"reserved": 1}, -5), ({"wq": None}, -1),
               ({"scale": None}, -1), ({"n": 0}, -2), ({"n": 1 << 30}, -2), ({"k": 96, "group": 32}, -2), ({"k": 65536 + 64}, -2),
               ({"group": 16}, -2), ({"group": 0}, -2), ({"group": -64}, -2), ({"group": 96, "k": 192}, -2),
               ({"group": 512}, -2), ({"wq": FAKE + 8}, -3), ({"scale": FAKE + 1}, -3), ({"scale": FAKE + 2, "scale_dtype": 0}, -3)]


@pytest.mark.parametrize("change,status", BAD_STRUCTS)
def test_weight_struct_refusals(L, change, status):
    assert L.nf4_int4_dequantize(_struct(**change), FAKE, 1, None) == status
    assert L.nf4_int4_linear(FAKE, 1, _struct(**change), FAKE, 1, None, 0, None) == status


def test_argument_refusals(L):
    dq, lin, qu = L.nf4_int4_dequantize, L.nf4_int4_linear, L.nf4_int4_quantize
    assert dq(None, FAKE, 1, None) == -1
    assert dq(_struct(), None, 1, None) == -1
    assert dq(_struct(), FAKE, 2, None) == -4
    assert dq(_struct(), FAKE + 8, 1, None) == -3
    assert lin(None, 1, _struct(), FAKE, 1, None, 0, None) == -1
    assert lin(FAKE, 1, _struct(), None, 1, None, 0, None) == -1
    assert lin(FAKE, 0, _struct(), FAKE, 1, None, 0, None) == -2
    assert lin(FAKE, -3, _struct(), FAKE, 1, None, 0, None) == -2
    assert lin(FAKE, 1, _struct(), FAKE, 3, None, 0, None) == -4
    assert lin(FAKE, 1, _struct(), FAKE, 1, None, 2, None) == -4
    assert lin(FAKE, 1, _struct(), FAKE, 1, None, _lib.NF4_LINEAR_TEST_TIMEOUT, None) == -4
    assert lin(FAKE + 2, 1, _struct(), FAKE, 1, None, 0, None) == -3
    assert lin(FAKE, 1, _struct(), FAKE + 4, 1, None, 0, None) == -3
    assert lin(FAKE, 1, _struct(), FAKE, 1, FAKE + 2, 0, None) == -3
    assert qu(None, 1, 8, 64, 64, 1, FAKE, FAKE, None, None) == -1
    assert qu(FAKE, 1, 8, 64, 64, 1, None, FAKE, None, None) == -1
    assert qu(FAKE, 1, 8, 64, 64, 1, FAKE, None, None, None) == -1
    assert qu(FAKE, 2, 8, 64, 64, 1, FAKE, FAKE, None, None) == -4
    assert qu(FAKE, 1, 8, 64, 64, 5, FAKE, FAKE, None, None) == -4
    assert qu(FAKE, 1, 8, 96, 32, 1, FAKE, FAKE, None, None) == -2
    assert qu(FAKE, 1, 0, 64, 64, 1, FAKE, FAKE, None, None) == -2
    assert qu(FAKE + 8, 1, 8, 64, 64, 1, FAKE, FAKE, None, None) == -3
    assert qu(FAKE, 1, 8, 64, 64, 0, FAKE, FAKE + 2, None, None) == -3


def test_struct_layout():
    assert ctypes.sizeof(_lib.nf4_int4_weight_t) == 64


def test_binding_refusals(nf4):
    with pytest.raises(ValueError):
        nf4.nf4_int4_quantize(torch.zeros(8, 64))                      # not on a GPU
    with pytest.raises(ValueError):
        nf4.Int4Weight(8, 64, 64, torch.zeros(256, dtype=torch.uint8), torch.zeros(1, 8))


# ------------------------------- quantization -------------------------------
@gpu
@pytest.mark.parametrize("n,k,group", [(1, 64, 32), (1, 64, 64), (7, 192, 192), (33, 128, 128), (5, 256, 256), (3, 640, 320),
                                       (1003, 1088, 32), (130, 4096, 64), (257, 2048, 2048), (64, 11008, 128)])
@pytest.mark.parametrize("dtype,scale_dtype,symmetric", [(torch.bfloat16, torch.bfloat16, True), (torch.float32, torch.float32, False),
                                                         (torch.bfloat16, torch.float32, False), (torch.float32, torch.bfloat16, True)])
def test_quantize_and_dequantize(nf4, n, k, group, dtype, scale_dtype, symmetric):
    g = torch.Generator(device="cuda").manual_seed(n * 7 + k)
    W = (torch.randn(n, k, device="cuda", generator=g) * 0.02)
    W[0, :group] = 0                                     # a group of zeros
    W[-1, -group:] = W[-1, -group:].abs() * 1e-30        # one sign, tiny
    W[n // 2, :group] *= 1e30
    W = W.to(dtype)
    wq, scale, zero = nf4.nf4_int4_quantize(W, group, symmetric, scale_dtype)
    q, s, z = _quantize(W, group, symmetric, scale_dtype)
    assert scale.shape == (k // group, n) and (zero is None) == symmetric
    assert np.array_equal(scale.float().cpu().numpy(), s)
    if not symmetric:
        assert np.array_equal(zero.cpu().numpy(), z)
    assert np.array_equal(_unpack(wq, n, k), q)
    w = nf4.Int4Weight(n, k, group, wq, scale, zero)
    zf = np.repeat(z.T.astype(np.float32), group, 1)
    ref = (q.astype(np.float32) - zf) * np.repeat(s.T, group, 1)
    assert np.array_equal(nf4.nf4_int4_dequantize(w, torch.float32).cpu().numpy(), ref)
    assert torch.equal(nf4.nf4_int4_dequantize(w, torch.bfloat16).cpu(), torch.from_numpy(ref).bfloat16())


@gpu
def test_quantize_ties_and_borders(nf4):
    """Quotients at and next to every half: the group's largest is 7, so the scale is 1
    and each weight is its own quotient."""
    v = np.arange(-7.5, 8, 0.5, dtype=np.float32)
    v = np.concatenate([v, np.nextafter(v, np.float32(9)), np.nextafter(v, np.float32(-9))])
    v = v[np.abs(v) <= 7]
    W = np.zeros((1, 128), np.float32)
    W[0, :len(v)] = v
    W = torch.from_numpy(W).cuda()
    wq, scale, _ = nf4.nf4_int4_quantize(W, 128, True, torch.float32)
    assert scale.item() == 1.0
    assert np.array_equal(_unpack(wq, 1, 128), _quantize(W, 128, True, torch.float32)[0])


@gpu
@pytest.mark.parametrize("group", [32, 64, 128, 256, 192])
@pytest.mark.parametrize("dtype,symmetric", [(torch.bfloat16, True), (torch.bfloat16, False), (torch.float32, True), (torch.float32, False)])
@pytest.mark.parametrize("size", [0.02, 1e-25])  # the second's divisors are out of the quotient's fast range
def test_quantize_not_finite(nf4, group, dtype, symmetric, size):
    """A NaN weight has code 15 and spoils no other weight of its word or group; where a
    group's scale is infinite a finite weight has the zero point's code."""
    n, k = 24, 4 * group
    g = torch.Generator(device="cuda").manual_seed(group)
    W = (torch.randn(n, k, device="cuda", generator=g) * size).to(dtype)
    clean = W.clone()
    for r in range(8):
        W[r, group + 8 + r] = float("nan")   # every place of a word
    W[8, :group] = float("nan")              # nothing but NaN
    W[9, 3:11] = float("nan")                # parts of two words
    W[10, 5], W[11, 6] = float("inf"), float("-inf")
    wq, scale, zero = nf4.nf4_int4_quantize(W, group, symmetric, torch.float32)
    q, s = _unpack(wq, n, k).reshape(n, 4, group), scale.cpu().numpy().T
    z = np.full((n, 4), 8) if symmetric else zero.cpu().numpy().T
    w = W.float().cpu().numpy()
    assert np.all(q.reshape(n, k)[np.isnan(w) | np.isinf(w)] == 15)
    for r, finite in ((10, np.arange(group) != 5), (11, np.arange(group) != 6)):
        assert np.isinf(s[r, 0]) and np.all(q[r, 0][finite] == z[r, 0])
    # as if the NaN had been zeros
    w[np.isnan(w)] = 0
    inf = np.isinf(w)
    w[inf] = clean.float().cpu().numpy()[inf]
    wantq, wants, wantz = _quantize(torch.from_numpy(w), group, symmetric, torch.float32)
    same = np.ones((n, 4), bool)
    same[10:12, 0] = False
    assert np.array_equal(s[same], wants.T[same]) and np.array_equal(z[same], wantz.T[same])
    same = np.repeat(same, group, 1) & ~np.isnan(W.float().cpu().numpy())
    assert np.array_equal(q.reshape(n, k)[same], wantq[same])


# ---------------------------------- linear ----------------------------------
SHAPES = [(1, 64, 64), (1, 64, 32), (15, 128, 128), (16, 192, 64), (17, 448, 448), (40, 1088, 32), (100, 4096, 128),
          (1003, 1088, 64), (2048, 640, 320), (129, 16384, 256), (8, 65536, 65536), (24, 57344, 32), (9000, 1024, 128), (60001, 128, 64)]


@gpu
@pytest.mark.parametrize("n,k,group", SHAPES)
@pytest.mark.parametrize("zero,scale_dtype", [(False, torch.bfloat16), (True, torch.float32)])
def test_linear_few_tokens(nf4, n, k, group, zero, scale_dtype):
    w = _weight(nf4, n, k, group, zero, scale_dtype, n + k)
    w64 = _dense64(w)
    for m, dtype in itertools.product((1, 2, 5, 8, 9, 16), (torch.float32, torch.bfloat16)):
        x = torch.randn(m, k, device="cuda").bfloat16()
        guard = torch.full((m + 2, n), 7.0, device="cuda", dtype=dtype)
        # rows before and behind the output keep what they held
        off = 1 if n * guard.element_size() % 16 == 0 else 0
        y = nf4.nf4_int4_linear(x, w, out=guard[off:off + m])
        _check(y, x, w64)
        assert torch.all(guard[:off] == 7) and torch.all(guard[off + m:] == 7)
        assert torch.equal(y, nf4.nf4_int4_linear(x, w, dtype, weights_early=True))


@gpu
@pytest.mark.parametrize("n,k,group", [(1, 64, 32), (100, 192, 64), (257, 1088, 32), (300, 512, 512), (1003, 1088, 64)])
@pytest.mark.parametrize("zero,scale_dtype", [(False, torch.bfloat16), (True, torch.float32)])
def test_linear_many_tokens(nf4, n, k, group, zero, scale_dtype):
    w = _weight(nf4, n, k, group, zero, scale_dtype, n + k)
    w64 = _dense64(w)
    for m, dtype in ((17, torch.float32), (64, torch.bfloat16), (100, torch.float32), (300, torch.float32)):
        x = torch.randn(m, k, device="cuda").bfloat16()
        _check(nf4.nf4_int4_linear(x, w, dtype), x, w64, rounded_weight=True)


@gpu
def test_linear_is_exact_on_integers(nf4):
    """Small integers and scales that are powers of two: every sum is exact, so any
    code in the wrong place shows."""
    n, k = 48, 512
    g = torch.Generator(device="cuda").manual_seed(5)
    for group, m in itertools.product((32, 64, 256), (3, 16, 20)):
        w = _weight(nf4, n, k, group, True, torch.float32, group)
        w = nf4.Int4Weight(n, k, group, w.wq, torch.full_like(w.scale, 0.25), w.zero)
        x = torch.randint(-4, 5, (m, k), device="cuda", generator=g).bfloat16()
        assert torch.equal(nf4.nf4_int4_linear(x, w, torch.float32).cpu().double(), x.cpu().double() @ _dense64(w).t())


@gpu
@pytest.mark.parametrize("group", [32, 64, 128])
def test_linear_ranges_of_x(nf4, group):
    """Tokens far from 1, and columns far apart in one token.  A token goes through fp16 times a
    power of two that brings its largest value (of a range of columns) to 2^14 or more: what
    is below fp16's normal numbers is off by 2^-25, 2^-39 of that largest value."""
    n, k = 300, 1152
    w = _weight(nf4, n, k, group, True, torch.float32, group)
    w64 = _dense64(w)
    g = torch.Generator(device="cuda").manual_seed(group)
    for m in (1, 7, 16):
        x = torch.randn(m, k, device="cuda", generator=g)
        x *= torch.exp2(torch.randint(-90, 91, (m, 1), device="cuda", generator=g).float())
        if m > 1:
            x[0] = 0
            x[1] *= torch.exp2(torch.randint(-30, 31, (k,), device="cuda", generator=g).float())
        x = x.bfloat16()
        y, x64 = nf4.nf4_int4_linear(x, w, torch.float32).cpu().double(), x.cpu().double()
        tol = k * 2.0 ** -23 * (x64.abs() @ w64.abs().t()) + 2.0 ** -39 * x64.abs().amax(1, keepdim=True) * w64.abs().sum(1) + 1e-37
        assert torch.all((y - x64 @ w64.t()).abs() <= tol)
        assert m == 1 or torch.all(y[0] == 0)


@gpu
def test_zero_points_beyond_four_bits(nf4):
    """Only the low four bits of a zero point count, on every path."""
    for group in (32, 64, 128):
        a = _weight(nf4, 96, 256, group, True, torch.bfloat16, group)
        b = nf4.Int4Weight(96, 256, group, a.wq, a.scale, a.zero + 16 * (a.zero % 7) + 128 * (a.zero % 2))
        assert torch.any(b.zero > 15)
        assert torch.equal(nf4.nf4_int4_dequantize(a), nf4.nf4_int4_dequantize(b))
        for m in (1, 12, 20, 200):
            x = torch.randn(m, 256, device="cuda").bfloat16()
            assert torch.equal(nf4.nf4_int4_linear(x, a), nf4.nf4_int4_linear(x, b))


@gpu
@pytest.mark.parametrize("m,n,k,group", [(300, 1003, 1088, 64), (130, 2048, 2048, 32), (700, 11008, 512, 128), (16, 5000, 4096, 128), (77, 130, 8192, 64)])
def test_linear_repeats_to_the_bit(nf4, m, n, k, group):
    """Many calls one after the other: a stage read before it is written, or after it is
    written again, would show."""
    w = _weight(nf4, n, k, group, True, torch.bfloat16, n)
    x = torch.randn(m, k, device="cuda").bfloat16()
    first = nf4.nf4_int4_linear(x, w)
    wrong = sum((nf4.nf4_int4_linear(x, w) != first).any() for _ in range(200))
    assert int(wrong) == 0


@gpu
@pytest.mark.parametrize("m,n,group,scale_dtype", [(40, 64, 64, torch.bfloat16), (300, 512, 32, torch.float32), (700, 11008, 128, torch.bfloat16), (600, 4096, 128, torch.bfloat16)])
def test_linear_waits_are_bounded(nf4, m, n, group, scale_dtype):
    """The GEMM's waits run out where nothing arrives, and the next call is right."""
    w = _weight(nf4, n, 512, group, False, scale_dtype, n)
    x = torch.randn(m, 512, device="cuda").bfloat16()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = torch.full((m, n), 7.0, device="cuda")
    nf4.nf4_int4_linear(x, w, out=y, dev_status=status, flags=_lib.NF4_LINEAR_TEST_TIMEOUT)
    assert status.item() == _lib.NF4_ERR_DEVICE_TIMEOUT and torch.all(y == 7)
    status.zero_()
    _check(nf4.nf4_int4_linear(x, w, torch.float32, dev_status=status), x, _dense64(w), rounded_weight=True)
    assert status.item() == 0


@gpu
def test_streams_graph_and_repeat(nf4):
    w = _weight(nf4, 1000, 2048, 128, False, torch.bfloat16, 3)
    x = torch.randn(4, 2048, device="cuda").bfloat16()
    ref = nf4.nf4_int4_linear(x, w)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    y = nf4.nf4_int4_linear(x, w, stream=side)
    side.synchronize()
    assert torch.equal(ref, y)
    out = torch.empty_like(ref)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        nf4.nf4_int4_linear(x, w, out=out)
        back = nf4.nf4_int4_dequantize(w)
    x.copy_(torch.randn(4, 2048, device="cuda").bfloat16())
    ref = nf4.nf4_int4_linear(x, w)
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(ref, out)
    assert torch.equal(back, nf4.nf4_int4_dequantize(w))


@gpu
@pytest.mark.parametrize("kind", ["int4", "nf4"])
def test_weights_are_copied_and_saved(nf4, kind):
    """A weight that was used is copied with its tensors and points to those."""
    W = torch.randn(64, 128, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
    w, fn = (nf4.int4_quantize_weight(W, 64), nf4.nf4_int4_linear) if kind == "int4" else (nf4.quantize_weight(W), nf4.nf4_linear)
    x = torch.randn(3, 128, device="cuda").bfloat16()
    want = fn(x, w)
    buf = io.BytesIO()
    torch.save(w, buf)
    buf.seek(0)
    for other in (copy.deepcopy(w), copy.copy(w), torch.load(buf, weights_only=False)):
        assert torch.equal(fn(x, other), want)
        assert other.struct().wq == other.wq.data_ptr()
    twin = copy.deepcopy(w)
    twin.wq.zero_()
    assert torch.equal(fn(x, w), want) and not torch.equal(fn(x, twin), want)


@gpu
def test_linear_from_few_to_many_tokens(nf4):
    """Around every change of path the result is within that of a weight rounded to bf16."""
    for n, k, group, zero, dtype in ((64, 4096, 128, True, torch.bfloat16), (4096, 1024, 128, False, torch.float32), (40000, 128, 128, True, torch.bfloat16),
                                     (333, 5184, 32, True, torch.float32), (1001, 8128, 64, False, torch.bfloat16), (96, 13440, 192, True, torch.float32)):
        w = _weight(nf4, n, k, group, zero, dtype, n)
        w64 = _dense64(w)
        for m in (16, 17, 31, 32, 33, 48, 64, 65, 96, 127, 128, 129, 256, 257):
            x = torch.randn(m, k, device="cuda").bfloat16()
            _check(nf4.nf4_int4_linear(x, w, torch.float32), x, w64, rounded_weight=True)


@gpu
def test_binding_refusals_on_device(nf4):
    w = _weight(nf4, 64, 128, 64, False, torch.bfloat16, 1)
    x = torch.randn(2, 128, device="cuda").bfloat16()
    bad = [lambda: nf4.nf4_int4_linear(x.float(), w), lambda: nf4.nf4_int4_linear(x[:, :64], w),
           lambda: nf4.nf4_int4_linear(x[0], w), lambda: nf4.nf4_int4_linear(torch.cat([x, x], 1)[:, :128], w),
           lambda: nf4.nf4_int4_linear(x, w, torch.float16), lambda: nf4.nf4_int4_linear(x, w, out=torch.empty(2, 63, device="cuda")),
           lambda: nf4.nf4_int4_linear(x, w, out=torch.empty(64, 2, device="cuda").t()),
           lambda: nf4.nf4_int4_dequantize(w, torch.float16), lambda: nf4.nf4_int4_dequantize(w, out=torch.empty(64, 64, device="cuda")),
           lambda: nf4.nf4_int4_quantize(x, 48), lambda: nf4.nf4_int4_quantize(x.half(), 64),
           lambda: nf4.nf4_int4_quantize(x, 64, zero=torch.empty(2, 2, device="cuda", dtype=torch.uint8)),
           lambda: nf4.Int4Weight(64, 128, 64, w.wq, w.scale.t().contiguous()), lambda: nf4.Int4Weight(64, 128, 64, w.wq[:-1], w.scale),
           lambda: nf4.Int4Weight(64, 128, 64, w.wq, w.scale.cpu()), lambda: nf4.Int4Weight(64, 128, 64, w.wq, w.scale, w.scale)]
    for f in bad:
        with pytest.raises(ValueError):
            f()
    with pytest.raises(nf4.NF4Error):
        nf4.nf4_int4_linear(torch.empty(0, 128, device="cuda").bfloat16(), w)
    with pytest.raises(nf4.NF4Error):  # not 16-byte aligned
        nf4.nf4_int4_linear(torch.empty(257, device="cuda").bfloat16()[1:].view(2, 128), w)


def test_status_refusals(nf4, monkeypatch):
    """A status that the kernel could not write (it does so when a wait runs out) is refused before
    anything is launched."""
    monkeypatch.setattr(nf4, "_need_cuda", lambda t, name: None)
    monkeypatch.setattr(nf4, "_launch", lambda *args: None)
    w = object.__new__(nf4.Int4Weight)
    w.__dict__.update(n=8, k=64, group=64, wq=torch.zeros(256, dtype=torch.uint8), scale=torch.zeros(1, 8), zero=None)
    x = torch.zeros(2, 64).bfloat16()
    for bad in (torch.zeros(1, dtype=torch.int64), torch.zeros(1), torch.zeros(0, dtype=torch.int32), torch.zeros(1, dtype=torch.int32, device="meta")):
        with pytest.raises(ValueError):
            nf4.nf4_int4_linear(x, w, dev_status=bad)
    nf4.nf4_int4_linear(x, w, dev_status=torch.zeros(1, dtype=torch.int32))
