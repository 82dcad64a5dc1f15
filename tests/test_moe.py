"""The mixture-of-experts layer for a few tokens against its definition in 64 bits."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

from quantized_linear_layers_nf4_b200 import _lib
from quantized_linear_layers_nf4_b200.build import CSRC, INCLUDE, NVCC_FLAGS, build, nvcc

gpu = pytest.mark.gpu
FAKE = 0x10000
U16, UBF = 2.0 ** -11, 2.0 ** -8  # half a step of fp16 and of bf16, relative


@pytest.fixture(scope="module")
def nf4():
    build()
    import quantized_linear_layers_nf4_b200 as m
    return m


@pytest.fixture(scope="module")
def L():
    build()
    return _lib.lib()


# ------------------------------ refusals (CPU) ------------------------------
def _w(n, k, **kw):
    w = _lib.nf4_weight_t(_lib.NF4_WEIGHT_MAGIC, _lib.NF4_WEIGHT_VERSION, n, k, 64, 256, FAKE, FAKE, FAKE, FAKE)
    for key, v in kw.items():
        setattr(w, key, v)
    return w


def _w4(n, k, **kw):
    w = _lib.nf4_int4_weight_t(_lib.NF4_INT4_WEIGHT_MAGIC, _lib.NF4_WEIGHT_VERSION, n, k, 64, 1, 0, FAKE, FAKE, None)
    for key, v in kw.items():
        setattr(w, key, v)
    return w


@pytest.mark.parametrize("which", ["nf4", "int4"])
def test_refusals(L, which):
    fn, mk = (L.nf4_moe, _w) if which == "nf4" else (L.nf4_int4_moe, _w4)
    E, h, f, top = 4, 128, 64, 2
    need = L.nf4_moe_workspace_bytes(h, f, E, top)
    assert need > 0

    def call(**kw):
        a = dict(X=FAKE, m=1, router=FAKE, E=E, gu=mk(E * 2 * f, h), dn=mk(E * h, f), top=top, Y=FAKE, ids=None, pr=None, flags=0,
                 ws=FAKE, n=need)
        a.update(kw)
        return fn(a["X"], a["m"], a["router"], a["E"], ctypes.byref(a["gu"]) if a["gu"] else None,
                  ctypes.byref(a["dn"]) if a["dn"] else None, a["top"], a["Y"], a["ids"], a["pr"], a["flags"], a["ws"], a["n"], None)

    for name in ("X", "router", "Y", "gu", "dn"):
        assert call(**{name: None}) == -1, name
    for name in ("X", "router", "Y", "ws"):
        assert call(**{name: FAKE + 8}) == -3, name
    assert call(ids=FAKE + 2) == -3 and call(pr=FAKE + 1) == -3
    for bad in (dict(m=0), dict(m=-1), dict(m=1 << 31), dict(E=0), dict(E=513), dict(E=5), dict(top=0), dict(top=5), dict(top=-1),
                dict(gu=mk(E * 2 * f + 64, h)), dict(dn=mk(E * h, 128)), dict(gu=mk(E * 2 * f, 192)), dict(dn=mk(E * h * 2, f))):
        assert call(**bad) == -2, bad
    assert call(gu=mk(E * 2 * f, h, magic=5)) == -5 and call(dn=mk(E * h, f, version=9)) == -5
    assert call(flags=2) == -4
    assert call(ws=None) == -6 and call(n=need - 1) == -6


def test_workspace_sizes(L):
    size = L.nf4_moe_workspace_bytes
    assert size(64, 64, 1, 1) > 0 and size(8192, 28672, 512, 16) > 0
    for bad in ((0, 64, 1, 1), (32, 64, 1, 1), (64, 96, 1, 1), (65600, 64, 1, 1), (64, 64, 0, 1), (64, 64, 513, 1), (64, 64, 4, 5),
                (64, 64, 32, 17), (64, 64, 4, 0), (-64, 64, 4, 1)):
        assert size(*bad) == 0, bad


# ------------------------------ the definition ------------------------------
def _dense64(nf4, w):
    """A weight in 64 bits from its parts, [n, k]."""
    b = w.wq.view(w.n, w.k // 2)
    q = torch.stack((b >> 4, b & 15), -1).view(w.n, w.k)
    if isinstance(w, nf4.Int4Weight):
        z = 8.0 if w.zero is None else w.zero.t().double().unsqueeze(-1)
        return ((q.double().view(w.n, -1, w.group) - z) * w.scale.t().double().unsqueeze(-1)).view(w.n, w.k)
    a = w.absmax_q.double() / 127 * w.absmax_scale.double().repeat_interleave(256)[:w.absmax_q.numel()] + w.absmax_offset.double()
    return (nf4.nf4_codebook(w.quant_type).cuda().double()[q.long()].view(w.n, -1, 64) * a.view(w.n, -1, 1)).view(w.n, w.k)


def _layer(nf4, E, h, f, fmt, seed, wscale=None):
    """(router, gate_up, down) of random weights: quantized ones, or drawn codes."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    router = (torch.randn(E, h, device="cuda", generator=g) * 2 * h ** -0.5).bfloat16()
    gu = torch.randn(E * 2 * f, h, device="cuda", generator=g) * (wscale or h ** -0.5)
    dn = torch.randn(E * h, f, device="cuda", generator=g) * f ** -0.5
    if fmt in ("nf4", "fp4"):
        return router, nf4.quantize_weight(gu, quant_type=fmt), nf4.quantize_weight(dn, quant_type=fmt)
    group, sym = {"int4_32": (32, False), "int4_64": (64, True), "int4_row": (0, False)}[fmt]
    sd = torch.float32 if fmt == "int4_32" else torch.bfloat16
    return router, nf4.int4_quantize_weight(gu, group or h, sym, sd), nf4.int4_quantize_weight(dn, group or f, sym, sd)


def _reference(nf4, x, router, gate_up, down, top, renorm):
    """y, ids, p, and how far a result in the kernels' precision may be from y."""
    E, h, f = router.shape[0], x.shape[1], down.k
    x = x.double()
    logits = x @ router.double().t()
    val, ids = logits.sort(dim=1, descending=True, stable=True)
    val, ids = val[:, :top], ids[:, :top]
    p = (val - val[:, :1]).exp()
    p = p / (p.sum(1, keepdim=True) if renorm else (logits - val[:, :1]).exp().sum(1, keepdim=True))
    G = _dense64(nf4, gate_up).view(E, 2 * f, h)
    D = _dense64(nf4, down).view(E, h, f)
    y, tol = torch.zeros_like(x), torch.zeros_like(x)
    lev = 0.0 if isinstance(gate_up, nf4.Int4Weight) else U16  # levels are rounded to fp16, codes are not
    # (the block's absmax and the scaling of sums: a few fp32 roundings, in the sums' share)
    for t in range(x.shape[0]):
        da_min = 0.0
        acts = []
        for j in range(top):
            e = ids[t, j]
            z, mag = G[e] @ x[t], G[e].abs() @ x[t].abs()
            dz = (lev + (h + 16) * 2.0 ** -23) * mag
            g, u, dg, du = z[:f], z[f:], dz[:f], dz[f:]
            silu = g * torch.sigmoid(g)
            # p: logits in fp32 sums, then exp: an error in the exponent counts as it is
            dp = ((h + 16) * 2.0 ** -23 * 2 * (router[ids[t]].double().abs() @ x[t].abs()).max() + 2.0 ** -20) * p[t, j]
            a = p[t, j] * silu * u
            # |silu'| < 1.1; expf and the division within 2^-20
            da = p[t, j] * (1.1 * dg * (u.abs() + du) + silu.abs() * du) + dp * (silu * u).abs() + (U16 + 2.0 ** -20) * a.abs()
            acts.append((e, a, da))
        # fp16 of a (scaled or not): below its normal range the step is 2^-24, and a token's
        # largest is at least 2^-6, or is brought to 2^14
        biggest = max(float(a.abs().max()) for _, a, _ in acts)
        step = 2.0 ** -25 if 2.0 ** -6 <= biggest < 2.0 ** 15 else 2.0 ** -38 * biggest
        for e, a, da in acts:
            y[t] += D[e] @ a
            da = da + step + da_min
            tol[t] += D[e].abs() @ (da * (1 + lev) + (lev + (top * f + 16) * 2.0 ** -23) * a.abs())
    return y, ids, p, tol * (1 + UBF) + UBF * y.abs() + 1e-37


def _check(nf4, x, layer, top, renorm, **kw):
    y, ids, p = nf4.nf4_moe(x, *layer, top, renorm, return_routing=True, **kw)
    ry, rids, rp, tol = _reference(nf4, x, *layer, top, renorm)
    assert torch.equal(ids.long(), rids)
    h = x.shape[1]
    mag = (x.double().abs() @ layer[0].double().abs().t()).max()
    assert torch.allclose(p.double(), rp, rtol=float(2 * (h + 16) * 2.0 ** -23 * mag) + 2.0 ** -19, atol=1e-30)
    bad = ((y.double() - ry).abs() > tol).nonzero()
    assert bad.numel() == 0, (bad.shape[0], bad[:4], y[bad[0][0], bad[0][1]], ry[bad[0][0], bad[0][1]], tol[bad[0][0], bad[0][1]])
    return y


CASES = [(1, 4, 1, 64, 64), (1, 1, 1, 128, 64), (3, 3, 3, 64, 192), (7, 40, 6, 448, 128), (8, 8, 2, 1024, 704), (9, 8, 2, 512, 320),
         (16, 64, 8, 320, 64), (16, 2, 1, 256, 1408), (5, 512, 16, 128, 64), (16, 300, 16, 64, 64), (17, 4, 2, 192, 128), (35, 10, 4, 128, 192),
         (16, 1, 1, 192, 64), (16, 3, 3, 128, 320), (13, 20, 16, 64, 128), (2, 2, 2, 65536, 64), (1, 1, 1, 64, 65536)]


@gpu
@pytest.mark.parametrize("m,E,top,h,f", CASES)
@pytest.mark.parametrize("fmt", ["nf4", "fp4", "int4_32", "int4_64", "int4_row"])
def test_layer(nf4, m, E, top, h, f, fmt):
    layer = _layer(nf4, E, h, f, fmt, seed=m + E)
    x = torch.randn(m, h, device="cuda", generator=torch.Generator(device="cuda").manual_seed(m * 31 + f)).bfloat16()
    _check(nf4, x, layer, top, renorm=(m + top) % 2 == 0)


@gpu
@pytest.mark.parametrize("fmt", ["nf4", "int4_32", "int4_64"])
@pytest.mark.parametrize("scale", [2.0 ** 40, 2.0 ** 12, 2.0 ** -12, 2.0 ** -60])
def test_range(nf4, fmt, scale):
    """Activations far out of fp16's range, of one token or of all."""
    layer = _layer(nf4, 4, 256, 192, fmt, seed=9)
    layer = (torch.zeros_like(layer[0]),) + layer[1:]  # large inputs, even choice: experts 0 and 1
    x = torch.randn(11, 256, device="cuda", generator=torch.Generator(device="cuda").manual_seed(2))
    _check(nf4, (x * scale).bfloat16(), layer, 2, True)
    x[3] *= scale
    x[5] = 0
    y = _check(nf4, x.bfloat16(), layer, 2, True)
    assert torch.all(y[5] == 0)


@gpu
def test_groups_of_the_two_weights_differ(nf4):
    a, b = _layer(nf4, 6, 384, 256, "int4_32", seed=1), _layer(nf4, 6, 384, 256, "int4_row", seed=2)
    x = torch.randn(9, 384, device="cuda", generator=torch.Generator(device="cuda").manual_seed(7)).bfloat16()
    _check(nf4, x, (a[0], a[1], b[2]), 3, True)
    _check(nf4, x, (a[0], b[1], a[2]), 3, False)


@gpu
def test_ties_go_to_the_lower_expert(nf4):
    """Integers: the logits are exact and many are equal, -0 and 0 among them."""
    E, h = 96, 64
    layer = _layer(nf4, E, h, 64, "nf4", seed=4)
    g = torch.Generator(device="cuda").manual_seed(1)
    router = torch.randint(-1, 2, (E, h), device="cuda", generator=g).bfloat16()
    x = torch.randint(-1, 2, (16, h), device="cuda", generator=g).bfloat16()
    x[:, 8:] = 0
    x[7] = 0
    x[8] = -0.0
    for top in (1, 5, 16):
        _, ids, p = nf4.nf4_moe(x, router, *layer[1:], top, return_routing=True)
        want = (x.double() @ router.double().t()).sort(dim=1, descending=True, stable=True).indices[:, :top]
        assert torch.equal(ids.long(), want)
        assert torch.allclose(p.sum(1), torch.ones(16, device="cuda"), atol=1e-5)


@gpu
def test_other_rows_and_memory_stay_as_they_are(nf4):
    """A row that is not finite spoils no other; rows around the output keep what they
    held; the workspace may hold anything."""
    layer = _layer(nf4, 16, 256, 128, "nf4", seed=6)
    x = torch.randn(10, 256, device="cuda").bfloat16()
    x[4, 3] = float("nan")
    x[6, 5] = float("inf")
    guard = torch.full((14, 256), 3.0, device="cuda").bfloat16()
    ws = torch.full_like(nf4.moe_workspace(256, 128, 16, 3), 255)
    y = nf4.nf4_moe(x, *layer, 3, out=guard[2:12], workspace=ws)
    keep = [0, 1, 2, 3, 5, 7, 8, 9]
    ry, _, _, tol = _reference(nf4, x[keep], *layer, 3, True)
    assert torch.all((y[keep].double() - ry).abs() <= tol)
    assert torch.all(guard[:2] == 3) and torch.all(guard[12:] == 3)


@gpu
def test_repeat_streams_and_graph(nf4):
    layer = _layer(nf4, 32, 512, 192, "nf4", seed=8)
    layer4 = _layer(nf4, 32, 512, 192, "int4_64", seed=8)
    x = torch.randn(12, 512, device="cuda").bfloat16()
    ref, ref4 = nf4.nf4_moe(x, *layer, 4), nf4.nf4_moe(x, *layer4, 4)
    torch.cuda.synchronize()
    # two calls at once, each with its workspace
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    ws1, ws2 = nf4.moe_workspace(512, 192, 32, 4), nf4.moe_workspace(512, 192, 32, 4)
    for _ in range(20):
        a = nf4.nf4_moe(x, *layer, 4, workspace=ws1, stream=s1)
        b = nf4.nf4_moe(x, *layer4, 4, workspace=ws2, stream=s2)
    c = nf4.nf4_moe(x, *layer, 4, stream=s1)  # a workspace of its own
    torch.cuda.synchronize()
    assert torch.equal(a, ref) and torch.equal(b, ref4) and torch.equal(c, ref)
    # captured: a chain of layers that share a workspace, replayed with new inputs
    graph, buf = torch.cuda.CUDAGraph(), torch.empty_like(x)
    with torch.cuda.graph(graph):
        mid = nf4.nf4_moe(x, *layer, 4, workspace=ws1)
        nf4.nf4_moe(mid, *layer4, 4, workspace=ws1, out=buf)
    for seed in range(3):
        x.copy_(torch.randn(12, 512, device="cuda", generator=torch.Generator(device="cuda").manual_seed(seed)))
        want = nf4.nf4_moe(nf4.nf4_moe(x, *layer, 4), *layer4, 4)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(buf, want)


@gpu
def test_decoder_block_step(nf4):
    """The operators together as a decoder's step uses them: an integer projection, then
    the experts on its result."""
    h, f, E = 256, 128, 8
    layer = _layer(nf4, E, h, f, "int4_64", seed=12)
    proj = nf4.int4_quantize_weight(torch.randn(h, h, device="cuda") * h ** -0.5, 64, False)
    x = torch.randn(6, h, device="cuda").bfloat16()
    mid = nf4.nf4_int4_linear(x, proj)
    dense = x.double() @ nf4.nf4_int4_dequantize(proj, torch.float32).double().t()
    assert torch.all((mid.double() - dense).abs() <= UBF * dense.abs() + h * 2.0 ** -22 * (x.double().abs() @ _dense64(nf4, proj).abs().t()))
    _check(nf4, mid, layer, 2, True)


@gpu
def test_binding_refusals(nf4):
    layer = _layer(nf4, 4, 128, 64, "nf4", seed=3)
    layer4 = _layer(nf4, 4, 128, 64, "int4_64", seed=3)
    x = torch.randn(2, 128, device="cuda").bfloat16()
    r, gu, dn = layer
    bad = [lambda: nf4.nf4_moe(x.float(), r, gu, dn, 1), lambda: nf4.nf4_moe(x[:, :64].contiguous(), r, gu, dn, 1),
           lambda: nf4.nf4_moe(x, r.float(), gu, dn, 1), lambda: nf4.nf4_moe(x, r[:3].contiguous(), gu, dn, 1),
           lambda: nf4.nf4_moe(x, r, dn, gu, 1), lambda: nf4.nf4_moe(x, r, layer4[1], dn, 1), lambda: nf4.nf4_moe(x, r, gu, dn, 5),
           lambda: nf4.nf4_moe(x, r, gu, dn, 0), lambda: nf4.nf4_moe(x, r, gu, dn, 1, out=x.float()),
           lambda: nf4.nf4_moe(x.cpu(), r, gu, dn, 1), lambda: nf4.nf4_moe(x, r.t().contiguous().t(), gu, dn, 1),
           lambda: nf4.moe_workspace(100, 64, 4, 1)]
    for f in bad:
        with pytest.raises(ValueError):
            f()
    with pytest.raises(nf4.NF4Error):
        nf4.nf4_moe(x, r, gu, dn, 1, workspace=torch.empty(64, device="cuda", dtype=torch.uint8))
    with pytest.raises(nf4.NF4Error):
        nf4.nf4_moe(x[:0], r, gu, dn, 1)


@pytest.mark.parametrize("limit", ["NF4_MOE_MAX_EXPERTS", "NF4_MOE_MAX_TOP_K"])
def test_header_limits_are_those_of_the_routing_tables(tmp_path, limit):
    """A header with a larger limit (its checks would let more through) does not build."""
    header = open(os.path.join(INCLUDE, "nf4.h")).read()
    value = int(re.search(r"#define %s (\d+)" % limit, header).group(1))
    assert value == getattr(_lib, limit)
    (tmp_path / "nf4.h").write_text(header.replace("#define %s %d" % (limit, value), "#define %s %d" % (limit, 4 * value)))
    r = subprocess.run([nvcc(), "-I" + str(tmp_path), *NVCC_FLAGS, "-c", os.path.join(CSRC, "nf4_moe.cu"), "-o", str(tmp_path / "o.o")],
                       capture_output=True, text=True)
    assert r.returncode != 0 and "static assertion" in r.stderr and "routing tables" in r.stderr
