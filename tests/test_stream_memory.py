"""With ``stream=`` a call runs on that stream, and what it allocates must belong to it:
a block of the current stream's memory may still be used by work queued there, and one
that is dropped goes back to its own stream alone."""
import contextlib
from types import SimpleNamespace

import pytest
import torch

from quantized_linear_layers_nf4_b200 import _lib
from quantized_linear_layers_nf4_b200.build import build

gpu = pytest.mark.gpu


@pytest.fixture(scope="module")
def nf4():
    build()
    import quantized_linear_layers_nf4_b200 as m
    return m


# ------------------- where the memory comes from (CPU) -------------------
def _int4(nf4, n, k, group):
    w = object.__new__(nf4.Int4Weight)
    w.__dict__.update(n=n, k=k, group=group, wq=torch.zeros(n * k // 2, dtype=torch.uint8), scale=torch.zeros(k // group, n), zero=None)
    return w


def _nf4(nf4, n, k):
    nb = n * k // 64
    return nf4.NF4Weight(n, k, torch.zeros(n * k // 2, dtype=torch.uint8), torch.zeros(nb, dtype=torch.int8),
                         torch.zeros((nb + 255) // 256), torch.zeros(1))


def _calls(nf4, weight4, weight):
    """(call of stream, number of tensors that it allocates) for every entry point that allocates."""
    x, y = torch.zeros(2, 128).bfloat16(), torch.zeros(2, 192).bfloat16()
    W = torch.zeros(64, 128)
    w4, w = weight4(nf4, 192, 128, 64), weight(nf4, 192, 128)
    up, down = weight(nf4, 4 * 2 * 64, 128), weight(nf4, 4 * 128, 64)
    up4, down4 = weight4(nf4, 4 * 2 * 64, 128, 64), weight4(nf4, 4 * 128, 64, 64)
    router = torch.zeros(4, 128).bfloat16()
    lora = torch.zeros(8, 128).bfloat16(), torch.zeros(192, 8).bfloat16()
    return {
        "int4_quantize": (lambda s: nf4.nf4_int4_quantize(W, 64, False, stream=s), 3),
        "int4_dequantize": (lambda s: nf4.nf4_int4_dequantize(w4, stream=s), 1),
        "int4_linear": (lambda s: nf4.nf4_int4_linear(x, w4, stream=s), 1),
        "moe": (lambda s: nf4.nf4_moe(x, router, up, down, 2, stream=s, return_routing=True), 4),
        "int4_moe": (lambda s: nf4.nf4_moe(x, router, up4, down4, 2, stream=s, return_routing=True), 4),
        "quantize": (lambda s: nf4.nf4_quantize(W, stream=s), 2),
        "double_quant": (lambda s: nf4.nf4_double_quant(torch.zeros(256), stream=s), 4),
        "quantize_weight": (lambda s: nf4.quantize_weight(W, stream=s), 6),
        "dequantize": (lambda s: nf4.nf4_dequantize(w, stream=s), 1),
        "dequantize_batch": (lambda s: nf4.nf4_dequantize_batch([w, w], stream=s), 2),
        "linear": (lambda s: nf4.nf4_linear(x, w, stream=s), 1),
        "linear_group": (lambda s: nf4.nf4_linear_group(x, [w, w], stream=s), 2),
        "linear_dx": (lambda s: nf4.nf4_linear_dx(y, w, stream=s), 1),
        "linear_lora": (lambda s: nf4.nf4_linear_lora(x, w, *lora, 1.0, torch.zeros(64), stream=s), 1),
        "merge_lora": (lambda s: nf4.nf4_merge_lora(w, *lora, 1.0, True, stream=s), 3),
    }


NAMES = ["int4_quantize", "int4_dequantize", "int4_linear", "moe", "int4_moe", "quantize", "double_quant", "quantize_weight",
         "dequantize", "dequantize_batch", "linear", "linear_group", "linear_dx", "linear_lora", "merge_lora"]


@pytest.mark.parametrize("name", NAMES)
def test_allocations_belong_to_the_stream(nf4, monkeypatch, name):
    call, count = _calls(nf4, _int4, _nf4)[name]
    now, seen = [None], []

    @contextlib.contextmanager
    def stream(s):
        before, now[0] = now[0], s
        yield
        now[0] = before

    def recorded(make):
        def f(*args, **kw):
            seen.append(now[0])
            return make(*args, **kw)
        return f

    real = _lib.lib()

    class Lib:  # sizes are the library's, launches do nothing
        def __getattr__(self, fn):
            return getattr(real, fn) if fn.endswith("_bytes") else lambda *args: _lib.NF4_OK

    monkeypatch.setattr(_lib, "lib", Lib)
    monkeypatch.setattr(nf4, "_need_cuda", lambda t, what: None)
    monkeypatch.setattr(nf4, "_launch", lambda *args: None)
    monkeypatch.setattr(nf4, "_stream", lambda s: None)
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch, "empty", recorded(torch.empty))
    monkeypatch.setattr(torch, "empty_like", recorded(torch.empty_like))
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: None)
    side = SimpleNamespace(cuda_stream=1)
    call(side)
    assert seen == [side] * count
    seen.clear()
    call(None)
    assert seen == [None] * count


# ------------------------------- on the device -------------------------------
def _flat(v):
    if isinstance(v, torch.Tensor):
        return [v]
    if isinstance(v, (tuple, list)):
        return [t for u in v for t in _flat(u)]
    return [] if v is None else [v.wq, v.absmax_q, v.absmax_scale, v.absmax_offset]


@gpu
@pytest.mark.parametrize("name", ["int4_quantize", "int4_dequantize", "int4_linear", "moe", "int4_moe", "quantize", "quantize_weight",
                                  "dequantize", "linear", "linear_dx"])
def test_results_survive_what_the_current_stream_still_has_to_do(nf4, name):
    g = torch.Generator(device="cuda").manual_seed(3)

    def rand(*shape):
        return torch.randn(*shape, device="cuda", generator=g)

    W, x, y = rand(512, 256), rand(8, 256).bfloat16(), rand(8, 512).bfloat16()
    w4, w = nf4.int4_quantize_weight(W, 64), nf4.quantize_weight(W)
    router, up, down = rand(8, 256).bfloat16(), rand(8 * 2 * 128, 256), rand(8 * 256, 128)
    up4, down4 = nf4.int4_quantize_weight(up, 64), nf4.int4_quantize_weight(down, 64)
    up, down = nf4.quantize_weight(up), nf4.quantize_weight(down)
    call = {
        "int4_quantize": lambda s: nf4.nf4_int4_quantize(W, 64, False, stream=s),
        "int4_dequantize": lambda s: nf4.nf4_int4_dequantize(w4, stream=s),
        "int4_linear": lambda s: nf4.nf4_int4_linear(x, w4, stream=s),
        "moe": lambda s: nf4.nf4_moe(x, router, up, down, 2, stream=s, return_routing=True),
        "int4_moe": lambda s: nf4.nf4_moe(x, router, up4, down4, 2, stream=s, return_routing=True),
        "quantize": lambda s: nf4.nf4_quantize(W, stream=s),
        "quantize_weight": lambda s: nf4.quantize_weight(W, stream=s),
        "dequantize": lambda s: nf4.nf4_dequantize(w, stream=s),
        "linear": lambda s: nf4.nf4_linear(x, w, stream=s),
        "linear_dx": lambda s: nf4.nf4_linear_dx(y, w, stream=s),
    }[name]
    want = _flat(call(None))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    # blocks of the results' sizes, dropped while the current stream has yet to write them
    torch.cuda._sleep(20_000_000)
    blocks = [torch.empty_like(t) for t in want] + [nf4.moe_workspace(256, 128, 8, 2)]
    for _ in range(50):
        for t in blocks:
            t.view(-1).view(torch.uint8).fill_(7)
    del blocks, t
    got = _flat(call(side))
    torch.cuda.synchronize()
    for a, b in zip(want, got, strict=True):
        assert torch.equal(a, b)
