"""NF4 (4-bit NormalFloat) weight quantization with double quantization, and the
fused dequantize + bf16 linear, for NVIDIA B200 (sm_100a).

The work is done by ``lib/libnf4.so`` (C ABI in ``include/nf4.h``); this module
only marshals PyTorch device tensors and the current CUDA stream into those
calls.  Functions carry the C names:

* ``nf4_quantize(W)`` -> ``(wq, absmax)``
* ``nf4_double_quant(absmax)`` -> ``(absmax_q, absmax_scale, absmax_offset)``
* ``nf4_dequantize(weight, dtype)`` -> dense tensor
* ``nf4_linear(X, weight, dtype)`` -> ``Y = X @ W_hat^T`` (optionally with a
  split-k ``workspace`` from ``linear_workspace``)
* ``nf4_linear_group(X, weights, dtype)`` -> ``[X @ W_i^T]`` for weights that
  share X (q/k/v, gate/up), in one launch
* ``nf4_linear_dx(dY, weight, dtype)`` -> ``dX = dY @ W_hat`` (backward through
  the frozen base)
* ``nf4_linear_lora(X, weight, down, up, scale, workspace=...)`` -> the QLoRA
  layer ``X @ W_hat^T + scale * (X @ down^T) @ up^T``
* ``nf4_merge_lora(weight, down, up, scale)`` -> ``(wq, absmax, w_new)``: the
  trained update folded into the weight and quantized again (``merge_lora``
  adds the double quantization and returns an ``NF4Weight``)

* ``nf4_int4_quantize(W, group)`` -> ``(wq, scale, zero)``, ``nf4_int4_dequantize``
  and ``nf4_int4_linear(X, weight)``: integer 4-bit weights with one scale (and
  zero point) per group (``int4_quantize_weight`` returns an ``Int4Weight``)

* ``nf4_moe(X, router, gate_up, down, top_k, workspace=...)``: a mixture-of-experts
  layer for a few tokens with NF4, FP4 or integer 4-bit experts

``quantize_weight(W)`` runs the first two and returns an ``NF4Weight``.  Every
quantizing call takes ``quant_type="nf4"`` (the default) or ``"fp4"``; an
``NF4Weight`` remembers which codebook its codes index.

With ``stream=`` a call runs on that stream, and the tensors it makes belong to it, as
under ``torch.cuda.stream(stream)``.  The usual rules follow: its inputs must be ready
there, and a tensor of one stream that another still uses when its last reference goes
needs ``Tensor.record_stream``.
"""
from __future__ import annotations

import contextlib
import ctypes
from dataclasses import dataclass

import torch

from . import _lib
from ._lib import NF4_BF16, NF4_F32, NF4Error, nf4_int4_weight_t, nf4_weight_t

__all__ = ["NF4Weight", "NF4Error", "nf4_quantize", "nf4_double_quant", "nf4_dequantize",
           "nf4_linear", "nf4_linear_ex", "nf4_linear_group", "nf4_linear_dx", "nf4_linear_lora", "lora_workspace",
           "nf4_merge_lora", "merge_lora", "nf4_dequantize_batch",
           "nf4_linear_workspace_bytes", "linear_workspace",
           "quantize_weight", "nf4_codebook", "library_path",
           "Int4Weight", "nf4_int4_quantize", "nf4_int4_dequantize", "nf4_int4_linear", "int4_quantize_weight",
           "nf4_moe", "moe_workspace"]

_DTYPES = {torch.float32: NF4_F32, torch.bfloat16: NF4_BF16}
_QUANT_TYPES = {"nf4": _lib.NF4_QUANT_NF4, "fp4": _lib.NF4_QUANT_FP4}


def _quant_type(quant_type: str) -> int:
    if quant_type not in _QUANT_TYPES:
        raise ValueError("quant_type must be 'nf4' or 'fp4'")
    return _QUANT_TYPES[quant_type]


def library_path() -> str:
    return _lib.LIB_PATH


def _stream(stream) -> ctypes.c_void_p:
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


_HERE = contextlib.nullcontext()


def _memory_of(stream):
    """What is allocated inside belongs to the stream that the call runs on.  A block of the
    current stream's would be one that work queued there may still use, and dropped it could go
    to a third stream while this one writes it."""
    return _HERE if stream is None else torch.cuda.stream(stream)


def _ptr(t: torch.Tensor) -> ctypes.c_void_p:
    return ctypes.c_void_p(t.data_ptr())


def _need_cuda(t: torch.Tensor, name: str) -> None:
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)


def nf4_codebook(quant_type: str = "nf4") -> torch.Tensor:
    """The 16 levels the library uses (host copy): NF4 ascending, FP4 in code order."""
    out = torch.zeros(16, dtype=torch.float32)
    _lib.check(_lib.lib().nf4_codebook_typed(_quant_type(quant_type), _ptr(out)), "nf4_codebook")
    return out


def nf4_quantize(W: torch.Tensor, wq: torch.Tensor | None = None, absmax: torch.Tensor | None = None,
                 stream=None, quant_type: str = "nf4"):
    """Blockwise NF4 (or FP4) quantization of a 2-D fp32/bf16 CUDA tensor [n, k]."""
    qt = _quant_type(quant_type)
    _need_cuda(W, "W")
    if W.dim() != 2 or W.dtype not in _DTYPES:
        raise ValueError("W must be a 2-D float32 or bfloat16 tensor")
    n, k = W.shape
    numel = n * k
    with _memory_of(stream):
        if wq is None:
            wq = torch.empty(numel // 2, dtype=torch.uint8, device=W.device)
        if absmax is None:
            absmax = torch.empty(numel // 64, dtype=torch.float32, device=W.device)
    _lib.check(_lib.lib().nf4_quantize_typed(_ptr(W), _DTYPES[W.dtype], n, k, qt, _ptr(wq), _ptr(absmax),
                                             _stream(stream)), "nf4_quantize")
    return wq, absmax


def nf4_double_quant(absmax: torch.Tensor, absmax_q: torch.Tensor | None = None,
                     absmax_scale: torch.Tensor | None = None,
                     absmax_offset: torch.Tensor | None = None,
                     workspace: torch.Tensor | None = None, stream=None):
    """Double quantization of the fp32 absmax vector."""
    _need_cuda(absmax, "absmax")
    nb = absmax.numel()
    L = _lib.lib()
    ws_bytes = L.nf4_double_quant_workspace_bytes(nb)
    with _memory_of(stream):
        if workspace is None:
            workspace = torch.empty(max(ws_bytes, 8) // 8 + 1, dtype=torch.float64, device=absmax.device)
        if absmax_q is None:
            absmax_q = torch.empty(nb, dtype=torch.int8, device=absmax.device)
        if absmax_scale is None:
            absmax_scale = torch.empty((nb + 255) // 256, dtype=torch.float32, device=absmax.device)
        if absmax_offset is None:
            absmax_offset = torch.empty(1, dtype=torch.float32, device=absmax.device)
    _lib.check(L.nf4_double_quant(_ptr(absmax), nb, _ptr(workspace),
                                  workspace.numel() * workspace.element_size(), _ptr(absmax_q),
                                  _ptr(absmax_scale), _ptr(absmax_offset), _stream(stream)),
               "nf4_double_quant")
    return absmax_q, absmax_scale, absmax_offset


class _KeptStruct:
    """The C struct that a weight's calls pass, kept beside its fields (not among them, so it
    is neither copied nor pickled) and built again when the key -- sizes and data pointers --
    is not that of the last time."""
    __slots__ = ("_kept",)

    def _struct_ref(self):
        """(key, C struct, reference to it); shared by all calls, not to be changed."""
        key = self._key()
        kept = getattr(self, "_kept", None)
        if kept is None or kept[0] != key:
            st = self._make(key)
            kept = (key, st, ctypes.byref(st))
            _set_kept(self, kept)
        return kept

    def struct(self):
        """A C struct of its own that borrows the weight's tensors."""
        return self._make(self._key())

    def __getstate__(self):
        return self.__dict__


_set_kept = _KeptStruct._kept.__set__  # past a frozen class's own


@dataclass
class NF4Weight(_KeptStruct):
    """A quantized [n, k] weight: device tensors plus the C struct that borrows them."""
    n: int
    k: int
    wq: torch.Tensor
    absmax_q: torch.Tensor
    absmax_scale: torch.Tensor
    absmax_offset: torch.Tensor
    quant_type: str = "nf4"

    def _key(self):
        return (self.n, self.k, self.quant_type, self.wq.data_ptr(), self.absmax_q.data_ptr(), self.absmax_scale.data_ptr(),
                self.absmax_offset.data_ptr())

    def _make(self, key) -> nf4_weight_t:
        magic = _lib.NF4_FP4_WEIGHT_MAGIC if self.quant_type == "fp4" else _lib.NF4_WEIGHT_MAGIC
        return nf4_weight_t(magic, _lib.NF4_WEIGHT_VERSION, self.n, self.k, _lib.NF4_BLOCKSIZE, _lib.NF4_BLOCKSIZE2, *key[3:])

    def nbytes(self) -> int:
        return (self.wq.numel() + self.absmax_q.numel() + 4 * self.absmax_scale.numel())


def quantize_weight(W: torch.Tensor, stream=None, quant_type: str = "nf4") -> NF4Weight:
    """nf4_quantize followed by nf4_double_quant; the fp32 absmax is dropped."""
    wq, absmax = nf4_quantize(W, stream=stream, quant_type=quant_type)
    q, s, mu = nf4_double_quant(absmax, stream=stream)
    return NF4Weight(W.shape[0], W.shape[1], wq, q, s, mu, quant_type)


def nf4_dequantize(weight: NF4Weight, dtype=torch.bfloat16, out: torch.Tensor | None = None,
                   stream=None) -> torch.Tensor:
    if dtype not in _DTYPES:
        raise ValueError("dtype must be float32 or bfloat16")
    if out is None:
        with _memory_of(stream):
            out = torch.empty((weight.n, weight.k), dtype=dtype, device=weight.wq.device)
    st = weight._struct_ref()[1]
    _lib.check(_lib.lib().nf4_dequantize(ctypes.byref(st), _ptr(out), _DTYPES[dtype],
                                         _stream(stream)), "nf4_dequantize")
    return out


def nf4_dequantize_batch(weights, dtype=torch.bfloat16, outs=None, stream=None):
    """[nf4_dequantize(w) for w in weights] in one launch (at most
    NF4_DEQUANT_BATCH_MAX weights; the same bits).  Returns the list of outputs."""
    if dtype not in _DTYPES:
        raise ValueError("dtype must be float32 or bfloat16")
    weights = list(weights)
    count = len(weights)
    if outs is None:
        with _memory_of(stream):
            outs = [torch.empty((w.n, w.k), dtype=dtype, device=w.wq.device) for w in weights]
    for o in outs:
        _need_cuda(o, "out")
    structs = [w._struct_ref()[1] for w in weights]
    wptrs = (ctypes.POINTER(nf4_weight_t) * max(count, 1))(*[ctypes.pointer(s) for s in structs])
    optrs = (ctypes.c_void_p * max(count, 1))(*[o.data_ptr() for o in outs])
    _lib.check(_lib.lib().nf4_dequantize_batch(wptrs, count, optrs, _DTYPES[dtype], _stream(stream)),
               "nf4_dequantize_batch")
    return outs


def nf4_linear_ex(X, weight, dtype=torch.bfloat16, out=None, dev_status=None, stream=None,
                  flags: int = 0, workspace=None):
    """Same as nf4_linear with the C flags word (NF4_LINEAR_WEIGHTS_EARLY,
    NF4_LINEAR_TEST_TIMEOUT)."""
    return nf4_linear(X, weight, dtype, out, dev_status, stream, workspace=workspace, flags=flags)


def nf4_linear_workspace_bytes(m: int, n: int, k: int) -> int:
    """Bytes of the optional split-k workspace of nf4_linear for these sizes on
    the current device (0: none needed)."""
    return int(_lib.lib().nf4_linear_workspace_bytes(m, n, k))


def linear_workspace(shapes, m: int = 16, device=None) -> torch.Tensor:
    """A zero-filled workspace large enough for nf4_linear at m tokens on every
    (n, k) in ``shapes`` (one buffer serves them all)."""
    nbytes = max([nf4_linear_workspace_bytes(m, n, k) for n, k in shapes] + [16])
    return torch.zeros((nbytes + 15) // 16 * 16, dtype=torch.uint8, device=device or "cuda")


def nf4_linear(X: torch.Tensor, weight: NF4Weight, dtype=torch.bfloat16,
               out: torch.Tensor | None = None, dev_status: torch.Tensor | None = None,
               stream=None, weights_early: bool = False,
               workspace: torch.Tensor | None = None, flags: int = 0) -> torch.Tensor:
    """Y = X @ W_hat^T for bf16 X [m, k]; Y [m, n] in ``dtype`` (bf16 or fp32).

    ``weights_early=True`` sets NF4_LINEAR_WEIGHTS_EARLY: the weight was not
    written by the work just before this call on the stream, so its loads may
    overlap that work (programmatic dependent launch).  ``workspace`` (from
    ``linear_workspace``) lets the decode path split the tiles of a weight over
    all SMs, with partial sums meeting in global memory; the results are the
    same bits as without it.  ``flags`` is OR'ed into the C flags word.  The
    call goes to ``nf4_linear_ws``."""
    _need_cuda(X, "X")
    if X.dtype != torch.bfloat16 or X.dim() != 2:
        raise ValueError("X must be a 2-D bfloat16 tensor")
    if dtype not in _DTYPES:
        raise ValueError("dtype must be float32 or bfloat16")
    m = X.shape[0]
    if out is None:
        with _memory_of(stream):
            out = torch.empty((m, weight.n), dtype=dtype, device=X.device)
    st = weight._struct_ref()[1]
    ds = ctypes.c_void_p(0) if dev_status is None else _ptr(dev_status)
    flags |= _lib.NF4_LINEAR_WEIGHTS_EARLY if weights_early else 0
    ws, ws_bytes = _ws(workspace)
    _lib.check(_lib.lib().nf4_linear_ws(_ptr(X), m, ctypes.byref(st), _ptr(out), _DTYPES[dtype], ds,
                                        flags, ws, ws_bytes, _stream(stream)), "nf4_linear_ws")
    return out


def _ws(workspace):
    if workspace is None:
        return ctypes.c_void_p(0), 0
    _need_cuda(workspace, "workspace")
    return _ptr(workspace), workspace.numel() * workspace.element_size()


def nf4_linear_group_launches(m: int, ns, k: int) -> int:
    """Kernel launches nf4_linear_group makes for weights of rows `ns` and width k
    at m tokens on the current device (1 when grouped into one launch)."""
    arr = (ctypes.c_int64 * len(ns))(*[int(n) for n in ns])
    r = _lib.lib().nf4_linear_group_launches(int(m), arr, len(ns), int(k))
    if r < 0:
        raise ValueError("invalid sizes or no usable device")
    return int(r)


def nf4_linear_group(X: torch.Tensor, weights, dtype=torch.bfloat16, outs=None,
                     dev_status: torch.Tensor | None = None, stream=None, weights_early: bool = False,
                     workspace: torch.Tensor | None = None, flags: int = 0):
    """[X @ W_i^T for W_i in weights] in one call for weights that share X and k
    (at most NF4_LINEAR_GROUP_MAX): one launch over all their row tiles when
    that is faster than one launch per weight.  Each output equals nf4_linear on
    that weight alone up to the fp32 summation order.  Returns the list of
    outputs."""
    _need_cuda(X, "X")
    if X.dtype != torch.bfloat16 or X.dim() != 2:
        raise ValueError("X must be a 2-D bfloat16 tensor")
    if dtype not in _DTYPES:
        raise ValueError("dtype must be float32 or bfloat16")
    weights = list(weights)
    count = len(weights)
    m = X.shape[0]
    if outs is None:
        with _memory_of(stream):
            outs = [torch.empty((m, w.n), dtype=dtype, device=X.device) for w in weights]
    structs = [w._struct_ref()[1] for w in weights]
    wptrs = (ctypes.POINTER(nf4_weight_t) * max(count, 1))(*[ctypes.pointer(s) for s in structs])
    yptrs = (ctypes.c_void_p * max(count, 1))(*[o.data_ptr() for o in outs])
    ds = ctypes.c_void_p(0) if dev_status is None else _ptr(dev_status)
    flags |= _lib.NF4_LINEAR_WEIGHTS_EARLY if weights_early else 0
    ws, ws_bytes = _ws(workspace)
    _lib.check(_lib.lib().nf4_linear_group(_ptr(X), m, wptrs, count, yptrs, _DTYPES[dtype], ds, flags, ws,
                                           ws_bytes, _stream(stream)), "nf4_linear_group")
    return outs


def nf4_linear_dx(dY: torch.Tensor, weight: NF4Weight, dtype=torch.bfloat16,
                  out: torch.Tensor | None = None, dev_status: torch.Tensor | None = None,
                  stream=None) -> torch.Tensor:
    """dX = dY @ W_hat for bf16 dY [m, n] (n % 8 == 0); dX [m, k] in ``dtype``."""
    _need_cuda(dY, "dY")
    if dY.dtype != torch.bfloat16 or dY.dim() != 2 or dY.shape[1] != weight.n:
        raise ValueError("dY must be a 2-D bfloat16 tensor with n columns")
    if dtype not in _DTYPES:
        raise ValueError("dtype must be float32 or bfloat16")
    m = dY.shape[0]
    if out is None:
        with _memory_of(stream):
            out = torch.empty((m, weight.k), dtype=dtype, device=dY.device)
    st = weight._struct_ref()[1]
    ds = ctypes.c_void_p(0) if dev_status is None else _ptr(dev_status)
    _lib.check(_lib.lib().nf4_linear_dx(_ptr(dY), m, ctypes.byref(st), _ptr(out), _DTYPES[dtype], ds,
                                        _stream(stream)), "nf4_linear_dx")
    return out


def lora_workspace(m: int, shapes, r: int, device=None) -> torch.Tensor:
    """A zero-filled workspace for nf4_linear_lora at m tokens and rank r on every
    (n, k) in ``shapes``."""
    L = _lib.lib()
    nbytes = max([int(L.nf4_linear_lora_workspace_bytes(m, n, k, r)) for n, k in shapes] + [16])
    return torch.zeros((nbytes + 15) // 16 * 16, dtype=torch.uint8, device=device or "cuda")


def nf4_linear_lora(X: torch.Tensor, weight: NF4Weight, down: torch.Tensor, up: torch.Tensor, scale: float,
                    workspace: torch.Tensor, dtype=torch.bfloat16, out: torch.Tensor | None = None,
                    dev_status: torch.Tensor | None = None, stream=None,
                    weights_early: bool = False) -> torch.Tensor:
    """Y = X @ W_hat^T + scale * (X @ down^T) @ up^T with down bf16 [r, k] and up
    bf16 [n, r]; ``workspace`` from ``lora_workspace``."""
    for t, name in ((X, "X"), (down, "down"), (up, "up"), (workspace, "workspace")):
        _need_cuda(t, name)
    if X.dtype != torch.bfloat16 or down.dtype != torch.bfloat16 or up.dtype != torch.bfloat16:
        raise ValueError("X, down and up must be bfloat16")
    r = down.shape[0]
    if down.shape != (r, weight.k) or up.shape != (weight.n, r) or X.shape[1] != weight.k:
        raise ValueError("shapes: X [m, k], down [r, k], up [n, r]")
    if dtype not in _DTYPES:
        raise ValueError("dtype must be float32 or bfloat16")
    m = X.shape[0]
    if out is None:
        with _memory_of(stream):
            out = torch.empty((m, weight.n), dtype=dtype, device=X.device)
    st = weight._struct_ref()[1]
    ds = ctypes.c_void_p(0) if dev_status is None else _ptr(dev_status)
    flags = _lib.NF4_LINEAR_WEIGHTS_EARLY if weights_early else 0
    _lib.check(_lib.lib().nf4_linear_lora(_ptr(X), m, ctypes.byref(st), _ptr(down), _ptr(up), r, float(scale),
                                          _ptr(out), _DTYPES[dtype], ds, flags, _ptr(workspace),
                                          workspace.numel() * workspace.element_size(), _stream(stream)),
               "nf4_linear_lora")
    return out


def nf4_merge_lora(weight: NF4Weight, down: torch.Tensor, up: torch.Tensor, scale: float,
                   want_bf16: bool = False, wq: torch.Tensor | None = None,
                   absmax: torch.Tensor | None = None, stream=None):
    """Dequantize to bf16, add scale * up @ down in bf16 and quantize again.
    Returns (wq, absmax fp32, w_new bf16 [n, k] or None)."""
    for t, name in ((down, "down"), (up, "up")):
        _need_cuda(t, name)
    if down.dtype != torch.bfloat16 or up.dtype != torch.bfloat16:
        raise ValueError("down and up must be bfloat16")
    r = down.shape[0]
    if down.dim() != 2 or down.shape != (r, weight.k) or up.shape != (weight.n, r):
        raise ValueError("shapes: down [r, k], up [n, r]")
    numel = weight.n * weight.k
    dev = weight.wq.device
    with _memory_of(stream):
        if wq is None:
            wq = torch.empty(numel // 2, dtype=torch.uint8, device=dev)
        if absmax is None:
            absmax = torch.empty(numel // 64, dtype=torch.float32, device=dev)
        w_new = torch.empty((weight.n, weight.k), dtype=torch.bfloat16, device=dev) if want_bf16 else None
    st = weight._struct_ref()[1]
    _lib.check(_lib.lib().nf4_merge_lora(ctypes.byref(st), _ptr(down), _ptr(up), r, float(scale),
                                         ctypes.c_void_p(0) if w_new is None else _ptr(w_new), _ptr(wq),
                                         _ptr(absmax), _stream(stream)), "nf4_merge_lora")
    return wq, absmax, w_new


def merge_lora(weight: NF4Weight, down: torch.Tensor, up: torch.Tensor, scale: float, stream=None) -> NF4Weight:
    """nf4_merge_lora followed by nf4_double_quant: the merged, requantized weight."""
    wq, absmax, _ = nf4_merge_lora(weight, down, up, scale, stream=stream)
    q, s, mu = nf4_double_quant(absmax, stream=stream)
    return NF4Weight(weight.n, weight.k, wq, q, s, mu, weight.quant_type)


def _check_out(out: torch.Tensor, shape, dtypes, device, name: str) -> None:
    if out.shape != shape or out.dtype not in dtypes or out.device != device or not out.is_contiguous():
        raise ValueError("%s must be a contiguous %s tensor on %s with one of the dtypes %s"
                         % (name, tuple(shape), device, tuple(dtypes)))


def _launch(index: int, stream, fn, where: str, *args) -> None:
    """fn(*args, stream) on device ``index``, which need not be the current one; the
    stream is that device's current one unless given."""
    if index != torch._C._cuda_getDevice():
        with torch.cuda.device(index):
            return _launch(index, stream, fn, where, *args)
    st = fn(*args, torch._C._cuda_getCurrentRawStream(index) if stream is None else stream.cuda_stream)
    if st != _lib.NF4_OK:
        _lib.check(st, where)


def _group_ok(k: int, group: int) -> bool:
    return k > 0 and group > 0 and k % 64 == 0 and (group == 32 or group % 64 == 0) and k % group == 0


_GROUP_RULE = "k must be a multiple of 64, group 32 or a multiple of 64 that divides k"


@dataclass(frozen=True)
class Int4Weight(_KeptStruct):
    """An integer 4-bit [n, k] weight with group scales: codes uint8 [n*k/2]
    (element 2i in the high nibble), ``scale`` [k/group, n] bf16 or fp32 and ``zero``
    uint8 [k/group, n], or None where every zero point is 8.  W ~ (q - zero) * scale."""
    n: int
    k: int
    group: int
    wq: torch.Tensor
    scale: torch.Tensor
    zero: torch.Tensor | None = None

    def __post_init__(self):
        n, k, group = self.n, self.k, self.group
        if n < 1 or not _group_ok(k, group):
            raise ValueError(_GROUP_RULE)
        wq, scale, zero = self.wq, self.scale, self.zero
        if not wq.is_cuda or wq.dtype != torch.uint8 or wq.numel() != n * k // 2 or not wq.is_contiguous():
            raise ValueError("wq must be a contiguous uint8 CUDA tensor of n * k / 2 bytes")
        dev = wq.device
        _check_out(scale, (k // group, n), _DTYPES, dev, "scale")
        if zero is not None:
            _check_out(zero, (k // group, n), (torch.uint8,), dev, "zero")

    def _key(self):
        return (self.wq.data_ptr(), self.scale.data_ptr(), None if self.zero is None else self.zero.data_ptr())

    def _make(self, key) -> nf4_int4_weight_t:
        return nf4_int4_weight_t(_lib.NF4_INT4_WEIGHT_MAGIC, _lib.NF4_WEIGHT_VERSION, self.n, self.k, self.group,
                                 _DTYPES[self.scale.dtype], 0, *key)

    def nbytes(self) -> int:
        return (self.wq.numel() + self.scale.numel() * self.scale.element_size() +
                (0 if self.zero is None else self.zero.numel()))


def _int4_outputs(n, k, group, symmetric, scale_dtype, wq, scale, zero, dev):
    """The outputs of a quantization: those given, checked, and new ones."""
    if wq is None:
        wq = torch.empty(n * k // 2, dtype=torch.uint8, device=dev)
    else:
        _check_out(wq, (n * k // 2,), (torch.uint8,), dev, "wq")
    if scale is None:
        scale = torch.empty(k // group, n, dtype=scale_dtype, device=dev)
    else:
        _check_out(scale, (k // group, n), (scale_dtype,), dev, "scale")
    if zero is not None:
        _check_out(zero, (k // group, n), (torch.uint8,), dev, "zero")
    elif not symmetric:
        zero = torch.empty(k // group, n, dtype=torch.uint8, device=dev)
    return wq, scale, zero


def nf4_int4_quantize(W: torch.Tensor, group: int = 128, symmetric: bool = True, scale_dtype=torch.bfloat16,
                      wq: torch.Tensor | None = None, scale: torch.Tensor | None = None,
                      zero: torch.Tensor | None = None, stream=None):
    """Integer codes with one scale per ``group`` weights of a row, for a 2-D fp32/bf16
    CUDA tensor [n, k].  Returns (wq, scale, zero); zero is None when ``symmetric``."""
    _need_cuda(W, "W")
    if W.dim() != 2 or W.dtype not in _DTYPES:
        raise ValueError("W must be a 2-D float32 or bfloat16 tensor")
    if scale_dtype not in _DTYPES:
        raise ValueError("scale_dtype must be float32 or bfloat16")
    if symmetric and zero is not None:
        raise ValueError("zero is an output of asymmetric quantization only")
    n, k = W.shape
    if not _group_ok(k, group):
        raise ValueError(_GROUP_RULE)
    dev = W.device
    if stream is None:
        wq, scale, zero = _int4_outputs(n, k, group, symmetric, scale_dtype, wq, scale, zero, dev)
    else:
        with _memory_of(stream):
            wq, scale, zero = _int4_outputs(n, k, group, symmetric, scale_dtype, wq, scale, zero, dev)
    _launch(dev.index, stream, _lib.lib().nf4_int4_quantize, "nf4_int4_quantize", W.data_ptr(), _DTYPES[W.dtype], n, k, group,
            _DTYPES[scale_dtype], wq.data_ptr(), scale.data_ptr(), None if zero is None else zero.data_ptr())
    return wq, scale, zero


def int4_quantize_weight(W: torch.Tensor, group: int = 128, symmetric: bool = True, scale_dtype=torch.bfloat16,
                         stream=None) -> Int4Weight:
    """nf4_int4_quantize as an Int4Weight."""
    wq, scale, zero = nf4_int4_quantize(W, group, symmetric, scale_dtype, stream=stream)
    return Int4Weight(W.shape[0], W.shape[1], group, wq, scale, zero)


def nf4_int4_dequantize(weight: Int4Weight, dtype=torch.bfloat16, out: torch.Tensor | None = None,
                        stream=None) -> torch.Tensor:
    """(q - zero) * scale as a dense [n, k] tensor of ``dtype`` (of ``out``, where given)."""
    dev = weight.wq.device
    if out is None:
        if dtype not in _DTYPES:
            raise ValueError("dtype must be float32 or bfloat16")
        if stream is None:
            out = torch.empty(weight.n, weight.k, dtype=dtype, device=dev)
        else:
            with _memory_of(stream):
                out = torch.empty(weight.n, weight.k, dtype=dtype, device=dev)
    else:
        _check_out(out, (weight.n, weight.k), _DTYPES, dev, "out")
    _launch(dev.index, stream, _lib.lib().nf4_int4_dequantize, "nf4_int4_dequantize", weight._struct_ref()[2], out.data_ptr(),
            _DTYPES[out.dtype])
    return out


def nf4_int4_linear(X: torch.Tensor, weight: Int4Weight, dtype=torch.bfloat16, out: torch.Tensor | None = None,
                    dev_status: torch.Tensor | None = None, stream=None, weights_early: bool = False,
                    flags: int = 0) -> torch.Tensor:
    """Y = X @ W_hat^T for bf16 X [m, k] and an integer 4-bit weight; Y [m, n] in
    ``dtype`` (in that of ``out``, where given).  For few tokens (up to 16, and more
    where that is faster) the weight is not rounded; otherwise it is restored on chip, to
    bf16 as in nf4_linear for a bf16 result and to twice that precision for an fp32 one
    (which takes up to 1.7 times as long).
    ``weights_early`` and ``flags`` as for nf4_linear."""
    _need_cuda(X, "X")
    dev = X.device
    if X.dtype != torch.bfloat16 or X.dim() != 2 or X.shape[1] != weight.k or weight.wq.device != dev:
        raise ValueError("X must be a 2-D bfloat16 tensor with k columns on the weight's device")
    m = X.shape[0]
    if out is None:
        if dtype not in _DTYPES:
            raise ValueError("dtype must be float32 or bfloat16")
        with _memory_of(stream):
            out = torch.empty(m, weight.n, dtype=dtype, device=dev)
    else:
        _check_out(out, (m, weight.n), _DTYPES, dev, "out")
    if dev_status is not None and (dev_status.dtype != torch.int32 or dev_status.device != dev or dev_status.numel() < 1):
        raise ValueError("dev_status must be an int32 tensor on the device of X")
    flags |= _lib.NF4_LINEAR_WEIGHTS_EARLY if weights_early else 0
    _launch(dev.index, stream, _lib.lib().nf4_int4_linear, "nf4_int4_linear", X.data_ptr(), m, weight._struct_ref()[2], out.data_ptr(),
            _DTYPES[out.dtype], None if dev_status is None else dev_status.data_ptr(), flags)
    return out


def moe_workspace(h: int, f: int, n_experts: int, top_k: int, device=None) -> torch.Tensor:
    """A workspace for nf4_moe on any number of tokens; its contents do not matter."""
    nbytes = int(_lib.lib().nf4_moe_workspace_bytes(h, f, n_experts, top_k))
    if nbytes == 0:
        raise ValueError("h and f must be multiples of 64, n_experts at most %d, top_k at most %d and n_experts"
                         % (_lib.NF4_MOE_MAX_EXPERTS, _lib.NF4_MOE_MAX_TOP_K))
    return torch.empty(nbytes, dtype=torch.uint8, device=device or "cuda")


def nf4_moe(X: torch.Tensor, router: torch.Tensor, gate_up, down, top_k: int, renormalize: bool = True,
            out: torch.Tensor | None = None, workspace: torch.Tensor | None = None, stream=None,
            return_routing: bool = False):
    """A mixture-of-experts layer for a few tokens: X bf16 [m, h] through router bf16
    [E, h], the ``top_k`` experts of each row and their gated feed-forward weights,
    gate_up [E * 2f, h] (each expert's gate rows, then its up rows) and down [E * h, f],
    both NF4Weight or both Int4Weight.  Returns Y bf16 [m, h], and with
    ``return_routing`` (Y, ids int32 [m, top_k], probabilities fp32 [m, top_k]).
    ``workspace`` from ``moe_workspace``; it must not serve two calls at once."""
    _need_cuda(X, "X")
    _need_cuda(router, "router")
    index = X.get_device()
    if X.dtype != torch.bfloat16 or X.dim() != 2 or router.dtype != torch.bfloat16 or router.dim() != 2:
        raise ValueError("X and router must be 2-D bfloat16 tensors")
    m, h = X.shape
    n_experts, f = router.shape[0], down.k
    integer = isinstance(gate_up, Int4Weight)
    if integer != isinstance(down, Int4Weight):
        raise ValueError("gate_up and down must both be NF4Weight or both be Int4Weight")
    if router.shape[1] != h or gate_up.k != h or gate_up.n != n_experts * 2 * f or down.n != n_experts * h:
        raise ValueError("shapes: X [m, h], router [E, h], gate_up [E * 2f, h], down [E * h, f]")
    if router.get_device() != index or gate_up.wq.get_device() != index or down.wq.get_device() != index:
        raise ValueError("X, router and the weights must be on one device")
    if out is None:
        with _memory_of(stream):
            out = torch.empty_like(X)
    else:
        _check_out(out, X.shape, (torch.bfloat16,), X.device, "out")
    if workspace is None:
        with _memory_of(stream):
            workspace = moe_workspace(h, f, n_experts, top_k, X.device)
    elif workspace.get_device() != index or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the device of X")
    ids = probs = None
    if return_routing:
        with _memory_of(stream):
            ids = torch.empty(m, top_k, dtype=torch.int32, device=X.device)
            probs = torch.empty(m, top_k, dtype=torch.float32, device=X.device)
    L = _lib.lib()
    if integer:
        fn, where, gu, dn = L.nf4_int4_moe, "nf4_int4_moe", gate_up._struct_ref()[2], down._struct_ref()[2]
    else:
        fn, where, gu, dn = L.nf4_moe, "nf4_moe", gate_up._struct_ref()[2], down._struct_ref()[2]
    _launch(index, stream, fn, where, X.data_ptr(), m, router.data_ptr(), n_experts, gu, dn, top_k, out.data_ptr(),
            None if ids is None else ids.data_ptr(), None if probs is None else probs.data_ptr(),
            _lib.NF4_MOE_RENORMALIZE if renormalize else 0, workspace.data_ptr(),
            workspace.numel() * workspace.element_size())
    return (out, ids, probs) if return_routing else out
