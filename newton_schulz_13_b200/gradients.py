"""The operators that make the gradients which muon_step and adamw_step take: the token embedding,
the root-mean-square norm, and 8-bit activation checkpoints with the weight gradient taken from them.

    y = ns.embedding(tokens, table, scale=s)                      # forward
    y, h, rstd, ck = ns.rms_norm(x, w, residual=r, checkpoint=True)
    dW = ns.weight_grad(dY, ck)                                   # muon_step's gradient of y @ W.T
    dx, dw = ns.rms_norm_grad(dy, h, w, rstd, dh=dh)              # adamw_step's gradient of a norm scale
    dE = ns.embedding_grad(tokens, dx, vocab, scale=s)            # adamw_step's gradient of the table

Argument marshalling only, as in the rest of the package; include/muon.h has the formulas. The plain
case of a call (contiguous tensors of the current device, outputs to be allocated, the current
stream) goes through the extension _plain (csrc/binding.cpp): 4-7 us of the interpreter's time instead of 10-23.
Any other, and any that is refused, takes the path below through ctypes. Inputs
are CUDA tensors whose last dimension is contiguous (rows may be strided); leading dimensions are
taken as rows. Outputs and workspaces come from torch's allocator on the stream the call runs on
(`stream`, or the current stream of the tensors' device), so calls on several streams, and calls
captured into several graphs, share nothing. Inputs that belong to another stream are the caller's to
keep until the call's work is done. Nothing is recorded for autograd: outputs are detached, and the
caller calls the backward operators.
"""
from __future__ import annotations

import ctypes
import functools
import importlib.machinery
import importlib.util
import warnings
from typing import NamedTuple, Optional

import torch

from . import BF16, FP32, MuonError, _check, last_error, lib

_vp, _i64, _int, _f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float
for _name, _args in {
        "muon_embedding": [_vp, _int, _i64, _vp, _int, _i64, _i64, _i64, _f32, _vp, _int, _i64, _vp],
        "muon_embedding_grad": [_vp, _int, _i64, _vp, _int, _i64, _i64, _i64, _f32, _vp, _int, _i64, _int, _vp, _i64, _vp],
        "muon_rms_norm": [_vp, _int, _i64, _vp, _int, _i64, _vp, _int, _i64, _i64, _f32, _vp, _i64, _vp, _i64, _vp, _i64,
                          _vp, _i64, _vp, _vp],
        "muon_rms_norm_grad": [_vp, _int, _i64, _vp, _int, _i64, _vp, _int, _vp, _vp, _i64, _i64, _i64, _vp, _i64, _vp,
                               _int, _vp, _i64, _vp],
        "muon_checkpoint_store": [_vp, _int, _i64, _i64, _i64, _vp, _i64, _vp, _i64, _vp],
        "muon_checkpoint_restore": [_vp, _i64, _vp, _i64, _i64, _i64, _vp, _int, _i64, _vp],
        "muon_weight_grad": [_vp, _int, _i64, _vp, _i64, _vp, _i64, _i64, _i64, _i64, _vp, _int, _i64, _int, _vp, _i64, _vp],
}.items():
    getattr(lib, _name).argtypes = _args
    getattr(lib, _name).restype = _int
for _name, _args in {"muon_embedding_grad_workspace": [_i64, _i64, _i64], "muon_rms_norm_grad_workspace": [_i64, _i64],
                     "muon_weight_grad_workspace": [_i64, _i64, _i64, _int]}.items():
    getattr(lib, _name).argtypes = _args
    getattr(lib, _name).restype = _i64



def _load_plain():
    """The extension, built if there is none for this interpreter and torch or it is older than its
    source; None where that fails: every call then takes the path through ctypes, to the same kernels."""
    from . import build as _build
    try:
        name, path = __package__ + "._plain", _build.build_binding()
        loader = importlib.machinery.ExtensionFileLoader(name, path)
        _plain = importlib.util.module_from_spec(importlib.util.spec_from_file_location(name, path, loader=loader))
        loader.exec_module(_plain)
    except Exception as e:  # noqa: BLE001
        warnings.warn(f"the extension of the plain calls is not usable ({e}); calls go through ctypes")
        return None
    _plain.bind(*(ctypes.cast(getattr(lib, "muon_" + n), _vp).value for n in (
        "embedding", "embedding_grad", "embedding_grad_workspace", "rms_norm", "rms_norm_grad", "rms_norm_grad_workspace",
        "checkpoint_store", "checkpoint_restore", "weight_grad", "weight_grad_workspace")))
    return _plain


_fast = _load_plain()

_CODE = {torch.bfloat16: BF16, torch.float32: FP32}
_Q, _S = torch.float8_e4m3fn, torch.float8_e8m0fnu
MX_BLOCK = 32


class ActCheckpoint(NamedTuple):
    """An activation in 8 bits: e4m3 values [..., dim] and e8m0 scales [..., ceil(dim / 32)], each
    scale for 32 consecutive values of a row."""
    q: torch.Tensor
    scales: torch.Tensor


class RmsNorm(NamedTuple):
    y: Optional[torch.Tensor]
    h: Optional[torch.Tensor]
    rstd: torch.Tensor
    checkpoint: Optional[ActCheckpoint]


def _code(dtype, name: str) -> int:
    c = _CODE.get(dtype)
    if c is None:
        raise TypeError(f"{name} must be bf16 or fp32, got {dtype}")
    return c


def _device(t, name: str) -> int:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    return t.get_device()


def _rows(t, name: str, dev: int, shape=None) -> int:
    """Row stride of a tensor [..., dim] on device `dev`, taken as a matrix; checks layout and shape."""
    if _device(t, name) != dev:
        raise ValueError(f"all tensors must be on one device: {name} is on {t.device}, not cuda:{dev}")
    have = t.shape
    if shape is not None and have != shape:
        raise ValueError(f"{name} has shape {tuple(have)}, expected {tuple(shape)}")
    if not have:
        raise ValueError(f"{name} must have at least one dimension")
    return have[-1] if t.is_contiguous() else _row_stride(t, name)


def _row_stride(t, name: str) -> int:
    shape, stride = t.shape, t.stride()
    d = shape[-1]
    if d > 1 and stride[-1] != 1:
        raise ValueError(f"the last dimension of {name} must be contiguous")
    # leading dimensions must collapse into one
    row, span = None, 1
    for n, s in zip(reversed(shape[:-1]), reversed(stride[:-1])):
        if n == 1:
            continue
        if row is None:
            row = s
        elif s != row * span:
            raise ValueError(f"the leading dimensions of {name} must be viewable as one")
        span *= n
    return max(d, 1) if row is None else row


# the current stream's handle without the Stream object that torch.cuda.current_stream makes (2 us)
_stream = torch._C._cuda_getCurrentRawStream


def _elsewhere(dev: int, stream):
    """None when a call may run on the current device's current stream as it is; else the context
    in which it has to."""
    if stream is None:
        return None if dev == torch.cuda.current_device() else torch.cuda.device(dev)
    if not isinstance(stream, torch.cuda.Stream):
        handle = int(getattr(stream, "cuda_stream", stream))
        stream = torch.cuda.default_stream(dev) if handle == 0 else torch.cuda.ExternalStream(handle, device=dev)
    if stream.device_index != dev:
        raise ValueError(f"the stream is on {stream.device}, the tensors on cuda:{dev}")
    return torch.cuda.stream(stream)


def _size(n: int) -> int:
    if n < 0:
        raise MuonError(int(n), last_error())
    return int(n)


@functools.lru_cache(maxsize=256)
def _embedding_grad_bytes(n: int, vocab: int, dim: int) -> int:
    return _size(lib.muon_embedding_grad_workspace(n, vocab, dim))


@functools.lru_cache(maxsize=256)
def _rms_norm_grad_bytes(rows: int, dim: int) -> int:
    return _size(lib.muon_rms_norm_grad_workspace(rows, dim))


@functools.lru_cache(maxsize=256)
def _weight_grad_bytes(rows: int, n: int, k: int, code: int) -> int:
    return _size(lib.muon_weight_grad_workspace(rows, n, k, code))


_BITS = {torch.int64: 64, torch.int32: 32}


def _tokens(tokens) -> int:
    if not tokens.is_contiguous():
        raise ValueError("tokens must be contiguous")
    bits = _BITS.get(tokens.dtype)
    if bits is None:
        raise TypeError(f"tokens must be int32 or int64, got {tokens.dtype}")
    return bits


def embedding(tokens, table, scale: float = 1.0, out=None, out_dtype=None, stream=None):
    """out[..., :] = scale * table[tokens]; tokens int32 or int64 of any shape, table [vocab, dim]
    bf16 or fp32, out in out_dtype (default: the table's). A negative id gives a row of zeros, and
    so does an id past the vocabulary, which check_status() then reports (WARN_TOKEN)."""
    if out is None and stream is None and _fast is not None:
        out = _fast.embedding(tokens, table, scale, out_dtype)
        if out is not None:
            return out
    dev = _device(tokens, "tokens")
    bits = _tokens(tokens)
    ts = _rows(table, "table", dev)
    if table.dim() != 2:
        raise ValueError("table must be a matrix")
    ctx = _elsewhere(dev, stream)
    if ctx is not None:
        with ctx:
            return embedding(tokens, table, scale, out, out_dtype)
    vocab, dim = table.shape
    if out is None:
        out = table.new_empty((*tokens.shape, dim), dtype=out_dtype or table.dtype)
        os_ = dim
    else:
        os_ = _rows(out, "out", dev, (*tokens.shape, dim))
        if out_dtype is not None and out.dtype != out_dtype:
            raise TypeError("out and out_dtype disagree")
    _check(lib.muon_embedding(tokens.data_ptr(), bits, tokens.numel(), table.data_ptr(), _code(table.dtype, "table"), ts,
                              vocab, dim, scale, out.data_ptr(), _code(out.dtype, "out"), os_, _stream(dev)))
    return out


def embedding_grad(tokens, dy, vocab: int, scale: float = 1.0, grad=None, grad_dtype=None, accumulate: bool = False,
                   stream=None):
    """Gradient of embedding() by its table: grad[v] = scale * sum of dy over the places of token v,
    [vocab, dim] in grad_dtype (default: dy's), zeros for absent tokens. With accumulate, added to
    `grad`, of which only the rows of present tokens are touched. The sums are fp32, in an order that
    goes by the tokens' places alone; negative and too large ids contribute nothing."""
    if stream is None and _fast is not None:
        got = _fast.embedding_grad(tokens, dy, vocab, scale, grad, grad_dtype, accumulate)
        if got is not None:
            return got if grad is None else grad
    dev = _device(tokens, "tokens")
    bits = _tokens(tokens)
    ds = _rows(dy, "dy", dev)
    dim = dy.shape[-1]
    if dy.shape[:-1] != tokens.shape:
        raise ValueError(f"dy has shape {tuple(dy.shape)}, expected {(*tokens.shape, dim)}")
    if accumulate and grad is None:
        raise ValueError("accumulate needs grad")
    ctx = _elsewhere(dev, stream)
    if ctx is not None:
        with ctx:
            return embedding_grad(tokens, dy, vocab, scale, grad, grad_dtype, accumulate)
    n = tokens.numel()
    nbytes = _embedding_grad_bytes(n, vocab, dim)
    if grad is None:
        grad = dy.new_empty((vocab, dim), dtype=grad_dtype or dy.dtype)
        gs = dim
    else:
        gs = _rows(grad, "grad", dev, (vocab, dim))
        if grad_dtype is not None and grad.dtype != grad_dtype:
            raise TypeError("grad and grad_dtype disagree")
    ws = dy.new_empty(nbytes, dtype=torch.uint8)
    _check(lib.muon_embedding_grad(tokens.data_ptr(), bits, n, dy.data_ptr(), _code(dy.dtype, "dy"), ds, vocab, dim, scale,
                                   grad.data_ptr(), _code(grad.dtype, "grad"), gs, int(accumulate), ws.data_ptr(), nbytes,
                                   _stream(dev)))
    return grad


def _new_checkpoint(x) -> ActCheckpoint:
    shape = x.shape
    return ActCheckpoint(x.new_empty(shape, dtype=_Q), x.new_empty((*shape[:-1], -(-shape[-1] // MX_BLOCK)), dtype=_S))


def _checkpoint(ck, name: str, shape=None):
    """Device and row strides of a checkpoint's two tensors, checked."""
    if not isinstance(ck, tuple) or len(ck) != 2:
        raise TypeError(f"{name} must be an ActCheckpoint")
    q, s = ck
    dev = _device(q, f"{name}.q")
    qs = _rows(q, f"{name}.q", dev, shape)
    have = q.shape
    ss = _rows(s, f"{name}.scales", dev, (*have[:-1], -(-have[-1] // MX_BLOCK)))
    if q.dtype != _Q or s.dtype != _S:
        raise TypeError(f"{name} must hold float8_e4m3fn values and float8_e8m0fnu scales, got {q.dtype} and {s.dtype}")
    return dev, qs, ss


def _contiguous(t, dtype=None):
    """An uninitialised contiguous tensor of t's shape."""
    if (dtype is None or dtype == t.dtype) and t.is_contiguous():
        return torch.empty_like(t)
    return t.new_empty(t.shape, dtype=dtype or t.dtype)


def rms_norm(x, weight, residual=None, eps: float = 1e-5, output: bool = True, checkpoint: bool = False, h=None, y=None,
             stream=None) -> RmsNorm:
    """h = x + residual (in the residual's type; x itself without one), y = h / rms(h) * weight in
    x's type, rstd = 1 / rms(h) per row (fp32), and with checkpoint=True an ActCheckpoint of y.
    output=False leaves y out (y None). `h` and `y` may be given as buffers: h may be the residual
    or, in its type, x; y may be x, and where there is no residual no h is left then (h None)."""
    if h is None and y is None and stream is None and _fast is not None:
        got = _fast.rms_norm(x, weight, residual, eps, output, checkpoint)
        if got is not None:
            y, h, rstd, q, s = got
            return RmsNorm(y, x if h is None else h, rstd, None if q is None else ActCheckpoint(q, s))
    dev = _device(x, "x")
    xs = _rows(x, "x", dev)
    shape = x.shape
    dim = shape[-1]
    _rows(weight, "weight", dev, shape[-1:])
    if not weight.is_contiguous():
        raise ValueError("weight must be contiguous")
    if not output and (not checkpoint or y is not None):
        raise ValueError("output=False needs checkpoint=True and no y")
    rs = hs = ys = ss = rc = 0
    if residual is not None:
        rs = _rows(residual, "residual", dev, shape)
        rc = _code(residual.dtype, "residual")
        if h is not None:
            hs = _rows(h, "h", dev, shape)
            if h.dtype != residual.dtype:
                raise TypeError("h must have the residual's type")
    elif h is not None:
        raise ValueError("h is written only where there is a residual")
    if y is not None:
        ys = _rows(y, "y", dev, shape)
        if y.dtype != x.dtype:
            raise TypeError("y must have x's type")
    ctx = _elsewhere(dev, stream)
    if ctx is not None:
        with ctx:
            return rms_norm(x, weight, residual, eps, output, checkpoint, h, y)
    xc, wc = _code(x.dtype, "x"), _code(weight.dtype, "weight")
    rp = hp = yp = qp = sp = None
    if residual is not None:
        rp = residual.data_ptr()
        if h is None:
            h, hs = _contiguous(residual), dim
        hp = h.data_ptr()
    if output:
        if y is None:
            y, ys = _contiguous(x), dim
        yp = y.data_ptr()
    rstd = x.new_empty(shape[:-1], dtype=torch.float32)
    ck = None
    if checkpoint:
        ck = _new_checkpoint(x)
        qp, sp, ss = ck[0].data_ptr(), ck[1].data_ptr(), -(-dim // MX_BLOCK)
    _check(lib.muon_rms_norm(x.data_ptr(), xc, xs, rp, rc, rs, weight.data_ptr(), wc, x.numel() // dim if dim else 0, dim, eps,
                             hp, hs, yp, ys, qp, dim, sp, ss, rstd.data_ptr(), _stream(dev)))
    if residual is None and (y is None or y.data_ptr() != x.data_ptr() or not x.numel()):
        h = x
    return RmsNorm(y, h, rstd, ck)


def rms_norm_grad(dy, h, weight, rstd, dh=None, dx=None, dweight=None, accumulate: bool = False, stream=None):
    """Gradient of rms_norm by h (and so by x and by the residual) and by weight, from what it
    returned: (dx, dweight), dx in h's type and dweight fp32. dh, in h's type, is the gradient that
    reaches h from elsewhere and is added to dx. With accumulate, dweight is added to the given
    `dweight`. dx may be one of dy, h and dh where the types agree."""
    if dx is None and dweight is None and not accumulate and stream is None and _fast is not None:
        got = _fast.rms_norm_grad(dy, h, weight, rstd, dh)
        if got is not None:
            return got
    dev = _device(h, "h")
    hs = _rows(h, "h", dev)
    shape = h.shape
    dim = shape[-1]
    ds = _rows(dy, "dy", dev, shape)
    _rows(weight, "weight", dev, shape[-1:])
    if _device(rstd, "rstd") != dev or rstd.shape != shape[:-1] or rstd.dtype != torch.float32 or not rstd.is_contiguous():
        raise ValueError("rstd must be the contiguous fp32 tensor that rms_norm returned")
    if not weight.is_contiguous():
        raise ValueError("weight must be contiguous")
    gs = xs = 0
    gp = None
    if dh is not None:
        gs, gp = _rows(dh, "dh", dev, shape), dh.data_ptr()
        if dh.dtype != h.dtype:
            raise TypeError("dh must have h's type")
    if dx is not None:
        xs = _rows(dx, "dx", dev, shape)
        if dx.dtype != h.dtype:
            raise TypeError("dx must have h's type")
    if dweight is not None:
        _rows(dweight, "dweight", dev, shape[-1:])
        if dweight.dtype != torch.float32 or not dweight.is_contiguous():
            raise TypeError("dweight must be fp32 and contiguous")
    elif accumulate:
        raise ValueError("accumulate needs dweight")
    ctx = _elsewhere(dev, stream)
    if ctx is not None:
        with ctx:
            return rms_norm_grad(dy, h, weight, rstd, dh, dx, dweight, accumulate)
    rows = h.numel() // dim if dim else 0
    nbytes = _rms_norm_grad_bytes(rows, dim)
    if dx is None:
        dx, xs = _contiguous(h), dim
    if dweight is None:
        dweight = h.new_empty(dim, dtype=torch.float32)
    ws = h.new_empty(nbytes, dtype=torch.uint8)
    _check(lib.muon_rms_norm_grad(dy.data_ptr(), _code(dy.dtype, "dy"), ds, h.data_ptr(), _code(h.dtype, "h"), hs,
                                  weight.data_ptr(), _code(weight.dtype, "weight"), rstd.data_ptr(), gp, gs, rows, dim,
                                  dx.data_ptr(), xs, dweight.data_ptr(), int(accumulate), ws.data_ptr(), nbytes,
                                  _stream(dev)))
    return dx, dweight


def checkpoint_store(x, out: Optional[ActCheckpoint] = None, stream=None) -> ActCheckpoint:
    """x [..., dim] (bf16 or fp32) in 8 bits: e4m3 values in blocks of 32 along a row, each under the
    smallest power of two that keeps its largest value within e4m3's range. A block with an
    infinity or a NaN becomes NaN."""
    if out is None and stream is None and _fast is not None:
        got = _fast.checkpoint_store(x)
        if got is not None:
            return ActCheckpoint(*got)
    dev = _device(x, "x")
    xs = _rows(x, "x", dev)
    dim = x.shape[-1]
    qs, ss = dim, -(-dim // MX_BLOCK)
    if out is not None:
        where, qs, ss = _checkpoint(out, "out", x.shape)
        if where != dev:
            raise ValueError("x and out must be on one device")
    ctx = _elsewhere(dev, stream)
    if ctx is not None:
        with ctx:
            return checkpoint_store(x, out)
    if out is None:
        out = _new_checkpoint(x)
    _check(lib.muon_checkpoint_store(x.data_ptr(), _code(x.dtype, "x"), xs, x.numel() // dim if dim else 0, dim,
                                     out[0].data_ptr(), qs, out[1].data_ptr(), ss, _stream(dev)))
    return out


def checkpoint_restore(checkpoint: ActCheckpoint, dtype=torch.bfloat16, out=None, stream=None):
    """The values of a checkpoint, in bf16 (exact for what checkpoint_store and rms_norm make) or fp32."""
    if out is None and stream is None and _fast is not None and type(checkpoint) is ActCheckpoint:
        x = _fast.checkpoint_restore(checkpoint[0], checkpoint[1], dtype)
        if x is not None:
            return x
    dev, qs, ss = _checkpoint(checkpoint, "checkpoint")
    q, s = checkpoint
    dim = xs = q.shape[-1]
    if out is not None:
        xs = _rows(out, "out", dev, q.shape)
    ctx = _elsewhere(dev, stream)
    if ctx is not None:
        with ctx:
            return checkpoint_restore(checkpoint, dtype, out)
    if out is None:
        _code(dtype, "dtype")
        out = q.new_empty(q.shape, dtype=dtype)
    _check(lib.muon_checkpoint_restore(q.data_ptr(), qs, s.data_ptr(), ss, q.numel() // dim if dim else 0, dim,
                                       out.data_ptr(), _code(out.dtype, "out"), xs, _stream(dev)))
    return out


def weight_grad(dy, checkpoint: ActCheckpoint, grad=None, grad_dtype=None, accumulate: bool = False, stream=None):
    """Gradient of y = x @ W.T by W, from dy [..., n] (bf16 or fp32) and the checkpoint of x [..., k]:
    grad[n, k] = sum over the rows of dy^T x, in grad_dtype (default: dy's), summed in fp32. With
    accumulate, added to `grad`. It is what muon_step takes as a gradient."""
    if stream is None and _fast is not None and type(checkpoint) is ActCheckpoint:
        got = _fast.weight_grad(dy, checkpoint[0], checkpoint[1], grad, grad_dtype, accumulate)
        if got is not None:
            return got if grad is None else grad
    dev, qs, ss = _checkpoint(checkpoint, "checkpoint")
    q, s = checkpoint
    ds = _rows(dy, "dy", dev)
    n, k = dy.shape[-1], q.shape[-1]
    if dy.shape[:-1] != q.shape[:-1]:
        raise ValueError(f"dy has shape {tuple(dy.shape)}, expected {(*q.shape[:-1], n)}")
    if accumulate and grad is None:
        raise ValueError("accumulate needs grad")
    ctx = _elsewhere(dev, stream)
    if ctx is not None:
        with ctx:
            return weight_grad(dy, checkpoint, grad, grad_dtype, accumulate)
    rows, code = dy.numel() // n if n else 0, _code(dy.dtype, "dy")
    nbytes = _weight_grad_bytes(rows, n, k, code)
    if grad is None:
        grad = dy.new_empty((n, k), dtype=grad_dtype or dy.dtype)
        gs = k
    else:
        gs = _rows(grad, "grad", dev, (n, k))
        if grad_dtype is not None and grad.dtype != grad_dtype:
            raise TypeError("grad and grad_dtype disagree")
    ws = dy.new_empty(nbytes, dtype=torch.uint8)
    _check(lib.muon_weight_grad(dy.data_ptr(), code, ds, q.data_ptr(), qs, s.data_ptr(), ss, rows, n, k, grad.data_ptr(),
                                _code(grad.dtype, "grad"), gs, int(accumulate), ws.data_ptr(), nbytes, _stream(dev)))
    return grad
