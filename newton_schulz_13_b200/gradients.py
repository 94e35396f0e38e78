"""The operators that make the gradients which muon_step and adamw_step take: the token embedding,
the root-mean-square norm, and 8-bit activation checkpoints with the weight gradient taken from them.

    y = ns.embedding(tokens, table, scale=s)                      # forward
    y, h, rstd, ck = ns.rms_norm(x, w, residual=r, checkpoint=True)
    dW = ns.weight_grad(dY, ck)                                   # muon_step's gradient of y @ W.T
    dx, dw = ns.rms_norm_grad(dy, h, w, rstd, dh=dh)              # adamw_step's gradient of a norm scale
    dE = ns.embedding_grad(tokens, dx, vocab, scale=s)            # adamw_step's gradient of the table

Argument marshalling only, as in the rest of the package; include/muon.h has the formulas. Inputs
are CUDA tensors whose last dimension is contiguous (rows may be strided); leading dimensions are
taken as rows. Outputs and workspaces come from torch's allocator on the stream the call runs on
(`stream`, or the current stream of the tensors' device), so calls on several streams, and calls
captured into several graphs, share nothing.
"""
from __future__ import annotations

import ctypes
import functools
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
    h: torch.Tensor
    rstd: torch.Tensor
    checkpoint: Optional[ActCheckpoint]


def _code(dtype, name: str) -> int:
    c = _CODE.get(dtype)
    if c is None:
        raise TypeError(f"{name} must be bf16 or fp32, got {dtype}")
    return c


def _rows(t, name: str, dim: Optional[int] = None, lead=None) -> int:
    """Row stride of a tensor [..., dim] taken as a matrix; checks its layout and shape."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    shape, stride = t.shape, t.stride()
    nd = len(shape)
    if nd == 0 or (dim is not None and shape[-1] != dim) or (lead is not None and shape[:-1] != lead):
        raise ValueError(f"{name} has shape {tuple(shape)}, expected {(*lead, dim) if lead is not None else ('...', dim)}")
    d = shape[-1]
    if d > 1 and stride[-1] != 1:
        raise ValueError(f"the last dimension of {name} must be contiguous")
    if nd == 2:
        return stride[0] if shape[0] > 1 else max(d, 1)
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


def _same_device(dev, *tensors) -> None:
    for t in tensors:
        if t is not None and t.device != dev:
            raise ValueError(f"all tensors must be on one device: got {dev} and {t.device}")


def _elsewhere(dev, stream):
    """None when a call may run on the current device's current stream as it is; else the context
    in which it has to."""
    if stream is not None:
        if not isinstance(stream, torch.cuda.Stream):
            handle = int(getattr(stream, "cuda_stream", stream))
            stream = torch.cuda.default_stream(dev) if handle == 0 else torch.cuda.ExternalStream(handle, device=dev)
        if stream.device != dev:
            raise ValueError(f"the stream is on {stream.device}, the tensors on {dev}")
        return torch.cuda.stream(stream)
    return torch.cuda.device(dev) if dev.index != torch.cuda.current_device() else None


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


def _tokens(tokens) -> int:
    if not isinstance(tokens, torch.Tensor) or not tokens.is_cuda:
        raise ValueError("tokens must be a CUDA tensor")
    if not tokens.is_contiguous():
        raise ValueError("tokens must be contiguous")
    if tokens.dtype == torch.int64:
        return 64
    if tokens.dtype == torch.int32:
        return 32
    raise TypeError(f"tokens must be int32 or int64, got {tokens.dtype}")


def embedding(tokens, table, scale: float = 1.0, out=None, out_dtype=None, stream=None):
    """out[..., :] = scale * table[tokens]; tokens int32 or int64 of any shape, table [vocab, dim]
    bf16 or fp32, out in out_dtype (default: the table's). A negative id gives a row of zeros, and
    so does an id past the vocabulary, which check_status() then reports (WARN_TOKEN)."""
    bits = _tokens(tokens)
    if table.dim() != 2:
        raise ValueError("table must be a matrix")
    ts = _rows(table, "table")
    dev = tokens.device
    _same_device(dev, table, out)
    ctx = _elsewhere(dev, stream)
    if ctx is not None:
        with ctx:
            return embedding(tokens, table, scale, out, out_dtype)
    vocab, dim = table.shape
    if out is None:
        out = torch.empty((*tokens.shape, dim), dtype=out_dtype or table.dtype, device=dev)
    elif out_dtype is not None and out.dtype != out_dtype:
        raise TypeError("out and out_dtype disagree")
    os_ = _rows(out, "out", dim, tokens.shape)
    _check(lib.muon_embedding(tokens.data_ptr(), bits, tokens.numel(), table.data_ptr(), _code(table.dtype, "table"), ts,
                              vocab, dim, scale, out.data_ptr(), _code(out.dtype, "out"), os_,
                              torch.cuda.current_stream(dev).cuda_stream))
    return out


def embedding_grad(tokens, dy, vocab: int, scale: float = 1.0, grad=None, grad_dtype=None, accumulate: bool = False,
                   stream=None):
    """Gradient of embedding() by its table: grad[v] = scale * sum of dy over the places of token v,
    [vocab, dim] in grad_dtype (default: dy's), zeros for absent tokens. With accumulate, added to
    `grad`, of which only the rows of present tokens are touched. The sums are fp32, in the order of
    the tokens; negative and too large ids contribute nothing."""
    bits = _tokens(tokens)
    ds = _rows(dy, "dy", None, tokens.shape)
    dev, dim = tokens.device, dy.shape[-1]
    _same_device(dev, dy, grad)
    if accumulate and grad is None:
        raise ValueError("accumulate needs grad")
    ctx = _elsewhere(dev, stream)
    if ctx is not None:
        with ctx:
            return embedding_grad(tokens, dy, vocab, scale, grad, grad_dtype, accumulate)
    n = tokens.numel()
    nbytes = _embedding_grad_bytes(n, vocab, dim)
    if grad is None:
        grad = torch.empty((vocab, dim), dtype=grad_dtype or dy.dtype, device=dev)
    elif grad_dtype is not None and grad.dtype != grad_dtype:
        raise TypeError("grad and grad_dtype disagree")
    gs = _rows(grad, "grad", dim, (vocab,))
    ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    _check(lib.muon_embedding_grad(tokens.data_ptr(), bits, n, dy.data_ptr(), _code(dy.dtype, "dy"), ds, vocab, dim, scale,
                                   grad.data_ptr(), _code(grad.dtype, "grad"), gs, int(accumulate), ws.data_ptr(), nbytes,
                                   torch.cuda.current_stream(dev).cuda_stream))
    return grad


def _new_checkpoint(lead, dim: int, dev) -> ActCheckpoint:
    return ActCheckpoint(torch.empty((*lead, dim), dtype=_Q, device=dev),
                         torch.empty((*lead, -(-dim // MX_BLOCK)), dtype=_S, device=dev))


def _checkpoint(ck, name: str, dim: Optional[int] = None, lead=None):
    """Row strides of a checkpoint's two tensors, checked."""
    if not isinstance(ck, tuple) or len(ck) != 2:
        raise TypeError(f"{name} must be an ActCheckpoint")
    q, s = ck
    qs = _rows(q, f"{name}.q", dim, lead)
    ss = _rows(s, f"{name}.scales", -(-q.shape[-1] // MX_BLOCK), q.shape[:-1])
    if q.dtype != _Q or s.dtype != _S:
        raise TypeError(f"{name} must hold float8_e4m3fn values and float8_e8m0fnu scales, got {q.dtype} and {s.dtype}")
    return qs, ss


def rms_norm(x, weight, residual=None, eps: float = 1e-5, output: bool = True, checkpoint: bool = False, h=None, y=None,
             stream=None) -> RmsNorm:
    """h = x + residual (in the residual's type; x itself without one), y = h / rms(h) * weight in
    x's type, rstd = 1 / rms(h) per row (fp32), and with checkpoint=True an ActCheckpoint of y.
    output=False leaves y out (y None). `h` and `y` may be given as buffers: h may be the residual,
    y may be x."""
    xs = _rows(x, "x")
    lead, dim, dev = x.shape[:-1], x.shape[-1], x.device
    _same_device(dev, weight, residual, h, y)
    _rows(weight, "weight", dim, ())
    if not output and (not checkpoint or y is not None):
        raise ValueError("output=False needs checkpoint=True and no y")
    rs = 0
    if residual is not None:
        rs = _rows(residual, "residual", dim, lead)
    elif h is not None:
        raise ValueError("h is written only where there is a residual")
    ctx = _elsewhere(dev, stream)
    if ctx is not None:
        with ctx:
            return rms_norm(x, weight, residual, eps, output, checkpoint, h, y)
    rows = x.numel() // dim if dim else 0
    hs = ys = qs = ss = 0
    rc = 0
    if residual is not None:
        rc = _code(residual.dtype, "residual")
        if h is None:
            h = torch.empty((*lead, dim), dtype=residual.dtype, device=dev)
        elif h.dtype != residual.dtype:
            raise TypeError("h must have the residual's type")
        hs = _rows(h, "h", dim, lead)
    if output:
        if y is None:
            y = torch.empty((*lead, dim), dtype=x.dtype, device=dev)
        elif y.dtype != x.dtype:
            raise TypeError("y must have x's type")
        ys = _rows(y, "y", dim, lead)
    rstd = torch.empty(lead, dtype=torch.float32, device=dev)
    ck = None
    if checkpoint:
        ck = _new_checkpoint(lead, dim, dev)
        qs, ss = _rows(ck.q, "q"), _rows(ck.scales, "scales")
    _check(lib.muon_rms_norm(x.data_ptr(), _code(x.dtype, "x"), xs, None if residual is None else residual.data_ptr(), rc, rs,
                             weight.data_ptr(), _code(weight.dtype, "weight"), rows, dim, eps,
                             None if h is None else h.data_ptr(), hs, None if y is None else y.data_ptr(), ys,
                             None if ck is None else ck.q.data_ptr(), qs, None if ck is None else ck.scales.data_ptr(), ss,
                             rstd.data_ptr(), torch.cuda.current_stream(dev).cuda_stream))
    return RmsNorm(y, x if h is None else h, rstd, ck)


def rms_norm_grad(dy, h, weight, rstd, dh=None, dx=None, dweight=None, accumulate: bool = False, stream=None):
    """Gradient of rms_norm by h (and so by x and by the residual) and by weight, from what it
    returned: (dx, dweight), dx in h's type and dweight fp32. dh, in h's type, is the gradient that
    reaches h from elsewhere and is added to dx. With accumulate, dweight is added to the given
    `dweight`. dx may be one of dy, h and dh where the types agree."""
    hs = _rows(h, "h")
    lead, dim, dev = h.shape[:-1], h.shape[-1], h.device
    ds = _rows(dy, "dy", dim, lead)
    _rows(weight, "weight", dim, ())
    _same_device(dev, dy, weight, rstd, dh, dx, dweight)
    if not rstd.is_cuda or rstd.shape != lead or rstd.dtype != torch.float32 or not rstd.is_contiguous():
        raise ValueError("rstd must be the contiguous fp32 CUDA tensor that rms_norm returned")
    gs = 0
    if dh is not None:
        gs = _rows(dh, "dh", dim, lead)
        if dh.dtype != h.dtype:
            raise TypeError("dh must have h's type")
    if accumulate and dweight is None:
        raise ValueError("accumulate needs dweight")
    ctx = _elsewhere(dev, stream)
    if ctx is not None:
        with ctx:
            return rms_norm_grad(dy, h, weight, rstd, dh, dx, dweight, accumulate)
    rows = h.numel() // dim if dim else 0
    nbytes = _rms_norm_grad_bytes(rows, dim)
    if dx is None:
        dx = torch.empty((*lead, dim), dtype=h.dtype, device=dev)
    elif dx.dtype != h.dtype:
        raise TypeError("dx must have h's type")
    xs = _rows(dx, "dx", dim, lead)
    if dweight is None:
        dweight = torch.empty(dim, dtype=torch.float32, device=dev)
    elif dweight.dtype != torch.float32:
        raise TypeError("dweight must be fp32")
    _rows(dweight, "dweight", dim, ())
    ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    _check(lib.muon_rms_norm_grad(dy.data_ptr(), _code(dy.dtype, "dy"), ds, h.data_ptr(), _code(h.dtype, "h"), hs,
                                  weight.data_ptr(), _code(weight.dtype, "weight"), rstd.data_ptr(),
                                  None if dh is None else dh.data_ptr(), gs, rows, dim, dx.data_ptr(), xs,
                                  dweight.data_ptr(), int(accumulate), ws.data_ptr(), nbytes,
                                  torch.cuda.current_stream(dev).cuda_stream))
    return dx, dweight


def checkpoint_store(x, out: Optional[ActCheckpoint] = None, stream=None) -> ActCheckpoint:
    """x [..., dim] (bf16 or fp32) in 8 bits: e4m3 values in blocks of 32 along a row, each under the
    smallest power of two that keeps its largest value within e4m3's range. A block with an
    infinity or a NaN becomes NaN."""
    xs = _rows(x, "x")
    lead, dim, dev = x.shape[:-1], x.shape[-1], x.device
    if out is not None:
        _checkpoint(out, "out", dim, lead)
        _same_device(dev, *out)
    ctx = _elsewhere(dev, stream)
    if ctx is not None:
        with ctx:
            return checkpoint_store(x, out)
    if out is None:
        out = _new_checkpoint(lead, dim, dev)
    qs, ss = _checkpoint(out, "out")
    _check(lib.muon_checkpoint_store(x.data_ptr(), _code(x.dtype, "x"), xs, x.numel() // dim if dim else 0, dim,
                                     out[0].data_ptr(), qs, out[1].data_ptr(), ss,
                                     torch.cuda.current_stream(dev).cuda_stream))
    return out


def checkpoint_restore(checkpoint: ActCheckpoint, dtype=torch.bfloat16, out=None, stream=None):
    """The values of a checkpoint, in bf16 (exact for what checkpoint_store and rms_norm make) or fp32."""
    qs, ss = _checkpoint(checkpoint, "checkpoint")
    q, s = checkpoint
    lead, dim, dev = q.shape[:-1], q.shape[-1], q.device
    _same_device(dev, s, out)
    ctx = _elsewhere(dev, stream)
    if ctx is not None:
        with ctx:
            return checkpoint_restore(checkpoint, dtype, out)
    if out is None:
        out = torch.empty((*lead, dim), dtype=dtype, device=dev)
    xs = _rows(out, "out", dim, lead)
    _check(lib.muon_checkpoint_restore(q.data_ptr(), qs, s.data_ptr(), ss, q.numel() // dim if dim else 0, dim,
                                       out.data_ptr(), _code(out.dtype, "out"), xs,
                                       torch.cuda.current_stream(dev).cuda_stream))
    return out


def weight_grad(dy, checkpoint: ActCheckpoint, grad=None, grad_dtype=None, accumulate: bool = False, stream=None):
    """Gradient of y = x @ W.T by W, from dy [..., n] (bf16 or fp32) and the checkpoint of x [..., k]:
    grad[n, k] = sum over the rows of dy^T x, in grad_dtype (default: dy's), summed in fp32. With
    accumulate, added to `grad`. It is what muon_step takes as a gradient."""
    qs, ss = _checkpoint(checkpoint, "checkpoint")
    q, s = checkpoint
    ds = _rows(dy, "dy", None, q.shape[:-1])
    n, k, dev = dy.shape[-1], q.shape[-1], dy.device
    _same_device(dev, q, s, grad)
    if accumulate and grad is None:
        raise ValueError("accumulate needs grad")
    ctx = _elsewhere(dev, stream)
    if ctx is not None:
        with ctx:
            return weight_grad(dy, checkpoint, grad, grad_dtype, accumulate)
    rows, code = dy.numel() // n if n else 0, _code(dy.dtype, "dy")
    nbytes = _weight_grad_bytes(rows, n, k, code)
    if grad is None:
        grad = torch.empty((n, k), dtype=grad_dtype or dy.dtype, device=dev)
    elif grad_dtype is not None and grad.dtype != grad_dtype:
        raise TypeError("grad and grad_dtype disagree")
    gs = _rows(grad, "grad", k, (n,))
    ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    _check(lib.muon_weight_grad(dy.data_ptr(), code, ds, q.data_ptr(), qs, s.data_ptr(), ss, rows, n, k, grad.data_ptr(),
                                _code(grad.dtype, "grad"), gs, int(accumulate), ws.data_ptr(), nbytes,
                                torch.cuda.current_stream(dev).cuda_stream))
    return grad
