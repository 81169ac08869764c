"""Layer operators of one rank: embedding lookup, layer norm, 8-bit
activations, and their gradients (the per-rank ends of a training step whose
weight gradients the collectives reduce).

Same two layers as the collectives: ``vcoll_*`` take integer device pointers
and return the status code, the functions without the prefix take CUDA (or
pinned host) tensors of fp32 or bf16 and raise ``VcollError``.  The formulas
and the conventions of every call are in ``include/vcoll.h``.

The last axis of a tensor is a row's columns and must be adjacent; the axes
before it are its rows, which may be parts of wider rows (a column slice of a
matrix is taken as it is, without a copy).  Outputs, and the workspaces that a
call takes when it is given none, are allocated on the stream that the call
runs on.

As with the collectives, autograd does not see these calls: a tensor that
requires grad is taken for its values, what comes back has no history, and an
in-place output's version is not counted up.  The gradients are the ``*_backward``
functions' to compute.
"""
from __future__ import annotations

import ctypes
import functools
from typing import NamedTuple

import torch

from . import BF16, ERR_INVALID_ARG, ERR_INVALID_TYPE, F32, VcollError, _check, lib

I32, I64 = 0, 1
CHECKPOINT8_BLOCK = 128

_P, _I, _L, _F, _Z = (ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float,
                      ctypes.c_size_t)
_ARGS = {
    "vcoll_embedding": [_P, _I, _L, _P, _L, _L, _L, _F, _P, _L, _I, _P],
    "vcoll_embedding_backward": [_P, _L, _I, _P, _I, _L, _L, _L, _F, _P, _L, _P, _L, _I, _P, _Z,
                                 _P],
    "vcoll_layer_norm": [_P, _L, _P, _P, _I, _L, _L, _F, _P, _L, _P, _P, _I, _P],
    "vcoll_layer_norm_backward": [_P, _L, _P, _L, _P, _P, _P, _I, _L, _L, _P, _L, _P, _P, _I, _P,
                                  _Z, _P],
    "vcoll_checkpoint8": [_P, _L, _L, _L, _P, _L, _P, _I, _P],
    "vcoll_checkpoint8_restore": [_P, _L, _P, _P, _P, _I, _L, _L, _P, _L, _I, _P],
    "vcoll_layer_norm_checkpoint8": [_P, _L, _P, _P, _I, _L, _L, _F, _P, _L, _P, _P, _L, _P, _I,
                                     _P],
    "vcoll_layer_norm_backward_checkpoint8": [_P, _L, _P, _L, _P, _P, _P, _I, _L, _L, _P, _L, _P,
                                              _P, _I, _P, _Z, _P],
    "vcoll_embedding_backward_workspace_bytes": [_L, _L, _L],
    "vcoll_layer_norm_workspace_bytes": [_L, _L],
}
_fns = {}


def _fn(name):
    f = _fns.get(name)
    if f is None:
        f = getattr(lib(), name)
        f.argtypes = _ARGS[name]
        f.restype = _Z if name.endswith("_bytes") else _I
        _fns[name] = f
    return f


# ----------------------------------------------------------- raw C ABI layer

def vcoll_embedding(tokens, index_type, N, table, table_ld, V, D, scale, out, out_ld, dtype,
                    stream=0) -> int:
    return _fn("vcoll_embedding")(tokens, index_type, N, table, table_ld, V, D, scale, out, out_ld,
                                  dtype, stream)


def vcoll_embedding_backward_workspace_bytes(N, V, D) -> int:
    return _fn("vcoll_embedding_backward_workspace_bytes")(N, V, D)


def vcoll_embedding_backward(grad, grad_ld, dtype, tokens, index_type, N, V, D, scale, base,
                             base_ld, table_grad, table_ld, table_dtype, workspace=0,
                             workspace_bytes=0, stream=0) -> int:
    return _fn("vcoll_embedding_backward")(grad, grad_ld, dtype, tokens, index_type, N, V, D,
                                           scale, base, base_ld, table_grad, table_ld, table_dtype,
                                           workspace, workspace_bytes, stream)


def vcoll_layer_norm(x, x_ld, weight, bias, weight_dtype, N, D, eps, y, y_ld, mean, rstd, dtype,
                     stream=0) -> int:
    return _fn("vcoll_layer_norm")(x, x_ld, weight, bias, weight_dtype, N, D, eps, y, y_ld, mean,
                                   rstd, dtype, stream)


def vcoll_layer_norm_workspace_bytes(N, D) -> int:
    return _fn("vcoll_layer_norm_workspace_bytes")(N, D)


def vcoll_layer_norm_backward(grad, grad_ld, x, x_ld, mean, rstd, weight, weight_dtype, N, D, dx,
                              dx_ld, dweight, dbias, dtype, workspace=0, workspace_bytes=0,
                              stream=0) -> int:
    return _fn("vcoll_layer_norm_backward")(grad, grad_ld, x, x_ld, mean, rstd, weight,
                                            weight_dtype, N, D, dx, dx_ld, dweight, dbias, dtype,
                                            workspace, workspace_bytes, stream)


def vcoll_checkpoint8(x, x_ld, N, D, codes, codes_ld, scales, dtype, stream=0) -> int:
    return _fn("vcoll_checkpoint8")(x, x_ld, N, D, codes, codes_ld, scales, dtype, stream)


def vcoll_checkpoint8_restore(codes, codes_ld, scales, weight, bias, weight_dtype, N, D, out,
                              out_ld, dtype, stream=0) -> int:
    return _fn("vcoll_checkpoint8_restore")(codes, codes_ld, scales, weight, bias, weight_dtype, N,
                                            D, out, out_ld, dtype, stream)


def vcoll_layer_norm_checkpoint8(x, x_ld, weight, bias, weight_dtype, N, D, eps, y, y_ld, rstd,
                                 codes, codes_ld, scales, dtype, stream=0) -> int:
    return _fn("vcoll_layer_norm_checkpoint8")(x, x_ld, weight, bias, weight_dtype, N, D, eps, y,
                                               y_ld, rstd, codes, codes_ld, scales, dtype, stream)


def vcoll_layer_norm_backward_checkpoint8(grad, grad_ld, codes, codes_ld, scales, rstd, weight,
                                          weight_dtype, N, D, dx, dx_ld, dweight, dbias, dtype,
                                          workspace=0, workspace_bytes=0, stream=0) -> int:
    return _fn("vcoll_layer_norm_backward_checkpoint8")(grad, grad_ld, codes, codes_ld, scales,
                                                        rstd, weight, weight_dtype, N, D, dx,
                                                        dx_ld, dweight, dbias, dtype, workspace,
                                                        workspace_bytes, stream)


# -------------------------------------------------------------- tensor layer
# A call on a few rows takes the GPU a few microseconds, so these functions
# keep the host's work short: the raw handle of the current stream, checks of
# the common case first, and one pass over each argument.

_TYPES = {torch.float32: F32, torch.bfloat16: BF16}
_INDEX = {torch.int32: I32, torch.int64: I64}
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
# torch.empty without the dispatcher: after a launch it takes the host 1.5 us
# where torch.empty takes 5.7 (a GB300's Grace CPU).  It is torch's own and may
# change, so it is tried once before it is used (_sound), and torch.empty takes
# its place where it is absent or does something else, and while a dispatch mode
# is on, which has to see what is allocated.
_new_cuda = getattr(getattr(getattr(torch._C, "_dynamo", None), "guards", None),
                    "_empty_strided_cuda", None)
_modes = getattr(torch._C, "_len_torch_dispatch_stack", None)
_tried = False


def _sound(new):
    """Whether new(shape, strides, dtype) allocates what _empty needs."""
    try:
        t = new((2, 3), (3, 1), torch.bfloat16)
        return (type(t) is torch.Tensor and t.shape == (2, 3) and t.stride() == (3, 1) and
                t.dtype == torch.bfloat16 and t.is_cuda and
                t.get_device() == torch.cuda.current_device() and not t.requires_grad)
    except Exception:
        return False


def _refuse(message, status=ERR_INVALID_ARG):
    raise VcollError(status, message)


def _handle(stream, device):
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is not None:
        return _raw_stream(device)
    return torch.cuda.current_stream().cuda_stream


def _strides(shape):
    strides, step = [], 1
    for size in reversed(shape):
        strides.append(step)
        step *= size if size > 1 else 1
    return tuple(reversed(strides))


def _empty(shape, dtype, stream):
    """A contiguous tensor allocated on the stream that the call runs on."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return torch.empty(shape, dtype=dtype, device="cuda")
    global _new_cuda, _tried
    if not _tried:
        _tried = True
        if _modes is None or (_new_cuda is not None and not _sound(_new_cuda)):
            _new_cuda = None
    if _new_cuda is None or _modes():
        return torch.empty(shape, dtype=dtype, device="cuda")
    shape = tuple(shape)
    n = len(shape)
    return _new_cuda(shape, (1,) if n == 1 else (shape[1], 1) if n == 2 and shape[1] else
                     _strides(shape), dtype)


@functools.lru_cache(maxsize=256)
def _embedding_need(N, vocab, D):
    return _fn("vcoll_embedding_backward_workspace_bytes")(N, vocab, D)


@functools.lru_cache(maxsize=256)
def _norm_need(N, D):
    return _fn("vcoll_layer_norm_workspace_bytes")(N, D)


def _dtype(t, what):
    code = _TYPES.get(t.dtype)
    if code is None:
        _refuse(f"{what}: unsupported dtype {t.dtype}", ERR_INVALID_TYPE)
    return code


def _place(t, what, device):
    """Refuses a tensor that the kernels of the current device cannot reach."""
    if t.is_cuda:
        _refuse(f"{what} is on device {t.get_device()}, the current device is {device}")
    if not t.is_pinned():
        _refuse(f"{what} is neither a CUDA tensor nor pinned host memory")


def _rows(t, what, device, width=None, rows=None):
    """(rows, columns, row stride in elements) of a tensor taken as a matrix."""
    if t.get_device() != device:
        _place(t, what, device)
    shape = t.shape
    if not shape:
        _refuse(f"{what} has no axes")
    d = shape[-1]
    if t.is_contiguous():
        n = shape[0] if len(shape) == 2 else shape[:-1].numel()
        ld = d
    else:
        try:
            m = t.view(-1, d) if d else t
        except RuntimeError:
            m = None
        if m is None or (d > 1 and m.stride(1) != 1) or (m.shape[0] > 1 and m.stride(0) < d):
            _refuse(f"{what} is not a matrix of rows with adjacent columns (not contiguous)")
        n = m.shape[0]
        ld = m.stride(0) if n > 1 else d
    if width is not None and d != width:
        _refuse(f"{what} has {d} columns, {width} are expected")
    if rows is not None and n != rows:
        _refuse(f"{what} has {n} rows, {rows} are expected")
    return n, d, ld


def _vector(t, what, device, length, dtype):
    if t.get_device() != device:
        _place(t, what, device)
    if t.numel() != length or not t.is_contiguous():
        _refuse(f"{what} is not a contiguous tensor of {length} elements")
    if t.dtype != dtype:
        _refuse(f"{what} is {t.dtype}, {dtype} is expected", ERR_INVALID_TYPE)
    return t.data_ptr()


def _tokens(tokens, device):
    code = _INDEX.get(tokens.dtype)
    if code is None:
        _refuse(f"tokens: unsupported dtype {tokens.dtype}", ERR_INVALID_TYPE)
    if tokens.get_device() != device:
        _place(tokens, "tokens", device)
    if not tokens.is_contiguous():
        _refuse("tokens is not contiguous")
    return code


def _workspace(given, need, device, stream):
    """(pointer, bytes, the tensor to hold on to)."""
    if given is None:
        if not need:
            return 0, 0, None
        given = _empty((need,), torch.uint8, stream)
        return given.data_ptr(), need, given
    if given.get_device() != device:
        _place(given, "workspace", device)
    if not given.is_contiguous():
        _refuse("workspace is not contiguous")
    return given.data_ptr(), given.numel() * given.element_size(), given


def embedding(tokens, table, scale=1.0, out=None, stream=None):
    """scale * table[tokens]: tokens (int32 or int64) of any shape, table
    [V, D].  A token outside [0, V) gives zeros.  Returns out, [*tokens.shape,
    D] of table's type."""
    device = torch.cuda.current_device()
    index = _tokens(tokens, device)
    dtype = _dtype(table, "table")
    if table.dim() != 2:
        _refuse("table is not a matrix")
    V, D, table_ld = _rows(table, "table", device)
    N = tokens.numel()
    if out is None:
        out = _empty((*tokens.shape, D), table.dtype, stream)
        out_ld = D
    else:
        _, _, out_ld = _rows(out, "out", device, D, N)
        if out.dtype != table.dtype:
            _refuse(f"out is {out.dtype}, table {table.dtype}", ERR_INVALID_TYPE)
    rc = _fn("vcoll_embedding")(tokens.data_ptr(), index, N, table.data_ptr(), table_ld, V, D,
                                scale, out.data_ptr(), out_ld, dtype, _handle(stream, device))
    if rc:
        _check(rc)
    return out


def embedding_workspace_bytes(N, vocab, width) -> int:
    return vcoll_embedding_backward_workspace_bytes(N, vocab, width)


def embedding_backward(grad, tokens, vocab, scale=1.0, base=None, out=None, dtype=None,
                       workspace=None, stream=None):
    """The gradient of ``embedding`` for its table: out[v] = base[v] + scale *
    (the sum of the rows of grad whose token is v), every row of out [vocab, D]
    written.  base: what the table's gradient holds from elsewhere (a tied
    projection, earlier micro-batches); ``out=base`` adds in place and touches
    only the rows of tokens that occur.  dtype: out's type (base's, or
    grad's).  workspace: a uint8 CUDA tensor of embedding_workspace_bytes(N,
    vocab, D) bytes, allocated here when omitted."""
    device = torch.cuda.current_device()
    vocab = int(vocab)
    index = _tokens(tokens, device)
    code = _dtype(grad, "grad")
    N, D, grad_ld = _rows(grad, "grad", device, None, tokens.numel())
    base_ptr, base_ld = 0, D
    if base is not None:
        _, _, base_ld = _rows(base, "base", device, D, vocab)
        base_ptr = base.data_ptr()
    if out is None:
        if vocab < 0:
            _refuse(f"vocab = {vocab} < 0")
        out = _empty((vocab, D), dtype or (base if base is not None else grad).dtype, stream)
        out_ld = D
    else:
        _, _, out_ld = _rows(out, "out", device, D, vocab)
        if dtype is not None and out.dtype != dtype:
            _refuse(f"out is {out.dtype}, {dtype} is asked for", ERR_INVALID_TYPE)
    table_code = _dtype(out, "out")
    if base is not None and base.dtype != out.dtype:
        _refuse(f"base is {base.dtype}, out {out.dtype}", ERR_INVALID_TYPE)
    need = _embedding_need(N, vocab, D)
    ws, ws_bytes, _hold = _workspace(workspace, need, device, stream)
    rc = _fn("vcoll_embedding_backward")(grad.data_ptr(), grad_ld, code, tokens.data_ptr(), index,
                                         N, vocab, D, scale, base_ptr, base_ld, out.data_ptr(),
                                         out_ld, table_code, ws, ws_bytes,
                                         _handle(stream, device))
    if rc:
        _check(rc)
    return out


def _weights(weight, bias, D, device):
    """(weight pointer, bias pointer, their type)."""
    w = weight if weight is not None else bias
    if w is None:
        return 0, 0, F32
    code = _dtype(w, "weight")
    return (_vector(weight, "weight", device, D, w.dtype) if weight is not None else 0,
            _vector(bias, "bias", device, D, w.dtype) if bias is not None else 0, code)


def _matrix_out(out, like, what, N, D, device, stream):
    """(tensor, row stride) of an output shaped and typed as `like`."""
    if out is None:
        return _empty(like.shape, like.dtype, stream), D
    _, _, ld = _rows(out, what, device, D, N)
    if out.dtype != like.dtype:
        _refuse(f"{what} is {out.dtype}, {like.dtype} is expected", ERR_INVALID_TYPE)
    return out, ld


def layer_norm(x, weight=None, bias=None, eps=1e-5, out=None, stream=None):
    """Layer norm over the last axis: (y, mean, rstd), y in x's type (in place
    with ``out=x``), mean and rstd fp32 of x's shape without its last axis."""
    device = torch.cuda.current_device()
    code = _dtype(x, "x")
    N, D, x_ld = _rows(x, "x", device)
    w, b, wcode = _weights(weight, bias, D, device)
    y, y_ld = _matrix_out(out, x, "out", N, D, device, stream)
    lead = x.shape[:-1]
    mean = _empty(lead, torch.float32, stream)
    rstd = _empty(lead, torch.float32, stream)
    rc = _fn("vcoll_layer_norm")(x.data_ptr(), x_ld, w, b, wcode, N, D, eps, y.data_ptr(), y_ld,
                                 mean.data_ptr(), rstd.data_ptr(), code, _handle(stream, device))
    if rc:
        _check(rc)
    return y, mean, rstd


def layer_norm_workspace_bytes(N, width) -> int:
    return vcoll_layer_norm_workspace_bytes(N, width)


def _gradients(grad, weight, dx, dweight, dbias, weight_grads, N, D, device, stream):
    """Output tensors and pointers of a layer norm's gradient."""
    w, _, wcode = _weights(weight, None, D, device)
    dx, dx_ld = _matrix_out(dx, grad, "dx", N, D, device, stream)
    wtype = weight.dtype if weight is not None else torch.float32
    pw = pb = 0
    if dweight is not None:
        pw = _vector(dweight, "dweight", device, D, wtype)
    elif weight_grads:
        dweight = _empty((D,), wtype, stream)
        pw = dweight.data_ptr()
    if dbias is not None:
        pb = _vector(dbias, "dbias", device, D, wtype)
    elif weight_grads:
        dbias = _empty((D,), wtype, stream)
        pb = dbias.data_ptr()
    return w, wcode, dx, dx_ld, dweight, dbias, pw, pb


def layer_norm_backward(grad, x, mean, rstd, weight=None, dx=None, dweight=None, dbias=None,
                        weight_grads=True, workspace=None, stream=None):
    """The gradient of ``layer_norm``: (dx, dweight, dbias) from its output's
    gradient, its input and the statistics that it returned.  dx may be grad or
    x (in place); dweight and dbias are of weight's type (fp32 without a
    weight) and may be slices of a fusion buffer; weight_grads=False leaves out
    (returns None for) those that are not given."""
    device = torch.cuda.current_device()
    code = _dtype(grad, "grad")
    N, D, grad_ld = _rows(grad, "grad", device)
    _, _, x_ld = _rows(x, "x", device, D, N)
    if x.dtype != grad.dtype:
        _refuse(f"x is {x.dtype}, grad {grad.dtype}", ERR_INVALID_TYPE)
    pm = _vector(mean, "mean", device, N, torch.float32)
    pr = _vector(rstd, "rstd", device, N, torch.float32)
    w, wcode, dx, dx_ld, dweight, dbias, pw, pb = _gradients(
        grad, weight, dx, dweight, dbias, weight_grads, N, D, device, stream)
    need = _norm_need(N, D)
    ws, ws_bytes, _hold = _workspace(workspace, need, device, stream)
    rc = _fn("vcoll_layer_norm_backward")(grad.data_ptr(), grad_ld, x.data_ptr(), x_ld, pm, pr, w,
                                          wcode, N, D, dx.data_ptr(), dx_ld, pw, pb, code, ws,
                                          ws_bytes, _handle(stream, device))
    if rc:
        _check(rc)
    return dx, dweight, dbias


class Checkpoint8(NamedTuple):
    """An activation kept in 8 bits: int8 codes (each row padded to a multiple
    of 16), one fp32 scale for each 128 columns of a row, and the activation's
    shape."""
    codes: torch.Tensor
    scales: torch.Tensor
    shape: torch.Size

    @property
    def nbytes(self) -> int:
        return self.codes.numel() + 4 * self.scales.numel()


def _kept_empty(shape, stream):
    """(codes, their row stride, scales) for an activation of that shape."""
    lead, D = shape[:-1], shape[-1]
    ld = (D + 15) // 16 * 16
    return (_empty((*lead, ld), torch.int8, stream), ld,
            _empty((*lead, -(-D // CHECKPOINT8_BLOCK)), torch.float32, stream))


def _kept(kept, device, D=None, N=None):
    """(rows, columns, codes pointer, their row stride, scales pointer)."""
    codes, scales, shape = kept
    width = shape[-1]
    rows = shape[0] if len(shape) == 2 else shape[:-1].numel()
    if (D is not None and width != D) or (N is not None and rows != N):
        _refuse(f"the kept activation has the shape {tuple(shape)}")
    ld = codes.shape[-1]
    if ld < width:
        _refuse("codes are not rows of the kept activation")
    return (rows, width, _vector(codes, "codes", device, rows * ld, torch.int8), ld,
            _vector(scales, "scales", device, rows * -(-width // CHECKPOINT8_BLOCK),
                    torch.float32))


def checkpoint8(x, stream=None) -> Checkpoint8:
    """x kept in 8 bits, with one scale for each 128 columns of a row."""
    device = torch.cuda.current_device()
    code = _dtype(x, "x")
    N, D, x_ld = _rows(x, "x", device)
    codes, ld, scales = _kept_empty(x.shape, stream)
    rc = _fn("vcoll_checkpoint8")(x.data_ptr(), x_ld, N, D, codes.data_ptr(), ld,
                                  scales.data_ptr(), code, _handle(stream, device))
    if rc:
        _check(rc)
    return Checkpoint8(codes, scales, x.shape)


def checkpoint8_restore(kept, weight=None, bias=None, dtype=torch.float32, out=None, stream=None):
    """What a Checkpoint8 stands for, times weight plus bias where given (the
    output of the layer norm that kept it).  dtype: of the result, unless out
    is given."""
    device = torch.cuda.current_device()
    N, D, codes, codes_ld, scales = _kept(kept, device)
    w, b, wcode = _weights(weight, bias, D, device)
    if out is None:
        out, out_ld = _empty(kept.shape, dtype, stream), D
    else:
        _, _, out_ld = _rows(out, "out", device, D, N)
    rc = _fn("vcoll_checkpoint8_restore")(codes, codes_ld, scales, w, b, wcode, N, D,
                                          out.data_ptr(), out_ld, _dtype(out, "out"),
                                          _handle(stream, device))
    if rc:
        _check(rc)
    return out


def layer_norm_checkpoint8(x, weight=None, bias=None, eps=1e-5, out=None, stream=None):
    """``layer_norm`` that keeps its normalised input in 8 bits on the way:
    (y, rstd, kept).  Neither x nor y is needed for the backward pass then:
    ``checkpoint8_restore(kept, weight, bias)`` gives y back, and
    ``layer_norm_backward_checkpoint8`` the gradients."""
    device = torch.cuda.current_device()
    code = _dtype(x, "x")
    N, D, x_ld = _rows(x, "x", device)
    w, b, wcode = _weights(weight, bias, D, device)
    y, y_ld = _matrix_out(out, x, "out", N, D, device, stream)
    rstd = _empty(x.shape[:-1], torch.float32, stream)
    codes, ld, scales = _kept_empty(x.shape, stream)
    rc = _fn("vcoll_layer_norm_checkpoint8")(x.data_ptr(), x_ld, w, b, wcode, N, D, eps,
                                             y.data_ptr(), y_ld, rstd.data_ptr(),
                                             codes.data_ptr(), ld, scales.data_ptr(), code,
                                             _handle(stream, device))
    if rc:
        _check(rc)
    return y, rstd, Checkpoint8(codes, scales, x.shape)


def layer_norm_backward_checkpoint8(grad, kept, rstd, weight=None, dx=None, dweight=None,
                                    dbias=None, weight_grads=True, workspace=None, stream=None):
    """``layer_norm_backward`` from what ``layer_norm_checkpoint8`` kept."""
    device = torch.cuda.current_device()
    code = _dtype(grad, "grad")
    N, D, grad_ld = _rows(grad, "grad", device)
    _, _, codes, codes_ld, scales = _kept(kept, device, D, N)
    pr = _vector(rstd, "rstd", device, N, torch.float32)
    w, wcode, dx, dx_ld, dweight, dbias, pw, pb = _gradients(
        grad, weight, dx, dweight, dbias, weight_grads, N, D, device, stream)
    need = _norm_need(N, D)
    ws, ws_bytes, _hold = _workspace(workspace, need, device, stream)
    rc = _fn("vcoll_layer_norm_backward_checkpoint8")(
        grad.data_ptr(), grad_ld, codes, codes_ld, scales, pr, w, wcode, N, D, dx.data_ptr(),
        dx_ld, pw, pb, code, ws, ws_bytes, _handle(stream, device))
    if rc:
        _check(rc)
    return dx, dweight, dbias
