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
"""
from __future__ import annotations

import ctypes
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

_TYPES = {torch.float32: F32, torch.bfloat16: BF16}
_INDEX = {torch.int32: I32, torch.int64: I64}


def _refuse(message, status=ERR_INVALID_ARG):
    raise VcollError(status, message)


def _dtype(t, what):
    code = _TYPES.get(t.dtype)
    if code is None:
        _refuse(f"{what}: unsupported dtype {t.dtype}", ERR_INVALID_TYPE)
    return code


def _place(t, what):
    """The tensor lies where the kernels of the current device may reach it."""
    if t.is_cuda:
        if t.get_device() != torch.cuda.current_device():
            _refuse(f"{what} is on device {t.get_device()}, the current device is "
                    f"{torch.cuda.current_device()}")
    elif not t.is_pinned():
        _refuse(f"{what} is neither a CUDA tensor nor pinned host memory")


def _rows(t, what, width=None, rows=None):
    """(rows, row stride in elements) of a tensor taken as a matrix."""
    _place(t, what)
    if t.dim() == 0:
        _refuse(f"{what} has no axes")
    d = t.shape[-1]
    if width is not None and d != width:
        _refuse(f"{what} has {d} columns, {width} are expected")
    if t.is_contiguous():
        n, ld = (t.numel() // d if d else t.shape[:-1].numel()), d
    else:
        try:
            m = t.view(-1, d) if d else t
        except RuntimeError:
            m = None
        if m is None or (d > 1 and m.stride(1) != 1) or (m.shape[0] > 1 and m.stride(0) < d):
            _refuse(f"{what} is not a matrix of rows with adjacent columns (not contiguous)")
        n = m.shape[0]
        ld = m.stride(0) if n > 1 else d
    if rows is not None and n != rows:
        _refuse(f"{what} has {n} rows, {rows} are expected")
    return n, ld


def _vector(t, what, length, dtype=None):
    _place(t, what)
    if t.numel() != length or not t.is_contiguous():
        _refuse(f"{what} is not a contiguous tensor of {length} elements")
    if dtype is not None and t.dtype != dtype:
        _refuse(f"{what} is {t.dtype}, {dtype} is expected", ERR_INVALID_TYPE)
    return t.data_ptr()


class _Call:
    """The stream of one call, and the tensors that it allocates there."""

    __slots__ = ("stream", "handle")

    def __init__(self, stream):
        self.stream = stream
        self.handle = (stream if stream is not None else torch.cuda.current_stream()).cuda_stream

    def empty(self, shape, dtype):
        if self.stream is None:
            return torch.empty(shape, dtype=dtype, device="cuda")
        with torch.cuda.stream(self.stream):
            return torch.empty(shape, dtype=dtype, device="cuda")

    def workspace(self, given, need):
        """(pointer, bytes, the tensor to hold on to)."""
        if given is None:
            if not need:
                return 0, 0, None
            given = self.empty(need, torch.uint8)
        _place(given, "workspace")
        return given.data_ptr(), given.numel() * given.element_size(), given


def _tokens(tokens):
    code = _INDEX.get(tokens.dtype)
    if code is None:
        _refuse(f"tokens: unsupported dtype {tokens.dtype}", ERR_INVALID_TYPE)
    _place(tokens, "tokens")
    if not tokens.is_contiguous():
        _refuse("tokens is not contiguous")
    return code


def embedding(tokens, table, scale=1.0, out=None, stream=None):
    """scale * table[tokens]: tokens (int32 or int64) of any shape, table
    [V, D].  A token outside [0, V) gives zeros.  Returns out, [*tokens.shape,
    D] of table's type."""
    index = _tokens(tokens)
    dtype = _dtype(table, "table")
    if table.dim() != 2:
        _refuse("table is not a matrix")
    V, D = table.shape
    _, table_ld = _rows(table, "table")
    N = tokens.numel()
    call = _Call(stream)
    if out is None:
        out = call.empty((*tokens.shape, D), table.dtype)
        out_ld = D
    else:
        _, out_ld = _rows(out, "out", D, N)
        if out.dtype != table.dtype:
            _refuse(f"out is {out.dtype}, table {table.dtype}", ERR_INVALID_TYPE)
    _check(vcoll_embedding(tokens.data_ptr(), index, N, table.data_ptr(), table_ld, V, D, scale,
                           out.data_ptr(), out_ld, dtype, call.handle))
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
    index = _tokens(tokens)
    N = tokens.numel()
    code = _dtype(grad, "grad")
    _, grad_ld = _rows(grad, "grad", None, N)
    D = grad.shape[-1]
    call = _Call(stream)
    base_ptr, base_ld = 0, D
    if base is not None:
        _, base_ld = _rows(base, "base", D, vocab)
        base_ptr = base.data_ptr()
    if out is None:
        want = dtype or (base if base is not None else grad).dtype
        out = call.empty((vocab, D), want)
        out_ld = D
    else:
        _, out_ld = _rows(out, "out", D, vocab)
        if dtype is not None and out.dtype != dtype:
            _refuse(f"out is {out.dtype}, {dtype} is asked for", ERR_INVALID_TYPE)
    table_code = _dtype(out, "out")
    if base is not None and base.dtype != out.dtype:
        _refuse(f"base is {base.dtype}, out {out.dtype}", ERR_INVALID_TYPE)
    ws, ws_bytes, _hold = call.workspace(
        workspace, vcoll_embedding_backward_workspace_bytes(N, vocab, D))
    _check(vcoll_embedding_backward(grad.data_ptr(), grad_ld, code, tokens.data_ptr(), index, N,
                                    vocab, D, scale, base_ptr, base_ld, out.data_ptr(), out_ld,
                                    table_code, ws, ws_bytes, call.handle))
    return out


def _weights(weight, bias, D):
    """(weight pointer, bias pointer, their type)."""
    w = weight if weight is not None else bias
    if w is None:
        return 0, 0, F32
    code = _dtype(w, "weight")
    return (_vector(weight, "weight", D) if weight is not None else 0,
            _vector(bias, "bias", D, w.dtype) if bias is not None else 0, code)


def _matrix_out(call, out, like, what, N, D):
    """(tensor, row stride) of an output shaped and typed as `like`."""
    if out is None:
        return call.empty(like.shape, like.dtype), D
    _, ld = _rows(out, what, D, N)
    if out.dtype != like.dtype:
        _refuse(f"{what} is {out.dtype}, {like.dtype} is expected", ERR_INVALID_TYPE)
    return out, ld


def layer_norm(x, weight=None, bias=None, eps=1e-5, out=None, stream=None):
    """Layer norm over the last axis: (y, mean, rstd), y in x's type (in place
    with ``out=x``), mean and rstd fp32 of x's shape without its last axis."""
    code = _dtype(x, "x")
    N, x_ld = _rows(x, "x")
    D = x.shape[-1]
    w, b, wcode = _weights(weight, bias, D)
    call = _Call(stream)
    y, y_ld = _matrix_out(call, out, x, "out", N, D)
    stats = call.empty((2, *x.shape[:-1]), torch.float32)
    mean, rstd = stats.unbind(0)
    at = stats.data_ptr()
    _check(vcoll_layer_norm(x.data_ptr(), x_ld, w, b, wcode, N, D, eps, y.data_ptr(), y_ld, at,
                            at + 4 * N, code, call.handle))
    return y, mean, rstd


def layer_norm_workspace_bytes(N, width) -> int:
    return vcoll_layer_norm_workspace_bytes(N, width)


def _gradients(call, grad, weight, dx, dweight, dbias, weight_grads, N, D):
    """Output tensors and pointers of a layer norm's gradient."""
    w, _, wcode = _weights(weight, None, D)
    dx, dx_ld = _matrix_out(call, dx, grad, "dx", N, D)
    wtype = weight.dtype if weight is not None else torch.float32
    if dweight is None and weight_grads:
        dweight = call.empty(D, wtype)
    if dbias is None and weight_grads:
        dbias = call.empty(D, wtype)
    pw = _vector(dweight, "dweight", D, wtype) if dweight is not None else 0
    pb = _vector(dbias, "dbias", D, wtype) if dbias is not None else 0
    return w, wcode, dx, dx_ld, dweight, dbias, pw, pb


def layer_norm_backward(grad, x, mean, rstd, weight=None, dx=None, dweight=None, dbias=None,
                        weight_grads=True, workspace=None, stream=None):
    """The gradient of ``layer_norm``: (dx, dweight, dbias) from its output's
    gradient, its input and the statistics that it returned.  dx may be grad or
    x (in place); dweight and dbias are of weight's type (fp32 without a
    weight) and may be slices of a fusion buffer; weight_grads=False leaves out
    (returns None for) those that are not given."""
    code = _dtype(grad, "grad")
    N, grad_ld = _rows(grad, "grad")
    D = grad.shape[-1]
    _, x_ld = _rows(x, "x", D, N)
    if x.dtype != grad.dtype:
        _refuse(f"x is {x.dtype}, grad {grad.dtype}", ERR_INVALID_TYPE)
    pm = _vector(mean, "mean", N, torch.float32)
    pr = _vector(rstd, "rstd", N, torch.float32)
    call = _Call(stream)
    w, wcode, dx, dx_ld, dweight, dbias, pw, pb = _gradients(call, grad, weight, dx, dweight,
                                                             dbias, weight_grads, N, D)
    ws, ws_bytes, _hold = call.workspace(workspace, vcoll_layer_norm_workspace_bytes(N, D))
    _check(vcoll_layer_norm_backward(grad.data_ptr(), grad_ld, x.data_ptr(), x_ld, pm, pr, w,
                                     wcode, N, D, dx.data_ptr(), dx_ld, pw, pb, code, ws, ws_bytes,
                                     call.handle))
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


def _kept_empty(call, shape):
    D = shape[-1]
    codes = call.empty((*shape[:-1], (D + 15) // 16 * 16), torch.int8)
    scales = call.empty((*shape[:-1], -(-D // CHECKPOINT8_BLOCK)), torch.float32)
    return Checkpoint8(codes, scales, shape)


def _kept(kept, D=None, N=None):
    """(rows, columns, codes pointer, their row stride, scales pointer)."""
    width = kept.shape[-1]
    rows = kept.shape[:-1].numel()
    if (D is not None and width != D) or (N is not None and rows != N):
        _refuse(f"the kept activation has the shape {tuple(kept.shape)}")
    ld = kept.codes.shape[-1]
    if kept.codes.dtype != torch.int8 or ld < width:
        _refuse("codes are not int8 rows of the kept activation", ERR_INVALID_TYPE)
    return (rows, width, _vector(kept.codes, "codes", rows * ld), ld,
            _vector(kept.scales, "scales", rows * -(-width // CHECKPOINT8_BLOCK), torch.float32))


def checkpoint8(x, stream=None) -> Checkpoint8:
    """x kept in 8 bits, with one scale for each 128 columns of a row."""
    code = _dtype(x, "x")
    N, x_ld = _rows(x, "x")
    call = _Call(stream)
    kept = _kept_empty(call, x.shape)
    _check(vcoll_checkpoint8(x.data_ptr(), x_ld, N, x.shape[-1], kept.codes.data_ptr(),
                             kept.codes.shape[-1], kept.scales.data_ptr(), code, call.handle))
    return kept


def checkpoint8_restore(kept, weight=None, bias=None, dtype=torch.float32, out=None, stream=None):
    """What a Checkpoint8 stands for, times weight plus bias where given (the
    output of the layer norm that kept it).  dtype: of the result, unless out
    is given."""
    N, D, codes, codes_ld, scales = _kept(kept)
    w, b, wcode = _weights(weight, bias, D)
    call = _Call(stream)
    if out is None:
        out, out_ld = call.empty(kept.shape, dtype), D
    else:
        _, out_ld = _rows(out, "out", D, N)
    _check(vcoll_checkpoint8_restore(codes, codes_ld, scales, w, b, wcode, N, D, out.data_ptr(),
                                     out_ld, _dtype(out, "out"), call.handle))
    return out


def layer_norm_checkpoint8(x, weight=None, bias=None, eps=1e-5, out=None, stream=None):
    """``layer_norm`` that keeps its normalised input in 8 bits on the way:
    (y, rstd, kept).  Neither x nor y is needed for the backward pass then:
    ``checkpoint8_restore(kept, weight, bias)`` gives y back, and
    ``layer_norm_backward_checkpoint8`` the gradients."""
    code = _dtype(x, "x")
    N, x_ld = _rows(x, "x")
    D = x.shape[-1]
    w, b, wcode = _weights(weight, bias, D)
    call = _Call(stream)
    y, y_ld = _matrix_out(call, out, x, "out", N, D)
    rstd = call.empty(x.shape[:-1], torch.float32)
    kept = _kept_empty(call, x.shape)
    _check(vcoll_layer_norm_checkpoint8(x.data_ptr(), x_ld, w, b, wcode, N, D, eps, y.data_ptr(),
                                        y_ld, rstd.data_ptr(), kept.codes.data_ptr(),
                                        kept.codes.shape[-1], kept.scales.data_ptr(), code,
                                        call.handle))
    return y, rstd, kept


def layer_norm_backward_checkpoint8(grad, kept, rstd, weight=None, dx=None, dweight=None,
                                    dbias=None, weight_grads=True, workspace=None, stream=None):
    """``layer_norm_backward`` from what ``layer_norm_checkpoint8`` kept."""
    code = _dtype(grad, "grad")
    N, grad_ld = _rows(grad, "grad")
    D = grad.shape[-1]
    _, _, codes, codes_ld, scales = _kept(kept, D, N)
    pr = _vector(rstd, "rstd", N, torch.float32)
    call = _Call(stream)
    w, wcode, dx, dx_ld, dweight, dbias, pw, pb = _gradients(call, grad, weight, dx, dweight,
                                                             dbias, weight_grads, N, D)
    ws, ws_bytes, _hold = call.workspace(workspace, vcoll_layer_norm_workspace_bytes(N, D))
    _check(vcoll_layer_norm_backward_checkpoint8(grad.data_ptr(), grad_ld, codes, codes_ld, scales,
                                                 pr, w, wcode, N, D, dx.data_ptr(), dx_ld, pw, pb,
                                                 code, ws, ws_bytes, call.handle))
    return dx, dweight, dbias
