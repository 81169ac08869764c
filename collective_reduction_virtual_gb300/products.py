"""Products of a rank's rows with weights, the element-wise part of the operator
in the product's epilogue: softmax cross entropy against a vocabulary without
keeping the logits, the gated feed-forward block, and their gradients.

Same conventions as ``layers``: ``vcoll_*`` take integer device pointers and
return the status code, the functions without the prefix take tensors and raise
``VcollError``; formulas and conventions are in ``include/vcoll.h``.  Autograd
does not see these calls.
"""
from __future__ import annotations

import functools

import torch

from . import ERR_INVALID_OP, ERR_INVALID_TYPE, _check
from .layers import (_ARGS, _I, _L, _P, _Z, _dtype, _empty, _fn, _handle, _matrix_out, _refuse,
                     _rows, _tokens, _vector, _workspace)

SILU, GELU, GELU_TANH = 0, 1, 2
_ACTIVATIONS = {"silu": SILU, "gelu": GELU, "gelu_tanh": GELU_TANH}

_ARGS.update({
    "vcoll_cross_entropy": [_P, _L, _P, _L, _P, _I, _L, _L, _L, _P, _P, _I, _P, _Z, _P],
    "vcoll_cross_entropy_backward": [_P, _L, _P, _L, _P, _L, _P, _I, _P, _L, _L, _L, _P, _L, _P, _L,
                                     _P, _L, _I, _P, _Z, _P],
    "vcoll_gated_ff": [_P, _L, _P, _L, _P, _L, _I, _L, _L, _L, _P, _L, _P, _L, _P, _L, _I, _P, _Z,
                       _P],
    "vcoll_gated_ff_backward": [_P, _L, _P, _L, _P, _L, _P, _L, _P, _L, _P, _L, _I, _L, _L, _L, _P,
                                _L, _P, _L, _P, _L, _I, _P, _Z, _P],
    "vcoll_cross_entropy_workspace_bytes": [_L, _L, _L, _I, _I],
    "vcoll_cross_entropy_backward_workspace_bytes": [_L, _L, _L, _I, _I],
    "vcoll_gated_ff_workspace_bytes": [_L, _L, _L, _I, _I],
    "vcoll_gated_ff_backward_workspace_bytes": [_L, _L, _L, _I, _I],
})


# ----------------------------------------------------------- raw C ABI layer

def vcoll_cross_entropy_workspace_bytes(N, V, D, dtype, direct) -> int:
    return _fn("vcoll_cross_entropy_workspace_bytes")(N, V, D, dtype, direct)


def vcoll_cross_entropy(x, x_ld, table, table_ld, targets, index_type, N, V, D, loss, lse, dtype,
                        workspace=0, workspace_bytes=0, stream=0) -> int:
    return _fn("vcoll_cross_entropy")(x, x_ld, table, table_ld, targets, index_type, N, V, D, loss,
                                      lse, dtype, workspace, workspace_bytes, stream)


def vcoll_cross_entropy_backward_workspace_bytes(N, V, D, dtype, direct) -> int:
    return _fn("vcoll_cross_entropy_backward_workspace_bytes")(N, V, D, dtype, direct)


def vcoll_cross_entropy_backward(dloss, dloss_count, x, x_ld, table, table_ld, targets, index_type,
                                 lse, N, V, D, dx, dx_ld, base, base_ld, dtable, dtable_ld, dtype,
                                 workspace=0, workspace_bytes=0, stream=0) -> int:
    return _fn("vcoll_cross_entropy_backward")(dloss, dloss_count, x, x_ld, table, table_ld,
                                               targets, index_type, lse, N, V, D, dx, dx_ld, base,
                                               base_ld, dtable, dtable_ld, dtype, workspace,
                                               workspace_bytes, stream)


def vcoll_gated_ff_workspace_bytes(N, D, F, dtype, direct) -> int:
    return _fn("vcoll_gated_ff_workspace_bytes")(N, D, F, dtype, direct)


def vcoll_gated_ff(x, x_ld, w_gate, w_gate_ld, w_up, w_up_ld, activation, N, D, F, h, h_ld, gate,
                   gate_ld, up, up_ld, dtype, workspace=0, workspace_bytes=0, stream=0) -> int:
    return _fn("vcoll_gated_ff")(x, x_ld, w_gate, w_gate_ld, w_up, w_up_ld, activation, N, D, F, h,
                                 h_ld, gate, gate_ld, up, up_ld, dtype, workspace, workspace_bytes,
                                 stream)


def vcoll_gated_ff_backward_workspace_bytes(N, D, F, dtype, direct) -> int:
    return _fn("vcoll_gated_ff_backward_workspace_bytes")(N, D, F, dtype, direct)


def vcoll_gated_ff_backward(dh, dh_ld, x, x_ld, w_gate, w_gate_ld, w_up, w_up_ld, gate, gate_ld, up,
                            up_ld, activation, N, D, F, dx, dx_ld, dw_gate, dw_gate_ld, dw_up,
                            dw_up_ld, dtype, workspace=0, workspace_bytes=0, stream=0) -> int:
    return _fn("vcoll_gated_ff_backward")(dh, dh_ld, x, x_ld, w_gate, w_gate_ld, w_up, w_up_ld,
                                          gate, gate_ld, up, up_ld, activation, N, D, F, dx, dx_ld,
                                          dw_gate, dw_gate_ld, dw_up, dw_up_ld, dtype, workspace,
                                          workspace_bytes, stream)


# -------------------------------------------------------------- tensor layer

@functools.lru_cache(maxsize=256)
def _need(name, a, b, c, dtype, direct):
    return _fn(name)(a, b, c, dtype, direct)


def _direct(*matrices):
    """1 where the products can read every (tensor, row stride) where it lies."""
    for t, ld in matrices:
        if not t.is_cuda or t.data_ptr() % 16 or (ld % 8 and t.numel() != t.shape[-1]):
            return 0
    return 1


def _same(t, like, what, name):
    if t.dtype != like.dtype:
        _refuse(f"{what} is {t.dtype}, {name} {like.dtype}", ERR_INVALID_TYPE)


def _loss_operands(x, table, targets, device):
    dtype = _dtype(x, "x")
    index = _tokens(targets, device)
    N, D, x_ld = _rows(x, "x", device, None, targets.numel())
    if table.dim() != 2:
        _refuse("table is not a matrix")
    V, _, table_ld = _rows(table, "table", device, D)
    _same(table, x, "table", "x")
    return dtype, index, N, V, D, x_ld, table_ld


def cross_entropy_workspace_bytes(N, vocab, width, dtype=torch.bfloat16, direct=0) -> int:
    return _need("vcoll_cross_entropy_workspace_bytes", N, vocab, width, 0 if dtype == torch.float32 else 1,
                 direct)


def cross_entropy(x, table, targets, loss=None, lse=None, workspace=None, stream=None):
    """Softmax cross entropy of rows x [..., D] against table [V, D] at targets
    (int32 or int64, x's shape without its last axis), the logits not kept:
    (loss, lse), both fp32 of targets' shape.  A target outside [0, V) has loss
    0.  lse, the logarithm of the sum of exponentials, is what
    ``cross_entropy_backward`` needs.  workspace: a uint8 CUDA tensor of
    cross_entropy_workspace_bytes(N, V, D, dtype) bytes, allocated here when
    omitted."""
    device = torch.cuda.current_device()
    dtype, index, N, V, D, x_ld, table_ld = _loss_operands(x, table, targets, device)
    if loss is None:
        loss = _empty(targets.shape, torch.float32, stream)
    else:
        _vector(loss, "loss", device, N, torch.float32)
    if lse is None:
        lse = _empty(targets.shape, torch.float32, stream)
    else:
        _vector(lse, "lse", device, N, torch.float32)
    need = _need("vcoll_cross_entropy_workspace_bytes", N, V, D, dtype,
                 _direct((x, x_ld), (table, table_ld)))
    ws, ws_bytes, _hold = _workspace(workspace, need, device, stream)
    rc = _fn("vcoll_cross_entropy")(x.data_ptr(), x_ld, table.data_ptr(), table_ld,
                                    targets.data_ptr(), index, N, V, D, loss.data_ptr(),
                                    lse.data_ptr(), dtype, ws, ws_bytes, _handle(stream, device))
    if rc:
        _check(rc)
    return loss, lse


def cross_entropy_backward_workspace_bytes(N, vocab, width, dtype=torch.bfloat16, direct=0) -> int:
    return _need("vcoll_cross_entropy_backward_workspace_bytes", N, vocab, width,
                 0 if dtype == torch.float32 else 1, direct)


def cross_entropy_backward(dloss, x, table, targets, lse, base=None, dx=None, dtable=None,
                           x_grad=True, table_grad=True, workspace=None, stream=None):
    """The gradient of ``cross_entropy``: (dx, dtable) from its loss's gradient
    (fp32 of targets' shape, or one value for all rows), its inputs and the lse
    that it returned.  dtable = base + the gradient; base: what the table's
    gradient holds from elsewhere (``dtable=base`` adds in place).  dx may be x
    (in place).  x_grad=False or table_grad=False leaves one out (None) unless
    its tensor is given.  Rows whose target is outside [0, V) give a row of
    zeros in dx and nothing to dtable, whatever they hold."""
    device = torch.cuda.current_device()
    dtype, index, N, V, D, x_ld, table_ld = _loss_operands(x, table, targets, device)
    count = dloss.numel()
    if count != 1 and count != N:
        _refuse(f"dloss has {count} values, {N} or 1 are expected")
    g = _vector(dloss, "dloss", device, count, torch.float32)
    plse = _vector(lse, "lse", device, N, torch.float32)
    base_ptr, base_ld = 0, D
    if base is not None:
        _, _, base_ld = _rows(base, "base", device, D, V)
        _same(base, table, "base", "table")
        base_ptr = base.data_ptr()
    pdx = pdt = 0
    dx_ld = dtable_ld = D
    if dx is not None or x_grad:
        dx, dx_ld = _matrix_out(dx, x, "dx", N, D, device, stream)
        pdx = dx.data_ptr()
    if dtable is not None or table_grad:
        dtable, dtable_ld = _matrix_out(dtable, table, "dtable", V, D, device, stream)
        pdt = dtable.data_ptr()
    need = _need("vcoll_cross_entropy_backward_workspace_bytes", N, V, D, dtype,
                 _direct((table, table_ld)))
    ws, ws_bytes, _hold = _workspace(workspace, need, device, stream)
    rc = _fn("vcoll_cross_entropy_backward")(
        g, count, x.data_ptr(), x_ld, table.data_ptr(), table_ld, targets.data_ptr(), index, plse,
        N, V, D, pdx, dx_ld, base_ptr, base_ld, pdt, dtable_ld, dtype, ws, ws_bytes,
        _handle(stream, device))
    if rc:
        _check(rc)
    return dx, dtable


def _block_operands(x, w_gate, w_up, activation, device):
    act = _ACTIVATIONS.get(activation)
    if act is None:
        _refuse(f"unknown activation {activation!r}", ERR_INVALID_OP)
    dtype = _dtype(x, "x")
    N, D, x_ld = _rows(x, "x", device)
    if w_gate.dim() != 2 or w_up.dim() != 2:
        _refuse("w_gate and w_up are not matrices")
    F, _, gate_ld = _rows(w_gate, "w_gate", device, D)
    _, _, up_ld = _rows(w_up, "w_up", device, D, F)
    _same(w_gate, x, "w_gate", "x")
    _same(w_up, x, "w_up", "x")
    return act, dtype, N, D, F, x_ld, gate_ld, up_ld


def gated_ff_workspace_bytes(N, width, inner, dtype=torch.bfloat16, direct=0) -> int:
    return _need("vcoll_gated_ff_workspace_bytes", N, width, inner, 0 if dtype == torch.float32 else 1,
                 direct)


def gated_ff(x, w_gate, w_up, activation="silu", keep=False, out=None, workspace=None, stream=None):
    """A gated feed-forward block: h = act(gate) * up with gate = x @ w_gate.T
    and up = x @ w_up.T, for rows x [..., D] and weights [F, D]; activation:
    "silu", "gelu" or "gelu_tanh".  Returns h [..., F], or with keep=True (h,
    gate, up), which ``gated_ff_backward`` needs.  out: where h goes.
    workspace: a uint8 CUDA tensor of gated_ff_workspace_bytes(N, D, F, dtype)
    bytes, allocated here when omitted."""
    device = torch.cuda.current_device()
    act, dtype, N, D, F, x_ld, wg_ld, wu_ld = _block_operands(x, w_gate, w_up, activation, device)
    shape = (*x.shape[:-1], F)
    if out is None:
        out, out_ld = _empty(shape, x.dtype, stream), F
    else:
        _, _, out_ld = _rows(out, "out", device, F, N)
        _same(out, x, "out", "x")
    gate = up = None
    pg = pu = 0
    if keep:
        gate, up = _empty(shape, x.dtype, stream), _empty(shape, x.dtype, stream)
        pg, pu = gate.data_ptr(), up.data_ptr()
    need = _need("vcoll_gated_ff_workspace_bytes", N, D, F, dtype,
                 _direct((x, x_ld), (w_gate, wg_ld), (w_up, wu_ld)))
    ws, ws_bytes, _hold = _workspace(workspace, need, device, stream)
    rc = _fn("vcoll_gated_ff")(x.data_ptr(), x_ld, w_gate.data_ptr(), wg_ld, w_up.data_ptr(), wu_ld,
                               act, N, D, F, out.data_ptr(), out_ld, pg, F, pu, F, dtype, ws,
                               ws_bytes, _handle(stream, device))
    if rc:
        _check(rc)
    return (out, gate, up) if keep else out


def gated_ff_backward_workspace_bytes(N, width, inner, dtype=torch.bfloat16, direct=0) -> int:
    return _need("vcoll_gated_ff_backward_workspace_bytes", N, width, inner,
                 0 if dtype == torch.float32 else 1, direct)


def gated_ff_backward(dh, x, w_gate, w_up, gate, up, activation="silu", dx=None, dw_gate=None,
                      dw_up=None, x_grad=True, weight_grads=True, workspace=None, stream=None):
    """The gradient of ``gated_ff``: (dx, dw_gate, dw_up) from its output's
    gradient, its inputs, and the gate and up that it kept.  x_grad=False or
    weight_grads=False leaves out (returns None for) those that are not given;
    dw_gate and dw_up may be slices of a fusion buffer."""
    device = torch.cuda.current_device()
    act, dtype, N, D, F, x_ld, wg_ld, wu_ld = _block_operands(x, w_gate, w_up, activation, device)
    lds = []
    for t, what in ((dh, "dh"), (gate, "gate"), (up, "up")):
        lds.append(_rows(t, what, device, F, N)[2])
        _same(t, x, what, "x")
    pdx = pg = pu = 0
    dx_ld = dg_ld = du_ld = D
    if dx is not None or x_grad:
        dx, dx_ld = _matrix_out(dx, x, "dx", N, D, device, stream)
        pdx = dx.data_ptr()
    if dw_gate is not None or weight_grads:
        dw_gate, dg_ld = _matrix_out(dw_gate, w_gate, "dw_gate", F, D, device, stream)
        pg = dw_gate.data_ptr()
    if dw_up is not None or weight_grads:
        dw_up, du_ld = _matrix_out(dw_up, w_up, "dw_up", F, D, device, stream)
        pu = dw_up.data_ptr()
    need = _need("vcoll_gated_ff_backward_workspace_bytes", N, D, F, dtype,
                 _direct((x, x_ld), (w_gate, wg_ld), (w_up, wu_ld)))
    ws, ws_bytes, _hold = _workspace(workspace, need, device, stream)
    rc = _fn("vcoll_gated_ff_backward")(
        dh.data_ptr(), lds[0], x.data_ptr(), x_ld, w_gate.data_ptr(), wg_ld, w_up.data_ptr(), wu_ld,
        gate.data_ptr(), lds[1], up.data_ptr(), lds[2], act, N, D, F, pdx, dx_ld, pg, dg_ld, pu,
        du_ld, dtype, ws, ws_bytes, _handle(stream, device))
    if rc:
        _check(rc)
    return dx, dw_gate, dw_up
