"""The two ends of a training step: embedding, layer norm, cross entropy.

Argument marshalling for the calls that include/nsortho.h describes under
"The two ends of a training step".  Like the other calls they run on the
current stream of their tensors' device, write new tensors (or the ``out``
given), never synchronize, and raise ValueError or TypeError for arguments
that the library could not use.  ``workspace`` is an optional device buffer of
the size that the matching ``*_workspace_size`` names; without it one is
allocated by torch.  ``status`` is the device int32 status word.  No call
builds an autograd graph: tensors that require a gradient are taken for their
values, results never require one, and the backward calls are made by hand.
"""

from __future__ import annotations

import ctypes
from typing import List, Optional, Tuple, Union

import torch

from . import _binding as B
from ._binding import NSError, _check, dtype_code, lib


def _stream_of(index: int) -> int:
    return torch.cuda.current_stream(index).cuda_stream


# The current stream's handle by device index, and the current device: the
# functions behind torch's public ones where this torch has them (1.2 us less
# in a call of 10 us).  A torch built for no GPU has not, and its tensors
# never get as far as a call.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _stream_of)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _call(name: str, device: torch.device, *args) -> None:
    """Calls an entry point on the current stream of ``device``, which is made
    the current device for its launches."""
    fn = getattr(lib(), name)
    index = device.index
    if index == _current_device():
        st = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(device):
            st = fn(*args, _raw_stream(index))
    if st != B.NS_OK:
        _check(st, name)


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _device(x: torch.Tensor) -> torch.device:
    if not x.is_cuda:
        raise ValueError("expects a device tensor")
    return x.device


def _same_device(device: torch.device, **tensors: Optional[torch.Tensor]) -> None:
    for name, t in tensors.items():
        if t is not None and t.device != device:
            raise ValueError(f"{name} must be on {device}")


def _rows(x: torch.Tensor, name: str) -> Tuple[int, int, int]:
    """(rows, cols, row stride) of a tensor seen as a matrix of its last axis.

    A 2-D tensor may have any row stride; one of another rank is contiguous.
    """
    shape = x.shape
    if not shape:
        raise ValueError(f"{name} must have at least one axis")
    cols = shape[-1]
    if cols < 1:
        raise ValueError(f"{name}'s last axis must not be empty")
    if x.is_contiguous():
        return (shape[0] if len(shape) == 2 else x.numel() // cols), cols, cols
    if len(shape) == 2:
        rows, (ld, step) = shape[0], x.stride()
        if step != 1 and cols > 1:
            raise ValueError(f"{name}'s rows must be contiguous (stride(-1) == 1)")
        if rows > 1 and ld < cols:
            raise ValueError(f"{name}'s rows must not overlap")
        return rows, cols, ld if rows > 1 else cols
    raise ValueError(f"{name} must be contiguous (or 2-D)")


def _output(out: Optional[torch.Tensor], shape, dtype: torch.dtype,
            device: torch.device, name: str) -> Tuple[torch.Tensor, int]:
    """The tensor to write and its row stride."""
    if out is None:
        return torch.empty(shape, dtype=dtype, device=device), shape[-1]
    return _given(out, shape, dtype, device, name)


def _output_like(out: Optional[torch.Tensor], x: torch.Tensor, cols: int,
                 device: torch.device, name: str) -> Tuple[torch.Tensor, int]:
    """The same for a result of x's shape and dtype (empty_like is a third
    cheaper than empty, which counts in calls of 10 us)."""
    if out is None and x.is_contiguous():
        return torch.empty_like(x), cols
    return _output(out, x.shape, x.dtype, device, name)


def _given(out: torch.Tensor, shape, dtype: torch.dtype,
           device: torch.device, name: str) -> Tuple[torch.Tensor, int]:
    if tuple(out.shape) != tuple(shape) or out.dtype != dtype or out.device != device:
        raise ValueError(f"{name} must have shape {tuple(shape)}, {dtype} and device {device}")
    return out, _rows(out, name)[2]


def _status_ptr(status: Optional[torch.Tensor], device: torch.device) -> Optional[int]:
    if status is None:
        return None
    if status.dtype != torch.int32 or not status.is_cuda:
        raise TypeError("status must be a device int32 tensor")
    if status.device != device or status.numel() < 1:
        raise ValueError(f"status must hold a word on {device}")
    return status.data_ptr()


def _workspace_args(need: int, device: torch.device,
                    workspace: Optional[torch.Tensor], query: str):
    if need == 0:
        raise NSError(1, query)
    return B._workspace(need, device, workspace)


def _ids(ids: torch.Tensor, device: torch.device, name: str) -> int:
    """1 for int64 ids, 0 for int32."""
    if ids.dtype not in (torch.int64, torch.int32):
        raise TypeError(f"{name} must be int64 or int32")
    if ids.device != device:
        raise ValueError(f"{name} must be on {device}")
    if not ids.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return 1 if ids.dtype == torch.int64 else 0


def _param(p: Optional[torch.Tensor], x: torch.Tensor, cols: int, name: str) -> None:
    if p is None:
        return
    if p.dtype != x.dtype and p.dtype != torch.float32:
        raise TypeError(f"{name} must have x's dtype or float32")
    if p.device != x.device or p.numel() != cols or not p.is_contiguous():
        raise ValueError(f"{name} must be a contiguous tensor of {cols} elements on {x.device}")


def _per_row(t: torch.Tensor, rows: int, device: torch.device, name: str) -> None:
    if t.dtype != torch.float32:
        raise TypeError(f"{name} must be float32")
    if t.device != device or t.numel() != rows or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous tensor of {rows} elements on {device}")


# ---------------------------------------------------------------------------
# Layer norm.
# ---------------------------------------------------------------------------

def layer_norm(x: torch.Tensor, weight: Optional[torch.Tensor] = None,
               bias: Optional[torch.Tensor] = None, eps: float = 1e-5,
               stats: bool = True, out: Optional[torch.Tensor] = None,
               status: Optional[torch.Tensor] = None):
    """Layer norm over the last axis: returns (y, mean, rstd).

    ``x``: a 2-D tensor with contiguous rows, or a contiguous one of any
    rank.  ``weight`` and ``bias``: x's dtype or float32, both the same.
    ``mean`` and ``rstd`` (fp32, one per row, x's leading axes) are what the
    backward pass takes; with ``stats=False`` they are None.  ``out`` may be
    ``x``.
    """
    device = _device(x)
    rows, cols, ldx = _rows(x, "x")
    code = dtype_code(x.dtype)
    _param(weight, x, cols, "weight")
    _param(bias, x, cols, "bias")
    if weight is not None and bias is not None and weight.dtype != bias.dtype:
        raise TypeError("weight and bias must have the same dtype")
    param = weight if weight is not None else bias
    pcode = code if param is None else dtype_code(param.dtype)
    y, ldy = _output_like(out, x, cols, device, "out")
    mean = rstd = None
    if stats:
        mean = torch.empty((rows,) if x.dim() == 2 else x.shape[:-1],
                           dtype=torch.float32, device=device)
        rstd = torch.empty_like(mean)
    _call("ns_layer_norm", device,
          x.data_ptr(), rows, cols, ldx, code,
          _ptr(weight),
          _ptr(bias), pcode, eps,
          y.data_ptr(), ldy, _ptr(mean),
          _ptr(rstd),
          _status_ptr(status, device))
    return y, mean, rstd


def layer_norm_workspace_size(rows: int, cols: int) -> int:
    return int(lib().ns_layer_norm_workspace_size(rows, cols))


def layer_norm_backward(dy: torch.Tensor, x: torch.Tensor, mean: torch.Tensor,
                        rstd: torch.Tensor,
                        weight: Optional[torch.Tensor] = None,
                        params: bool = True,
                        out: Optional[torch.Tensor] = None,
                        status: Optional[torch.Tensor] = None,
                        workspace: Optional[torch.Tensor] = None):
    """Gradients of layer_norm: returns (dx, dweight, dbias).

    ``mean`` and ``rstd`` as returned by layer_norm.  dweight and dbias have
    weight's dtype (x's without a weight); with ``params=False`` they are
    None.  ``out`` receives dx and may be ``dy``.
    """
    device = _device(x)
    rows, cols, ldx = _rows(x, "x")
    if dy.shape != x.shape or dy.dtype != x.dtype:
        raise ValueError("dy must have x's shape and dtype")
    _same_device(device, dy=dy)
    lddy = _rows(dy, "dy")[2]
    code = dtype_code(x.dtype)
    _per_row(mean, rows, device, "mean")
    _per_row(rstd, rows, device, "rstd")
    _param(weight, x, cols, "weight")
    pdtype = x.dtype if weight is None else weight.dtype
    dx, lddx = _output_like(out, x, cols, device, "out")
    dweight = dbias = keep = None
    wptr, wbytes = None, 0
    if params:
        dweight = torch.empty(cols, dtype=pdtype, device=device)
        dbias = torch.empty_like(dweight)
        wptr, wbytes, keep = _workspace_args(
            int(lib().ns_layer_norm_workspace_size(rows, cols)), device,
            workspace, "ns_layer_norm_workspace_size")
    _call("ns_layer_norm_backward", device,
          dy.data_ptr(), lddy, x.data_ptr(), ldx, rows, cols, code,
          mean.data_ptr(), rstd.data_ptr(),
          _ptr(weight), dtype_code(pdtype),
          dx.data_ptr(), lddx, _ptr(dweight),
          _ptr(dbias),
          _status_ptr(status, device), wptr, wbytes)
    return dx, dweight, dbias


# ---------------------------------------------------------------------------
# Embedding.
# ---------------------------------------------------------------------------

def embedding(ids: torch.Tensor, table: torch.Tensor, scale: float = 1.0,
              out: Optional[torch.Tensor] = None,
              status: Optional[torch.Tensor] = None) -> torch.Tensor:
    """scale * table[ids], of shape ids.shape + (cols,).

    ``ids``: contiguous int64 or int32, any shape; ``table``: [vocab, cols]
    with contiguous rows.  An id outside the table gives a row of zeros and
    sets STATUS_BAD_INDEX in ``status``.
    """
    device = _device(table)
    if table.dim() != 2:
        raise ValueError("table must be 2-D")
    vocab, cols, ldt = _rows(table, "table")
    ids64 = _ids(ids, device, "ids")
    code = dtype_code(table.dtype)
    y, ldo = _output(out, tuple(ids.shape) + (cols,), table.dtype, device, "out")
    _call("ns_embedding", device,
          ids.data_ptr(), ids64, ids.numel(), table.data_ptr(), vocab, cols,
          ldt, code, scale, y.data_ptr(), ldo, _status_ptr(status, device))
    return y


def embedding_workspace_size(n: int, vocab: int, cols: int) -> int:
    return int(lib().ns_embedding_workspace_size(n, vocab, cols))


def embedding_backward(ids: torch.Tensor, dy: torch.Tensor, vocab: int,
                       scale: float = 1.0, out: Optional[torch.Tensor] = None,
                       accumulate: bool = False,
                       status: Optional[torch.Tensor] = None,
                       workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The table's gradient, [vocab, cols]: rows of ``dy`` summed by id.

    ``dy`` has the shape ids.shape + (cols,).  ``out`` receives the gradient;
    with ``accumulate`` it is added to what ``out`` holds (tied embeddings),
    and rows without an id are left alone.
    """
    device = _device(dy)
    ids64 = _ids(ids, device, "ids")
    n, cols, lddy = _rows(dy, "dy")
    if tuple(dy.shape[:-1]) != tuple(ids.shape):
        raise ValueError("dy must have the shape of ids and one more axis")
    if accumulate and out is None:
        raise ValueError("accumulate needs out")
    code = dtype_code(dy.dtype)
    dt, ldt = _output(out, (vocab, cols), dy.dtype, device, "out")
    wptr, wbytes, keep = _workspace_args(
        int(lib().ns_embedding_workspace_size(n, vocab, cols)), device,
        workspace, "ns_embedding_workspace_size")
    _call("ns_embedding_backward", device,
          ids.data_ptr(), ids64, n, dy.data_ptr(), lddy, vocab, cols, code,
          scale, dt.data_ptr(), ldt, 1 if accumulate else 0,
          _status_ptr(status, device), wptr, wbytes)
    return dt


# ---------------------------------------------------------------------------
# Cross entropy of the output projection.
# ---------------------------------------------------------------------------

def _projection(h: torch.Tensor, w: torch.Tensor, targets: torch.Tensor):
    device = _device(h)
    if h.dim() != 2 or w.dim() != 2:
        raise ValueError("h and w must be 2-D")
    rows, cols, ldh = _rows(h, "h")
    vocab, wcols, ldw = _rows(w, "w")
    if wcols != cols or w.dtype != h.dtype:
        raise ValueError("w must have h's dtype and number of columns")
    if vocab < 1:
        raise ValueError("w must have at least one row")
    _same_device(device, w=w)
    t64 = _ids(targets, device, "targets")
    if targets.numel() != rows:
        raise ValueError("targets must have one entry per row of h")
    size = h.element_size()
    aligned = (h.data_ptr() % 16 == 0 and w.data_ptr() % 16 == 0
               and ldh * size % 128 == 0 and ldw * size % 128 == 0)
    return device, rows, cols, ldh, vocab, ldw, t64, 1 if aligned else 0


def linear_cross_entropy_workspace_size(rows: int, cols: int, vocab: int,
                                        dtype: torch.dtype = torch.bfloat16,
                                        aligned: bool = True,
                                        backward: bool = False) -> int:
    """``aligned``: h and w start on 16-byte boundaries and their row strides
    are multiples of 128 bytes (contiguous rows of 64 16-bit or 32 fp32
    elements are)."""
    return int(lib().ns_linear_cross_entropy_workspace_size(
        rows, cols, vocab, dtype_code(dtype), 1 if aligned else 0,
        1 if backward else 0))


def plan_linear_cross_entropy(rows: int, cols: int, vocab: int,
                              dtype: torch.dtype = torch.bfloat16,
                              aligned: bool = True,
                              backward: bool = False) -> List[str]:
    """The kernel builds one call would launch, and for the gradients the
    pieces of the vocabulary and dH's splits (host only, no device)."""
    args = (rows, cols, vocab, dtype_code(dtype), 1 if aligned else 0,
            1 if backward else 0)
    need = int(lib().ns_plan_linear_cross_entropy(*args, None, 0))
    if need < 0:
        raise NSError(1, "ns_plan_linear_cross_entropy")
    buf = ctypes.create_string_buffer(need)
    lib().ns_plan_linear_cross_entropy(*args, buf, need)
    return buf.value.decode().split()


def linear_cross_entropy(h: torch.Tensor, w: torch.Tensor, targets: torch.Tensor,
                         ignore_index: int = -100,
                         status: Optional[torch.Tensor] = None,
                         workspace: Optional[torch.Tensor] = None
                         ) -> Tuple[torch.Tensor, torch.Tensor]:
    """Softmax cross entropy of the logits h w^T: returns (loss, lse), fp32.

    ``h``: [rows, cols] hidden states, ``w``: [vocab, cols] weights, of one
    dtype; ``targets``: rows ids (int64 or int32).  The logits are not
    stored.  A row whose target is ``ignore_index`` has loss 0; another
    target outside the vocabulary gives NaN and sets STATUS_BAD_INDEX.
    """
    device, rows, cols, ldh, vocab, ldw, t64, aligned = _projection(h, w, targets)
    code = dtype_code(h.dtype)
    loss = torch.empty(rows, dtype=torch.float32, device=device)
    lse = torch.empty_like(loss)
    wptr, wbytes, keep = _workspace_args(
        int(lib().ns_linear_cross_entropy_workspace_size(
            rows, cols, vocab, code, aligned, 0)), device, workspace,
        "ns_linear_cross_entropy_workspace_size")
    _call("ns_linear_cross_entropy", device,
          h.data_ptr(), ldh, w.data_ptr(), ldw, targets.data_ptr(), t64, rows,
          cols, vocab, code, ignore_index, loss.data_ptr(), lse.data_ptr(),
          _status_ptr(status, device), wptr, wbytes)
    return loss, lse


def linear_cross_entropy_backward(h: torch.Tensor, w: torch.Tensor,
                                  targets: torch.Tensor, lse: torch.Tensor,
                                  dloss: Union[torch.Tensor, float],
                                  ignore_index: int = -100, need_dh: bool = True,
                                  need_dw: bool = True,
                                  out_dh: Optional[torch.Tensor] = None,
                                  out_dw: Optional[torch.Tensor] = None,
                                  status: Optional[torch.Tensor] = None,
                                  workspace: Optional[torch.Tensor] = None):
    """Gradients of linear_cross_entropy: returns (dh, dw).

    ``lse`` as returned by linear_cross_entropy; ``dloss``: the losses'
    gradients, fp32, one per row, or one number for all of them (1 / valid
    rows for a mean).  ``need_dh`` / ``need_dw`` False skip a gradient and
    return None for it.  The workspace holds a piece of the logits' gradients
    twice and transposed copies of h and of that piece of w, about a copy of w
    however few the rows.
    """
    device, rows, cols, ldh, vocab, ldw, t64, aligned = _projection(h, w, targets)
    code = dtype_code(h.dtype)
    _per_row(lse, rows, device, "lse")
    if not isinstance(dloss, torch.Tensor):
        dloss = torch.full((rows,), float(dloss), dtype=torch.float32, device=device)
    _per_row(dloss, rows, device, "dloss")
    dh = dw = None
    lddh = lddw = cols
    if need_dh:
        dh, lddh = _output_like(out_dh, h, cols, device, "out_dh")
    if need_dw:
        dw, lddw = _output_like(out_dw, w, cols, device, "out_dw")
    wptr, wbytes, keep = _workspace_args(
        int(lib().ns_linear_cross_entropy_workspace_size(
            rows, cols, vocab, code, aligned, 1)), device, workspace,
        "ns_linear_cross_entropy_workspace_size")
    _call("ns_linear_cross_entropy_backward", device,
          h.data_ptr(), ldh, w.data_ptr(), ldw, targets.data_ptr(), t64, rows,
          cols, vocab, code, ignore_index, lse.data_ptr(), dloss.data_ptr(),
          _ptr(dh), lddh,
          _ptr(dw), lddw,
          _status_ptr(status, device), wptr, wbytes)
    return dh, dw
