"""The rest of a block's training step: AdamW beside Muon, norms, feed-forward.

Argument marshalling for the calls that include/nsortho.h describes under
"The rest of a block's training step", with the conventions of
``_training.py``: the current stream of the tensors' device, no
synchronization, no autograd graph, ValueError or TypeError for arguments
that the library could not use.
"""

from __future__ import annotations

import ctypes
import importlib
from typing import List, Optional, Sequence, Tuple, Union

import torch

from . import _binding as B
from ._binding import NSError, dtype_code, lib
from ._training import _call, _current_device, _device, _raw_stream, _status_ptr

_MARSHAL = None


def _marshal():
    """The host module that checks the arguments of small calls (csrc/marshal.cpp)."""
    global _MARSHAL
    if _MARSHAL is None:
        try:
            _MARSHAL = importlib.import_module("._marshal", __package__)
        except ImportError as e:
            raise RuntimeError("_marshal.so is not built for this Python and torch; run "
                               "`python -m newton_schulz_matrix_amd.build` first") from e
    return _MARSHAL


_ADDRESS = {}  # the entry points' addresses


def _address(name: str) -> int:
    got = _ADDRESS.get(name)
    if got is None:
        got = _ADDRESS[name] = ctypes.cast(getattr(lib(), name), ctypes.c_void_p).value
    return got


def _run(name: str, device: torch.device, status: Optional[torch.Tensor], *args):
    """Checks the arguments of an entry point in the host module and calls it
    on the current stream of ``device``, which is made the current device."""
    args += (None if status is None else _status_ptr(status, device), _raw_stream(device.index))
    fn = getattr(_marshal(), name[3:])
    if device.index == _current_device():
        got = fn(_address(name), *args)
    else:
        with torch.cuda.device(device):
            got = fn(_address(name), *args)
    if type(got) is int:
        B._check(got, name)
    return got


# ---------------------------------------------------------------------------
# AdamW.
# ---------------------------------------------------------------------------
STATE_BLOCK = 256  # elements of an 8-bit moment that share a scale


def adamw_states(params: Sequence[torch.Tensor], bits: int = 32):
    """Zero moments for ``params``: (m, v, scales), lists of one entry each.

    ``bits`` 32: fp32 moments, scales None.  8: e4m3 codes (of m and of
    sqrt(v)) and fp32 scales [2, ceil(numel / 256)], the largest magnitude of
    m and of sqrt(v) in each block of 256 elements; a code stands for
    code * scale / 448.
    """
    if bits not in (8, 32):
        raise ValueError("bits must be 8 or 32")
    dtype = torch.float32 if bits == 32 else torch.float8_e4m3fn
    m = [torch.zeros(p.shape, dtype=dtype, device=p.device) for p in params]
    v = [torch.zeros_like(t) for t in m]
    if bits == 32:
        return m, v, None
    scales = [torch.zeros(2, -(-p.numel() // STATE_BLOCK), dtype=torch.float32, device=p.device)
              for p in params]
    return m, v, scales


def _scalar(t: Optional[torch.Tensor], dtype: torch.dtype, device: torch.device,
            name: str) -> Optional[int]:
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or t.dtype != dtype:
        raise TypeError(f"{name} must be a device {dtype} tensor")
    if t.device != device or t.numel() != 1:
        raise ValueError(f"{name} must hold one element on {device}")
    return t.data_ptr()


def adamw_step(params: Sequence[torch.Tensor], grads: Sequence[torch.Tensor],
               m: Sequence[torch.Tensor], v: Sequence[torch.Tensor],
               lr: Union[float, Sequence[float]], step: Union[int, torch.Tensor],
               betas: Tuple[float, float] = (0.9, 0.95), eps: float = 1e-8,
               weight_decay: Union[float, Sequence[float]] = 0.1,
               scales: Optional[Sequence[Optional[torch.Tensor]]] = None,
               copies: Optional[Sequence[Optional[torch.Tensor]]] = None,
               grad_scale: Optional[torch.Tensor] = None,
               lr_scale: Optional[torch.Tensor] = None,
               status: Optional[torch.Tensor] = None) -> None:
    """One AdamW step over all of ``params``, in place.

    ``params`` and ``grads``: contiguous tensors of bf16, fp16 or fp32, each
    pair of one shape (types may differ).  ``m``, ``v`` and, for 8-bit
    moments, ``scales``: as made by adamw_states (of any shape with as many
    elements); fp32 and 8-bit tensors may
    be mixed, with None in scales for the former.  ``lr`` and
    ``weight_decay``: a number, or one per tensor.  ``step``: 1 for the first
    step, or a device int32 tensor holding it (a captured step reads it when
    it runs; the caller counts it up).  ``copies``: tensors (or None) that
    receive the new parameters in their own type, as the 16-bit weights
    beside fp32 masters.  ``grad_scale`` and ``lr_scale``: device fp32
    factors of all gradients and of all learning rates.
    """
    count = len(params)
    if count == 0:
        return
    device = _device(params[0])
    table = _marshal().adamw_table(params, grads, m, v, scales, copies, lr, weight_decay)
    if isinstance(step, torch.Tensor):
        step_ptr, step = _scalar(step, torch.int32, device, "step"), 0
    else:
        step_ptr = None
        if step < 1:
            raise ValueError("step must be 1 or more")
    _call("ns_adamw_step", device, table, count,
          betas[0], betas[1], eps, int(step), step_ptr,
          _scalar(grad_scale, torch.float32, device, "grad_scale"),
          _scalar(lr_scale, torch.float32, device, "lr_scale"),
          _status_ptr(status, device))


# ---------------------------------------------------------------------------
# Norms before and after a block.
# ---------------------------------------------------------------------------

def residual_norm(residual: torch.Tensor, branch: Optional[torch.Tensor] = None,
                  gate: Optional[torch.Tensor] = None, scale: float = 1.0,
                  branch_weight: Optional[torch.Tensor] = None,
                  weight: Optional[torch.Tensor] = None, norm_branch: bool = True,
                  norm_out: bool = True, eps: float = 1e-6, stats: bool = True,
                  out: Optional[torch.Tensor] = None,
                  out_norm: Optional[torch.Tensor] = None,
                  status: Optional[torch.Tensor] = None):
    """scale * residual + gate * rms_norm(branch), and its RMS norm.

    Returns (stream, normed, branch_rstd, rstd): the new residual stream, the
    next block's input, and what the backward pass takes (fp32, one per row;
    None with ``stats=False`` or without that norm).  ``residual`` and
    ``branch`` (the block's output): one shape and dtype, 2-D with contiguous
    rows or contiguous of any rank.  ``gate``: contiguous, last axis as the
    data's; each of its rows is shared by as many consecutive rows of the
    data (one row: a layer scale; one per sequence; one per token).
    ``branch_weight`` and ``weight`` scale the two norms.  Gate and weights
    have the data's dtype or float32, all the same.  ``norm_branch=False``
    takes the branch as it is (times branch_weight), ``norm_out=False`` gives
    no normed.  Without ``branch`` only normed is computed, the norm of
    ``residual`` itself, which is returned as the stream.  ``out`` (the
    stream) may be ``residual`` and ``out_norm`` may be ``branch``.
    """
    return _run("ns_residual_norm", _device(residual), status, residual, branch, gate, scale, branch_weight, weight,
                norm_branch, norm_out, eps, stats, out, out_norm)


def residual_norm_workspace_size(rows: int, cols: int) -> int:
    return int(lib().ns_residual_norm_workspace_size(rows, cols))


def residual_norm_backward(dstream: Optional[torch.Tensor], dnormed: Optional[torch.Tensor],
                           stream: torch.Tensor, branch: Optional[torch.Tensor] = None,
                           branch_rstd: Optional[torch.Tensor] = None,
                           rstd: Optional[torch.Tensor] = None,
                           gate: Optional[torch.Tensor] = None, scale: float = 1.0,
                           branch_weight: Optional[torch.Tensor] = None,
                           weight: Optional[torch.Tensor] = None, params: bool = True,
                           out: Optional[torch.Tensor] = None,
                           out_branch: Optional[torch.Tensor] = None,
                           status: Optional[torch.Tensor] = None,
                           workspace: Optional[torch.Tensor] = None):
    """Gradients of residual_norm: returns (dresidual, dbranch, dgate, dbranch_weight, dweight).

    ``dstream`` and ``dnormed``: the gradients of stream and normed, either
    None for zeros.  ``stream``, ``branch_rstd`` and ``rstd`` as returned by
    residual_norm (branch_rstd None if the branch was not normed, rstd None
    without dnormed), the other arguments as given to it.  dgate and the
    weights' gradients have their parameter's shape and dtype; they are None
    without that parameter or with ``params=False``.  ``out`` receives
    dresidual and may be ``dstream``; ``out_branch`` receives dbranch and may
    be ``dnormed``.
    """
    return _run("ns_residual_norm_backward", _device(stream), status, _address("ns_residual_norm_workspace_size"),
                dstream, dnormed, stream, branch, branch_rstd, rstd, gate, scale, branch_weight, weight, params, out,
                out_branch, workspace)


# ---------------------------------------------------------------------------
# The gated feed-forward block.
# ---------------------------------------------------------------------------
_ACTIVATIONS = {"silu": 0, "gelu": 1, "gelu_tanh": 2, "relu": 3}


def _activation(name: str) -> int:
    try:
        return _ACTIVATIONS[name]
    except KeyError:
        raise ValueError(f"activation must be one of {', '.join(_ACTIVATIONS)}") from None


def gated_mlp_workspace_size(rows: int, cols: int, inner: int, dtype: torch.dtype = torch.bfloat16,
                             aligned: bool = True, backward: bool = False) -> int:
    """``aligned``: the operands whose rows are whole 128 bytes (x, w_gate and
    w_up by cols, w_down by inner; backward: dy) start on 16-byte boundaries,
    their row strides are multiples of 128 bytes and w_gate's and w_up's are
    the same."""
    return int(lib().ns_gated_mlp_workspace_size(rows, cols, inner, dtype_code(dtype), 1 if aligned else 0,
                                                 1 if backward else 0))


def plan_gated_mlp(rows: int, cols: int, inner: int, dtype: torch.dtype = torch.bfloat16, aligned: bool = True,
                   backward: bool = False) -> List[str]:
    """The kernel builds one call would launch (host only, no device)."""
    args = (rows, cols, inner, dtype_code(dtype), 1 if aligned else 0, 1 if backward else 0)
    need = int(lib().ns_plan_gated_mlp(*args, None, 0))
    if need < 0:
        raise NSError(1, "ns_plan_gated_mlp")
    buf = ctypes.create_string_buffer(need)
    lib().ns_plan_gated_mlp(*args, buf, need)
    return buf.value.decode().split()


def gated_mlp(x: torch.Tensor, w_gate: torch.Tensor, w_up: torch.Tensor, w_down: torch.Tensor,
              activation: str = "silu", save: Union[bool, torch.dtype] = True,
              out: Optional[torch.Tensor] = None,
              status: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None):
    """A gated feed-forward block, (act(x w_gate^T) * (x w_up^T)) w_down^T: returns (y, gate, up).

    ``x``: [..., cols], 2-D with contiguous rows or contiguous of any rank;
    ``w_gate`` and ``w_up``: [inner, cols], ``w_down``: [cols, inner], all of
    x's dtype.  ``activation``: "silu", "gelu", "gelu_tanh" or "relu".
    ``gate`` and ``up``, [..., inner], are the two projections that the
    backward pass takes, in float32; ``save`` may name x's dtype instead,
    which halves their memory and doubles the gradients' rounding error.
    With ``save=False`` they are None.
    """
    device, act = _device(x), _activation(activation)
    if save is True:
        save = torch.float32
    if save is False:
        save = None
    elif save != torch.float32 and save != x.dtype:
        raise TypeError("save must be True, False, torch.float32 or x's dtype")
    else:
        save = save == torch.float32
    return _run("ns_gated_mlp", device, status, _address("ns_gated_mlp_workspace_size"), x, w_gate, w_up, w_down, act,
                save, out, workspace)


def gated_mlp_backward(dy: torch.Tensor, x: torch.Tensor, w_gate: torch.Tensor, w_up: torch.Tensor,
                       w_down: torch.Tensor, gate: torch.Tensor, up: torch.Tensor, activation: str = "silu",
                       need_dx: bool = True, need_dw: bool = True, out_dx: Optional[torch.Tensor] = None,
                       out_dw_gate: Optional[torch.Tensor] = None, out_dw_up: Optional[torch.Tensor] = None,
                       out_dw_down: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
                       workspace: Optional[torch.Tensor] = None):
    """Gradients of gated_mlp: returns (dx, dw_gate, dw_up, dw_down).

    ``gate`` and ``up`` as returned by gated_mlp.  ``need_dx`` / ``need_dw``
    False skip dx or the weights' gradients and return None for them.  The
    workspace holds the gradients of gate and up twice, h, and transposed
    copies of x, dy and the weights.
    """
    return _run("ns_gated_mlp_backward", _device(x), status, _address("ns_gated_mlp_workspace_size"), x, w_gate, w_up,
                w_down, dy, gate, up, _activation(activation), need_dx, need_dw, out_dx, out_dw_gate, out_dw_up,
                out_dw_down, workspace)
