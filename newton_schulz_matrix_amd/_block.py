"""The rest of a block's training step: AdamW beside Muon, norms, feed-forward.

Argument marshalling for the calls that include/nsortho.h describes under
"The rest of a block's training step", with the conventions of
``_training.py``: the current stream of the tensors' device, no
synchronization, no autograd graph, ValueError or TypeError for arguments
that the library could not use.
"""

from __future__ import annotations

import ctypes
import struct
from typing import List, Optional, Sequence, Tuple, Union

import torch

from . import _binding as B
from ._training import _call, _device, _status_ptr

# ---------------------------------------------------------------------------
# AdamW.
# ---------------------------------------------------------------------------
STATE_BLOCK = 256  # elements of an 8-bit moment that share a scale

_TENSOR = struct.Struct("=6Qq2f4i")  # ns_adamw_tensor

_MOMENT_TYPES = {torch.float32: False, torch.float8_e4m3fn: True}


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


def _per_tensor(value, count: int, name: str) -> Sequence[float]:
    if isinstance(value, (int, float)):
        return (value,) * count
    if len(value) != count:
        raise ValueError(f"{name} must be one number or one per tensor")
    return value


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
    moments, ``scales``: as made by adamw_states; fp32 and 8-bit tensors may
    be mixed, with None in scales for the former.  ``lr`` and
    ``weight_decay``: a number, or one per tensor.  ``step``: 1 for the first
    step, or a device int32 tensor holding it (a captured step reads it when
    it runs; the caller counts it up).  ``copies``: tensors (or None) that
    receive the new parameters in their own type, as the 16-bit weights
    beside fp32 masters.  ``grad_scale`` and ``lr_scale``: device fp32
    factors of all gradients and of all learning rates.
    """
    count = len(params)
    if not (len(grads) == len(m) == len(v) == count):
        raise ValueError("params, grads, m and v must have one entry per tensor")
    for name, given in (("scales", scales), ("copies", copies)):
        if given is not None and len(given) != count:
            raise ValueError(f"{name} must have one entry (or None) per tensor")
    rates = _per_tensor(lr, count, "lr")
    decays = _per_tensor(weight_decay, count, "weight_decay")
    if count == 0:
        return
    device = _device(params[0])
    codes = B._DTYPE_CODE
    table = bytearray(_TENSOR.size * count)
    pack, size = _TENSOR.pack_into, _TENSOR.size
    written = []
    for i in range(count):
        p, g, mi, vi = params[i], grads[i], m[i], v[i]
        n, shape = p.numel(), p.shape
        if not (p.dtype in codes and g.dtype in codes):
            raise TypeError("params and grads must be bf16, fp16 or fp32")
        coded = _MOMENT_TYPES.get(mi.dtype)
        if coded is None or vi.dtype != mi.dtype:
            raise TypeError("m and v must both be float32 or both float8_e4m3fn")
        if not (g.shape == shape and mi.shape == shape and vi.shape == shape):
            raise ValueError("grads, m and v must have their parameter's shape")
        if not (p.device == device and g.device == device and mi.device == device and vi.device == device):
            raise ValueError(f"every tensor must be on {device}")
        if not (p.is_contiguous() and g.is_contiguous() and mi.is_contiguous() and vi.is_contiguous()):
            raise ValueError("every tensor must be contiguous")
        pp, pm, pv, ps, pc, ct = p.data_ptr(), mi.data_ptr(), vi.data_ptr(), 0, 0, 0
        si = scales[i] if scales is not None else None
        if (si is not None) != coded:
            raise ValueError("scales go with float8_e4m3fn moments, one tensor each")
        if coded:
            blocks = -(-n // STATE_BLOCK)
            if si.dtype != torch.float32 or si.numel() != 2 * blocks or not si.is_contiguous() or si.device != device:
                raise ValueError(f"scales must be contiguous float32 tensors [2, ceil(numel / {STATE_BLOCK})] "
                                 f"on {device}")
            ps = si.data_ptr()
        ci = copies[i] if copies is not None else None
        if ci is not None:
            if ci.dtype not in codes or ci.shape != shape or ci.device != device or not ci.is_contiguous():
                raise ValueError("copies must be contiguous bf16, fp16 or fp32 tensors of their parameter's shape")
            pc, ct = ci.data_ptr(), codes[ci.dtype]
        if n:
            written += (pp, pm, pv)
            if ps:
                written.append(ps)
            if pc:
                written.append(pc)
        pack(table, i * size, pp, g.data_ptr(), pm, pv, ps, pc, n, rates[i], decays[i], codes[p.dtype],
             codes[g.dtype], ct, 0)
    if len(set(written)) != len(written):
        raise ValueError("a tensor is given twice")
    if isinstance(step, torch.Tensor):
        step_ptr, step = _scalar(step, torch.int32, device, "step"), 0
    else:
        step_ptr = None
        if step < 1:
            raise ValueError("step must be 1 or more")
    _call("ns_adamw_step", device, (ctypes.c_char * len(table)).from_buffer(table), count,
          betas[0], betas[1], eps, int(step), step_ptr,
          _scalar(grad_scale, torch.float32, device, "grad_scale"),
          _scalar(lr_scale, torch.float32, device, "lr_scale"),
          _status_ptr(status, device))
