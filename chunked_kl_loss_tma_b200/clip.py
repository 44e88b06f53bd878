"""The global gradient norm over many tensors, and clipping.

    norm = clip_grad_norm_(grads, 1.0)                      # in place, as a training loop does
    norm = clip_grad_norm_([out["dW"], *rest], 1.0,         # the head's fp32 gradient and the
                           out=[W_grad_bf16, *rest_grads])  # others, clipped into other tensors

Everything is enqueued on the current stream of the tensors' device, and the norm
stays on the device: no synchronisation."""
from __future__ import annotations

import array
import math

import torch
from torch.autograd.graph import increment_version

from . import _lib as L
from .ops import on_device

_DT = {torch.bfloat16: L.KL_DTYPE_BF16, torch.float32: L.KL_DTYPE_F32,
       torch.float16: L.KL_DTYPE_F16}
_PAIR = {t: k | k << 32 for t, k in _DT.items()}  # source and destination alike


def _dense(t):
    """Whether t's elements fill one block of memory, each once, in some order."""
    order = sorted(range(t.dim()), key=t.stride, reverse=True)
    return t.permute(order).is_contiguous()


def _gradient_dtype(t):
    """t's type, where t requires grad: refuses parameters, whose weights would be scaled
    (or overwritten) in place of their gradients."""
    if t.is_leaf:
        raise ValueError("a leaf that requires grad: pass its gradient (p.grad), not the "
                         "parameter")
    return t.dtype


def _list(ts, name, kinds, clip):
    """The tensors' device and what `kinds` names their types; clip: no parameters."""
    if not ts:
        raise ValueError(f"no {name}")
    try:
        where = set(map(torch.Tensor.get_device, ts))
    except TypeError:
        raise ValueError(f"{name} must be tensors") from None
    if len(where) != 1 or where == {-1}:
        raise ValueError(f"{name} must be on one CUDA device")
    try:
        if not clip:
            return ts[0].device, [kinds[t.dtype] for t in ts]
        return ts[0].device, [kinds[_gradient_dtype(t) if t.requires_grad else t.dtype]
                              for t in ts]
    except KeyError:
        raise TypeError(f"{name} must be float32, bfloat16 or float16") from None


def _table(src, dst=None, clip=False):
    """The library's table of the tensors in the lists (an array that stays alive for the
    call), their number and device."""
    if dst is None:
        dev, kinds = _list(src, "gradients", _PAIR, clip)
        if not all(map(torch.Tensor.is_contiguous, src)) and not all(
                t.is_contiguous() or _dense(t) for t in src):
            raise ValueError("a gradient with gaps or repeats in memory")
        to = at = array.array("q", map(torch.Tensor.data_ptr, src))
    else:
        dev, st = _list(src, "gradients", _DT, clip)
        dev_d, dt = _list(dst, "destinations", _DT, clip)
        if len(src) != len(dst) or dev_d != dev:
            raise ValueError(f"{len(src)} gradients on {dev}, {len(dst)} destinations on {dev_d}")
        for s, d in zip(src, dst):
            if s.shape != d.shape or not s.is_contiguous() or not d.is_contiguous():
                raise ValueError("a destination must be contiguous, of its gradient's shape")
        at, to = (array.array("q", map(torch.Tensor.data_ptr, ts)) for ts in (src, dst))
        kinds = [a | b << 32 for a, b in zip(st, dt)]
    # kl_grad: src, dst, n, and the two 32-bit types in one word
    table = array.array("q", bytes(32 * len(src)))
    table[::4], table[1::4] = at, to
    table[2::4] = array.array("q", map(torch.Tensor.numel, src))
    table[3::4] = array.array("q", kinds)
    return table, len(src), dev


def _as_list(ts):
    return [ts] if isinstance(ts, torch.Tensor) else list(ts)


def _norm_type(norm_type):
    if norm_type == 2:
        return L.KL_NORM_2
    if norm_type in (math.inf, "inf"):
        return L.KL_NORM_INF
    raise ValueError("norm_type must be 2 or inf")


def _scratch(n, dev):
    return torch.empty(L.kl_grad_workspace_bytes(n), dtype=torch.uint8, device=dev)


def _norm(grads, norm_type, dtype):
    table, n, dev = _table(_as_list(grads))
    kind, ws = _norm_type(norm_type), _scratch(n, dev)
    out = torch.empty((), dtype=dtype, device=dev)
    total, norm = (out.data_ptr(), None) if dtype == torch.float64 else (None, out.data_ptr())
    on_device(dev, "kl_grad_norm", table.buffer_info()[0], n, kind, ws.data_ptr(), ws.numel(),
              total, norm)
    return out


def grad_norm(grads, *, norm_type=2.0):
    """Norm of all values of the tensors (float32 device scalar): the root of the sum
    of squares, or with norm_type inf the largest magnitude.  Squares beyond float32's
    range count too."""
    return _norm(grads, norm_type, torch.float32)


def grad_total(grads, *, norm_type=2.0):
    """The sum of squares (norm_type 2) or the largest magnitude as a float64 device
    scalar: what ranks that hold parts of the gradients join, for clip_grad_norm_."""
    return _norm(grads, norm_type, torch.float64)


def clip_grad_norm_(grads, max_norm, *, norm_type=2.0, out=None, total=None):
    """Scales the gradients by min(1, max_norm / (norm + 1e-6)) and returns the norm
    before (float32 device scalar).  grads are the gradients themselves, not the
    parameters: a leaf that requires grad is refused.  In place, or into the tensors
    `out`, each rounded once to its type.  In place nothing is written while the norm
    stays under max_norm.  total: the float64 device scalar that grad_total gives (joined
    over ranks, say) in place of the tensors' own.  A NaN norm gives NaN everywhere, an
    infinite one zeros (NaN where a gradient is infinite)."""
    grads, out = _as_list(grads), None if out is None else _as_list(out)
    table, n, dev = _table(grads, out, clip=True)
    kind, ws = _norm_type(norm_type), _scratch(n, dev)
    if total is not None and (not isinstance(total, torch.Tensor) or total.numel() != 1 or
                              total.dtype != torch.float64 or total.device != dev):
        raise ValueError("total must be a float64 scalar on the gradients' device")
    norm = torch.empty((), dtype=torch.float32, device=dev)
    on_device(dev, "kl_grad_clip", table.buffer_info()[0], n, kind, float(max_norm),
              None if total is None else total.data_ptr(), ws.data_ptr(), ws.numel(),
              norm.data_ptr())
    increment_version(grads if out is None else out)  # autograd refuses what was saved before
    return norm
