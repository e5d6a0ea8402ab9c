"""The global L2 norm of many gradient tensors, and clipping: wrappers over the
C ABI in include/tp_grad.h.  csrc/pycall.cpp checks the tensors; all arithmetic
happens in libtpmlp's kernels.

Gradients are contiguous bf16 or fp32 CUDA tensors of one device, of any number
and shape, in a list or in a dict; of a dict as the ``backward`` methods of the
blocks and of QKNormRotary return it, the gradients of the activations (``dX``;
``dq`` and ``dk``) are left out.

With ``stream`` the work, and the norm's memory, belong to that stream;
otherwise to the current one of the tensors' device."""
from __future__ import annotations

import torch

from . import binding as B_


_ACTIVATIONS = ("dX", "dq", "dk")


def _listed(tensors):
    if isinstance(tensors, dict):
        return [t for n, t in tensors.items() if n not in _ACTIVATIONS]
    if isinstance(tensors, torch.Tensor):
        return [tensors]
    return tensors if isinstance(tensors, (list, tuple)) else list(tensors)


def grad_norm(tensors, stream=None) -> torch.Tensor:
    """The L2 norm of all elements of all tensors: a 0-dim fp32 tensor on their
    device (the call does not wait for it)."""
    return B_.tensor_calls().grads(_listed(tensors), None, 0, 0.0, 0.0, stream)


def clip_grad_norm(tensors, max_norm: float, eps: float = 1e-6, out=None,
                   stream=None) -> torch.Tensor:
    """Scale all tensors by min(1, max_norm / (norm + eps)), in place or into
    ``out`` (a list of as many tensors, or for a dict a dict with its names), and
    return the norm they had, as grad_norm.  A norm that is not finite is
    returned and scales nothing."""
    if isinstance(tensors, dict) and isinstance(out, dict):
        names = [n for n in tensors if n not in _ACTIVATIONS]
        missing = [n for n in names if n not in out]
        if missing:
            raise ValueError(f"out has no {missing}")
        out = [out[n] for n in names]
    return B_.tensor_calls().grads(
        _listed(tensors), None if out is None else _listed(out), 1, max_norm,
        eps, stream)
