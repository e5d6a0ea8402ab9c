"""The global L2 norm of many gradient tensors, and clipping: wrappers over the
C ABI in include/tp_grad.h.  All arithmetic happens in libtpmlp's kernels.

Gradients are contiguous bf16 or fp32 CUDA tensors of one device, of any number
and shape, in a list or in a dict; of a dict as the blocks' ``backward`` methods
return it, the entry ``dX`` (the gradient of the activations) is left out."""
from __future__ import annotations

import torch

from . import binding as B_
from .rotary import _DTYPES, _on


def _listed(tensors):
    if isinstance(tensors, dict):
        return [t for n, t in tensors.items() if n != "dX"]
    if isinstance(tensors, torch.Tensor):
        return [tensors]
    return list(tensors)


def _table(grads, out):
    """The C table of the tensors, which are checked."""
    device = grads[0].device
    if device.type != "cuda":
        raise ValueError("gradients must be CUDA tensors")
    rows = []
    for i, g in enumerate(grads):
        code = _DTYPES.get(g.dtype)
        if code is None or g.device != device or not g.is_contiguous():
            raise ValueError(f"gradient {i}: expected a contiguous bf16 or "
                             f"fp32 tensor on {device}, got {tuple(g.shape)} "
                             f"{g.dtype} on {g.device}")
        p = g.data_ptr()
        if out is None:
            rows.append((p, p, g.numel(), code))
            continue
        o = out[i]
        if (o.shape != g.shape or o.dtype != g.dtype or o.device != device or
                not o.is_contiguous()):
            raise ValueError(f"out {i}: expected a contiguous "
                             f"{tuple(g.shape)} {g.dtype} tensor on {device}")
        rows.append((p, o.data_ptr(), g.numel(), code))
    return (B_.tp_grad_tensor * len(rows))(*rows)


def _call(tensors, out, stream, call):
    grads = _listed(tensors)
    if not grads:
        raise ValueError("no gradients")
    if out is not None:
        out = _listed(out)
        if len(out) != len(grads):
            raise ValueError(f"out: expected {len(grads)} tensors, got "
                             f"{len(out)}")
    device = grads[0].device
    table = _table(grads, out)

    def run():
        norm = torch.empty((), dtype=torch.float32, device=device)
        nbytes = B_.tp_grad_workspace_bytes(len(grads))
        # of this call alone, as in rotary.py
        ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
        call(len(grads), table, norm, ws, nbytes)
        return norm

    if stream is None and device.index == torch.cuda.current_device():
        return run()
    with _on(device, stream):
        return run()


def grad_norm(tensors, stream=None) -> torch.Tensor:
    """The L2 norm of all elements of all tensors: a 0-dim fp32 tensor on their
    device (the call does not wait for it)."""
    return _call(tensors, None, stream,
                 lambda n, t, norm, ws, size:
                 B_.tp_grad_norm(n, t, norm, ws, size))


def clip_grad_norm(tensors, max_norm: float, eps: float = 1e-6, out=None,
                   stream=None) -> torch.Tensor:
    """Scale all tensors by min(1, max_norm / (norm + eps)), in place or into
    ``out`` (a list or dict of as many tensors), and return the norm they had,
    as grad_norm.  A norm that is not finite is returned and scales nothing."""
    return _call(tensors, out, stream,
                 lambda n, t, norm, ws, size:
                 B_.tp_grad_clip(n, t, max_norm, eps, norm, ws, size))
