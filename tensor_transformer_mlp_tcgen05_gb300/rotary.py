"""Rotary positions and the per-head norm of queries and keys: object wrappers
over the C ABI in include/tp_rope.h, which check shapes, types and devices.  All
arithmetic happens in libtpmlp's kernels.

Queries and keys are bf16 or fp32 CUDA tensors whose head elements are
consecutive, with any strides otherwise: ``[T, heads, d]``, or ``[T, shards,
heads per shard, d]``, as a view of the attention block's projection has them
(``qkv.view(T, t, 3, H // t, d)[:, :, 0]`` are the queries).  T counts tokens.

Every call takes the tokens' positions in one of three ways: ``positions``, an
int32 or int64 tensor [T]; ``seq_len``, so that token t is at ``offset + t %
seq_len``; or neither, for ``offset + t``.

Outputs are made new unless given (``q_out``, ``k_out``; the input itself for a
call in place).  With ``stream`` the work, and the outputs' memory, belong to
that stream; otherwise to the current one of the tensors' device.  The caller
keeps the inputs alive until that stream has read them.
"""
from __future__ import annotations

import contextlib
import ctypes

import torch

from . import binding as B_

_DTYPES = {torch.bfloat16: B_.TPMLP_BF16, torch.float32: B_.TPMLP_FP32}
_SCALINGS = {"none": B_.TPROPE_SCALE_NONE, "linear": B_.TPROPE_SCALE_LINEAR,
             "ntk": B_.TPROPE_SCALE_NTK, "yarn": B_.TPROPE_SCALE_YARN}
_NORMS = {"rms": B_.TPQK_RMSNORM, "layer": B_.TPQK_LAYERNORM}


@contextlib.contextmanager
def _on(device, stream):
    """The device and the stream (None: the device's current one) that a call
    belongs to."""
    with torch.cuda.device(device):
        if stream is None:
            stream = torch.cuda.current_stream(device)
        elif isinstance(stream, int):
            stream = torch.cuda.ExternalStream(stream, device=device)
        if stream.device != device:
            raise ValueError(f"the stream belongs to {stream.device}, the "
                             f"tensors to {device}")
        with torch.cuda.stream(stream):
            yield


def _heads(name, x, d, like=None):
    """(tp_heads of x, tokens); like: the tensor that x has to match."""
    shape, stride = x.shape, x.stride()
    if like is not None:
        if shape != like.shape or x.dtype != like.dtype:
            raise ValueError(f"{name}: expected {tuple(like.shape)} "
                             f"{like.dtype}, got {tuple(shape)} {x.dtype}")
        if x.device != like.device:
            raise ValueError(f"{name} is on {x.device}, not {like.device}")
    elif x.dtype not in _DTYPES or x.device.type != "cuda":
        raise ValueError(f"{name} must be a bf16 or fp32 CUDA tensor")
    n = len(shape)
    if n not in (3, 4) or shape[-1] != d or (stride[-1] != 1 and d != 1):
        raise ValueError(
            f"{name}: expected [T, heads, {d}] or [T, shards, heads, {d}] with "
            f"consecutive head elements, got {tuple(shape)}, strides {stride}")
    if n == 3:
        h = shape[1]
        return B_.tp_heads(x.data_ptr(), stride[0], 0, stride[1], h, h)
    return B_.tp_heads(x.data_ptr(), stride[0], stride[1], stride[2],
                       shape[1] * shape[2], shape[2])


class RotaryEmbedding:
    """Rotary positions: the first ``rotary_dim`` elements (default: all) of
    every head turn pair by pair, pairs (i, i + rotary_dim / 2), or (2i, 2i + 1)
    with ``interleaved``.

    Frequencies: base^(-2i / rotary_dim), scaled for contexts longer than the
    trained one by ``scaling``: "linear" (divided by ``factor``), "ntk" (the
    base raised) or "yarn" (by the turns a pair makes over
    ``original_length``, see include/tp_rope.h); or any ``inv_freq``, a
    sequence of rotary_dim / 2 numbers.  ``amplitude`` scales the rotated
    elements (default 1; "yarn": 0.1 ln(factor) + 1)."""

    def __init__(self, head_dim: int, rotary_dim: int | None = None,
                 base: float = 10000.0, interleaved: bool = False,
                 scaling: str = "none", factor: float = 1.0,
                 original_length: float = 0.0, slow_turns: float = 1.0,
                 fast_turns: float = 32.0, amplitude: float = 0.0,
                 inv_freq=None):
        if scaling not in _SCALINGS:
            raise ValueError(f"scaling must be one of {sorted(_SCALINGS)}")
        r = head_dim if rotary_dim is None else rotary_dim
        freqs, code = None, _SCALINGS[scaling]
        if inv_freq is not None:
            if scaling != "none":
                raise ValueError("inv_freq excludes scaling")
            values = [float(f) for f in inv_freq]
            if len(values) != r // 2:
                raise ValueError(f"inv_freq: expected {r // 2} values, got "
                                 f"{len(values)}")
            freqs, code = (ctypes.c_double * max(1, len(values)))(*values), \
                B_.TPROPE_SCALE_CUSTOM
        self.cfg = B_.tp_rope_config(
            head_dim=head_dim, rot_dim=r, interleaved=1 if interleaved else 0,
            scaling=code, base=base, factor=factor,
            original_length=original_length, slow_turns=slow_turns,
            fast_turns=fast_turns, amplitude=amplitude, inv_freq=freqs)
        self.handle = None
        self.handle = B_.tp_rope_create(self.cfg)
        self.head_dim, self.rotary_dim = head_dim, r

    def close(self):
        if self.handle:
            B_.tp_rope_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def frequencies(self):
        """(the rotary_dim / 2 angles per position in radians, amplitude)."""
        return B_.tp_rope_frequencies(self.handle, self.rotary_dim)

    def _where(self, q, positions, offset, seq_len):
        if positions is None:
            return B_.tp_positions(None, 0, offset, seq_len)
        T = q.shape[0]
        if (positions.shape != (T,) or positions.device != q.device or
                positions.dtype not in (torch.int32, torch.int64) or
                not positions.is_contiguous()):
            raise ValueError(f"positions: expected a contiguous int32 or int64 "
                             f"tensor [{T}] on {q.device}")
        return B_.tp_positions(positions.data_ptr(),
                               1 if positions.dtype == torch.int64 else 0, 0, 0)

    def _views(self, q, k, q_out, k_out):
        """The views of a call's tensors, and its outputs."""
        d = self.head_dim
        vq = _heads("q", q, d)
        if q_out is None:
            q_out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        wq = _heads("q_out", q_out, d, q)
        if k is None:
            if k_out is not None:
                raise ValueError("k_out without k")
            return vq, wq, None, None, q_out, None
        vk = _heads("k", k, d)
        if (k.shape[0] != q.shape[0] or k.dtype != q.dtype or
                k.device != q.device):
            raise ValueError("q and k differ in tokens, type or device")
        if k_out is None:
            k_out = torch.empty(k.shape, dtype=k.dtype, device=k.device)
        return vq, wq, vk, _heads("k_out", k_out, d, k), q_out, k_out

    def _apply(self, inverse, q, k, positions, offset, seq_len, q_out, k_out,
               stream):
        if stream is not None or q.device.index != torch.cuda.current_device():
            with _on(q.device, stream):
                return self._apply(inverse, q, k, positions, offset, seq_len,
                                   q_out, k_out, None)
        vq, wq, vk, wk, q_out, k_out = self._views(q, k, q_out, k_out)
        B_.tp_rope_apply(self.handle, q.shape[0], _DTYPES[q.dtype], inverse,
                         vq, wq, vk, wk,
                         self._where(q, positions, offset, seq_len))
        return q_out, k_out

    def forward(self, q, k=None, positions=None, offset: int = 0,
                seq_len: int = 0, q_out=None, k_out=None, stream=None):
        """(q, k) rotated; k may be None."""
        return self._apply(0, q, k, positions, offset, seq_len, q_out, k_out,
                           stream)

    def backward(self, dq, dk=None, positions=None, offset: int = 0,
                 seq_len: int = 0, q_out=None, k_out=None, stream=None):
        """The gradients with respect to forward's q and k."""
        return self._apply(1, dq, dk, positions, offset, seq_len, q_out, k_out,
                           stream)


class QKNormRotary:
    """Every head of the queries and keys normalised ("rms", or "layer": with
    the mean taken off) and then rotated, in one pass.  ``gamma`` [d] and
    ``beta`` [d] (fp32, None for ones and zeros; "rms" has no beta) are shared
    by the heads of q, and others by those of k.  ``rotary`` None: no
    rotation."""

    def __init__(self, head_dim: int, norm: str = "rms", eps: float = 1e-6,
                 rotary: RotaryEmbedding | None = None):
        if norm not in _NORMS:
            raise ValueError(f"norm must be one of {sorted(_NORMS)}")
        if rotary is None:
            rotary = RotaryEmbedding(head_dim, rotary_dim=0)
        if rotary.head_dim != head_dim:
            raise ValueError(f"rotary is for heads of {rotary.head_dim}, not "
                             f"{head_dim}")
        self.rotary, self.head_dim, self.norm, self.eps = (rotary, head_dim,
                                                           norm, eps)

    def _param(self, name, p, q):
        if p is None:
            return None
        if (p.dtype != torch.float32 or p.shape != (self.head_dim,) or
                p.device != q.device or not p.is_contiguous()):
            raise ValueError(f"{name}: expected a contiguous fp32 tensor "
                             f"[{self.head_dim}] on {q.device}")
        return p.data_ptr()

    def _norm(self, q, q_gamma, k_gamma, q_beta, k_beta):
        return B_.tp_qk_norm(
            _NORMS[self.norm], self.eps, self._param("q_gamma", q_gamma, q),
            self._param("q_beta", q_beta, q),
            self._param("k_gamma", k_gamma, q),
            self._param("k_beta", k_beta, q))

    def forward(self, q, k=None, q_gamma=None, k_gamma=None, q_beta=None,
                k_beta=None, positions=None, offset: int = 0, seq_len: int = 0,
                q_out=None, k_out=None, stream=None):
        """(q, k) normalised and rotated; k may be None."""
        if stream is not None or q.device.index != torch.cuda.current_device():
            with _on(q.device, stream):
                return self.forward(q, k, q_gamma, k_gamma, q_beta, k_beta,
                                    positions, offset, seq_len, q_out, k_out)
        r = self.rotary
        vq, wq, vk, wk, q_out, k_out = r._views(q, k, q_out, k_out)
        B_.tp_qk_norm_forward(
            r.handle, q.shape[0], _DTYPES[q.dtype],
            self._norm(q, q_gamma, k_gamma, q_beta, k_beta), vq, wq, vk, wk,
            r._where(q, positions, offset, seq_len))
        return q_out, k_out

    def backward(self, dq, dk, q, k, q_gamma=None, k_gamma=None,
                 positions=None, offset: int = 0, seq_len: int = 0,
                 param_grads: bool = True, out=None, stream=None):
        """Gradients from dq, dk (of the rotated heads) and forward's q, k: a
        dict with dq, dk and (with param_grads) dq_gamma, dk_gamma and, for
        "layer", dq_beta, dk_beta.  ``out`` may hold any of them; out["dq"] may
        be dq or q themselves.  dk and k are None together."""
        if stream is not None or dq.device.index != torch.cuda.current_device():
            with _on(dq.device, stream):
                return self.backward(dq, dk, q, k, q_gamma, k_gamma, positions,
                                     offset, seq_len, param_grads, out)
        if (dk is None) != (k is None):
            raise ValueError("dk and k must be given together")
        d, r = self.head_dim, self.rotary
        g = out if out is not None else {}
        vq, wq, vk, wk, g["dq"], dk_out = r._views(dq, dk, g.get("dq"),
                                                   g.get("dk"))
        xq = _heads("q", q, d, dq)
        xk = None
        if k is not None:
            xk = _heads("k", k, d, dk)
            g["dk"] = dk_out
        grads = ws = None
        nbytes = 0
        if param_grads:
            grads = B_.tp_qk_norm_grads()
            names = ("q_gamma", "q_beta", "k_gamma", "k_beta")
            for name in names[:2 if k is None else 4]:
                if name.endswith("beta") and self.norm != "layer":
                    continue
                if g.get("d" + name) is None:
                    g["d" + name] = torch.empty(d, dtype=torch.float32,
                                                device=dq.device)
                setattr(grads, name, self._param("d" + name, g["d" + name], dq))
            nbytes = B_.tp_qk_norm_workspace_bytes(r.handle)
            # of this call alone: calls on several streams, and captured
            # graphs, share no partial sums
            ws = torch.empty(nbytes, dtype=torch.uint8, device=dq.device)
        B_.tp_qk_norm_backward(
            r.handle, dq.shape[0], _DTYPES[dq.dtype],
            self._norm(dq, q_gamma, k_gamma, None, None), vq, xq, wq, vk, xk,
            wk, r._where(dq, positions, offset, seq_len), grads, ws, nbytes)
        return g
