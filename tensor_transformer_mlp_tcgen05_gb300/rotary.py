"""Rotary positions and the per-head norm of queries and keys: object wrappers
over the C ABI in include/tp_rope.h.  csrc/pycall.cpp checks shapes, types and
devices; all arithmetic happens in libtpmlp's kernels.

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

import ctypes

import torch   # noqa: F401  (the tensor calls need its libraries loaded)

from . import binding as B_

_SCALINGS = {"none": B_.TPROPE_SCALE_NONE, "linear": B_.TPROPE_SCALE_LINEAR,
             "ntk": B_.TPROPE_SCALE_NTK, "yarn": B_.TPROPE_SCALE_YARN}
_GRADS = ("dq", "dk", "dq_gamma", "dq_beta", "dk_gamma", "dk_beta")
_NORMS = {"rms": B_.TPQK_RMSNORM, "layer": B_.TPQK_LAYERNORM}


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
        self._calls = B_.tensor_calls()

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

    def forward(self, q, k=None, positions=None, offset: int = 0,
                seq_len: int = 0, q_out=None, k_out=None, stream=None):
        """(q, k) rotated; k may be None."""
        return self._calls.rope(self.handle, self.head_dim, 0, q, k, positions,
                                offset, seq_len, q_out, k_out, stream)

    def backward(self, dq, dk=None, positions=None, offset: int = 0,
                 seq_len: int = 0, q_out=None, k_out=None, stream=None):
        """The gradients with respect to forward's q and k."""
        return self._calls.rope(self.handle, self.head_dim, 1, dq, dk,
                                positions, offset, seq_len, q_out, k_out,
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
        self._code = _NORMS[norm]

    def forward(self, q, k=None, q_gamma=None, k_gamma=None, q_beta=None,
                k_beta=None, positions=None, offset: int = 0, seq_len: int = 0,
                q_out=None, k_out=None, stream=None):
        """(q, k) normalised and rotated; k may be None."""
        r = self.rotary
        return r._calls.norm_forward(
            r.handle, self.head_dim, self._code, self.eps, q, k, q_gamma,
            q_beta, k_gamma, k_beta, positions, offset, seq_len, q_out, k_out,
            stream)

    def backward(self, dq, dk, q, k, q_gamma=None, k_gamma=None,
                 positions=None, offset: int = 0, seq_len: int = 0,
                 param_grads: bool = True, out=None, stream=None):
        """Gradients from dq, dk (of the rotated heads) and forward's q, k: a
        dict with dq, dk and (with param_grads) dq_gamma, dk_gamma and, for
        "layer", dq_beta, dk_beta.  ``out`` may hold any of them, and no gradient
        that the call does not have; out["dq"] may be dq or q themselves.  dk and
        k are None together."""
        r = self.rotary
        g = out if out is not None else {}
        get = g.get
        made = r._calls.norm_backward(
            r.handle, self.head_dim, self._code, self.eps, dq, dk, q, k,
            q_gamma, k_gamma, positions, offset, seq_len, get("dq"), get("dk"),
            param_grads, get("dq_gamma"), get("dq_beta"), get("dk_gamma"),
            get("dk_beta"), stream)
        for name, t in zip(_GRADS, made):
            if t is not None:
                g[name] = t
        return g
