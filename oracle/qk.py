"""fp64 CPU oracle for rotary positions, the per-head norm of queries and keys,
and gradient clipping.

TEST INFRASTRUCTURE ONLY (never on the product path).

Rotation: the first r elements of a head form r / 2 pairs, (i, i + r/2) or
(2i, 2i + 1) when interleaved; at position p pair i is multiplied, as the
complex number a + i b, by amp exp(i p f_i).  Norm: xh = (x - mu) rstd with mu
= mean(x) ("layer") or 0 ("rms"), rstd = 1 / sqrt(mean((x - mu)^2) + eps), y =
xh gamma + beta, then the rotation.  Written element by element where that is
affordable, and with complex products, unlike the kernels.
"""
from __future__ import annotations

import math

import numpy as np

from . import attention as A


def frequencies(r, base=10000.0, scaling="none", factor=1.0,
                original_length=0.0, slow_turns=1.0, fast_turns=32.0):
    """(f_i [r / 2], amplitude)."""
    if scaling == "ntk" and r > 2:
        base = base * factor ** (r / (r - 2.0))
    out = []
    for i in range(r // 2):
        f = base ** (-2.0 * i / r)
        if scaling == "linear":
            f = f / factor
        if scaling == "yarn":
            turns = original_length * f / (2.0 * math.pi)
            k = (turns - slow_turns) / (fast_turns - slow_turns)
            k = min(1.0, max(0.0, k))
            f = k * f + (1.0 - k) * f / factor
        out.append(f)
    amp = 0.1 * math.log(factor) + 1.0 if scaling == "yarn" else 1.0
    return np.array(out), amp


def rotate(x, positions, freqs, interleaved=False, amp=1.0, inverse=False):
    """x [T, H, d] rotated at positions [T] (the gradient with inverse)."""
    x = np.array(x, dtype=np.float64)
    r = 2 * len(freqs)
    if r == 0:
        return x
    # p f_i modulo a turn, in extended precision where the machine has it
    p = np.asarray(positions).astype(np.longdouble)[:, None]
    angle = np.fmod(p * np.asarray(freqs).astype(np.longdouble),
                    2 * np.longdouble(math.pi)).astype(np.float64)
    z = amp * np.exp((-1j if inverse else 1j) * angle)[:, None, :]
    if interleaved:
        w = (x[..., 0:r:2] + 1j * x[..., 1:r:2]) * z
        x[..., 0:r:2], x[..., 1:r:2] = w.real, w.imag
    else:
        w = (x[..., :r // 2] + 1j * x[..., r // 2:r]) * z
        x[..., :r // 2], x[..., r // 2:r] = w.real, w.imag
    return x


def normal(x, norm, eps):
    """(xh, rstd [.., 1])."""
    x = np.array(x, dtype=np.float64)
    if norm == "layer":
        x = x - x.mean(-1, keepdims=True)
    rstd = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    return x * rstd, rstd


def forward(x, positions, freqs, norm, eps, gamma=None, beta=None,
            interleaved=False, amp=1.0):
    y, _ = normal(x, norm, eps)
    if gamma is not None:
        y = y * np.asarray(gamma, dtype=np.float64)
    if beta is not None:
        y = y + np.asarray(beta, dtype=np.float64)
    return rotate(y, positions, freqs, interleaved, amp)


def backward(dy, x, positions, freqs, norm, eps, gamma=None,
             interleaved=False, amp=1.0):
    """dict dx, dgamma, dbeta."""
    g = rotate(dy, positions, freqs, interleaved, amp, inverse=True)
    xh, rstd = normal(x, norm, eps)
    axes = tuple(range(g.ndim - 1))
    u = g if gamma is None else g * np.asarray(gamma, dtype=np.float64)
    dx = u - xh * (u * xh).mean(-1, keepdims=True)
    if norm == "layer":
        dx = dx - u.mean(-1, keepdims=True)
    return dict(dx=dx * rstd, dgamma=(g * xh).sum(axes), dbeta=g.sum(axes))


def clip(grads, max_norm, eps=1e-6):
    """(norm, factor, scaled gradients); a norm that is not finite scales
    nothing."""
    total = 0.0
    for g in grads:
        total += float(np.sum(np.asarray(g, dtype=np.float64) ** 2))
    norm = math.sqrt(total)
    c = min(1.0, max_norm / (norm + eps)) if math.isfinite(norm) else 1.0
    return norm, c, [np.asarray(g, dtype=np.float64) * c for g in grads]


# ------------------------------------------------- in the attention block --

def attention_forward(X, Wqkv, Wo, heads, seq_len, shards=1, bqkv=None, bo=None,
                      gamma=None, beta=None, eps=1e-5, causal=True,
                      residual=False, positions=None, freqs=(),
                      interleaved=False, amp=1.0, norm=None, qk_eps=1e-6,
                      q_gamma=None, q_beta=None, k_gamma=None, k_beta=None):
    """The unsharded attention block of ``attention.forward`` with each head of
    Q and K normalised (norm "rms" or "layer") and rotated between the
    projection and the core."""
    fwd = A.forward(X, Wqkv, Wo, heads, seq_len, shards, bqkv, bo, gamma, beta,
                    eps, causal, residual)
    T = fwd["QKV"].shape[0]
    if positions is None:
        positions = np.arange(T) % seq_len
    q, k, v = A._split(fwd["QKV"], heads, shards)
    rot = {}
    for name, x, g, b in (("q", q, q_gamma, q_beta), ("k", k, k_gamma, k_beta)):
        rot[name] = (rotate(x, positions, freqs, interleaved, amp)
                     if norm is None else
                     forward(x, positions, freqs, norm, qk_eps, g, b,
                             interleaved, amp))
    o, probs, lse = A.attention_core(rot["q"], rot["k"], v, seq_len, causal)
    ctx = o.reshape(T, -1)
    Z = ctx @ np.asarray(Wo, dtype=np.float64)
    if bo is not None:
        Z = Z + np.asarray(bo, dtype=np.float64)[None, :]
    if residual:
        Z = Z + np.asarray(X, dtype=np.float64)
    return dict(fwd, Z=Z, Ctx=ctx, P=probs, lse=lse, Qr=rot["q"], Kr=rot["k"],
                positions=positions)


def attention_backward(dZ, X, Wqkv, Wo, fwd, heads, seq_len, shards=1,
                       gamma=None, causal=True, residual=False, freqs=(),
                       interleaved=False, amp=1.0, norm=None, qk_eps=1e-6,
                       q_gamma=None, k_gamma=None):
    """Gradients of attention_forward, as ``attention.backward`` plus dq_gamma,
    dq_beta, dk_gamma, dk_beta."""
    f = lambda a: np.asarray(a, dtype=np.float64)
    dZ, X, Wqkv, Wo = f(dZ), f(X), f(Wqkv), f(Wo)
    T = X.shape[0]
    dctx = dZ @ Wo.T
    q, k, v = A._split(fwd["QKV"], heads, shards)
    dqr, dkr, dv = A.core_backward(fwd["Qr"], fwd["Kr"], v,
                                   dctx.reshape(T, heads, -1), fwd["P"],
                                   seq_len)
    out = {}
    grads = {}
    for name, dy, x, g in (("q", dqr, q, q_gamma), ("k", dkr, k, k_gamma)):
        if norm is None:
            grads[name] = rotate(dy, fwd["positions"], freqs, interleaved, amp,
                                 inverse=True)
        else:
            b = backward(dy, x, fwd["positions"], freqs, norm, qk_eps, g,
                         interleaved, amp)
            grads[name] = b["dx"]
            out["d" + name + "_gamma"] = b["dgamma"]
            out["d" + name + "_beta"] = b["dbeta"]
    dqkv = A._merge(grads["q"], grads["k"], dv, shards)
    dXn = dqkv @ Wqkv.T
    dgamma = dbeta = None
    dX = dXn
    if gamma is not None:
        dX, dgamma, dbeta = A.layernorm_backward(dXn, X, fwd["mean"],
                                                 fwd["rstd"], gamma)
    if residual:
        dX = dX + dZ
    return dict(out, dX=dX, dWqkv=fwd["Xn"].T @ dqkv, dbqkv=dqkv.sum(axis=0),
                dWo=fwd["Ctx"].T @ dZ, dbo=dZ.sum(axis=0), dgamma=dgamma,
                dbeta=dbeta, dQKV=dqkv, dCtx=dctx)
