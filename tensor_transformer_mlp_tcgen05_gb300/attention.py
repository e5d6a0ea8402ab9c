"""A small object wrapper over the attention block's C ABI (tp_attn_*):
owns a handle and a workspace tensor, checks shapes, dtypes and devices, and
calls tp_attn_forward / tp_attn_backward.  All arithmetic happens in
libtpmlp's kernels; PyTorch only provides device memory and the stream."""
from __future__ import annotations

import torch

from . import binding as B_
from .rotary import _NORMS


class TensorParallelAttention:
    """Head-parallel self-attention block with t logical shards: W_qkv split
    by columns head group by head group ([Q_i | K_i | V_i] per shard), W_o by
    rows, the shard partials summed in a fixed order.  Optionally the whole
    pre-LN sub-block X + Attn(LN(X)); with ``rotary`` (a
    rotary.RotaryEmbedding for heads of hidden / heads) rotary positions on Q
    and K, with ``qk_norm`` ("rms" or "layer") their heads normalised before
    that."""

    def __init__(self, hidden: int, heads: int, shards: int, max_tokens: int,
                 seq_len: int, causal: bool = True, layernorm: bool = False,
                 ln_eps: float = 1e-5, residual: bool = False, device=None,
                 ln_prologue: bool = True, rotary=None,
                 qk_norm: str | None = None, qk_norm_eps: float = 1e-6):
        if qk_norm is not None and qk_norm not in _NORMS:
            raise ValueError(f"qk_norm must be one of {sorted(_NORMS)} or None")
        self.handle = None
        self.cfg = B_.tp_attn_config(
            hidden=hidden, heads=heads, shards=shards, max_tokens=max_tokens,
            seq_len=seq_len, causal=1 if causal else 0,
            use_layernorm=1 if layernorm else 0, ln_eps=ln_eps,
            use_residual=1 if residual else 0)
        self.handle = B_.tp_attn_create(self.cfg)
        if not ln_prologue:   # the LayerNorm as its own launch before QKV
            B_.tp_attn_set_ln_prologue(self.handle, False)
        if rotary is not None:
            B_.tp_attn_set_rope(self.handle, rotary.cfg)
        if qk_norm is not None:
            B_.tp_attn_set_qk_norm(self.handle, _NORMS[qk_norm], qk_norm_eps)
        self.rotary, self.qk_norm = rotary, qk_norm
        self.hidden, self.heads, self.shards = hidden, heads, shards
        self.seq_len = seq_len
        self.layernorm = layernorm
        self.device = torch.device(device or "cuda")
        self._ws = None

    def close(self):
        if self.handle:
            B_.tp_attn_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def workspace(self, tokens: int, training: bool = True) -> torch.Tensor:
        need = B_.tp_attn_workspace_bytes(self.handle, tokens,
                                          1 if training else 0)
        if self._ws is None or self._ws.numel() < need:
            self._ws = torch.empty(max(need, 256), dtype=torch.uint8,
                                   device=self.device)
        return self._ws

    def saved(self, tokens: int, which: str, training: bool = True):
        """A view of an intermediate kept in the workspace: "qkv" [T, 3h]
        bf16, "ctx" [T, h] bf16, "lse2" [H, T] fp32 (base-2 log-sum-exp of
        the scores scaled by log2(e)/sqrt(d)), "dqkv" [T, 3h] bf16, or "qkr"
        [T, 3h] bf16: Q and K as the core reads them (see TPATTN_WS_QKR in
        include/tp_attn.h)."""
        code = {"qkr": B_.TPATTN_WS_QKR, "qkv": B_.TPATTN_WS_QKV, "ctx": B_.TPATTN_WS_CTX,
                "lse2": B_.TPATTN_WS_LSE, "dqkv": B_.TPATTN_WS_DQKV}[which]
        off = B_.tp_attn_workspace_offset(self.handle, tokens,
                                          1 if training else 0, code)
        if off < 0 or self._ws is None:
            raise ValueError(f"{which} is not in this workspace")
        h, H = self.hidden, self.heads
        shape, dt = {"qkr": ((tokens, 3 * h), torch.bfloat16),
                     "qkv": ((tokens, 3 * h), torch.bfloat16),
                     "ctx": ((tokens, h), torch.bfloat16),
                     "lse2": ((H, tokens), torch.float32),
                     "dqkv": ((tokens, 3 * h), torch.bfloat16)}[which]
        n = shape[0] * shape[1] * (2 if dt == torch.bfloat16 else 4)
        return self._ws[off:off + n].view(dt).view(*shape)

    @staticmethod
    def _chk(name, t, shape, dtype):
        if t is None:
            return
        if tuple(t.shape) != tuple(shape) or t.dtype != dtype:
            raise ValueError(f"{name}: expected {tuple(shape)} {dtype}, got "
                             f"{tuple(t.shape)} {t.dtype}")
        if not t.is_contiguous() or t.device.type != "cuda":
            raise ValueError(f"{name} must be a contiguous CUDA tensor")

    def _qk(self, T, q_gamma, k_gamma, q_beta, k_beta, positions):
        """The tp_attn_qk of a call (None without norm and rotation)."""
        given = (q_gamma, k_gamma, q_beta, k_beta, positions)
        if all(t is None for t in given):
            return None
        d = (self.hidden // self.heads,)
        for name, t in zip(("q_gamma", "k_gamma", "q_beta", "k_beta"), given):
            if t is not None and self.qk_norm is None:
                raise ValueError(f"{name} without qk_norm")
            self._chk(name, t, d, torch.float32)
        if positions is not None:
            if self.rotary is None:
                raise ValueError("positions without rotary")
            self._chk("positions", positions, (T,),
                      torch.int64 if positions.dtype == torch.int64
                      else torch.int32)
        ptr = lambda t: None if t is None else t.data_ptr()
        return B_.tp_attn_qk(
            ptr(positions),
            1 if positions is not None and positions.dtype == torch.int64 else 0,
            ptr(q_gamma), ptr(q_beta), ptr(k_gamma), ptr(k_beta))

    def forward(self, X, Wqkv, Wo, bqkv=None, bo=None, gamma=None, beta=None,
                training: bool = True, out=None, stream=None, q_gamma=None,
                k_gamma=None, q_beta=None, k_beta=None, positions=None):
        """``positions`` (int32 or int64 [T], with ``rotary``) default to each
        token's place in its sequence; q_gamma .. k_beta (fp32 [d], with
        ``qk_norm``) to ones and zeros."""
        T = X.shape[0]
        h = self.hidden
        bf = torch.bfloat16
        self._chk("X", X, (T, h), bf)
        self._chk("Wqkv", Wqkv, (h, 3 * h), bf)
        self._chk("Wo", Wo, (h, h), bf)
        self._chk("bqkv", bqkv, (3 * h,), torch.float32)
        self._chk("bo", bo, (h,), torch.float32)
        self._chk("gamma", gamma, (h,), torch.float32)
        self._chk("beta", beta, (h,), torch.float32)
        Z = out if out is not None else torch.empty((T, h), dtype=bf,
                                                   device=X.device)
        self._chk("Z", Z, (T, h), bf)
        qk = self._qk(T, q_gamma, k_gamma, q_beta, k_beta, positions)
        ws = self.workspace(T, training)
        B_.tp_attn_forward_qk(self.handle, T, X, Wqkv, Wo, bqkv, bo, gamma,
                              beta, Z, ws, ws.numel(), 1 if training else 0,
                              qk, stream)
        return Z

    def backward(self, dZ, X, Wqkv, Wo, gamma=None, bias_grads: bool = True,
                 out=None, stream=None, q_gamma=None, k_gamma=None,
                 positions=None):
        """Gradients after a training forward on the same workspace (with the
        same q_gamma, k_gamma and positions): a dict with dX, dWqkv, dWo and
        (optionally) dbqkv, dbo, dgamma, dbeta, and with ``qk_norm`` dq_gamma,
        dk_gamma and, for "layer", dq_beta, dk_beta; ``out`` may hold any of
        them, but none of the last four that the block does not have."""
        T = dZ.shape[0]
        h = self.hidden
        names = {None: (), "rms": ("q_gamma", "k_gamma"),
                 "layer": ("q_gamma", "k_gamma", "q_beta", "k_beta")}[self.qk_norm]
        for n in ("q_gamma", "k_gamma", "q_beta", "k_beta"):
            if out and out.get("d" + n) is not None and n not in names:
                raise ValueError(f"out: this block has no d{n}")
        self._chk("dZ", dZ, (T, h), torch.bfloat16)
        dev = dZ.device
        f32 = torch.float32
        g = out if out is not None else {}
        g.setdefault("dX", torch.empty((T, h), dtype=torch.bfloat16, device=dev))
        g.setdefault("dWqkv", torch.empty((h, 3 * h), dtype=f32, device=dev))
        g.setdefault("dWo", torch.empty((h, h), dtype=f32, device=dev))
        if bias_grads:
            g.setdefault("dbqkv", torch.empty(3 * h, dtype=f32, device=dev))
            g.setdefault("dbo", torch.empty(h, dtype=f32, device=dev))
        if self.layernorm:
            g.setdefault("dgamma", torch.empty(h, dtype=f32, device=dev))
            g.setdefault("dbeta", torch.empty(h, dtype=f32, device=dev))
        qk_grads = None
        if self.qk_norm is not None:
            d = h // self.heads
            qk_grads = B_.tp_qk_norm_grads()
            for n in names:
                g.setdefault("d" + n, torch.empty(d, dtype=f32, device=dev))
                self._chk("d" + n, g["d" + n], (d,), f32)
                setattr(qk_grads, n, g["d" + n].data_ptr())
        qk = self._qk(T, q_gamma, k_gamma, None, None, positions)
        ws = self.workspace(T, True)
        B_.tp_attn_backward_qk(self.handle, T, dZ, X, Wqkv, Wo, gamma, ws,
                               ws.numel(), g["dX"], g["dWqkv"], g["dWo"],
                               g.get("dbqkv"), g.get("dbo"), g.get("dgamma"),
                               g.get("dbeta"), qk, qk_grads, stream)
        return g

    def check(self, stream=None) -> int:
        """Synchronise and return the device status (TPMLP_OK or an error)."""
        if self._ws is None:
            return B_.TPMLP_OK
        return B_.tp_attn_check(self.handle, self._ws, stream)
