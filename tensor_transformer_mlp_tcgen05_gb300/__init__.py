"""Megatron-LM intra-layer tensor-parallel MLP block on one GB300 (sm_103a).

The compute path is libtpmlp.so (hand-written tcgen05/TMA CUDA kernels behind
a C ABI, see include/tp_mlp.h, tp_attn.h, tp_rope.h, tp_grad.h and tp_fp4.h);
``binding`` is its ctypes binding with the same names, ``mlp.TensorParallelMLP``
and ``attention.TensorParallelAttention`` thin object wrappers, and so are
``rotary.RotaryEmbedding`` and ``rotary.QKNormRotary`` (rotary positions and the
per-head norm of queries and keys), ``clip.clip_grad_norm`` (the global
gradient norm, and clipping) and ``fp4`` (four-bit quantisation, products and the
linear layer ``fp4.Fp4Linear``).  Submodules
load lazily, so importing the package (e.g. for ``workloads``) does not load
the shared library.
"""
import importlib

__all__ = ["attention", "binding", "build", "clip", "fp4", "mlp", "rotary",
           "workloads", "Fp4Linear", "QKNormRotary", "RotaryEmbedding",
           "TensorParallelAttention", "TensorParallelMLP", "clip_grad_norm",
           "grad_norm"]


def __getattr__(name):
    if name in ("attention", "binding", "build", "clip", "fp4", "mlp",
                "rotary", "workloads"):
        return importlib.import_module(f".{name}", __name__)
    if name == "TensorParallelMLP":
        return importlib.import_module(".mlp", __name__).TensorParallelMLP
    if name == "TensorParallelAttention":
        return importlib.import_module(".attention",
                                       __name__).TensorParallelAttention
    if name == "Fp4Linear":
        return importlib.import_module(".fp4", __name__).Fp4Linear
    if name in ("QKNormRotary", "RotaryEmbedding"):
        return getattr(importlib.import_module(".rotary", __name__), name)
    if name in ("clip_grad_norm", "grad_norm"):
        return getattr(importlib.import_module(".clip", __name__), name)
    raise AttributeError(name)
