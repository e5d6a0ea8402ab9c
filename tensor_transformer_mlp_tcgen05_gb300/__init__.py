"""Megatron-LM intra-layer tensor-parallel MLP block on one GB300 (sm_103a).

The compute path is libtpmlp.so (hand-written tcgen05/TMA CUDA kernels behind
a C ABI, see include/tp_mlp.h, tp_attn.h, tp_rope.h and tp_grad.h);
``binding`` is its ctypes binding with the same names, ``mlp.TensorParallelMLP``
and ``attention.TensorParallelAttention`` thin object wrappers, and so are
``rotary.RotaryEmbedding`` and ``rotary.QKNormRotary`` (rotary positions and the
per-head norm of queries and keys) and ``clip.clip_grad_norm`` (the global
gradient norm, and clipping).  Submodules
load lazily, so importing the package (e.g. for ``workloads``) does not load
the shared library.
"""
import importlib

__all__ = ["attention", "binding", "build", "clip", "mlp", "rotary",
           "workloads", "QKNormRotary", "RotaryEmbedding",
           "TensorParallelAttention", "TensorParallelMLP", "clip_grad_norm",
           "grad_norm"]


def __getattr__(name):
    if name in ("attention", "binding", "build", "clip", "mlp", "rotary",
                "workloads"):
        return importlib.import_module(f".{name}", __name__)
    if name == "TensorParallelMLP":
        return importlib.import_module(".mlp", __name__).TensorParallelMLP
    if name == "TensorParallelAttention":
        return importlib.import_module(".attention",
                                       __name__).TensorParallelAttention
    if name in ("QKNormRotary", "RotaryEmbedding"):
        return getattr(importlib.import_module(".rotary", __name__), name)
    if name in ("clip_grad_norm", "grad_norm"):
        return getattr(importlib.import_module(".clip", __name__), name)
    raise AttributeError(name)
