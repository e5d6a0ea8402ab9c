"""Calls of the four-bit operators that need no GPU."""
import contextlib
import os
import re

import pytest
import torch

from tensor_transformer_mlp_tcgen05_gb300 import binding as B
from tensor_transformer_mlp_tcgen05_gb300 import build as build_mod
from tensor_transformer_mlp_tcgen05_gb300 import fp4
from tensor_transformer_mlp_tcgen05_gb300.mlp import TensorParallelMLP


def block(**kw):
    build_mod.build()
    return TensorParallelMLP(128, 512, 1, 16, **kw)


class Memory:
    """Of a workspace on a device that is not the current one."""

    def __init__(self, index):
        self.device = torch.device("cuda", index)


def test_check_runs_on_its_workspaces_device(monkeypatch):
    m, current, seen = block(), [0], []

    @contextlib.contextmanager
    def device(d):
        current.append(d.index)
        yield
        current.pop()

    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(B, "tp_mlp_check", lambda handle, ws, stream=None:
                        seen.append((ws.device.index, current[-1])) or 0)
    m._fp4_ws, m._ws = Memory(1), Memory(2)
    assert m.check() == B.TPMLP_OK
    assert seen == [(1, 1), (2, 2)] and current == [0]


def test_status_of_a_block_and_its_refusals():
    """A status word has to be aligned, and lies in nothing that a call writes."""
    m = block()

    def refused(code, call):
        with pytest.raises(B.TPMLPError) as e:
            call()
        assert e.value.code == code

    X, P, Z, W, S = (i << 32 for i in range(1, 6))   # far apart

    def forward(status):
        B.tp_fp4_mlp_set_status(m.handle, status)
        B.tp_fp4_mlp_forward(m.handle, 10, B.TPFP4_NV, X, P, None, None, None, None,
                             1.0, 1.0, Z, W, 1 << 30, stream=0)

    refused(B.TPMLP_ERR_ALIGN, lambda: B.tp_fp4_mlp_set_status(m.handle, S + 8))
    refused(B.TPMLP_ERR_ARG, lambda: B.tp_fp4_mlp_set_status(None, S))
    refused(B.TPMLP_ERR_ARG, lambda: forward(Z + 16))
    refused(B.TPMLP_ERR_ARG, lambda: forward(W))
    B.tp_fp4_mlp_set_status(m.handle, None)


def test_a_matrix_of_no_rows_has_no_scale(monkeypatch):
    """Quantising one writes nothing, its header included: what lies there is not
    taken for g."""
    none = fp4.Fp4Tensor(torch.empty(4096, dtype=torch.uint8), 0, 64, "nvfp4")
    monkeypatch.setattr(B, "tensor_calls", lambda: pytest.fail("the call was made"))
    with pytest.raises(ValueError):
        fp4.quantize(torch.zeros(4, 64), scale=none)
    with pytest.raises(ValueError):
        none.tensor_scale()
    assert none.check() == B.TPMLP_OK


def test_kernels_that_start_early_read_memory_that_may_change():
    """They run while the launch before them still writes, so that no load may be one
    of memory that stays the same as long as the kernel runs."""
    csrc = os.path.dirname(build_mod.__file__) + "/csrc/"
    for name in sorted(n for n in os.listdir(csrc) if n.startswith("fp4")):
        text = re.sub(r"//[^\n]*", "", open(csrc + name).read())
        assert not re.search(r"__ldg|global\.nc|const \w+\s*\*\s*__restrict__", text), name
