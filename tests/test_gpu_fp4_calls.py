"""The four-bit operators' calls on streams, from threads, on empty and on wrong
inputs: what belongs to whom, and which errors are reported when."""
import pytest
import torch

from tensor_transformer_mlp_tcgen05_gb300 import binding as B
from tensor_transformer_mlp_tcgen05_gb300 import fp4
from tensor_transformer_mlp_tcgen05_gb300.mlp import Fp4Weights, TensorParallelMLP

pytestmark = pytest.mark.gpu

FORMATS = ["nvfp4", "mxfp4"]
BF, F32 = torch.bfloat16, torch.float32


def randn(*shape, seed=0, dtype=BF, scale=1.0):
    g = torch.Generator("cuda").manual_seed(seed)
    return (scale * torch.randn(shape, generator=g, device="cuda")).to(dtype)


def block_case(T, h, f, **kw):
    m = TensorParallelMLP(h, f, 1, T, **kw)
    return (m, randn(T, h, seed=1), randn(h, f, seed=2, scale=h ** -0.5),
            randn(f, h, seed=3, scale=f ** -0.5))


def owner(t):
    """The handle of the stream that t's memory belongs to."""
    for s in torch.cuda.memory_snapshot():
        if s["address"] <= t.data_ptr() < s["address"] + s["total_size"]:
            return s["stream"]
    raise AssertionError("memory of no segment")


@pytest.mark.parametrize("fmt", FORMATS)
def test_packed_weights_belong_to_the_stream_that_writes_them(fmt):
    """(Of the current stream's memory, a block that its pending kernels still use
    could be overwritten.)"""
    m, X, A, Bw = block_case(40, 256, 512)
    want = m.pack_fp4_weights(A, Bw, format=fmt)
    assert owner(want.buffer) == torch.cuda.current_stream().cuda_stream
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for stream in (side, side.cuda_stream):
        p = m.pack_fp4_weights(A, Bw, format=fmt, stream=stream)
        assert owner(p.buffer) == side.cuda_stream
        assert p.shape == (256, 512) and p.format == fmt
        Z = m.forward_fp4(X, p, stream=stream)
        assert owner(Z) == side.cuda_stream
        side.synchronize()
        assert torch.equal(Z, m.forward_fp4(X, want))
    for bad in ((A.cpu(), Bw), (A, Bw.cpu()), (A.float(), Bw), (A.t(), Bw),
                (A, Bw[:, :8])):
        with pytest.raises(ValueError):
            m.pack_fp4_weights(*bad, format=fmt)


@pytest.mark.parametrize("fmt", FORMATS)
def test_gradients_of_no_tokens(fmt):
    """Their zeros are written on the call's stream and belong to it, and the arguments
    are checked as for any number of tokens."""
    lin = fp4.Fp4Linear(randn(64, 48), randn(48, dtype=F32), format=fmt)
    x, dy = randn(0, 64), randn(0, 48)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for stream in (side, side.cuda_stream):
        g = lin.backward(dy, x, stream=stream)
        side.synchronize()
        assert owner(g["dw"]) == owner(g["db"]) == side.cuda_stream
        assert g["dx"].shape == (0, 64) and g["dx"].dtype == BF
        assert g["dw"].shape == (64, 48) and g["db"].shape == (48,)
        assert g["dw"].dtype == g["db"].dtype == F32
        assert not g["dw"].any() and not g["db"].any()
    assert lin.backward(dy, x, bias_grad=False)["db"] is None
    assert lin.backward(dy, x, dtype=F32)["dx"].dtype == F32
    for bad in (lambda: lin.backward(dy.half(), x), lambda: lin.backward(dy, x.half()),
                lambda: lin.backward(dy.cpu(), x), lambda: lin.backward(dy, x.cpu()),
                lambda: lin.backward(dy, x, dtype=torch.float16),
                lambda: lin.backward(dy, x, x_scale=-1.0)):
        with pytest.raises(ValueError):
            bad()
    for kw in (dict(dy_scale=3.0), dict(x_scale=3.0)):
        with pytest.raises(B.TPMLPError) as e:
            lin.backward(dy, x, **kw)
        assert e.value.code == B.TPMLP_ERR_ARG


def test_weights_of_too_few_bytes_are_refused():
    """As after a checkpoint that was cut off, or was written in another format: the
    products would read past the buffer."""
    m, X, A, Bw = block_case(10, 256, 512)
    mx = m.pack_fp4_weights(A, Bw, format="mxfp4").buffer
    nv = m.pack_fp4_weights(A, Bw, format="nvfp4").buffer
    assert mx.numel() < nv.numel()
    for buffer, fmt in ((mx, "nvfp4"), (nv[:-1], "nvfp4"), (mx[:4096], "mxfp4"),
                        (mx.view(torch.int32), "mxfp4"), (nv[:0], "nvfp4"),
                        (mx.repeat(2)[::2], "mxfp4")):
        with pytest.raises(ValueError):
            m.forward_fp4(X, Fp4Weights(buffer, fmt, (256, 512)))
    want = m.forward_fp4(X, Fp4Weights(mx, "mxfp4", (256, 512)))
    assert torch.equal(m.forward_fp4(X, Fp4Weights(mx.clone(), "mxfp4", (256, 512))),
                       want)


def test_a_block_keeps_its_first_error_until_it_is_asked():
    """A call that gave up, and right ones after it."""
    T, h, f = 2000, 2048, 8192
    m, X, A, Bw = block_case(T, h, f)
    p = m.pack_fp4_weights(A, Bw)
    q = m.pack_fp4_weights(A, Bw, format="mxfp4")   # keeps the status there is
    want = m.forward_fp4(X, p)
    assert m.check() == B.TPMLP_OK
    B.tp_mlp_set_wait_budget(m.handle, 1)
    m.forward_fp4(X, p)
    torch.cuda.synchronize()
    B.tp_mlp_set_wait_budget(m.handle, 2_000_000_000)
    assert torch.equal(m.forward_fp4(X, p), want)
    m.forward_fp4(X[:3], q)
    assert m.forward_fp4(X[:0], p).shape == (0, h)
    assert m.check() == B.TPMLP_ERR_TIMEOUT
    assert m.check() == B.TPMLP_OK
    assert torch.equal(m.forward_fp4(X, p), want) and m.check() == B.TPMLP_OK


def test_a_block_that_packed_nothing_reports_its_last_call():
    """Weights of another block, and weights packed in a captured graph."""
    T, h, f = 2000, 2048, 8192
    m, X, A, Bw = block_case(T, h, f)
    p = m.pack_fp4_weights(A, Bw)
    want = m.forward_fp4(X, p)
    other = TensorParallelMLP(h, f, 1, T)
    assert torch.equal(other.forward_fp4(X, p), want) and other.check() == B.TPMLP_OK
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        Z = other.forward_fp4(X, other.pack_fp4_weights(A, Bw))
    g.replay()
    assert torch.equal(Z, want) and other._fp4_status is None
    B.tp_mlp_set_wait_budget(other.handle, 1)
    other.forward_fp4(X, p)
    assert other.check() == B.TPMLP_ERR_TIMEOUT
    assert other.check() == B.TPMLP_OK and m.check() == B.TPMLP_OK


@pytest.mark.parametrize("fmt", FORMATS)
def test_a_budget_counts_waits_of_its_own_kernel(fmt):
    """The block's second product is resident while the first one runs (48 places of
    304 are left by the first's 256 CTAs).  A budget that each of the two fits in, but
    not both together: nothing is stuck, and nothing is reported.  (Both read 604 MB
    of weights, MX 570: about 100 us each, of which the budget is one and a half.)"""
    h = f = 32768
    m, X, A, Bw = block_case(16, h, f)
    p = m.pack_fp4_weights(A, Bw, format=fmt)
    del A, Bw
    want = m.forward_fp4(X, p)
    assert m.check() == B.TPMLP_OK
    times = []
    for _ in range(5):
        start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        start.record()
        m.forward_fp4(X, p)
        end.record()
        end.synchronize()
        times.append(start.elapsed_time(end) * 1e6)
    B.tp_mlp_set_wait_budget(m.handle, int(0.75 * min(times)))
    for _ in range(5):
        Z = m.forward_fp4(X, p)
        assert m.check() == B.TPMLP_OK
        assert torch.equal(Z, want)
