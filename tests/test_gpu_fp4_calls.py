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


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T", [8, 300])
def test_memory_that_is_written_and_read_again_and_again(fmt, T):
    """One buffer that a product writes and the next launches read, over and over, and
    one packed matrix likewise: every launch starts while the one before it runs, and
    none reads what an earlier round left (in a cache of its SM, say)."""
    N, K, rounds = 1024, 512, 12
    b = fp4.quantize(randn(N, K, seed=1, scale=K ** -0.5), fmt)
    As = [fp4.quantize(randn(T, K, seed=10 + i), fmt) for i in range(rounds)]
    biases = [randn(N, seed=30 + i, dtype=F32) for i in range(rounds)]
    one = 1.0 if fmt == "nvfp4" else None
    buf = torch.empty(T, N, dtype=BF, device="cuda")
    bias = torch.empty(N, device="cuda")
    P = fp4.quantize(torch.zeros(T, N, device="cuda"), fmt)

    def launches(step):
        out = []
        for a, v in zip(As, biases):
            bias.copy_(v)
            step()
            fp4.matmul(a, b, bias, out=buf)
            step()
            p = fp4.quantize(buf, fmt, scale=one, out=P)
            step()
            out.append(p.dequantize())
            step()
            for x in fp4.quantize_both(buf, fmt):
                step()
                out.append(x.dequantize(F32))
            step()
            fp4.matmul(a, b, out=buf)
            step()
            out.append(fp4.quantize(buf, fmt, transpose=True).dequantize(F32))
            step()
        return out

    want = launches(torch.cuda.synchronize)
    for _ in range(5):
        got = launches(lambda: None)
        assert all(torch.equal(x, y) for x, y in zip(got, want))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = launches(lambda: None)
    for _ in range(20):
        g.replay()
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    assert all(a.check() == 0 for a in As)


# ------------------------------------------------------- the block's calls --

def test_the_block_on_given_streams_and_from_several_threads():
    """forward_fp4 of one block on several streams at once, from one thread and from
    several, in both formats: the results of the calls one by one."""
    from concurrent.futures import ThreadPoolExecutor
    m, _, A, Bw = block_case(900, 256, 1024)
    b1, b2 = randn(1024, seed=4, dtype=F32), randn(256, seed=5, dtype=F32)
    packed = [m.pack_fp4_weights(A, Bw, format=f) for f in FORMATS]
    xs = [randn(t, 256, seed=t) for t in (1, 8, 20, 100, 300, 900)]
    want = [[m.forward_fp4(x, p, b1, b2) for p in packed] for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    got = [m.forward_fp4(x, p, b1, b2, stream=(s, s.cuda_stream)[i % 2])
           for i in range(6) for x, s in zip(xs, streams) for p in packed]
    torch.cuda.synchronize()
    assert all(torch.equal(z, w) for z, w in zip(got, 6 * sum(want, [])))

    def work(i):
        s = torch.cuda.Stream()
        for n in range(20):
            z = m.forward_fp4(xs[i], packed[n % 2], b1, b2, stream=s)
            s.synchronize()
            assert torch.equal(z, want[i][n % 2])

    with ThreadPoolExecutor(6) as ex:
        list(ex.map(work, range(6)))
    assert m.check() == B.TPMLP_OK


@pytest.mark.parametrize("dtype,N,pad", [(BF, 55, 1), (BF, 1501, 3), (BF, 1502, 2),
                                         (BF, 1500, 4), (BF, 1500, 12), (BF, 1504, 8),
                                         (F32, 3, 1), (F32, 1501, 3), (F32, 1502, 2),
                                         (F32, 1503, 1), (F32, 1503, 5),
                                         (F32, 1504, 4)])
@pytest.mark.parametrize("T", [7, 74, 700])
def test_rows_that_end_off_16_bytes_leave_what_lies_behind_them(dtype, N, pad, T):
    """Columns of a wider matrix whose rows are 16-byte aligned: products of every kind
    write them, and neither the columns behind them nor what follows the last row."""
    K = 320
    x, w = whole(T, K, 1), whole(N, K, 2)
    a, b = fp4.quantize(x), fp4.quantize(w)
    lin = fp4.Fp4Linear(w.t().contiguous())
    want = exact_product(x, w).to(dtype)
    for call in (lambda out: fp4.matmul(a, b, dtype=dtype, out=out),
                 lambda out: lin.forward(x, dtype=dtype, out=out)):
        buf = torch.full((T * (N + pad) + 16,), 5.0, dtype=dtype, device="cuda")
        rows = buf[:T * (N + pad)].view(T, N + pad)
        assert torch.equal(call(rows[:, :N]), want)
        assert torch.equal(rows[:, :N], want)
        assert (rows[:, N:] == 5).all() and (buf[rows.numel():] == 5).all()


# ------------------------------------------------- exact sums, large offsets --

VALUES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def whole(rows, cols, seed, dtype=BF):
    """E2M1 values of random signs, a 6 in every 16 columns: a matrix that is its own
    quantisation (every scale is 1) in both formats, along its rows."""
    g = torch.Generator("cuda").manual_seed(seed)
    v = torch.tensor(VALUES, dtype=dtype, device="cuda")
    x = v[torch.randint(0, 8, (rows, cols), generator=g, device="cuda")]
    x[:, ::16] = 6
    sign = torch.randint(0, 2, (rows, cols), generator=g, device="cuda")
    return torch.where(sign.bool(), x, -x)


def exact_product(a, b):
    """a b^T in 64 bits."""
    return a.double() @ b.double().t()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T,N,K", [(1, 1, 1), (1, 4096, 1024), (2, 300, 20480),
                                   (8, 700, 16500), (16, 64, 512), (33, 129, 1000),
                                   (64, 257, 2100), (128, 600, 4200),
                                   (300, 700, 16500), (257, 300, 33), (700, 1001, 600),
                                   (1500, 2500, 256), (1100, 2600, 16500),
                                   (2100, 5000, 1040), (4096, 4096, 768)])
def test_products_of_whole_numbers_are_exact(fmt, T, N, K):
    """Multiples of 1/4, sums below 36 K = 2^19.5 (in quarters 2^21.5): fp32 holds every
    one, in whatever order, so that one k-tile, row or scale out of place shows."""
    x, w = whole(T, K, 1), whole(N, K, 2)
    want = exact_product(x, w)
    a, b = fp4.quantize(x, fmt), fp4.quantize(w, fmt)
    assert torch.equal(a.dequantize(), x) and torch.equal(b.dequantize(), w)
    assert torch.equal(fp4.matmul(a, b, dtype=F32).double(), want)
    assert torch.equal(fp4.matmul(a, b), want.to(BF))
    lin = fp4.Fp4Linear(w.t().contiguous(), format=fmt)
    assert torch.equal(lin.weight.dequantize(), w)
    assert torch.equal(lin.forward(x, dtype=F32).double(), want)


@pytest.mark.parametrize("fmt", FORMATS)
def test_offsets_past_32_bits_of_unlike_rows(fmt):
    """A matrix of 8.7e9 elements (17 GB of bf16, more than 4.3 GB of codes) whose rows
    past 2^31 and 2^32 bytes, elements and bytes of codes are like no others: a read or
    a write that wrapped would not find them.  Quantised along rows, columns and both,
    read back, and in products as the many rows and as the weight, whose sums are exact
    (at most 36 x 65536 = 2^21.2, in quarters 2^23.2)."""
    rows, cols, some = 132096, 65536, 256
    # rows at these wrap to row 0 or to one another: 2^31 and 2^32 bytes, 2^32 elements
    # (2^31 bytes of codes), 2^32 bytes of codes; the last ends with the matrix
    starts = (16384, 32768, 65536, 131072, rows - some)
    one = 1.0 if fmt == "nvfp4" else None
    x = whole(512, cols, 1).repeat(rows // 512, 1)
    own = {}
    for i, at in enumerate((0, *starts)):
        own[at] = whole(some, cols, 10 + i)
        x[at:at + some] = own[at]
    q = fp4.quantize(x, fmt, scale=one)
    assert q.buffer.numel() > 2 ** 32
    r, t = fp4.quantize_both(x, fmt, one)
    for p in (q, r):
        out = p.dequantize()
        assert all(torch.equal(out[at:at + some], v) for at, v in own.items())
        del out
    del r
    # along the columns the blocks are of 16 or 32 rows, and starts multiples of 256
    out = t.dequantize()
    for at, v in own.items():
        u = fp4.quantize(v, fmt, scale=one, transpose=True)
        assert torch.equal(out[:, at:at + some], u.dequantize())
    del out
    t2 = fp4.quantize(x, fmt, scale=one, transpose=True)
    kt = 16384 * 512 * (rows // 256)      # bytes of codes
    assert torch.equal(t.buffer[4096:4096 + kt], t2.buffer[4096:4096 + kt])
    del t, t2
    w = whole(300, cols, 3)
    got = fp4.matmul(q, fp4.quantize(w, fmt, scale=one), dtype=F32)
    for at, v in own.items():
        assert torch.equal(got[at:at + some].double(), exact_product(v, w))
    for T in (2, 30, 300):    # quantised by the product, split, on pairs
        a = whole(T, cols, 5)
        got = fp4.matmul(fp4.quantize(a, fmt, scale=one), q, dtype=F32)
        for at, v in own.items():
            assert torch.equal(got[:, at:at + some].double(), exact_product(a, v))
    del x, q


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 16), (300, 70), (129, 515),
                                       (256, 256), (700, 1100), (257, 1000)])
def test_both_ways_over_any_memory(fmt, rows, cols):
    """quantize_both over packed buffers full of ones: everything that its products
    read is written, and only the matrix's own."""
    code, x = fp4._FORMATS[fmt], randn(rows, cols, seed=rows)
    sizes = B.tp_fp4_bytes(rows, cols, code), B.tp_fp4_bytes(cols, rows, code)
    res = []
    for fill in (0xff, 0):
        bufs = [torch.full((n + 256,), fill, dtype=torch.uint8, device="cuda")
                for n in sizes]
        B.tp_fp4_quantize_both(rows, cols, B.TPMLP_BF16, x, cols, code, 0.0, bufs[0],
                               sizes[0], bufs[1], sizes[1])
        assert all((b[n:] == fill).all() for b, n in zip(bufs, sizes))
        r = fp4.Fp4Tensor(bufs[0][:sizes[0]], rows, cols, fmt)
        t = fp4.Fp4Tensor(bufs[1][:sizes[1]], cols, rows, fmt)
        assert r.check() == 0 and t.check() == 0
        res.append((r, t))
    for p, o, ref in zip(*res, (fp4.quantize(x, fmt),
                                fp4.quantize(x, fmt, transpose=True))):
        # codes to the end of the last k-tile, and its scales past the columns
        assert torch.equal(p.codes(), o.codes()) and torch.equal(p.codes(), ref.codes())
        assert torch.equal(p.scales(), ref.scales())
        assert torch.equal(p.tensor_scale(), ref.tensor_scale())
        block = 16 if fmt == "nvfp4" else 32
        wide = [fp4.Fp4Tensor(m.buffer, m.rows, -(-m.cols // 256) * 256, fmt)
                for m in (p, o, ref)]
        past = [m.scales()[:, -(-p.cols // block):] for m in wide]
        assert (past[0] == (0 if fmt == "nvfp4" else 127)).all()
        assert torch.equal(past[0], past[1]) and torch.equal(past[0], past[2])
        assert torch.equal(fp4.matmul(p, p), fp4.matmul(ref, ref))
