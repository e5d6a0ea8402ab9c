"""GPU parity of the four-bit operators against the oracle: codes, scales and
packed layout bit for bit; products, the linear layer and its gradients, and the
block's forward against fp64 sums of the values that the packed operands stand
for."""
import math

import numpy as np
import pytest
import torch

from oracle import fp4 as O
from oracle import mlp as OM
from tensor_transformer_mlp_tcgen05_gb300 import binding as B
from tensor_transformer_mlp_tcgen05_gb300 import fp4
from tensor_transformer_mlp_tcgen05_gb300.mlp import TensorParallelMLP

pytestmark = pytest.mark.gpu

FORMATS = ["nvfp4", "mxfp4"]
BF, F32 = torch.bfloat16, torch.float32
HALF_STEP = {BF: 2.0 ** -8, F32: 2.0 ** -24}


def f64(t):
    return t.detach().cpu().double().numpy()


def randn(*shape, seed=0, dtype=BF, scale=1.0):
    g = torch.Generator("cuda").manual_seed(seed)
    return (scale * torch.randn(shape, generator=g, device="cuda")).to(dtype)


def unsigned_zero(codes):
    """A code of zero may have either sign."""
    return np.where(codes == 8, 0, codes)


def nibbles(q):
    """q's codes [rows, cols], and what lies past the columns."""
    b = q.codes().cpu().numpy()
    full = np.empty((b.shape[0], 2 * b.shape[1]), dtype=np.int64)
    full[:, 0::2], full[:, 1::2] = b & 15, b >> 4
    return full[:, :q.cols], full[:, q.cols:]


def check_quantized(q, x, scale=None):
    """q against the oracle's quantisation of x [rows, cols] (fp64)."""
    c, b, g = O.quantize(x, q.format, scale)
    bad = np.repeat(b == (127 if q.format == "nvfp4" else 255),
                    O.BLOCK[q.format], 1)[:, :x.shape[1]]
    assert float(q.tensor_scale()) == g
    assert np.array_equal(q.scales().cpu().numpy(), b)
    got, past = nibbles(q)
    assert np.array_equal(np.where(bad, 0, unsigned_zero(got)),
                          np.where(bad, 0, unsigned_zero(c)))
    assert not past.any()
    # (a scale may be rounded up, and 6 times it pass the type's largest number:
    # infinity; or fall below its smallest: rounded)
    v = torch.from_numpy(O.values(np.where(bad, 0, c), b, g, q.format)).float()
    for dt in (F32, BF):
        assert np.array_equal(f64(q.dequantize(dt)), f64(v.to(dt)), equal_nan=True)
    # the scales of a k-tile past the columns: products read them, with codes
    # of zero
    per = 256 // O.BLOCK[q.format]
    rt, kt = -(-q.rows // 128), -(-q.cols // 256)
    at = B.tp_fp4_offset(q.rows, q.cols, q._code, B.TPFP4_SCALES)
    s = q.buffer[at:at + rt * kt * 128 * per].view(rt, kt, per // 4, 32, 4, 4)
    s = s.permute(0, 4, 3, 1, 2, 5).reshape(rt * 128, kt * per)
    rest = s[:q.rows, b.shape[1]:].cpu().numpy()
    assert (rest == (0 if q.format == "nvfp4" else 127)).all()


# ------------------------------------------------------------- quantise --

@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 16), (17, 33), (130, 256),
                                       (65, 257), (1, 1000), (129, 515)])
@pytest.mark.parametrize("transpose", [False, True])
def test_codes_and_scales(fmt, dtype, rows, cols, transpose):
    x = randn(rows, cols, seed=rows + cols, dtype=dtype, scale=3.0)
    x[0, 0] = 0
    for scale in ((None, 1.0) if fmt == "nvfp4" else (None,)):
        q = fp4.quantize(x, fmt, scale=scale, transpose=transpose)
        check_quantized(q, f64(x.t() if transpose else x), scale)


@pytest.mark.parametrize("fmt", FORMATS)
def test_large_matrices(fmt):
    """More rows than one pass of the row kernel takes, in both directions
    (spot rows; every row against the other direction)."""
    x = randn(5000, 1096, seed=5, dtype=BF)
    q = fp4.quantize(x, fmt)
    t = fp4.quantize(x.t().contiguous(), fmt, transpose=True)
    assert torch.equal(q.codes(), t.codes()) and torch.equal(q.scales(), t.scales())
    assert torch.equal(q.tensor_scale(), t.tensor_scale())
    some = [0, 63, 64, 127, 128, 2500, 4999]
    c, b, _ = O.quantize(f64(x[some]), fmt, float(q.tensor_scale()))
    got, _ = nibbles(q)
    assert np.array_equal(unsigned_zero(got[some]), unsigned_zero(c))
    assert np.array_equal(q.scales()[some].cpu().numpy(), b)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_borders(fmt, dtype):
    """Elements on, just below and just above every border of the codes for
    many scales, and block maxima on and around the borders of the scales."""
    size = O.BLOCK[fmt]
    eps = torch.finfo(dtype).eps
    rows = []
    mids = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]
    for m in range(8, 16):
        for e in (-9, -6, 0, 7):
            s = m * 2.0 ** e
            for f in (1.0, 1 - eps, 1 + eps):
                rows.append([6 * s] + [v * s * f * (-1) ** i
                                       for i, v in enumerate(mids)])
    for k in range(60):
        lo, hi = O.E4M3[60 + k], O.E4M3[61 + k]
        for f in (1.0, 1 - eps, 1 + eps):
            rows.append([6 * (lo + hi) / 2 * f, lo, hi, -lo])
            rows.append([2.0 ** (k - 30) * f, 2.0 ** (k - 32)])
    x = torch.zeros(len(rows), size, dtype=torch.float64)
    for i, r in enumerate(rows):
        x[i, :len(r)] = torch.tensor(r)
    x = x.to(dtype).cuda()
    scale = 1.0 if fmt == "nvfp4" else None
    check_quantized(fp4.quantize(x, fmt, scale=scale), f64(x), scale)
    check_quantized(fp4.quantize(x.t().contiguous(), fmt, scale=scale,
                                 transpose=True), f64(x), scale)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_extremes(fmt, dtype):
    """Largest and smallest numbers, zeros, and values that are not finite."""
    big = torch.finfo(dtype).max
    tiny = torch.finfo(dtype).smallest_normal
    x = randn(12, 96, seed=9, dtype=dtype)
    x[0] = 0
    x[1] *= 0
    x[1, 5] = big
    x[2] = tiny * 2.0 ** -5
    x[3] = tiny
    x[4, 40] = math.inf
    x[5, 70] = -math.inf
    x[6, 0] = math.nan
    x[7] = big
    x[8] = -x[8].abs() * tiny * 8
    x[9] = 2.0 ** -133
    for scale in ((None, 1.0, 2.0 ** 100, 2.0 ** -126, 2.0 ** 127)
                  if fmt == "nvfp4" else (None,)):
        check_quantized(fp4.quantize(x, fmt, scale=scale), f64(x), scale)
        check_quantized(fp4.quantize(x.t().contiguous(), fmt, scale=scale,
                                     transpose=True), f64(x), scale)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("off,pad", [(0, 0), (1, 0), (8, 8), (3, 5), (16, 16)])
def test_strides_and_alignment(fmt, dtype, off, pad):
    """Views into a larger buffer: any row stride, any alignment."""
    rows, cols = 37, 272
    buf = randn(rows * (cols + pad) + off + 64, seed=3, dtype=dtype)
    x = buf[off:off + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
    check_quantized(fp4.quantize(x, fmt), f64(x))
    check_quantized(fp4.quantize(x, fmt, transpose=True), f64(x.t()))
    q = fp4.quantize(x, fmt)
    out = torch.full_like(buf, 7.0)
    view = out[off:off + rows * (cols + pad)].view(rows, cols + pad)
    q.dequantize(dtype, out=view[:, :cols])
    assert torch.equal(view[:, :cols], q.dequantize(dtype))
    assert (view[:, cols:] == 7).all() and (out[:off] == 7).all()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,cols", [(70, 515), (2500, 4099)])
def test_any_alignment_is_the_same(fmt, dtype, rows, cols):
    """Rows that start on every boundary (an odd stride, and every first element of
    a 32-byte piece): the same codes and the same values as of an aligned copy."""
    wide = -(-cols // 16) * 16
    x = torch.zeros(rows, wide, dtype=dtype, device="cuda")[:, :cols]
    x.copy_(randn(rows, cols, seed=cols, dtype=dtype))
    x[0, 0], x[-1, -1] = 1e3, -2e3
    auto = fp4.quantize(x, fmt)
    want = auto.codes(), auto.scales(), auto.dequantize(dtype)
    for off in range(0, 32 // x.element_size(), 1 if rows < 100 else 5):
        # (the view ends where its memory does)
        buf = torch.full((off + rows * (cols + 2) - 2,), math.nan, dtype=dtype,
                         device="cuda")
        y = buf.as_strided((rows, cols), (cols + 2, 1), off)
        y.copy_(x)
        q = fp4.quantize(y, fmt)
        r, t = fp4.quantize_both(y, fmt)
        for p in (q, r):
            assert float(p.tensor_scale()) == float(auto.tensor_scale())
            assert torch.equal(p.codes(), want[0]) and torch.equal(p.scales(), want[1])
        assert torch.equal(t.dequantize(F32), fp4.quantize(x, fmt, transpose=True)
                           .dequantize(F32))
        buf.fill_(7.0)
        assert torch.equal(q.dequantize(dtype, out=y), want[2])
        y.fill_(7.0)
        assert (buf == 7).all()   # nothing beside the rows


def test_scale_of_another_matrix():
    """g taken from a packed matrix on the device: codes as with that power of
    two given."""
    x, y = randn(70, 300, seed=1, scale=100.0), randn(40, 200, seed=2)
    q = fp4.quantize(x)
    for t in (False, True):
        got = fp4.quantize(y, scale=q, transpose=t)
        check_quantized(got, f64(y.t() if t else y), float(q.tensor_scale()))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_both_ways_in_one_pass(fmt, dtype):
    """quantize_both is quantize along the rows and along the columns, in memory
    full of ones before; odd sizes, strides and alignments; g given or x's own."""
    for rows, cols, off, pad in ((1, 1, 0, 0), (3, 16, 1, 0), (300, 70, 0, 2),
                                 (129, 515, 3, 5), (1000, 257, 0, 0), (256, 256, 0, 0),
                                 (700, 1100, 16, 16)):
        buf = randn(rows * (cols + pad) + off, seed=rows, dtype=dtype)
        x = buf[off:].view(rows, cols + pad)[:, :cols]
        x[rows // 2, cols // 3] = (math.nan, 0.0, 3e4)[rows % 3]
        for scale in (None, 4.0) if fmt == "nvfp4" else (None,):
            torch.full((4 << 20,), 255, dtype=torch.uint8, device="cuda")
            r, t = fp4.quantize_both(x, fmt, scale)
            check_quantized(r, f64(x), scale)
            check_quantized(t, f64(x.t()), scale)
            assert r.check() == 0 and t.check() == 0
    code = fp4._FORMATS[fmt]
    x = randn(700, 130, dtype=dtype)   # with the sums of its columns
    n, nt = B.tp_fp4_bytes(700, 130, code), B.tp_fp4_bytes(130, 700, code)
    ws = B.tp_fp4_colsum_workspace_bytes(700, 130)
    got = [torch.empty(k, dtype=torch.uint8, device="cuda")
           for k in (n, nt, nt, 520, 520, ws)]
    dt = B.TPMLP_BF16 if dtype == BF else B.TPMLP_FP32
    B.tp_fp4_quantize_both(700, 130, dt, x, 130, code, 1.0, got[0], n, got[1], nt,
                           got[3], got[5], ws)
    B.tp_fp4_quantize(700, 130, dt, x, 130, 1, code, 1.0, None, got[2], nt, got[4],
                      got[5], ws)
    assert torch.equal(got[3], got[4])


def test_column_sums():
    """The bias gradient of Fp4Linear.backward: 32 rows in order, 8 such sums, then
    256-row sums; each addition off by at most 2^-24 of the sum of magnitudes so
    far: at most (32 + 8 + tiles) additions deep."""
    for T, N, dtype in ((1, 5, F32), (700, 130, F32), (513, 64, BF)):
        dy = randn(T, N, seed=T, dtype=dtype)
        lin = fp4.Fp4Linear(randn(32, N, dtype=dtype), torch.zeros(N, device="cuda"))
        db = lin.backward(dy, randn(T, 32, dtype=dtype))["db"]
        w = f64(dy)
        depth = 32 + 8 + -(-T // 256)
        assert (np.abs(f64(db) - w.sum(0)) <=
                depth * 2.0 ** -24 * np.abs(w).sum(0)).all()


# -------------------------------------------------------------- products --

def close_product(got, a, b, bias=None):
    """got against a b^T (+ bias) in fp64.  Products of codes and scales are
    exact in fp32 (2 + 2 bits of codes, 4 + 4 of scales); K sums of fp32, of
    which each addition may be truncated: off by at most 2^-23 of the sum of
    magnitudes; the bias is one more; then the rounding to got's type."""
    want = a @ b.T
    mag = np.abs(a) @ np.abs(b).T
    if bias is not None:
        want, mag = want + bias, mag + np.abs(bias)
    K = a.shape[1]
    tol = (HALF_STEP[got.dtype] * np.abs(want) * (1 + 2.0 ** -8) +
           (K + 2) * 2.0 ** -23 * mag)
    err = np.abs(f64(got) - want)
    assert (err <= tol).all(), (float((err - tol).max()), float(err.max()))


def operands(T, N, K, fmt, seed=0, dtype=BF):
    a = fp4.quantize(randn(T, K, seed=seed, dtype=dtype), fmt)
    b = fp4.quantize(randn(N, K, seed=seed + 1, dtype=dtype), fmt)
    return a, b, f64(a.dequantize(F32)), f64(b.dequantize(F32))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T,N,K", [(5, 128, 256), (1, 1, 1), (16, 64, 512),
                                   (17, 100, 300), (33, 129, 1000), (1, 4096, 1024),
                                   (65, 257, 33), (128, 640, 2048), (200, 300, 4096),
                                   (8, 1280, 5120), (64, 257, 2100), (128, 600, 4200),
                                   (300, 700, 16500)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_product_of_few_rows(fmt, T, N, K, dtype):
    a, b, va, vb = operands(T, N, K, fmt, seed=T + N)
    bias = randn(N, seed=4, dtype=F32)
    close_product(fp4.matmul(a, b, dtype=dtype), va, vb)
    close_product(fp4.matmul(a, b, bias, dtype=dtype), va, vb, f64(bias))
    assert a.check() == 0


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T,N,K", [(300, 256, 512), (257, 300, 33), (700, 1001, 600),
                                   (1500, 2500, 256), (2100, 5000, 1040),
                                   (4096, 4096, 768)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_product_of_many_rows(fmt, T, N, K, dtype):
    a, b, va, vb = operands(T, N, K, fmt, seed=T + N)
    bias = randn(N, seed=4, dtype=F32)
    got = fp4.matmul(a, b, bias, dtype=dtype)
    close_product(got, va, vb, f64(bias))
    assert a.check() == 0
    assert torch.equal(got, fp4.matmul(a, b, bias, dtype=dtype))


@pytest.mark.parametrize("T", [1, 20, 600])
def test_scales_of_whole_matrices_far_from_one(T):
    """g_A g_B below and above fp32's range, the results within it (or zero)."""
    N, K = 300, 640
    for sx, sw in ((1e-20, 1e-19), (1e-25, 1e-12), (1e25, 1e10), (1e-30, 1e30)):
        x, W = randn(T, K, seed=T, dtype=F32), randn(K, N, seed=1, dtype=F32)
        x[0, :300] = 0
        lin = fp4.Fp4Linear(W * sw)
        q = fp4.quantize(x * sx)
        va, vb = f64(q.dequantize(F32)), f64(lin.weight.dequantize(F32))
        for y in (fp4.matmul(q, lin.weight, dtype=F32),
                  lin.forward(x * sx, x_scale=None, dtype=F32),
                  lin.forward(x * sx, x_scale=float(q.tensor_scale()), dtype=F32)):
            close_product(y, va, vb)
    # 2^127 and 2^120: the codes of small x are zeros, and so is y
    x, W = randn(T, K, seed=T), torch.full((K, N), 2.0 ** 126, device="cuda")
    lin = fp4.Fp4Linear(W)
    assert not fp4.matmul(fp4.quantize(x, scale=2.0 ** 127), lin.weight).any()
    assert not lin.forward(x, x_scale=2.0 ** 127).any()


def test_every_pair_of_codes_and_scales():
    """Each row of A holds one code in one block, B all codes: every product of
    two codes under many scales, exact in fp32."""
    for fmt in FORMATS:
        size = O.BLOCK[fmt]
        lo, hi = (1, 127) if fmt == "nvfp4" else (90, 160)
        T, K = 16 * 8, 256
        r = np.random.default_rng(0)
        ca = np.zeros((T, K), dtype=np.int64)
        for t in range(T):
            ca[t, r.integers(K)] = t % 16
        cb = r.integers(0, 16, (64, K))
        q = []
        for c in (ca, cb):
            byte = r.integers(lo, hi, (c.shape[0], K // size))
            packed, scales = O.pack(c, byte, fmt)
            t = fp4.quantize(torch.zeros(c.shape, device="cuda"), fmt)
            for part, data in ((B.TPFP4_CODES, packed), (B.TPFP4_SCALES, scales)):
                at = B.tp_fp4_offset(t.rows, t.cols, t._code, part)
                t.buffer[at:at + data.size].copy_(torch.from_numpy(data))
            q.append((t, O.values(c, byte, 1.0, fmt)))
        (a, va), (b, vb) = q
        assert np.array_equal(f64(a.dequantize(F32)), va)
        assert np.array_equal(f64(fp4.matmul(a, b, dtype=F32)), va @ vb.T)


@pytest.mark.parametrize("fmt", FORMATS)
def test_sums_are_held_in_fp32(fmt):
    """Small terms next to large ones: a sum of fewer bits would lose them."""
    for T, N, K in ((16, 64, 8192), (512, 4096, 8192)):
        x = torch.full((T, K), 2.0 ** -9, device="cuda")
        x[:, 0] = 6.0
        x[:, 1:32] = 0
        w = torch.ones(N, K, device="cuda")
        a = fp4.quantize(x, fmt, scale=2.0 ** -9 if fmt == "nvfp4" else None)
        b = fp4.quantize(w, fmt)
        va, vb = f64(a.dequantize(F32)), f64(b.dequantize(F32))
        got = f64(fp4.matmul(a, b, dtype=F32))
        assert np.array_equal(got, va @ vb.T)     # 22 bits: exact in fp32


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T", [3, 2000])
def test_a_block_that_is_nan_reaches_its_row_only(fmt, T):
    x = randn(T, 400, seed=1)
    x[1, 300] = math.nan
    w = randn(500, 400, seed=2)
    w[7, 3] = math.inf
    a, b = fp4.quantize(x, fmt), fp4.quantize(w, fmt)
    got = f64(fp4.matmul(a, b))
    want = np.zeros(got.shape, dtype=bool)
    want[1], want[:, 7] = True, True
    assert np.array_equal(np.isnan(got), want)
    x[1, 300], w[7, 3] = 0, 0
    ok = ~want
    ref = f64(fp4.matmul(fp4.quantize(x, fmt, scale=float(a.tensor_scale())
                                      if fmt == "nvfp4" else None),
                         fp4.quantize(w, fmt, scale=float(b.tensor_scale())
                                      if fmt == "nvfp4" else None)))
    assert np.array_equal(got[ok], ref[ok])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T", [7, 700, 3000])
@pytest.mark.parametrize("off,pad", [(0, 0), (0, 8), (1, 1), (3, 4), (8, 0)])
def test_output_strides_and_alignment(dtype, T, off, pad):
    N, K = 1500 if T > 256 else 200, 320
    a, b, va, vb = operands(T, N, K, "nvfp4")
    buf = torch.full((T * (N + pad) + off + 16,), 5.0, dtype=dtype, device="cuda")
    out = buf[off:off + T * (N + pad)].view(T, N + pad)
    bias = randn(N + 3, seed=8, dtype=F32)[3:]      # off 16 bytes
    assert fp4.matmul(a, b, bias, dtype=dtype, out=out[:, :N]) is not None
    close_product(out[:, :N], va, vb, f64(bias))
    assert (out[:, N:] == 5).all() and (buf[:off] == 5).all()
    assert (buf[off + T * (N + pad):] == 5).all()


def test_poisoned_buffers():
    """Packed matrices over memory full of NaNs (codes, scales of rows past the
    matrix, headers): nothing of it is read."""
    for fmt in FORMATS:
        for T, N, K in ((5, 200, 300), (600, 1100, 300), (3000, 3000, 300)):
            res = []
            for fill in (0, 0xff):
                x, w = randn(T, K, seed=1), randn(N, K, seed=2)
                q = []
                for m in (x, w):
                    n = B.tp_fp4_bytes(*m.shape, fp4._FORMATS[fmt])
                    t = fp4.Fp4Tensor(torch.full((n,), fill, dtype=torch.uint8,
                                                 device="cuda"), *m.shape, fmt)
                    q.append(fp4.quantize(m, fmt, out=t))
                res.append(fp4.matmul(*q))
                assert q[0].check() == 0
            assert torch.equal(*res)


# ---------------------------------------------------------- linear layer --

@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T,K,N", [(1, 128, 96), (16, 1000, 130), (9, 2055, 640),
                                   (3, 5, 4), (40, 300, 200), (777, 1024, 1000)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_linear_layer_and_its_gradients(fmt, T, K, N, dtype):
    W = randn(K, N, seed=1, dtype=dtype, scale=K ** -0.5)
    bias = randn(N, seed=2, dtype=F32)
    x, dy = randn(T, K, seed=3, dtype=dtype), randn(T, N, seed=4, dtype=dtype,
                                                    scale=1e-3)
    lin = fp4.Fp4Linear(W, bias, format=fmt)
    one = 1.0 if fmt == "nvfp4" else None
    w_cols = O.quantized(f64(W).T, fmt)
    close_product(lin.forward(x), O.quantized(f64(x), fmt, one), w_cols, f64(bias))
    g = lin.backward(dy, x)
    close_product(g["dx"], O.quantized(f64(dy), fmt), O.quantized(f64(W), fmt))
    close_product(g["dw"], O.quantized(f64(x).T, fmt, one),
                  O.quantized(f64(dy).T, fmt))
    assert np.allclose(f64(g["db"]), f64(dy).sum(0), rtol=0,
                       atol=(T + 8) * 2.0 ** -24 * np.abs(f64(dy)).sum(0).max())
    # another scale of the activations, taken from them
    if fmt == "nvfp4":
        close_product(lin.forward(x, x_scale=None), O.quantized(f64(x), fmt),
                      w_cols, f64(bias))
    # as the steps one by one
    y = fp4.matmul(fp4.quantize(x, fmt, scale=one), lin.weight, bias)
    assert torch.equal(y, lin.forward(x))
    assert fp4.Fp4Linear(W, format=fmt).backward(dy, x)["db"] is None


def test_gradients_by_differences():
    """Where quantisation loses nothing (whole numbers whose blocks have the
    largest code), the layer is linear: its gradients are differences of a loss
    sum(dy * y)."""
    r = np.random.default_rng(0)
    pick = lambda *s: torch.from_numpy(r.choice([0.0, 1, -1, 2, -3, 4], s)).float()
    T, K, N = 32, 64, 32
    x, W, dy = pick(T, K), pick(K, N), pick(T, N)
    for m in (x, W, dy):     # a 6 in every block, along rows and columns
        m[::16, :] = 6
        m[:, ::16] = 6
    x, W, dy = x.cuda(), W.cuda(), dy.cuda()
    for fmt in FORMATS:
        loss = lambda x, W: float((fp4.Fp4Linear(W, format=fmt).forward(
            x, dtype=F32) * dy).double().sum())
        g = fp4.Fp4Linear(W, format=fmt).backward(dy, x, dtype=F32)
        base = loss(x, W)
        for _ in range(6):
            t, k, n = (int(r.integers(1, m)) for m in (T, K, N))
            t, k, n = t | 1, k | 1, n | 1        # not where a block's 6 stands
            t, k, n = t % T, k % K, n % N
            x2, W2 = x.clone(), W.clone()
            x2[t, k] = -x[t, k] if x[t, k] else 2.0
            W2[k, n] = -W[k, n] if W[k, n] else 2.0
            assert loss(x2, W) - base == float(g["dx"][t, k] * (x2 - x)[t, k])
            assert loss(x, W2) - base == float(g["dw"][k, n] * (W2 - W)[k, n])


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_few_rows_quantised_by_the_product(fmt, dtype):
    """1 to 10 rows, strided and unaligned, with borders, zeros and values that are
    not finite: the same bits as the two steps one by one."""
    N, K = 200, 1100
    lin = fp4.Fp4Linear(randn(K, N, seed=1, scale=K ** -0.5), randn(N, dtype=F32),
                        format=fmt)
    one = 1.0 if fmt == "nvfp4" else None
    for T in range(1, 11):
        for off, pad in ((0, 0), (0, 4), (3, 1)):
            buf = randn(T * (K + pad) + off, seed=T, dtype=dtype)
            x = buf[off:].view(T, K + pad)[:, :K]
            x[0, :64] = 0
            x[-1, 64:80] = torch.arange(16, device="cuda") * 0.25
            x[T // 2, 500] = (math.inf, math.nan, 1e30)[T % 3]
            want = fp4.matmul(fp4.quantize(x, fmt, scale=one), lin.weight, lin.bias)
            assert torch.equal(lin.forward(x).nan_to_num(7.0), want.nan_to_num(7.0))
            got = lin.forward(x, dtype=F32)
            want = fp4.matmul(fp4.quantize(x, fmt, scale=one), lin.weight, lin.bias,
                              dtype=F32)
            assert torch.equal(got.nan_to_num(7.0), want.nan_to_num(7.0))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_few_rows_over_a_long_ring(fmt, dtype):
    """More k-tiles a CTA than twice the stages (N of 130 x 128: K is not split),
    rows quantised by the product and before it."""
    N, K = 130 * 128, 5200
    lin = fp4.Fp4Linear(randn(K, N, seed=1, scale=K ** -0.5), format=fmt)
    one = 1.0 if fmt == "nvfp4" else None
    for T in (1, 3, 4, 7, 8, 16):
        x = randn(T, K, seed=T, dtype=dtype)
        q = fp4.quantize(x, fmt, scale=one)
        want = fp4.matmul(q, lin.weight, dtype=F32)
        for _ in range(5):
            assert torch.equal(lin.forward(x, dtype=F32), want)
        some = slice(5000, 5100)
        w = fp4.quantize(randn(K, N, seed=1, scale=K ** -0.5)[:, some].t().contiguous(),
                         fmt, scale=lin.weight if fmt == "nvfp4" else None)
        close_product(want[:, some], f64(q.dequantize(F32)), f64(w.dequantize(F32)))


def test_no_tokens():
    lin = fp4.Fp4Linear(randn(64, 48), randn(48, dtype=F32))
    x = randn(0, 64)
    assert lin.forward(x).shape == (0, 48)
    g = lin.backward(randn(0, 48), x)
    assert g["dx"].shape == (0, 64) and g["dx"].dtype == BF
    assert g["dw"].shape == (64, 48) and not g["dw"].any() and not g["db"].any()
    assert fp4.quantize(x).dequantize().shape == (0, 64)
    q = fp4.quantize(x)
    assert fp4.matmul(q, lin.weight).shape == (0, 48)
    assert q.check() == 0 and lin.check() == 0


def test_offsets_past_32_bits():
    """A matrix of 8.6e9 elements (17 GB of bf16, 4.3 GB of codes): its last rows,
    quantised and read back, and in products as the many rows and as the weight."""
    rows, cols, fresh = 132096, 65536, 512
    part = randn(fresh, cols, seed=1)
    x = part.repeat(rows // fresh, 1)
    last = slice(rows - fresh, rows)
    want = fp4.quantize(part, scale=1.0)
    q = fp4.quantize(x, scale=1.0)
    assert q.buffer.numel() > 2 ** 32
    tail = rows // 128 * 256     # tiles; those of the last rows
    codes = q.buffer[4096:4096 + tail * 16384].view(-1, 16384)
    assert torch.equal(codes[-1024:], want.buffer[4096:4096 + 1024 * 16384]
                       .view(-1, 16384))
    out = q.dequantize()
    assert torch.equal(out[last], want.dequantize())
    del out
    qt = fp4.quantize(x, scale=1.0, transpose=True)     # [cols, rows]
    rows_of = qt.dequantize()[:, last]
    assert torch.equal(rows_of, fp4.quantize(part, scale=1.0, transpose=True)
                       .dequantize())
    del qt, rows_of, x
    w = fp4.quantize(randn(300, cols, seed=2), scale=1.0)
    got = fp4.matmul(q, w, dtype=F32)
    vp, vw = f64(want.dequantize(F32)), f64(w.dequantize(F32))
    close_product(got[:fresh], vp, vw)
    close_product(got[last], vp, vw)
    for T in (2, 30, 300):
        a = fp4.quantize(randn(T, cols, seed=3), scale=1.0)
        got = fp4.matmul(a, q, dtype=F32)
        va = f64(a.dequantize(F32))
        close_product(got[:, :fresh], va, vp)
        close_product(got[:, last], va, vp)


# -------------------------------------------------------------- MLP block --

def block_case(T, h, f, t, seed=0, bias=True, **kw):
    X = randn(T, h, seed=seed)
    A = randn(h, f, seed=seed + 1, scale=h ** -0.5)
    Bw = randn(f, h, seed=seed + 2, scale=f ** -0.5)
    b1 = randn(f, seed=seed + 3, dtype=F32, scale=0.1) if bias else None
    b2 = randn(h, seed=seed + 4, dtype=F32, scale=0.1) if bias else None
    m = TensorParallelMLP(h, f, t, T, **kw)
    return m, X, A, Bw, b1, b2


def up(n):
    return (n + 255) // 256 * 256


def check_block(m, Z, X, Xn, A, Bw, b1, b2, fmt, gelu="erf", residual=False):
    """Z step by step, on what the kernels left in the workspace: Xq's codes are
    those of Xn (bf16); Yq's those of the fp64 GeLU of Xq A + b1, but for values
    next to a rounding border, which fp32 may put on its other side (the device's
    GeLU is within 1e-6 of the largest |H|, H within K 2^-23 of its sum of
    magnitudes: 2e-5 allowed); Z the product of that Yq."""
    T, h = X.shape
    f = A.shape[1]
    one = 1.0 if fmt == "nvfp4" else None
    code = fp4._FORMATS[fmt]
    # (up to 8 rows are quantised inside the product)
    xq = (fp4.quantize(Xn, fmt, scale=one) if T <= 8
          else fp4.Fp4Tensor(m._fp4_ws, T, h, fmt))
    yq = fp4.Fp4Tensor(m._fp4_ws[up(B.tp_fp4_bytes(T, h, code)):], T, f, fmt)
    check_quantized(xq, f64(Xn), one)
    H = f64(xq.dequantize(F32)) @ O.quantized(f64(A).T, fmt).T
    H = H if b1 is None else H + f64(b1)
    Y = OM.gelu(H, gelu)
    codes, byte, g = O.quantize(Y, fmt, one)
    want, got = O.values(codes, byte, g, fmt), f64(yq.dequantize(F32))
    same = np.repeat(yq.scales().cpu().numpy() == byte, O.BLOCK[fmt], 1)[:, :f]
    assert same.mean() > 0.999
    differ = (np.abs(got) != np.abs(want)) & same
    assert differ.mean() < 1e-3
    for i, j in np.argwhere(differ)[:200]:
        assert abs(Y[i, j] - (got[i, j] + want[i, j]) / 2) <= \
            2e-5 * max(1.0, np.abs(H).max())
    bias = f64(b2) if b2 is not None else np.zeros(h)
    close_product(Z, got, O.quantized(f64(Bw).T, fmt),
                  bias + f64(X) if residual else bias)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T,h,f,t", [(1, 64, 64, 1), (8, 128, 512, 2),
                                     (4, 256, 1088, 1), (33, 192, 320, 1),
                                     (50, 2048, 320, 1), (100, 4096, 576, 1),
                                     (130, 256, 1088, 1),
                                     (300, 320, 640, 2), (700, 512, 2048, 4),
                                     (2500, 256, 4160, 1)])
@pytest.mark.parametrize("gelu", ["erf", "tanh"])
def test_block_forward(fmt, T, h, f, t, gelu):
    m, X, A, Bw, b1, b2 = block_case(T, h, f, t, gelu=gelu)
    packed = m.pack_fp4_weights(A, Bw, format=fmt)
    Z = m.forward_fp4(X, packed, b1, b2)
    assert m.check() == 0
    check_block(m, Z, X, X, A, Bw, b1, b2, fmt, gelu)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T", [9, 600, 2600])
def test_block_with_layernorm_and_residual(fmt, T):
    h, f = (256, 1024) if T < 1000 else (1024, 2048)
    m, X, A, Bw, b1, b2 = block_case(T, h, f, 2, layernorm=True, residual=True)
    gamma = 1 + randn(h, seed=8, dtype=F32, scale=0.2)
    beta = randn(h, seed=9, dtype=F32, scale=0.1)
    packed = m.pack_fp4_weights(A, Bw, format=fmt)
    Z = m.forward_fp4(X, packed, b1, b2, gamma, beta)
    assert m.check() == 0
    code = fp4._FORMATS[fmt]
    at = up(B.tp_fp4_bytes(T, h, code)) + up(B.tp_fp4_bytes(T, f, code))
    Xn = m._fp4_ws[at:at + 2 * T * h].view(BF).view(T, h)
    want = OM.layernorm_forward(f64(X), f64(gamma), f64(beta))[0]
    # one rounding to bf16, and fp32's: a few in 2^-24 of values of order 4
    assert (np.abs(f64(Xn) - want) <= 2.0 ** -8 * np.abs(want) + 1e-5).all()
    check_block(m, Z, X, Xn, A, Bw, b1, b2, fmt, residual=True)


def test_block_does_not_depend_on_shards_and_repeats():
    res = []
    for t in (1, 2, 4, 8):
        m, X, A, Bw, b1, b2 = block_case(500, 512, 2048, t)
        p = m.pack_fp4_weights(A, Bw)
        res += [m.forward_fp4(X, p, b1, b2) for _ in range(2)]
    assert all(torch.equal(res[0], z) for z in res[1:])


def test_block_scales_and_no_tokens():
    """X 2^12 and g 2^12: the same codes, so that Z is that of X with y_scale as
    given where GeLU is linear or zero; checked against the oracle in norm (what
    next to a border goes the other way is below 1e-3 of the elements, each off by
    at most a quarter of itself)."""
    m, X, A, Bw, b1, b2 = block_case(40, 128, 256, 1, bias=False)
    p = m.pack_fp4_weights(A, Bw)
    X2 = X * 2.0 ** 12
    Z = m.forward_fp4(X2, p, x_scale=2.0 ** 12, y_scale=2.0 ** 10)
    ref = O.mlp_forward(f64(X2), f64(A), f64(Bw), "nvfp4", x_scale=2.0 ** 12,
                        y_scale=2.0 ** 10)
    assert np.linalg.norm(f64(Z) - ref["Z"]) < 1e-2 * np.linalg.norm(ref["Z"])
    assert m.forward_fp4(X[:0], p).shape == (0, 128) and m.check() == 0


# ---------------------------------------------- streams, graphs, threads --

def test_block_in_two_graphs_and_beside_a_training_step():
    """Two captured graphs of one block, replayed at the same time; and a
    forward_fp4 between a training forward and its backward changes no gradient."""
    m, X, A, Bw, b1, b2 = block_case(300, 256, 1024, 2)
    p = m.pack_fp4_weights(A, Bw)
    graphs = []
    for i in range(2):
        xi, g = X.clone(), torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = m.forward_fp4(xi, p, b1, b2)
        graphs.append((g, xi, out, torch.cuda.Stream()))
    for rep in range(5):
        new = [randn(300, 256, seed=20 + 2 * rep + i) for i in range(2)]
        for (g, xi, out, s), n in zip(graphs, new):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                xi.copy_(n)
                g.replay()
        torch.cuda.synchronize()
        for (g, xi, out, s), n in zip(graphs, new):
            assert torch.equal(out, m.forward_fp4(n, p, b1, b2))
    dZ = randn(300, 256, seed=40)
    m.forward(X, A, Bw, b1, b2)
    want = {k: v.clone() for k, v in m.backward(dZ, X, A, Bw).items()}
    m.forward(X, A, Bw, b1, b2)
    m.forward_fp4(randn(300, 256, seed=41), p, b1, b2)
    got = m.backward(dZ, X, A, Bw)
    assert all(torch.equal(got[k], want[k]) for k in want)
    assert m.check() == 0


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T,h,f", [(2, 16384, 32768), (8, 16384, 32768),
                                   (16, 16384, 32768),
                                   (2000, 2048, 8192)])
def test_wait_timeout_is_reported_and_context_survives(fmt, T, h, f):
    """Every kind of product: its bounded waits give up, the status says so, and the
    same block then computes what it did before.  (A wait gives up after two tries,
    which last up to 20 us each: the weights of few rows are read in 45 us or more,
    300 MB at 6.7 TB/s.)"""
    m, X, A, Bw, b1, b2 = block_case(T, h, f, 1)
    p = m.pack_fp4_weights(A, Bw, format=fmt)
    want = m.forward_fp4(X, p, b1, b2)
    assert m.check() == B.TPMLP_OK
    B.tp_mlp_set_wait_budget(m.handle, 1)
    m.forward_fp4(X, p, b1, b2)
    assert m.check() == B.TPMLP_ERR_TIMEOUT
    assert m.check() == B.TPMLP_OK
    B.tp_mlp_set_wait_budget(m.handle, 2_000_000_000)
    assert torch.equal(m.forward_fp4(X, p, b1, b2), want)
    assert m.check() == B.TPMLP_OK


def test_a_layer_keeps_its_first_error_until_it_is_asked():
    """An error in the layer's status word (as a product would leave it) stays over
    further calls, which are right, and is gone once it was read."""
    lin = fp4.Fp4Linear(randn(256, 320), randn(320, dtype=F32))
    x = randn(20, 256)
    want = lin.forward(x)
    assert lin.check() == B.TPMLP_OK
    lin._status[0] = B.TPMLP_ERR_TIMEOUT
    lin.forward(x[:1])
    assert torch.equal(lin.forward(x), want)
    lin.backward(randn(20, 320), x)
    assert lin.check() == B.TPMLP_ERR_TIMEOUT
    assert lin.check() == B.TPMLP_OK


def test_products_at_once_on_the_same_operands():
    a, b, va, vb = operands(700, 900, 640, "nvfp4")
    few = fp4.quantize(randn(20, 640, seed=5))
    want = [fp4.matmul(a, b), fp4.matmul(few, b), fp4.matmul(a, a)]
    streams = [torch.cuda.Stream() for _ in range(6)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [fp4.matmul((a, few, a)[i % 3], (b, b, a)[i % 3], stream=s)
           for _ in range(10) for i, s in enumerate(streams)]
    torch.cuda.synchronize()
    assert all(torch.equal(g, want[i % 3]) for i, g in enumerate(got))
    assert a.check() == 0 and few.check() == 0


def test_other_streams_and_captured_graphs():
    T, K, N = 600, 512, 1300
    lin = fp4.Fp4Linear(randn(K, N, seed=1), randn(N, seed=2, dtype=F32))
    x, dy = randn(T, K, seed=3), randn(T, N, seed=4)
    want, grads = lin.forward(x), lin.backward(dy, x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for s in (side, side.cuda_stream):
        got = lin.forward(x, stream=s)
        side.synchronize()
        assert torch.equal(got, want)
    # two captured graphs of the same layer, replayed on two streams at once
    graphs = []
    for i in range(2):
        xi, di = x.clone(), dy.clone()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = lin.forward(xi, x_scale=None), lin.backward(di, xi)
        graphs.append((g, xi, di, out))
    for rep in range(3):
        streams = [torch.cuda.Stream() for _ in graphs]
        new = [randn(T, K, seed=10 + rep + i) for i in range(2)]
        for (g, xi, di, out), s, n in zip(graphs, streams, new):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                xi.copy_(n)
                g.replay()
        torch.cuda.synchronize()
        for (g, xi, di, out), n in zip(graphs, new):
            assert torch.equal(out[0], lin.forward(n, x_scale=None))
            ref = lin.backward(di, n)
            for k in ref:
                assert torch.equal(out[1][k], ref[k])
    assert torch.equal(grads["dw"], lin.backward(dy, x)["dw"])


def test_launches_among_other_work():
    """The kernels start early only where what they read is complete: weights packed
    right before they are used, copies and joined streams before a call, many calls
    in a row, eagerly and in a captured graph."""
    T, h = 32, 1024
    Ws = [randn(h, h, seed=i, scale=h ** -0.5) for i in range(4)]
    x = randn(T, h, seed=9)
    rows = (1, 4, 8, 32)

    def chain(x, side):
        out = []
        for n in rows:
            y = torch.empty_like(x[:n]).copy_(x[:n])
            for W in Ws:      # packed, used, overwritten in the next round
                lin = fp4.Fp4Linear(W)
                y = lin.forward(y)
            main = torch.cuda.current_stream()
            side.wait_stream(main)
            with torch.cuda.stream(side):
                z = fp4.quantize(y).dequantize()
            main.wait_stream(side)
            m = fp4.matmul(fp4.quantize(z), fp4.quantize(Ws[0]))
            m.record_stream(main)
            out.append(m)
        return out

    def steps(x):
        """The same, one by one."""
        out = []
        for n in rows:
            y = x[:n].clone()
            for W in Ws:
                w = fp4.quantize(W, transpose=True)
                torch.cuda.synchronize()
                q = fp4.quantize(y, scale=1.0)
                torch.cuda.synchronize()
                y = fp4.matmul(q, w)
                torch.cuda.synchronize()
            z = fp4.quantize(y).dequantize()
            torch.cuda.synchronize()
            a, b = fp4.quantize(z), fp4.quantize(Ws[0])
            torch.cuda.synchronize()
            out.append(fp4.matmul(a, b))
        return out

    side = torch.cuda.Stream()
    want = steps(x)
    for _ in range(10):
        assert all(torch.equal(a, b) for a, b in zip(chain(x, side), want))
    g, xi = torch.cuda.CUDAGraph(), x.clone()
    with torch.cuda.graph(g):
        got = chain(xi, side)
    for i in range(10):
        xi.copy_(randn(T, h, seed=50 + i))
        g.replay()
        assert all(torch.equal(a, b) for a, b in zip(got, steps(xi)))


def test_several_threads():
    from concurrent.futures import ThreadPoolExecutor
    lin = fp4.Fp4Linear(randn(300, 700, seed=1))
    xs = [randn(t, 300, seed=t) for t in (1, 3, 20, 64, 300, 900)]
    want = [lin.forward(x) for x in xs]
    torch.cuda.synchronize()

    def work(i):
        s = torch.cuda.Stream()
        for _ in range(20):
            got = lin.forward(xs[i], stream=s)
            s.synchronize()
            assert torch.equal(got, want[i])

    with ThreadPoolExecutor(6) as ex:
        list(ex.map(work, range(6)))


def test_one_after_another_as_a_training_step():
    """Two layers, forward and backward, and the gradients clipped: the operators
    as they are used together."""
    from tensor_transformer_mlp_tcgen05_gb300 import clip_grad_norm
    T, h, f = 320, 256, 512
    l1 = fp4.Fp4Linear(randn(h, f, seed=1, scale=h ** -0.5),
                       randn(f, seed=2, dtype=F32))
    l2 = fp4.Fp4Linear(randn(f, h, seed=3, scale=f ** -0.5),
                       randn(h, seed=4, dtype=F32), format="mxfp4")
    x, dz = randn(T, h, seed=5), randn(T, h, seed=6, scale=1e-3)
    y = l1.forward(x)
    z = l2.forward(y)
    g2 = l2.backward(dz, y)
    g1 = l1.backward(g2["dx"], x)
    fq = lambda m, fmt, s=None: O.quantized(f64(m), fmt, s)
    close_product(z, fq(y, "mxfp4"), f64(l2.weight.dequantize(F32)), f64(l2.bias))
    close_product(g1["dx"], fq(g2["dx"], "nvfp4"),
                  f64(l1.weight_rows.dequantize(F32)))
    close_product(g1["dw"], fq(x.t(), "nvfp4", 1.0), fq(g2["dx"].t(), "nvfp4"))
    grads = [g1["dw"], g1["db"], g2["dw"], g2["db"]]
    norm = math.sqrt(sum(float((g.double() ** 2).sum()) for g in grads))
    assert abs(float(clip_grad_norm(grads, 0.5 * norm)) - norm) < 1e-5 * norm


def test_refusals_on_tensors():
    x = randn(8, 64)
    q = fp4.quantize(x)
    bad = [
        lambda: fp4.quantize(x.cpu()),
        lambda: fp4.quantize(x.half()),
        lambda: fp4.quantize(x[0]),
        lambda: fp4.quantize(x[:, ::2]),
        lambda: fp4.quantize(x[:1].expand(8, 64)),
        lambda: fp4.quantize(x, "fp4"),
        lambda: fp4.quantize(x, scale=-1.0),
        lambda: fp4.quantize(x, scale=0.0),
        lambda: fp4.quantize(x, out=fp4.quantize(x, "mxfp4")),
        lambda: fp4.quantize(x, out=fp4.quantize(randn(8, 32))),
        lambda: fp4.quantize(x[:0], transpose=True),
        lambda: fp4.quantize_both(x[:0]),
        lambda: fp4.quantize_both(x, "nvfp4", 0.0),
        lambda: fp4.quantize_both(x.half()),
        lambda: fp4.matmul(q, fp4.quantize(randn(4, 32))),
        lambda: fp4.matmul(q, fp4.quantize(randn(4, 64), "mxfp4")),
        lambda: fp4.matmul(q, q, bias=randn(8)),
        lambda: fp4.matmul(q, q, bias=randn(9, dtype=F32)),
        lambda: fp4.matmul(q, q, out=randn(8, 9)),
        lambda: fp4.matmul(q, q, out=randn(8, 8, dtype=F32)),
        lambda: fp4.matmul(q, q, dtype=torch.float16),
        lambda: q.dequantize(torch.float16),
        lambda: q.dequantize(out=randn(8, 63)),
        lambda: fp4.quantize(x, scale=fp4.quantize(x, "mxfp4")),
        lambda: fp4.matmul(fp4.Fp4Tensor(q.buffer[:256], 8, 64, "nvfp4"), q),
        lambda: fp4.Fp4Linear(randn(64, 8)).forward(randn(2, 63)),
        lambda: fp4.Fp4Linear(randn(64, 8)).backward(randn(2, 8), randn(3, 64)),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} was accepted")
    for call in (lambda: fp4.quantize(x, scale=3.0),
                 lambda: fp4.quantize(x, "mxfp4", scale=2.0),
                 lambda: fp4.matmul(q, q, out=q.buffer.view(BF)[128:192].view(8, 8))):
        with pytest.raises(B.TPMLPError) as e:
            call()
        assert e.value.code == B.TPMLP_ERR_ARG
    m = TensorParallelMLP(64, 128, 1, 8)
    p = m.pack_fp4_weights(randn(64, 128), randn(128, 64))
    for call in (lambda: m.forward_fp4(x, p.buffer),
                 lambda: m.forward_fp4(x.float(), p),
                 lambda: TensorParallelMLP(128, 128, 1, 8).forward_fp4(
                     randn(8, 128), p),
                 lambda: TensorParallelMLP(64, 128, 1, 8, dropout_p=0.1)
                 .pack_fp4_weights(randn(64, 128), randn(128, 64)),
                 lambda: m.pack_fp4_weights(randn(64, 128), randn(128, 64), "fp4")):
        with pytest.raises(ValueError):
            call()
    for kw in (dict(x_scale=0.0), dict(y_scale=3.0), dict(x_scale=math.inf)):
        with pytest.raises(B.TPMLPError):
            m.forward_fp4(x, p, **kw)
