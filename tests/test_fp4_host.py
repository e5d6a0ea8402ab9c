"""Host-side checks of the four-bit C ABI (no GPU): sizes and offsets, and every
refusal before a device is touched."""
import os
import re

import pytest

from tensor_transformer_mlp_tcgen05_gb300 import binding as B
from tensor_transformer_mlp_tcgen05_gb300 import build as build_mod
from tensor_transformer_mlp_tcgen05_gb300 import fp4

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
NV, MX = B.TPFP4_NV, B.TPFP4_MX
BF, F32 = B.TPMLP_BF16, B.TPMLP_FP32
X, P, P2, C, W = 1 << 32, 2 << 32, 3 << 32, 4 << 32, 5 << 32   # far apart


@pytest.fixture(scope="module", autouse=True)
def lib():
    build_mod.build()
    return B.lib()


def test_every_declared_symbol_is_exported(lib):
    text = open(os.path.join(ROOT, "include", "tp_fp4.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = sorted(set(re.findall(r"\b(tp_fp4_\w+)\s*\(", text)))
    assert names == sorted(B.EXPORTED_FP4)
    assert all(hasattr(lib, n) for n in names)


@pytest.mark.parametrize("fmt,tile", [(NV, 2048), (MX, 1024)])
def test_sizes_and_offsets(fmt, tile):
    for rows, cols in ((1, 1), (0, 5), (128, 256), (129, 257), (7, 1000),
                       (1 << 20, 1 << 15)):
        tiles = (rows + 127) // 128 * ((cols + 255) // 256)
        at = 4096 + tiles * 16384
        assert B.tp_fp4_bytes(rows, cols, fmt) == at + tiles * tile
        assert B.tp_fp4_offset(rows, cols, fmt, B.TPFP4_CODES) == 4096
        assert B.tp_fp4_offset(rows, cols, fmt, B.TPFP4_SCALES) == at
        assert B.tp_fp4_offset(rows, cols, fmt, 2) == -1
    for rows, cols, f in ((-1, 5, fmt), (5, 0, fmt), (5, 5, 2),
                          ((1 << 28) + 1, 5, fmt), (5, (1 << 28) + 1, fmt)):
        assert B.tp_fp4_bytes(rows, cols, f) == 0
        assert B.tp_fp4_offset(rows, cols, f, 0) == -1
    assert B.tp_fp4_colsum_workspace_bytes(257, 10) == 80
    assert B.tp_fp4_colsum_workspace_bytes(0, 10) == 0


def quantize(rows=100, cols=300, dtype=BF, x=X, stride=300, transpose=0,
             fmt=NV, scale=1.0, like=None, packed=P, nbytes=None, colsum=None,
             ws=None, ws_bytes=0):
    if nbytes is None:
        r, c = (cols, rows) if transpose else (rows, cols)
        nbytes = B.tp_fp4_bytes(r, c, fmt)
    B.tp_fp4_quantize(rows, cols, dtype, x, stride, transpose, fmt, scale, like,
                      packed, nbytes, colsum, ws, ws_bytes, stream=0)


def refused(code, call):
    with pytest.raises(B.TPMLPError) as e:
        call()
    assert e.value.code == code, e.value


ARG, SHAPE, ALIGN, WS = (B.TPMLP_ERR_ARG, B.TPMLP_ERR_SHAPE, B.TPMLP_ERR_ALIGN,
                         B.TPMLP_ERR_WORKSPACE)


@pytest.mark.parametrize("code,kw", [
    (ARG, dict(fmt=7, nbytes=1 << 30)), (ARG, dict(dtype=5)),
    (ARG, dict(transpose=2, nbytes=1 << 30)),
    (SHAPE, dict(rows=-1, nbytes=1 << 30)), (SHAPE, dict(cols=0, nbytes=1 << 30)),
    (SHAPE, dict(rows=0, transpose=1, nbytes=1 << 30)),
    (SHAPE, dict(rows=(1 << 28) + 1, nbytes=1 << 40)),
    (SHAPE, dict(cols=(1 << 28) + 1, stride=1 << 30, nbytes=1 << 40)),
    (SHAPE, dict(stride=299)), (SHAPE, dict(stride=1 << 41)),
    (ARG, dict(scale=3.0)), (ARG, dict(scale=-1.0)),
    (ARG, dict(scale=float("inf"))), (ARG, dict(scale=float("nan"))),
    (ARG, dict(scale=2.0 ** 128)), (ARG, dict(scale=2.0 ** -127)),
    (ARG, dict(fmt=MX, scale=2.0)),
    (ARG, dict(like=P2)), (ARG, dict(fmt=MX, scale=0.0, like=P2)),
    (ALIGN, dict(scale=0.0, like=P2 + 16)), (ARG, dict(scale=0.0, like=P)),
    (ARG, dict(packed=None)), (ALIGN, dict(packed=P + 16)), (WS, dict(nbytes=100)),
    (ARG, dict(x=None)), (ALIGN, dict(x=X + 1)), (ALIGN, dict(x=X + 2, dtype=F32)),
    (ARG, dict(colsum=C, ws=W, ws_bytes=1 << 20)),
    (ARG, dict(transpose=1, colsum=C)),
    (WS, dict(transpose=1, colsum=C, ws=W, ws_bytes=100)),
    (ALIGN, dict(transpose=1, colsum=C + 2, ws=W, ws_bytes=1 << 20)),
    (ALIGN, dict(transpose=1, colsum=C, ws=W + 8, ws_bytes=1 << 20)),
    (ARG, dict(transpose=1, colsum=X + 1000, ws=W, ws_bytes=1 << 20)),
    (ARG, dict(transpose=1, colsum=P + 1000, ws=W, ws_bytes=1 << 20)),
    (ARG, dict(transpose=1, colsum=W + 1000, ws=W, ws_bytes=1 << 20)),
    (ARG, dict(transpose=1, colsum=C, ws=P + 256, ws_bytes=1 << 20)),
    (ARG, dict(packed=X)), (ARG, dict(packed=X - 4096)),
    (ARG, dict(packed=X + 100 * 300 * 2 // 256 * 256)),
])
def test_quantize_refusals(code, kw):
    refused(code, lambda: quantize(**kw))


def both(rows=100, cols=300, dtype=BF, x=X, stride=300, fmt=NV, scale=1.0, packed=P,
         n=1 << 20, packed_t=P2, nt=1 << 20, colsum=None, ws=None, ws_bytes=0):
    B.tp_fp4_quantize_both(rows, cols, dtype, x, stride, fmt, scale, packed, n,
                           packed_t, nt, colsum, ws, ws_bytes, stream=0)


@pytest.mark.parametrize("code,kw", [
    (ARG, dict(fmt=7)), (ARG, dict(dtype=5)), (SHAPE, dict(rows=0)),
    (SHAPE, dict(cols=0)), (SHAPE, dict(stride=299)), (ARG, dict(scale=3.0)),
    (ARG, dict(fmt=MX, scale=2.0)), (ARG, dict(packed=None)),
    (ARG, dict(packed_t=None)), (ALIGN, dict(packed=P + 16)),
    (ALIGN, dict(packed_t=P2 + 16)), (WS, dict(n=100)), (WS, dict(nt=100)),
    (ARG, dict(x=None)), (ALIGN, dict(x=X + 1)), (ARG, dict(packed=X)),
    (ARG, dict(packed_t=X)), (ARG, dict(packed_t=P + 4096)),
    (WS, dict(colsum=C, ws=W, ws_bytes=100)), (ARG, dict(colsum=C)),
    (ARG, dict(colsum=P + 64, ws=W, ws_bytes=1 << 20)),
    (ARG, dict(colsum=P2 + 64, ws=W, ws_bytes=1 << 20)),
    (ARG, dict(colsum=C, ws=P + 64, ws_bytes=1 << 20)),
    (SHAPE, dict(rows=1 << 28, cols=1 << 28, stride=1 << 28, x=1 << 60,
                 packed=1 << 56, n=1 << 56, packed_t=1 << 58, nt=1 << 56)),
])
def test_quantize_both_refusals(code, kw):
    refused(code, lambda: both(**kw))


def test_calls_of_no_rows_touch_nothing():
    quantize(rows=0)
    quantize(rows=0, x=None, scale=0.0)
    B.tp_fp4_dequantize(0, 5, NV, P, 4096, BF, None, 5, stream=0)
    matmul(T=0, C=None)


@pytest.mark.parametrize("code,a", [
    (ARG, (8, 64, 9, P, 1 << 16, BF, X, 64)), (ARG, (8, 64, NV, P, 1 << 16, 3, X, 64)),
    (SHAPE, (-1, 64, NV, P, 1 << 16, BF, X, 64)), (SHAPE, (8, 0, NV, P, 1 << 16, BF, X, 64)),
    (SHAPE, (8, 64, NV, P, 1 << 16, BF, X, 63)), (ARG, (8, 64, NV, None, 1 << 16, BF, X, 64)),
    (ALIGN, (8, 64, NV, P + 128, 1 << 16, BF, X, 64)), (WS, (8, 64, NV, P, 700, BF, X, 64)),
    (ARG, (8, 64, NV, P, 1 << 16, BF, None, 64)), (ALIGN, (8, 64, NV, P, 1 << 16, F32, X + 2, 64)),
    (ARG, (8, 64, NV, P, 1 << 16, BF, P + 512, 64)),
])
def test_dequantize_refusals(code, a):
    refused(code, lambda: B.tp_fp4_dequantize(*a, stream=0))


def matmul(T=20, N=30, K=100, fmt=NV, A=P, na=None, Bp=P2, nb=None, bias=None,
           dtype=BF, C=C, ldc=30, st=None):
    na = B.tp_fp4_bytes(max(T, 0), K, fmt) if na is None else na
    nb = B.tp_fp4_bytes(N, K, fmt) if nb is None else nb
    B.tp_fp4_matmul(T, N, K, fmt, A, na, Bp, nb, bias, dtype, C, ldc, st, stream=0)


@pytest.mark.parametrize("code,kw", [
    (ARG, dict(fmt=3, na=1 << 20, nb=1 << 20)), (ARG, dict(dtype=9)),
    (SHAPE, dict(T=-1)), (SHAPE, dict(N=0, nb=1 << 20)),
    (SHAPE, dict(K=0, na=1 << 20, nb=1 << 20)), (SHAPE, dict(ldc=29)),
    (SHAPE, dict(ldc=1 << 41)),
    (ARG, dict(A=None)), (ARG, dict(Bp=None)), (ALIGN, dict(A=P + 64)),
    (WS, dict(na=10)), (WS, dict(nb=10)), (ARG, dict(C=None)),
    (ALIGN, dict(C=C + 1)), (ALIGN, dict(C=C + 2, dtype=F32)),
    (ALIGN, dict(bias=W + 2)), (ARG, dict(C=P + 256)), (ARG, dict(C=P2 + 512)),
    (ARG, dict(bias=C + 8)), (ALIGN, dict(st=W + 8)), (ARG, dict(st=C + 32)),
    (ARG, dict(st=P)), (ARG, dict(st=P2 + 64)), (ARG, dict(st=W, bias=W)),
    (SHAPE, dict(T=1 << 28, N=1 << 28, K=1, na=1 << 50, nb=1 << 50, ldc=1 << 28,
                 A=1 << 50, Bp=1 << 53, C=1 << 59)),
    (SHAPE, dict(T=1 << 28, K=1 << 28, na=1 << 60, nb=1 << 60, A=1 << 57,
                 Bp=1 << 50, C=1 << 59)),
])
def test_matmul_refusals(code, kw):
    refused(code, lambda: matmul(**kw))


def linear(T=20, N=30, K=100, xd=BF, x=X, xs=100, fmt=NV, scale=1.0, xq=P,
           nq=1 << 20, Wp=P2, nw=1 << 20, bias=None, dtype=BF, C=C, ldc=30, st=None):
    B.tp_fp4_linear(T, N, K, xd, x, xs, fmt, scale, xq, nq, Wp, nw, bias, dtype, C,
                    ldc, st, stream=0)


@pytest.mark.parametrize("code,kw", [
    (ARG, dict(fmt=3)), (ARG, dict(xd=4)), (ARG, dict(dtype=4)),
    (SHAPE, dict(T=-1)), (SHAPE, dict(N=0)), (SHAPE, dict(K=0)),
    (SHAPE, dict(xs=99)), (SHAPE, dict(ldc=29)), (ARG, dict(scale=3.0)),
    (ARG, dict(x=None)), (ARG, dict(xq=None)), (ARG, dict(Wp=None)),
    (ARG, dict(C=None)), (ALIGN, dict(x=X + 1)), (ALIGN, dict(xq=P + 16)),
    (ALIGN, dict(Wp=P2 + 16)), (WS, dict(nq=100)), (WS, dict(nw=100)),
    (ARG, dict(xq=X)), (ARG, dict(xq=P2)), (ARG, dict(C=X + 100)),
    (ARG, dict(C=P + 1024)), (ARG, dict(C=P2 + 1024)), (ARG, dict(bias=C + 4)),
    (ARG, dict(bias=P + 1024)), (ALIGN, dict(st=W + 4)), (ARG, dict(st=C)),
    (ARG, dict(st=P + 16)),
])
def test_linear_refusals(code, kw):
    refused(code, lambda: linear(**kw))
    linear(T=0)


def block(**kw):
    cfg = dict(hidden=128, ffn=512, shards=2, max_tokens=256, dtype=BF,
               use_layernorm=0, ln_eps=1e-5, gelu_mode=B.TPMLP_GELU_ERF)
    cfg.update(kw)
    return B.tp_mlp_create(B.tp_mlp_config(**cfg))


def test_block_sizes_and_refusals():
    up = lambda n: (n + 255) // 256 * 256
    for fmt in (NV, MX):
        h = block()
        assert B.tp_fp4_mlp_weights_bytes(h, fmt) == \
            up(B.tp_fp4_bytes(512, 128, fmt)) + up(B.tp_fp4_bytes(128, 512, fmt))
        assert B.tp_fp4_mlp_workspace_bytes(h, 10, fmt) == \
            up(B.tp_fp4_bytes(10, 128, fmt)) + up(B.tp_fp4_bytes(10, 512, fmt))
        n = block(use_layernorm=1)
        assert B.tp_fp4_mlp_workspace_bytes(n, 10, fmt) == \
            B.tp_fp4_mlp_workspace_bytes(h, 10, fmt) + up(2560) + 2 * up(40)
        assert B.tp_fp4_mlp_workspace_bytes(h, -1, fmt) == 0
    h = block()
    for other in (block(dropout_p=0.1), block(dtype=F32)):
        assert B.tp_fp4_mlp_weights_bytes(other, NV) == 0
        assert B.tp_fp4_mlp_workspace_bytes(other, 1, NV) == 0
        refused(ARG, lambda: forward(other))
    assert B.tp_fp4_mlp_weights_bytes(h, 5) == 0
    assert B.tp_fp4_mlp_weights_bytes(None, NV) == 0
    big = 1 << 30
    for code, kw in (
            (ARG, dict(fmt=4)), (SHAPE, dict(T=-1)), (SHAPE, dict(T=257)),
            (ARG, dict(X=None)), (ARG, dict(Z=None)), (ARG, dict(packed=None)),
            (ARG, dict(ws=None)), (ALIGN, dict(X=X + 8)), (ALIGN, dict(Z=C + 2)),
            (ALIGN, dict(b1=W + 4)), (ALIGN, dict(packed=P + 16)),
            (ALIGN, dict(ws=P2 + 16)), (WS, dict(ws_bytes=100)),
            (ARG, dict(Z=X)), (ARG, dict(Z=P + 512)), (ARG, dict(Z=P2 + 512)),
            (ARG, dict(ws=X - 256)), (ARG, dict(ws=P)), (ARG, dict(b1=P2 + 64)),
            (ARG, dict(b2=C)),
            (ARG, dict(xs=0.0)), (ARG, dict(ys=5.0)), (ARG, dict(fmt=MX, xs=2.0))):
        refused(code, lambda: forward(h, **kw))
    refused(ARG, lambda: forward(block(use_layernorm=1)))
    pack = lambda **k: B.tp_fp4_mlp_pack_weights(
        k.get("h", h), k.get("fmt", NV), k.get("A", X), k.get("B", C),
        k.get("packed", P), k.get("n", big), stream=0)
    for code, kw in ((ARG, dict(h=None)), (ARG, dict(fmt=2)), (ARG, dict(A=None)),
                     (ARG, dict(B=None)), (ARG, dict(packed=None)),
                     (ALIGN, dict(A=X + 8)), (ALIGN, dict(packed=P + 32)),
                     (WS, dict(n=1000)), (ARG, dict(packed=X + 256)),
                     (ARG, dict(packed=C))):
        refused(code, lambda: pack(**kw))


def forward(h, T=10, fmt=NV, X=X, packed=P, b1=None, b2=None, xs=1.0, ys=1.0,
            Z=C, ws=P2, ws_bytes=1 << 30):
    B.tp_fp4_mlp_forward(h, T, fmt, X, packed, b1, b2, None, None, xs, ys, Z, ws,
                         ws_bytes, stream=0)


def test_python_refusals_without_a_gpu():
    import torch
    x = torch.zeros(4, 32)
    for call in (lambda: fp4.quantize(x), lambda: fp4.quantize(x, "fp8"),
                 lambda: fp4.quantize(x, scale=-2.0),
                 lambda: fp4.Fp4Tensor(x, 4, 32, "int4"),
                 lambda: fp4.Fp4Linear(x, format="e2m1")):
        with pytest.raises(ValueError):
            call()
