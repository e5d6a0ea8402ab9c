"""CPU oracle for the four-bit formats: quantisation, its inverse, the packed
layout and products, in fp64 and integer arithmetic.

TEST INFRASTRUCTURE ONLY (never on the product path).

E2M1: sign, values 0 .5 1 1.5 2 3 4 6 (codes 0-7).  E4M3: 4-bit exponent of bias 7,
3-bit mantissa, largest value 448, code 0x7f NaN.  E8M0: 2^(code - 127), 255 NaN.
Roundings are found by comparing with the half-way points, whose products with the
scales are exact.
"""
from __future__ import annotations

import math

import numpy as np

E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
BLOCK = {"nvfp4": 16, "mxfp4": 32}


def e4m3_table():
    """The 127 values of codes 0 .. 126."""
    out = []
    for code in range(127):
        e, m = code >> 3, code & 7
        out.append(m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10))
    return np.array(out)


E4M3 = e4m3_table()


def round_e4m3(num, den=1.0):
    """Codes of num / den >= 0 to the nearest value, ties to the even code, at
    most 448: num is compared with den times the half-way points."""
    num = np.asarray(num, dtype=np.float64)
    mid = (E4M3[1:] + E4M3[:-1]) / 2 * den
    above = np.searchsorted(mid, num, side="left")     # mids strictly below num
    tie = np.isin(num, mid) & (above % 2 == 1)         # code `above` is odd: up
    return np.minimum(above + tie, 126).astype(np.int64)


def round_e2m1(mag, unit):
    """Codes of mag / unit (mag >= 0, unit > 0, or 0: code 0), ties to even."""
    code = np.zeros(mag.shape, dtype=np.int64)
    for i in range(7):
        border = (E2M1[i] + E2M1[i + 1]) / 2 * unit    # exact: 3 x 4 bits
        code += (mag > border) | ((mag == border) & (i % 2 == 1))
    return np.where(unit > 0, code, 0)


def auto_scale(x):
    """The smallest power of two g with max |x| <= 2688 g over finite x."""
    x = np.abs(np.asarray(x, dtype=np.float64))
    top = x[np.isfinite(x)].max(initial=0.0)
    if top == 0:
        return 1.0
    e = math.frexp(top)[1] - 13
    while top > 2688.0 * 2.0 ** e:
        e += 1
    return 2.0 ** max(e, -126)


def quantize(x, fmt, scale=None):
    """x [R, C]: (codes [R, C] with the sign in bit 3, scale codes [R, blocks],
    g)."""
    x = np.asarray(x, dtype=np.float64)
    R, C = x.shape
    size = BLOCK[fmt]
    n = -(-C // size)
    pad = np.zeros((R, n * size))
    pad[:, :C] = x
    b = pad.reshape(R, n, size)
    bad = ~np.isfinite(b).all(-1)
    b = np.where(bad[..., None], 0.0, b)
    amax = np.abs(b).max(-1)
    if fmt == "mxfp4":
        g = 1.0
        e = np.frexp(np.where(amax > 0, amax, 4.0))[1] - 1 - 2
        e = np.maximum(e, -127)
        byte = e + 127
        unit = np.ldexp(1.0, e)
        nan = 255
    else:
        g = auto_scale(x) if scale is None else float(scale)
        byte = round_e4m3(amax, 6.0 * g)
        unit = E4M3[byte] * g
        nan = 127
    codes = round_e2m1(np.abs(b), np.broadcast_to(unit[..., None], b.shape))
    codes = codes | (np.signbit(b) << 3)
    byte = np.where(bad, nan, byte)
    return codes.reshape(R, -1)[:, :C], byte.astype(np.int64), g


def scale_values(byte, fmt):
    if fmt == "mxfp4":
        return np.where(byte == 255, np.nan, np.ldexp(1.0, byte - 127))
    return np.where(byte == 127, np.nan, E4M3[np.minimum(byte, 126)])


def values(codes, byte, g, fmt):
    """What codes and scales stand for."""
    mag = E2M1[codes & 7] * np.where(codes >> 3, -1.0, 1.0)
    s = np.repeat(scale_values(byte, fmt), BLOCK[fmt], axis=1)[:, :codes.shape[1]]
    return mag * s * g


def quantized(x, fmt, scale=None):
    return values(*quantize(x, fmt, scale), fmt)


def pack(codes, byte, fmt):
    """The code section and the scale section as bytes (those of rows past the
    matrix are left 0)."""
    R, C = codes.shape
    per = 256 // BLOCK[fmt]
    rt, kt = -(-R // 128), -(-C // 256)
    full = np.zeros((rt * 128, kt * 256), dtype=np.uint8)
    full[:R, :C] = codes
    out = np.zeros((rt, kt, 128 * 128), dtype=np.uint8)
    for i in range(rt):
        for j in range(kt):
            t = full[128 * i:128 * i + 128, 256 * j:256 * j + 256]
            b = t[:, 0::2] | (t[:, 1::2] << 4)
            for r in range(128):
                for u in range(8):
                    at = r * 128 + (u ^ (r % 8)) * 16
                    out[i, j, at:at + 16] = b[r, 16 * u:16 * u + 16]
    empty = 127 if fmt == "mxfp4" else 0
    scales = np.zeros((rt, kt, 128 * per), dtype=np.uint8)
    for r in range(R):
        for b in range(kt * per):
            v = byte[r, b] if b < byte.shape[1] else empty
            at = b % per // 4 * 512 + r % 32 * 16 + r % 128 // 32 * 4 + b % 4
            scales[r // 128, b // per, at] = v
    return out.reshape(-1), scales.reshape(-1)


def matmul(a, b, bias=None):
    """Values a [T, K] times b [N, K]^T (+ bias)."""
    y = a @ b.T
    return y if bias is None else y + bias


def mlp_forward(X, A, B, fmt, b1=None, b2=None, x_scale=1.0, y_scale=1.0,
                gelu=None):
    """The block's forward (without LayerNorm): dict with Xq, H, Y, Yq (values)
    and Z."""
    from . import mlp as O
    scale = (lambda s: None) if fmt == "mxfp4" else (lambda s: s)
    Xq = quantized(X, fmt, scale(x_scale))
    H = matmul(Xq, quantized(A.T, fmt), b1)
    Y = (gelu or O.gelu)(H)
    Yq = quantized(Y, fmt, scale(y_scale))
    Z = matmul(Yq, quantized(B.T, fmt), b2)
    return dict(Xq=Xq, H=H, Y=Y, Yq=Yq, Z=Z)
