"""GPU parity of rotary positions and of the per-head norm of queries and keys
against the fp64 oracle (oracle/qk.py): both layouts, part of the head, every
vector width (aligned, odd and shifted rows), head dims up to 256, one token to
thousands, far and negative positions, strided and in-place calls, gradients,
repeats, streams and captured graphs."""
import math

import numpy as np
import pytest
import torch

from oracle import qk as O
from tensor_transformer_mlp_tcgen05_gb300 import binding as B
from tensor_transformer_mlp_tcgen05_gb300.rotary import (QKNormRotary,
                                                         RotaryEmbedding)

pytestmark = pytest.mark.gpu

# Tolerances.  A result is rounded once to its type: at most half a step,
# eps / 2 of its value (bf16 2^-8, fp32 2^-24).  Before that, in units u =
# 2^-24 of the largest value M of the head row:
#   rotation: the angle is within pi u (its conversion to fp32) + 2^-33 turns,
#   sincospif within 2 ulp, times amp 1 u: each of two products is off by at
#   most (3.2 + 2 + 1 + 1) u M, their sum by one more, amp <= 1.4: under 32 u M.
#   norm: the mean and the sum of squares add d / 8 values in a lane (<= 16)
#   and 4 rounds of a tree, each rounding u of the sum: the mean is off by 20 u
#   max |x|, the root of the mean square by 10 u of itself, rsqrtf 2 ulp, two
#   products and one sum: under 64 u M with M = max |x| rstd max |gamma| + max
#   |beta| (the rotation included: another 32).
# K_ROPE and K_NORM below are these.
U = 2.0 ** -24
K_ROPE, K_NORM = 32, 96
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def f64(t):
    return t.detach().cpu().double().numpy()


def flat(t):
    """[T, H, d] of a [T, H, d] or [T, t, H / t, d] tensor."""
    return f64(t).reshape(t.shape[0], -1, t.shape[-1])


def within(got, want, big, k, dtype):
    """|got - want| <= half a step of want + k u M per head row; big: M."""
    err = np.abs(got - want)
    tol = HALF_STEP[dtype] * np.abs(want) * (1 + 2 * k * U) + k * U * big
    assert np.isfinite(got).all()
    assert (err <= tol).all(), (err.max(), (err / np.maximum(tol, 1e-300)).max())


def rows_max(x):
    return np.abs(x).max(axis=-1, keepdims=True)


def make(T, hq, hk, d, dtype, seed, layout="plain"):
    g = torch.Generator("cuda").manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=g, device="cuda").to(dtype)
    if layout == "shards":            # hq == hk, two shards
        x = n(T, 2, 3, hq // 2, d)
        return x[:, :, 0], x[:, :, 1]
    if layout == "fused":             # [T, hq + hk + 1, d], rows one apart
        x = n(T, hq + hk + 1, d)
        return x[:, :hq], x[:, hq:hq + hk]
    if layout == "major":             # [H, T, d]
        return n(hq, T, d).transpose(0, 1), n(hk, T, d).transpose(0, 1)
    if layout == "shifted":           # off by one element, odd row pitch
        a = n(T * (hq * (d + 3)) + 1)[1:].view(T, hq, d + 3)[..., :d]
        b = n(T * (hk * (d + 3)) + 1)[1:].view(T, hk, d + 3)[..., :d]
        return a, b
    return n(T, hq, d), n(T, hk, d)


# (d, r): rows of whole 16-byte vectors that fill lanes exactly and that do not,
# rows moved element by element in pieces of 16, 8, 4 and 2 bytes, few and many
# elements past r, the smallest and the largest
DIMS = [(64, 64), (128, 128), (96, 96), (80, 40), (128, 32), (256, 256),
        (256, 64), (72, 72), (100, 100), (40, 20), (36, 12), (24, 10), (10, 6),
        (2, 2), (7, 4), (1, 0), (64, 0), (192, 48), (250, 250), (255, 254),
        (160, 160), (32, 32), (16, 16), (48, 32), (112, 112), (256, 2), (8, 8),
        (4, 2), (128, 126), (192, 192), (224, 128)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("d,r", DIMS)
def test_rotation(d, r, inter, dtype):
    T, hq, hk = 37, 6, 2
    q, k = make(T, hq, hk, d, dtype, d + r)
    rope = RotaryEmbedding(d, rotary_dim=r, interleaved=inter)
    f, amp = O.frequencies(r)
    pos = torch.randint(-50, 5000, (T,), device="cuda",
                        generator=torch.Generator("cuda").manual_seed(1))
    yq, yk = rope.forward(q, k, positions=pos)
    gq, gk = rope.backward(q, k, positions=pos.to(torch.int32))
    for x, y, g in ((q, yq, gq), (k, yk, gk)):
        m = rows_max(flat(x))
        p = pos.cpu().numpy()
        within(flat(y), O.rotate(flat(x), p, f, inter, amp), m, K_ROPE, dtype)
        within(flat(g), O.rotate(flat(x), p, f, inter, amp, inverse=True), m,
               K_ROPE, dtype)
        assert torch.equal(y[..., r:], x[..., r:])


@pytest.mark.parametrize("norm", ["rms", "layer"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("d,r", DIMS)
def test_norm_and_rotation(d, r, inter, dtype, norm):
    T, hq, hk = 29, 3, 5
    q, k = make(T, hq, hk, d, dtype, 3 * d + r)
    g = torch.Generator("cuda").manual_seed(d)
    par = [torch.randn(d, generator=g, device="cuda") for _ in range(4)]
    bq, bk = (par[2], par[3]) if norm == "layer" else (None, None)
    rope = RotaryEmbedding(d, rotary_dim=r, interleaved=inter, base=500.0)
    op = QKNormRotary(d, norm=norm, eps=1e-5, rotary=rope)
    f, _ = O.frequencies(r, base=500.0)
    yq, yk = op.forward(q, k, par[0], par[1], bq, bk, offset=3, seq_len=11)
    pos = 3 + np.arange(T) % 11
    for x, y, ga, be in ((q, yq, par[0], bq), (k, yk, par[1], bk)):
        n = None if be is None else f64(be)
        want = O.forward(flat(x), pos, f, norm, 1e-5, f64(ga), n, inter)
        rstd = O.normal(flat(x), norm, 1e-5)[1]
        big = (rows_max(flat(x)) * rstd * np.abs(f64(ga)).max() +
               (0 if n is None else np.abs(n).max()))
        within(flat(y), want, big, K_NORM, dtype)


def check_gradients(op, q, k, dq, dk, gq, gk, pos, f, inter, dtype, got,
                    amp=1.0, params=True):
    """dx within half a step plus, in units u of M = rstd (max |u| + max |xh|
    |mean(u xh)| + |mean u|): g and u as the rotation (32), the two means over
    d <= 256 values 20 each of at most max |u| max |xh|, xh as the norm (64) and
    four more roundings: 256 u M with the mean taken as max |u xh|.  Parameter
    gradients: the sum's chain of roundings is at most the rows of a lane, the
    row slots of a block (128), 20 blocks and 32 partial sums, each u of sum |g
    xh|, and the terms themselves are off by 100 u."""
    d = q.shape[-1]
    for n, dy, x, ga in (("q", dq, q, gq), ("k", dk, k, gk)):
        if dy is None:
            continue
        gamma = None if ga is None else f64(ga)
        want = O.backward(flat(dy), flat(x), pos, f, op.norm, op.eps, gamma,
                          inter, amp)
        g = O.rotate(flat(dy), pos, f, inter, amp, inverse=True)
        xh, rstd = O.normal(flat(x), op.norm, op.eps)
        u = g if gamma is None else g * gamma
        umax = rows_max(flat(dy)) * 1.5 * amp * (
            1 if gamma is None else np.abs(gamma).max())
        big = rstd * umax * (2 + rows_max(xh) ** 2)
        within(flat(got["d" + n]), want["dx"], big, 256, dtype)
        if not params:
            continue
        T, H = flat(x).shape[:2]
        chain = T * H // 2000 + H + 180 + 100
        for name, terms in (("gamma", g * xh), ("beta", g)):
            key = "d%s_%s" % (n, name)
            if name == "beta" and op.norm != "layer":
                assert key not in got
                continue
            tol = chain * U * np.abs(terms).sum((0, 1)) + 1e-30
            if name == "gamma":      # xh of a row is off by 64 u of its largest
                tol = tol + 64 * U * (np.abs(g) * rows_max(xh)).sum((0, 1))
            # a pair's elements are off by u of either
            tol = tol.max() if len(f) else tol
            assert (np.abs(f64(got[key]) - want["d" + name]) <= tol).all(), key


@pytest.mark.parametrize("norm", ["rms", "layer"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("d,r", DIMS)
def test_norm_gradients(d, r, inter, dtype, norm):
    T, hq, hk = 45, 6, 2
    q, k = make(T, hq, hk, d, dtype, 5 * d + r)
    dq, dk = make(T, hq, hk, d, dtype, 7 * d + r)
    g = torch.Generator("cuda").manual_seed(d)
    gq, gk = (1 + 0.3 * torch.randn(d, generator=g, device="cuda")
              for _ in range(2))
    rope = RotaryEmbedding(d, rotary_dim=r, interleaved=inter)
    op = QKNormRotary(d, norm=norm, eps=1e-4, rotary=rope)
    got = op.backward(dq, dk, q, k, gq, gk, offset=-4)
    check_gradients(op, q, k, dq, dk, gq, gk, np.arange(T) - 4,
                    O.frequencies(r)[0], inter, dtype, got)


@pytest.mark.parametrize("layout", ["shards", "fused", "major", "shifted"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d,r", [(96, 48), (64, 64), (7, 6), (128, 2)])
def test_strided_views(layout, dtype, d, r):
    T, H = 130, 6
    q, k = make(T, H, H, d, dtype, 11, layout)
    dq, dk = make(T, H, H, d, dtype, 12, layout)
    rope = RotaryEmbedding(d, rotary_dim=r)
    op = QKNormRotary(d, norm="layer", rotary=rope)
    f, _ = O.frequencies(r)
    pos = np.arange(T) % 50
    y = rope.forward(q, k, seq_len=50)
    z = op.forward(q, k, seq_len=50)
    for x, a, b in ((q, y[0], z[0]), (k, y[1], z[1])):
        assert a.is_contiguous() and a.shape == x.shape
        within(flat(a), O.rotate(flat(x), pos, f), rows_max(flat(x)), K_ROPE,
               dtype)
        rstd = O.normal(flat(x), "layer", op.eps)[1]
        within(flat(b), O.forward(flat(x), pos, f, "layer", op.eps),
               rows_max(flat(x)) * rstd, K_NORM, dtype)
    got = op.backward(dq, dk, q, k, seq_len=50)
    check_gradients(op, q, k, dq, dk, None, None, pos, f, False, dtype, got)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("d,r", DIMS)
def test_rotation_in_place(d, r, inter, dtype):
    """Equal to out of place; the elements past r stay as they were."""
    T, hq, hk = 23, 5, 3
    q, k = make(T, hq, hk, d, dtype, d + 2 * r)
    rope = RotaryEmbedding(d, rotary_dim=r, interleaved=inter)
    want = rope.forward(q, k, offset=9)
    got = rope.forward(q, k, offset=9, q_out=q, k_out=k)
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_parameters_off_16_bytes():
    d = 128
    q, k = make(50, 4, 4, d, torch.bfloat16, 6)
    dq, dk = make(50, 4, 4, d, torch.bfloat16, 7)
    g = torch.Generator("cuda").manual_seed(8)
    par = [torch.randn(d, generator=g, device="cuda") for _ in range(4)]
    room = torch.empty(4, d + 1, device="cuda")
    off = [room[i, 1:].copy_(p) if (i % 2 == 0) else p.clone()
           for i, p in enumerate(par)]
    assert any(p.data_ptr() % 16 for p in off)
    op = QKNormRotary(d, norm="layer", rotary=RotaryEmbedding(d))
    for a, b in zip(op.forward(q, k, *par), op.forward(q, k, *off)):
        assert torch.equal(a, b)
    a = op.backward(dq, dk, q, k, *par[:2])
    b = op.backward(dq, dk, q, k, *off[:2],
                    out={"dq_gamma": room.view(-1)[3:3 + d]})
    for n in a:
        assert torch.equal(a[n], b[n]), n


@pytest.mark.parametrize("r", [96, 40])
def test_in_place_equals_out_of_place_and_leaves_the_rest(r):
    T, H, d = 200, 4, 96
    g = torch.Generator("cuda").manual_seed(4)
    qkv = torch.randn((T, 2, 3, H // 2, d), generator=g,
                      device="cuda").to(torch.bfloat16)
    before = qkv.clone()
    rope = RotaryEmbedding(d, rotary_dim=r, interleaved=True)
    op = QKNormRotary(d, rotary=rope)
    for call in (rope.forward, op.forward):
        qkv.copy_(before)
        q, k = qkv[:, :, 0], qkv[:, :, 1]
        want = call(q, k, seq_len=100)
        call(q, k, seq_len=100, q_out=q, k_out=k)
        assert torch.equal(q, want[0]) and torch.equal(k, want[1])
        assert torch.equal(qkv[:, :, 2], before[:, :, 2])
    # gradients over dq, and over q
    qkv.copy_(before)
    dqkv = torch.randn_like(before)
    args = [qkv[:, :, 0], qkv[:, :, 1]]
    grad = lambda: [dqkv[:, :, 0], dqkv[:, :, 1]]
    want = op.backward(*grad(), *args)
    keep = dqkv.clone()
    over = dict(dq=dqkv[:, :, 0], dk=dqkv[:, :, 1])
    op.backward(*grad(), *args, out=over)
    assert torch.equal(over["dq"], want["dq"])
    assert torch.equal(dqkv[:, :, 1], want["dk"])
    assert torch.equal(dqkv[:, :, 2], keep[:, :, 2])
    for n in ("dq_gamma", "dk_gamma"):
        assert torch.equal(over[n], want[n])
    dqkv.copy_(keep)
    op.backward(*grad(), *args, out=dict(dq=args[0], dk=args[1]))
    assert torch.equal(args[0], want["dq"]) and torch.equal(args[1], want["dk"])


def test_outputs_touch_nothing_else():
    # an output with room between its rows: the room stays as it was
    T, H, d = 33, 3, 40
    q, _ = make(T, H, 1, d, torch.bfloat16, 5)
    buf = torch.full((T + 2, H + 1, d + 8), 7.0, device="cuda",
                     dtype=torch.bfloat16)
    out = buf[1:T + 1, :H, 8:]
    RotaryEmbedding(d).forward(q, q_out=out)
    want, _ = RotaryEmbedding(d).forward(q)
    assert torch.equal(out, want)
    out.fill_(7.0)
    assert (buf == 7.0).all()


@pytest.mark.parametrize("T", [1, 2, 3, 31, 32, 33, 1000, 5000])
@pytest.mark.parametrize("hq,hk", [(1, 1), (40, 40), (7, 3)])
def test_token_and_head_counts(T, hq, hk):
    d = 64
    q, k = make(T, hq, hk, d, torch.bfloat16, T)
    dq, dk = make(T, hq, hk, d, torch.bfloat16, T + 1)
    rope = RotaryEmbedding(d)
    op = QKNormRotary(d, rotary=rope)
    f, _ = O.frequencies(d)
    pos = np.arange(T) + 17
    y = op.forward(q, k, offset=17)
    for x, a in ((q, y[0]), (k, y[1])):
        rstd = O.normal(flat(x), "rms", op.eps)[1]
        within(flat(a), O.forward(flat(x), pos, f, "rms", op.eps),
               rows_max(flat(x)) * rstd, K_NORM, torch.bfloat16)
    got = op.backward(dq, dk, q, k, offset=17)
    check_gradients(op, q, k, dq, dk, None, None, pos, f, False,
                    torch.bfloat16, got)


def test_queries_alone():
    q, _ = make(50, 5, 1, 64, torch.float32, 8)
    dq, _ = make(50, 5, 1, 64, torch.float32, 9)
    op = QKNormRotary(64, norm="layer")
    y, none = op.forward(q)
    assert none is None
    within(flat(y), O.forward(flat(q), np.arange(50), [], "layer", op.eps),
           rows_max(flat(q)) * O.normal(flat(q), "layer", op.eps)[1], K_NORM,
           torch.float32)
    got = op.backward(dq, None, q, None)
    assert sorted(got) == ["dq", "dq_beta", "dq_gamma"]
    check_gradients(op, q, None, dq, None, None, None, np.arange(50),
                    np.zeros(0), False, torch.float32, got)


def test_no_tokens():
    q = torch.empty((0, 4, 64), dtype=torch.bfloat16, device="cuda")
    op = QKNormRotary(64, norm="layer", rotary=RotaryEmbedding(64))
    assert op.rotary.forward(q, q)[1].shape == (0, 4, 64)
    assert op.forward(q, q)[0].shape == (0, 4, 64)
    g = op.backward(q, q, q, q)
    for n in ("dq_gamma", "dk_gamma", "dq_beta", "dk_beta"):
        assert (g[n] == 0).all()


@pytest.mark.parametrize("kw", [
    dict(scaling="linear", factor=8.0), dict(scaling="ntk", factor=8.0),
    dict(scaling="yarn", factor=8.0, original_length=4096)])
def test_far_positions(kw):
    # angles keep 2^-33 of a turn at any position: the fp32 tolerance holds at
    # 2^31 and beyond (the oracle's own angle, pos f in extended or double
    # precision, is off by 2^-53 pos f: 2^-19 u at 2^33, nothing)
    T, d = 64, 128
    q, k = make(T, 2, 1, d, torch.float32, 21)
    g = torch.Generator("cuda").manual_seed(2)
    pos = torch.randint(-(1 << 31), 1 << 31, (T,), generator=g, device="cuda")
    rope = RotaryEmbedding(d, **kw)
    f, amp = O.frequencies(d, **kw)
    # the frequencies themselves are held to 2^-53 of a turn: 2^31 2^-54 turns
    # is 2^-23 turns, 6.3 u 2 of an angle, and the oracle's as much again
    y, _ = rope.forward(q, k, positions=pos)
    within(flat(y), O.rotate(flat(q), pos.cpu().numpy(), f, amp=amp),
           rows_max(flat(q)) * amp, K_ROPE + 32, torch.float32)
    lim = torch.tensor([2 ** 62, -2 ** 62], device="cuda")
    z, _ = rope.forward(q[:2], positions=lim)
    n = lambda t: np.sqrt((f64(t) ** 2).sum(-1))
    assert np.allclose(n(z), n(q[:2]) * amp, rtol=1e-5)


def test_whole_turns_drop_out():
    # a quarter turn per position: positions 4 n + m are m exactly
    q, _ = make(8, 1, 1, 2, torch.float32, 1)
    rope = RotaryEmbedding(2, inv_freq=[math.pi / 2])
    a, _ = rope.forward(q, offset=0)
    b, _ = rope.forward(q, offset=4 * 12345)
    assert torch.equal(a, b)


def test_gradient_against_differences():
    # <dx, v> against (L(x + h v) - L(x - h v)) / 2h, L = <dy, y>: L is about
    # sqrt(n) = 100 and rounded, as its terms are, to u of their sum of
    # magnitudes n = 1e4: 2 u n / 2h = 0.06 for h = 1e-2; the third derivative
    # adds h^2 / 6 of about the same size as the sum (100): 2e-3
    T, H, d = 20, 4, 128
    q, _ = make(T, H, 1, d, torch.float32, 31)
    dy, _ = make(T, H, 1, d, torch.float32, 32)
    v, _ = make(T, H, 1, d, torch.float32, 33)
    for norm in ("rms", "layer"):
        op = QKNormRotary(d, norm=norm, rotary=RotaryEmbedding(d))
        ga = 1 + 0.1 * torch.randn(d, device="cuda", generator=torch.Generator(
            "cuda").manual_seed(3))
        h = 1e-2
        loss = lambda x: float((op.forward(x, q_gamma=ga)[0].double() *
                                dy.double()).sum())
        num = (loss(q + h * v) - loss(q - h * v)) / (2 * h)
        got = op.backward(dy, None, q, None, ga)
        assert abs(num - float((got["dq"].double() * v.double()).sum())) < 0.1
        w = torch.randn(d, device="cuda",
                        generator=torch.Generator("cuda").manual_seed(4))
        at = lambda gam: float((op.forward(q, q_gamma=gam)[0].double() *
                                dy.double()).sum())
        num = (at(ga + h * w) - at(ga - h * w)) / (2 * h)
        assert abs(num - float((got["dq_gamma"].double() * w.double()).sum())) \
            < 0.1


def test_values_that_are_not_finite_stay_in_their_row():
    T, H, d = 9, 5, 96
    q, k = make(T, H, H, d, torch.bfloat16, 41)
    clean = [QKNormRotary(d, rotary=RotaryEmbedding(d)).forward(q, k),
             RotaryEmbedding(d).forward(q, k)]
    q2 = q.clone()
    q2[3, 2, 7] = float("nan")
    q2[4, 1, 95] = float("inf")
    dirty = [QKNormRotary(d, rotary=RotaryEmbedding(d)).forward(q2, k),
             RotaryEmbedding(d).forward(q2, k)]
    rows = torch.ones(T, H, dtype=torch.bool, device="cuda")
    rows[3, 2] = rows[4, 1] = False
    for c, n in zip(clean, dirty):
        assert torch.equal(c[0][rows], n[0][rows])
        assert torch.equal(c[1], n[1])
        assert not torch.isfinite(n[0][3, 2]).all()


@pytest.mark.parametrize("d,r", [(128, 64), (96, 48), (128, 32), (100, 50),
                                 (64, 0), (72, 18)])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_values_that_are_not_finite_stay_with_their_pair(d, r, inter, bad):
    """One bad value at a time: the rotation makes its pair bad (or, past r, the
    value alone), the RMS norm the same (the others become zero beside an
    infinity, and are not numbers beside a NaN), as the formula has it."""
    q = torch.ones((d, 1, d), dtype=torch.bfloat16, device="cuda")
    i = torch.arange(d, device="cuda")
    q[i, 0, i] = bad                       # token t: element t
    rope = RotaryEmbedding(d, rotary_dim=r, interleaved=inter)
    f = torch.tensor(rope.frequencies()[0], device="cuda")
    ang = (i + 1)[:, None] * f

    def rotate(x, sign=1.0):
        x = x[:, 0].double()
        c, s = torch.cos(ang), sign * torch.sin(ang)
        a, b = ((x[:, 0:r:2], x[:, 1:r:2]) if inter
                else (x[:, :r // 2], x[:, r // 2:r]))
        y = x.clone()
        ya, yb = a * c - b * s, a * s + b * c
        if inter:
            y[:, 0:r:2], y[:, 1:r:2] = ya, yb
        else:
            y[:, :r // 2], y[:, r // 2:r] = ya, yb
        return y

    def kinds(t):
        return torch.isnan(t), torch.isposinf(t), torch.isneginf(t)

    y, _ = rope.forward(q, offset=1)
    for a, b in zip(kinds(y[:, 0]), kinds(rotate(q))):
        assert torch.equal(a, b)
    op = QKNormRotary(d, rotary=rope)
    y, _ = op.forward(q, offset=1)
    x = q.float()
    want = rotate(x * torch.rsqrt((x * x).mean(-1, keepdim=True) + op.eps))
    assert torch.equal(torch.isnan(y[:, 0]), torch.isnan(want))
    # the gradient of beta: a bad value of dy reaches its pair's columns only
    op = QKNormRotary(d, norm="layer", rotary=rope)
    x, _ = make(1, 1, 1, d, torch.bfloat16, d)
    for t in (0, max(r - 1, 0), min(r, d - 1), d - 1):
        g = op.backward(q[t:t + 1], None, x, None, offset=t + 1)
        want = rotate(q, -1.0)[t]
        assert torch.equal(torch.isfinite(g["dq_beta"]), torch.isfinite(want))


def test_rows_of_zeros():
    # rstd = 1 / sqrt(eps): zero rows give beta, and finite gradients
    q = torch.zeros((4, 2, 64), dtype=torch.bfloat16, device="cuda")
    dy = torch.ones_like(q)
    be = torch.full((64,), 0.5, device="cuda")
    for norm in ("rms", "layer"):
        op = QKNormRotary(64, norm=norm)
        y, _ = op.forward(q, q_beta=be if norm == "layer" else None)
        assert (y == (0.5 if norm == "layer" else 0.0)).all()
        g = op.backward(dy, None, q, None)
        want = 0.0 if norm == "layer" else 1e3     # 1 / sqrt(1e-6)
        assert torch.allclose(g["dq"].float(), torch.full_like(
            g["dq"], want).float(), rtol=2 ** -8)
        assert (g["dq_gamma"] == 0).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d", [64, 96, 10])
@pytest.mark.parametrize("norm", ["rms", "layer"])
def test_rows_of_zeros_with_the_smallest_eps(dtype, d, norm):
    """eps = 2^-130: rstd = 2^65, whose square is past fp32's range."""
    q = torch.zeros((4, 2, d), dtype=dtype, device="cuda")
    g = QKNormRotary(d, norm=norm, eps=2.0 ** -130).backward(
        torch.ones_like(q), None, q, None)
    want = 2.0 ** 65 if norm == "rms" else 0.0
    # rsqrt is off by two steps at most; the mean of d ones by d / 2 of them
    assert torch.allclose(g["dq"].double(), torch.full_like(g["dq"], want).double(),
                          rtol=HALF_STEP[dtype] + (2 + d) * U, atol=2.0 ** 65 * (2 + d) * U)
    assert (g["dq_gamma"] == 0).all()


def test_offsets_past_32_bits():
    # token stride 2^26 elements: token 33's row starts past 2^31 elements
    T, H, d = 36, 2, 64
    buf = torch.empty(T * (1 << 26), dtype=torch.bfloat16, device="cuda")
    x = buf.as_strided((T, H, d), (1 << 26, d, 1))
    src, _ = make(T, H, 1, d, torch.bfloat16, 51)
    x.copy_(src)
    rope = RotaryEmbedding(d)
    want, _ = rope.forward(src)
    got, _ = rope.forward(x, q_out=x)
    assert torch.equal(got, want)


def test_repeats_are_bit_identical():
    q, k = make(3000, 12, 4, 80, torch.bfloat16, 61)
    dq, dk = make(3000, 12, 4, 80, torch.bfloat16, 62)
    op = QKNormRotary(80, norm="layer", rotary=RotaryEmbedding(80))
    a = op.backward(dq, dk, q, k)
    for _ in range(3):
        b = op.backward(dq, dk, q, k)
        for n in a:
            assert torch.equal(a[n], b[n]), n


def test_streams_side_by_side():
    """Two calls of one object on two streams share nothing."""
    op = QKNormRotary(128, rotary=RotaryEmbedding(128))
    data = [make(2000, 8, 8, 128, torch.bfloat16, 70 + i) +
            make(2000, 8, 8, 128, torch.bfloat16, 80 + i) for i in range(2)]
    want = [op.backward(d[2], d[3], d[0], d[1]) for d in data]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for i, d in enumerate(data):
            got[i].append(op.backward(d[2], d[3], d[0], d[1],
                                      stream=streams[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for g in got[i]:
            for n in g:
                assert torch.equal(g[n], want[i][n])
    # a raw stream handle
    y, _ = op.forward(data[0][0], stream=streams[0].cuda_stream)
    streams[0].synchronize()
    assert torch.equal(y, op.forward(data[0][0])[0])


def test_captured_graphs():
    op = QKNormRotary(64, norm="layer", rotary=RotaryEmbedding(64))
    q, k = make(100, 4, 4, 64, torch.bfloat16, 91)
    dq, dk = make(100, 4, 4, 64, torch.bfloat16, 92)
    pos = torch.arange(100, device="cuda")
    runs = lambda: (op.forward(q, k, positions=pos),
                    op.backward(dq, dk, q, k, positions=pos))
    runs()
    torch.cuda.synchronize()
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(runs())
        graphs.append(g)
    for step in range(3):
        fresh = make(100, 4, 4, 64, torch.bfloat16, 93 + step)
        q.copy_(fresh[0])
        k.copy_(fresh[1])
        pos.add_(13)
        for g in graphs:
            g.replay()
        (y, z), g1 = runs()
        torch.cuda.synchronize()
        for (a, b), g2 in outs:
            assert torch.equal(a, y) and torch.equal(b, z)
            for n in g1:
                assert torch.equal(g1[n], g2[n]), n


def test_refusals_of_the_wrappers():
    q, k = make(8, 4, 2, 64, torch.bfloat16, 95)
    rope = RotaryEmbedding(64)
    op = QKNormRotary(64, rotary=rope)
    one = torch.ones(64, device="cuda")
    bad = [
        lambda: rope.forward(q.cpu(), k),
        lambda: rope.forward(q.half(), k.half()),
        lambda: rope.forward(q, k.float()),
        lambda: rope.forward(q, k[:4]),
        lambda: rope.forward(q[..., :32], k),
        lambda: rope.forward(q[..., ::2], k),
        lambda: rope.forward(q[0], k[0]),
        lambda: rope.forward(q, k, positions=torch.arange(7, device="cuda")),
        lambda: rope.forward(q, k, positions=torch.arange(8)),
        lambda: rope.forward(q, k, positions=torch.zeros(8, device="cuda")),
        lambda: rope.forward(q, k, positions=torch.arange(
            16, device="cuda")[::2]),
        lambda: rope.forward(q, q_out=k),
        lambda: rope.forward(q, k_out=k),
        lambda: op.forward(q, k, q_gamma=torch.ones(32, device="cuda")),
        lambda: op.forward(q, k, q_gamma=torch.ones(64)),
        lambda: op.backward(q, None, q, k),
        lambda: op.backward(q, k, q, None),
        lambda: op.backward(q, k, q[:4], k),
        lambda: op.backward(q, k, q, k, out={"dq_beta": one}),
        lambda: op.backward(q, None, q, None, out={"dk_gamma": one}),
    ]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    lib_bad = [
        lambda: rope.forward(q, k, seq_len=-1),
        lambda: rope.forward(q, q_out=q[:1].expand(8, 4, 64)),
        lambda: rope.forward(q[:, :2], q[:, 2:], q_out=q[:, 1:3],
                             k_out=q[:, 2:]),
        lambda: op.forward(q, k, q_beta=torch.ones(64, device="cuda")),
    ]
    for call in lib_bad:
        with pytest.raises(B.TPMLPError):
            call()


def test_lazy_copies_as_outputs_get_memory_of_their_own():
    d = 64
    q, k = make(50, 4, 2, d, torch.bfloat16, 101)
    dq, dk = make(50, 4, 2, d, torch.bfloat16, 102)
    keep = [t.clone() for t in (q, k, dq, dk)]
    rope = RotaryEmbedding(d, rotary_dim=32)
    op = QKNormRotary(d, norm="layer", rotary=rope)
    for call in (rope.forward, op.forward, rope.backward):
        want = call(q, k, offset=5)
        outs = [torch._lazy_clone(t) for t in (q, k)]
        got = call(q, k, offset=5, q_out=outs[0], k_out=outs[1])
        for a, b, c in zip(outs, want, got):
            assert torch.equal(a, b) and torch.equal(c, b)
        # in place in a tensor that another one still shares
        outs = [torch._lazy_clone(t) for t in (q, k)]
        call(outs[0], outs[1], offset=5, q_out=outs[0], k_out=outs[1])
        for a, b in zip(outs, want):
            assert torch.equal(a, b)
    want = op.backward(dq, dk, q, k)
    par = {n: torch.full((d,), 3.0, device="cuda")
           for n in ("dq_gamma", "dk_gamma", "dq_beta", "dk_beta")}
    out = {n: torch._lazy_clone(t) for n, t in par.items()}
    out.update(dq=torch._lazy_clone(q), dk=torch._lazy_clone(dk))
    op.backward(dq, dk, q, k, out=out)
    for n in want:
        assert torch.equal(out[n], want[n]), n
    for t in par.values():
        assert (t == 3.0).all()
    for a, b in zip((q, k, dq, dk), keep):
        assert torch.equal(a, b)


@pytest.mark.parametrize("norm", ["rms", "layer"])
def test_without_parameter_gradients(norm):
    """param_grads=False: dq and dk alone, the same bits; parameter gradients
    that are given all the same are refused, not handed back unwritten."""
    q, k = make(40, 4, 2, 64, torch.bfloat16, 103)
    dq, dk = make(40, 4, 2, 64, torch.bfloat16, 104)
    op = QKNormRotary(64, norm=norm, rotary=RotaryEmbedding(64))
    want = op.backward(dq, dk, q, k)
    got = op.backward(dq, dk, q, k, param_grads=False)
    assert sorted(got) == ["dk", "dq"]
    for n in got:
        assert torch.equal(got[n], want[n])
    for n in ("dq_gamma", "dk_gamma", "dq_beta", "dk_beta"):
        given = torch.full((64,), 5.0, device="cuda")
        with pytest.raises(ValueError):
            op.backward(dq, dk, q, k, param_grads=False, out={n: given})
        assert (given == 5.0).all()


def _turns(positions, freqs):
    """p f / 2 pi modulo one turn, exact integer arithmetic on the doubles f and
    1 / 2 pi to 300 bits (pi by Machin's formula), as floats of [-1/2, 1/2)."""
    from fractions import Fraction
    bits = 320

    def arctan_inverse(n):
        total, term, k, sign = 0, (1 << bits) // n, 1, 1
        while term:
            total += sign * (term // k)
            term //= n * n
            k += 2
            sign = -sign
        return total

    two_pi = 8 * (4 * arctan_inverse(5) - arctan_inverse(239))
    assert abs(two_pi / (1 << bits) - 2 * math.pi) < 1e-15
    out = np.empty((len(positions), len(freqs)))
    for j, f in enumerate(freqs):
        per = Fraction(f) * (1 << bits) / two_pi      # turns per position
        for i, p in enumerate(positions):
            t = (per * int(p)) % 1
            out[i, j] = float(t if t < Fraction(1, 2) else t - 1)
    return out


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("base", [10000.0, 500000.0, None])
def test_angles_of_the_furthest_positions(base, inter):
    """The angle of the frequencies as they are reported, at positions of 2^20
    to 2^36: the phase is within 2^-33 of a turn (its 32 bits), and |p| 2^-64 from
    the frequency's 64, 2^-28 at 2^36, together under 2^-27.9 turns, which is
    2^-25.2 or 0.43 u of an angle.  Of the rotation's tolerance, by its own
    derivation, (3.2 + 2 + 1 + 1) u M for each product and 1.5 u M for their sum,
    15.9 u M, 0.9 more."""
    d = 64
    kw = dict(base=base) if base else dict(
        inv_freq=[(-1) ** i * 2.0 ** (3 - i) / 3 for i in range(d // 2)])
    rope = RotaryEmbedding(d, interleaved=inter, **kw)
    f, amp = rope.frequencies()
    g = torch.Generator("cuda").manual_seed(5)
    pos = torch.cat([torch.randint(-(1 << b), 1 << b, (12,), generator=g,
                                   device="cuda") for b in (20, 24, 28, 31, 36)] +
                    [torch.tensor([(1 << 31) - 1, -(1 << 31), 4000000],
                                  device="cuda")])
    q, _ = make(len(pos), 2, 1, d, torch.float32, 105)
    y, _ = rope.forward(q, positions=pos)
    ang = 2 * math.pi * _turns(pos.tolist(), f)
    c, s = np.cos(ang)[:, None], np.sin(ang)[:, None]
    x, want = flat(q), flat(q)
    ia, ib = ((slice(0, d, 2), slice(1, d, 2)) if inter
              else (slice(0, d // 2), slice(d // 2, d)))
    want[..., ia] = x[..., ia] * c - x[..., ib] * s
    want[..., ib] = x[..., ia] * s + x[..., ib] * c
    within(flat(y), amp * want, rows_max(x) * amp, 17, torch.float32)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("d,r", [(128, 64), (96, 48), (100, 50), (64, 0),
                                 (72, 18)])
@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_a_bias_that_is_not_finite_stays_with_its_element(d, r, inter, dtype,
                                                          bad):
    """Past r a bias reaches its own element only; before, its pair."""
    rope = RotaryEmbedding(d, rotary_dim=r, interleaved=inter)
    op = QKNormRotary(d, norm="layer", rotary=rope)
    q, _ = make(1, 3, 1, d, dtype, 106)
    for e in sorted({0, max(r - 1, 0), min(r, d - 1), (r + d) // 2, d - 1}):
        beta = torch.zeros(d, device="cuda")
        beta[e] = bad
        y, _ = op.forward(q, q_beta=beta, offset=1)
        hit = torch.zeros(d, dtype=torch.bool, device="cuda")
        hit[e] = True
        if e < r:
            hit[e ^ 1 if inter else (e + r // 2) % r] = True
        assert torch.equal(~torch.isfinite(y), hit.expand_as(y)), e


# rows of 31 units of fp32: one lane of the warp idle, 62 pieces of 16 bytes
@pytest.mark.parametrize("norm", ["rms", "layer"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("d,r", [(248, 248), (248, 64), (240, 240), (232, 80)])
def test_rows_of_nearly_a_warp(d, r, inter, dtype, norm):
    T, hq, hk = 21, 5, 3
    q, k = make(T, hq, hk, d, dtype, d + r)
    dq, dk = make(T, hq, hk, d, dtype, d + r + 1)
    rope = RotaryEmbedding(d, rotary_dim=r, interleaved=inter)
    op = QKNormRotary(d, norm=norm, eps=1e-5, rotary=rope)
    f, pos = O.frequencies(r)[0], np.arange(T) + 2
    turned, y = rope.forward(q, k, offset=2), op.forward(q, k, offset=2)
    for x, a, b in zip((q, k), turned, y):
        within(flat(a), O.rotate(flat(x), pos, f, inter), rows_max(flat(x)),
               K_ROPE, dtype)
        rstd = O.normal(flat(x), norm, 1e-5)[1]
        within(flat(b), O.forward(flat(x), pos, f, norm, 1e-5, None, None, inter),
               rows_max(flat(x)) * rstd, K_NORM, dtype)
    got = op.backward(dq, dk, q, k, offset=2)
    check_gradients(op, q, k, dq, dk, None, None, pos, f, inter, dtype, got)


def test_the_bindings_of_the_c_abi():
    """The ctypes binding's functions give what the tensor calls give."""
    T, H, d = 33, 4, 64
    q, k = make(T, H, H, d, torch.bfloat16, 107)
    dq, dk = make(T, H, H, d, torch.bfloat16, 108)
    gamma = torch.linspace(0.5, 1.5, d, device="cuda")
    rope = RotaryEmbedding(d)
    op = QKNormRotary(d, norm="rms", rotary=rope)
    heads = lambda t: B.tp_heads(t.data_ptr(), H * d, 0, d, H, H)
    at = B.tp_positions(None, 0, 3, 10)
    where = dict(offset=3, seq_len=10)
    out = [torch.empty_like(q) for _ in range(2)]
    v = [heads(t) for t in (q, out[0], k, out[1])]
    for inverse, call in ((0, rope.forward), (1, rope.backward)):
        B.tp_rope_apply(rope.handle, T, B.TPMLP_BF16, inverse, *v, at)
        for a, b in zip(out, call(q, k, **where)):
            assert torch.equal(a, b)
    n = B.tp_qk_norm(B.TPQK_RMSNORM, 1e-6, gamma.data_ptr(), None,
                     gamma.data_ptr(), None)
    B.tp_qk_norm_forward(rope.handle, T, B.TPMLP_BF16, n, *v, at)
    for a, b in zip(out, op.forward(q, k, gamma, gamma, **where)):
        assert torch.equal(a, b)
    par = [torch.empty(d, device="cuda") for _ in range(2)]
    grads = B.tp_qk_norm_grads(par[0].data_ptr(), None, par[1].data_ptr(), None)
    nbytes = B.tp_qk_norm_workspace_bytes(rope.handle)
    ws = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    B.tp_qk_norm_backward(rope.handle, T, B.TPMLP_BF16, n, heads(dq), heads(q),
                          v[1], heads(dk), heads(k), v[3], at, grads, ws, nbytes)
    want = op.backward(dq, dk, q, k, gamma, gamma, **where)
    for a, name in zip(out + par, ("dq", "dk", "dq_gamma", "dk_gamma")):
        assert torch.equal(a, want[name]), name
    with pytest.raises(B.TPMLPError):
        B.tp_rope_apply(rope.handle, T, B.TPMLP_BF16, 2, *v, at)


def test_millions_of_tokens():
    """2^22 tokens of one short head: the same bits as in pieces of 2^16."""
    T, d = 1 << 22, 8
    g = torch.Generator("cuda").manual_seed(109)
    q, dq = (torch.randn((T, 1, d), generator=g, device="cuda").bfloat16()
             for _ in range(2))
    op = QKNormRotary(d, rotary=RotaryEmbedding(d, rotary_dim=4))
    y, _ = op.forward(q)
    dx = op.backward(dq, None, q, None, param_grads=False)["dq"]
    for t in range(0, T, 1 << 16):
        part = slice(t, t + (1 << 16))
        assert torch.equal(y[part], op.forward(q[part], offset=t)[0])
        assert torch.equal(dx[part], op.backward(
            dq[part], None, q[part], None, offset=t, param_grads=False)["dq"])


@pytest.mark.parametrize("d,r", [(64, 64), (96, 48), (10, 6)])
def test_broadcast_inputs(d, r):
    """One row (or one token, or one head) shown as many by strides of zero."""
    T, H = 19, 5
    g = torch.Generator("cuda").manual_seed(110)
    n = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()
    op = QKNormRotary(d, norm="layer", rotary=RotaryEmbedding(d, rotary_dim=r))
    for shape in ((1, 1, d), (1, H, d), (T, 1, d)):
        q, k = n(*shape).expand(T, H, d), n(*shape).expand(T, H, d)
        dq, dk = n(*shape).expand(T, H, d), n(*shape).expand(T, H, d)
        full = [t.contiguous() for t in (q, k, dq, dk)]
        for call in (op.rotary.forward, op.forward):
            for a, b in zip(call(q, k), call(*full[:2])):
                assert torch.equal(a, b)
        a = op.backward(dq, dk, q, k)
        b = op.backward(full[2], full[3], full[0], full[1])
        for name in a:
            assert torch.equal(a[name], b[name]), name


def test_threads_side_by_side():
    """One object called from several threads, each with a stream of its own."""
    import threading
    op = QKNormRotary(96, norm="layer", rotary=RotaryEmbedding(96))
    data = [make(500, 8, 4, 96, torch.bfloat16, 120 + i) +
            make(500, 8, 4, 96, torch.bfloat16, 130 + i) for i in range(4)]
    want = [op.backward(d[2], d[3], d[0], d[1], offset=i)
            for i, d in enumerate(data)]
    streams = [torch.cuda.Stream() for _ in data]
    torch.cuda.synchronize()
    got = [[] for _ in data]

    def work(i):
        d = data[i]
        for _ in range(30):
            got[i].append(op.backward(d[2], d[3], d[0], d[1], offset=i,
                                      stream=streams[i]))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert len(g) == 30
        for made in g:
            for n in w:
                assert torch.equal(made[n], w[n])
