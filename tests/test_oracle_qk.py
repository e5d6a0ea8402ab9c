"""Pins of the fp64 oracle for rotary positions, the per-head norm and gradient
clipping (no GPU): element-by-element loops, invariants and central
differences."""
import math

import numpy as np
import pytest

from oracle import attention as A
from oracle import qk as O


def rng(seed):
    return np.random.default_rng(seed)


@pytest.mark.parametrize("inter", [False, True])
def test_rotation_is_the_plane_rotation_of_each_pair(inter):
    x = rng(1).normal(size=(3, 2, 10))
    f, _ = O.frequencies(6, base=50.0)
    pos = [0, 5, -2]
    y = O.rotate(x, pos, f, inter, amp=1.5)
    for t in range(3):
        for h in range(2):
            want = x[t, h].copy()
            for i in range(3):
                a, b = (2 * i, 2 * i + 1) if inter else (i, i + 3)
                c, s = math.cos(pos[t] * f[i]), math.sin(pos[t] * f[i])
                want[a] = 1.5 * (x[t, h, a] * c - x[t, h, b] * s)
                want[b] = 1.5 * (x[t, h, a] * s + x[t, h, b] * c)
            assert np.allclose(y[t, h], want, rtol=0, atol=1e-14)


def test_scores_depend_on_the_distance_only():
    q, k = rng(2).normal(size=(2, 1, 1, 16))
    f, _ = O.frequencies(16)
    dot = lambda m, n: float(np.sum(O.rotate(q, [m], f) * O.rotate(k, [n], f)))
    assert abs(dot(1000, 993) - dot(7, 0)) < 1e-12


def test_far_positions_keep_their_fraction_of_a_turn():
    # 2 pi / 8 per position: position 8 n + 3 turns by 3/8 of a turn
    x = np.array([[[1.0, 0.0]]])
    y = O.rotate(x, [8 * (1 << 20) + 3], [2 * math.pi / 8])
    assert np.allclose(y[0, 0], [math.cos(0.75 * math.pi),
                                 math.sin(0.75 * math.pi)], atol=1e-8)


def test_scalings():
    plain, one = O.frequencies(8)
    assert one == 1.0 and plain[0] == 1.0
    assert np.allclose(O.frequencies(8, scaling="linear", factor=4.0)[0],
                       plain / 4)
    ntk = O.frequencies(8, scaling="ntk", factor=4.0)[0]
    assert ntk[0] == 1.0 and np.isclose(ntk[-1], plain[-1] / 4)
    yarn, amp = O.frequencies(8, scaling="yarn", factor=4.0,
                              original_length=2000)
    assert np.isclose(yarn[0], plain[0]) and np.isclose(yarn[-1], plain[-1] / 4)
    assert np.isclose(amp, 0.1 * math.log(4) + 1)


@pytest.mark.parametrize("norm", ["rms", "layer"])
@pytest.mark.parametrize("inter", [False, True])
def test_norm_gradients_against_central_differences(norm, inter):
    g = rng(3)
    x, dy = g.normal(size=(2, 4, 2, 6))
    gamma, beta = 1 + 0.3 * g.normal(size=6), g.normal(size=6)
    f, amp = O.frequencies(4, base=7.0)[0], 1.25
    pos = np.array([0, 1, 9, 30])
    b = beta if norm == "layer" else None
    loss = lambda x_, ga, be: float(np.sum(dy * O.forward(
        x_, pos, f, norm, 1e-3, ga, be, inter, amp)))
    got = O.backward(dy, x, pos, f, norm, 1e-3, gamma, inter, amp)
    h = 1e-5
    for name, base in (("dx", x), ("dgamma", gamma), ("dbeta", b)):
        if base is None:
            continue
        num = np.zeros_like(base)
        for idx in np.ndindex(base.shape):
            up, dn = base.copy(), base.copy()
            up[idx] += h
            dn[idx] -= h
            args = {"dx": (x, gamma, b), "dgamma": (x, gamma, b),
                    "dbeta": (x, gamma, b)}[name]
            at = ("dx", "dgamma", "dbeta").index(name)
            a1, a2 = list(args), list(args)
            a1[at], a2[at] = up, dn
            num[idx] = (loss(*a1) - loss(*a2)) / (2 * h)
        assert np.allclose(got[name], num, rtol=0, atol=1e-8), name


def test_norm_rows_by_hand():
    x = np.array([[[3.0, 4.0]]])
    xh, _ = O.normal(x, "rms", 0.0)
    assert np.allclose(xh, x / math.sqrt(12.5))
    xh, _ = O.normal(x, "layer", 0.0)
    assert np.allclose(xh, [[[-1.0, 1.0]]])


def test_clip_by_hand():
    n, c, out = O.clip([np.array([3.0]), np.array([[4.0]])], 1.0, eps=0.0)
    assert n == 5.0 and c == 0.2 and np.allclose(out[1], 0.8)
    assert O.clip([np.array([0.3])], 1.0)[1] == 1.0
    assert O.clip([np.array([np.inf])], 1.0)[1] == 1.0


def test_attention_block_gradients_against_central_differences():
    g = rng(5)
    T, h, H = 6, 8, 2
    X, dZ = g.normal(size=(2, T, h))
    Wqkv, Wo = 0.5 * g.normal(size=(h, 3 * h)), g.normal(size=(h, h))
    qg, kg = 1 + 0.2 * g.normal(size=(2, 4))
    kw = dict(freqs=O.frequencies(4)[0], norm="rms")

    def loss(X_, W_, qg_, kg_):
        return float(np.sum(dZ * O.attention_forward(
            X_, W_, Wo, H, 3, shards=2, q_gamma=qg_, k_gamma=kg_, **kw)["Z"]))

    fwd = O.attention_forward(X, Wqkv, Wo, H, 3, shards=2, q_gamma=qg,
                              k_gamma=kg, **kw)
    got = O.attention_backward(dZ, X, Wqkv, Wo, fwd, H, 3, shards=2,
                               q_gamma=qg, k_gamma=kg, **kw)
    args = [X, Wqkv, qg, kg]
    for at, name in enumerate(("dX", "dWqkv", "dq_gamma", "dk_gamma")):
        base = args[at]
        v = g.normal(size=base.shape)
        up, dn = list(args), list(args)
        up[at], dn[at] = base + 1e-5 * v, base - 1e-5 * v
        num = (loss(*up) - loss(*dn)) / 2e-5
        assert abs(num - float(np.sum(got[name] * v))) < 1e-6, name


def test_attention_block_without_positions_is_the_plain_block():
    g = rng(6)
    X = g.normal(size=(4, 8))
    W, Wo = g.normal(size=(8, 24)), g.normal(size=(8, 8))
    a = A.forward(X, W, Wo, 2, 2)["Z"]
    b = O.attention_forward(X, W, Wo, 2, 2)["Z"]
    assert np.allclose(a, b, rtol=0, atol=1e-13)
