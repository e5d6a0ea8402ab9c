"""Host side of the query/key operators and of gradient clipping, without a
GPU: exported symbols, frequencies, and every refusal, which is decided before
any device work (stand-in addresses are never dereferenced)."""
import ctypes
import math
import os
import re

import numpy as np
import pytest
import torch

from oracle import qk as O
from tensor_transformer_mlp_tcgen05_gb300 import binding as B
from tensor_transformer_mlp_tcgen05_gb300 import build as build_mod
from tensor_transformer_mlp_tcgen05_gb300 import clip as C
from tensor_transformer_mlp_tcgen05_gb300 import rotary as R

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 1 << 24


@pytest.fixture(scope="module")
def lib():
    build_mod.build()
    return B.lib()


def declared(header, prefix):
    text = open(os.path.join(ROOT, "include", header)).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(tp_(?:%s)_\w+)\s*\(" % prefix, text)))


def test_every_declared_symbol_is_exported(lib):
    for header, prefix, names in (("tp_rope.h", "rope|qk", B.EXPORTED_ROPE),
                                  ("tp_grad.h", "grad", B.EXPORTED_GRAD)):
        assert declared(header, prefix) == sorted(names)
        for n in names:
            assert hasattr(lib, n), n


# ---------------------------------------------------------- frequencies --

@pytest.mark.parametrize("kw", [
    {}, dict(base=500000.0), dict(scaling="linear", factor=3.0),
    dict(scaling="ntk", factor=8.0),
    dict(scaling="yarn", factor=4.0, original_length=4096),
    dict(scaling="yarn", factor=2.0, original_length=512, slow_turns=2.0,
         fast_turns=9.0)])
@pytest.mark.parametrize("r", [0, 2, 10, 128])
def test_frequencies_match_the_oracle(lib, kw, r):
    rope = R.RotaryEmbedding(128, rotary_dim=r, **kw)
    f, amp = rope.frequencies()
    want, amp_want = O.frequencies(r, **kw)
    assert np.allclose(f, want, rtol=1e-14, atol=0)
    assert math.isclose(amp, amp_want, rel_tol=1e-15)


def test_custom_frequencies_and_amplitude(lib):
    rope = R.RotaryEmbedding(8, rotary_dim=4, inv_freq=[2.5, -0.125],
                             amplitude=0.75)
    assert rope.frequencies() == ([2.5, -0.125], 0.75)


def rope_cfg(**kw):
    base = dict(head_dim=64, rot_dim=64, interleaved=0, scaling=0,
                base=10000.0, factor=1.0, original_length=0.0, slow_turns=1.0,
                fast_turns=32.0, amplitude=0.0, inv_freq=None)
    base.update(kw)
    return B.tp_rope_config(**base)


@pytest.mark.parametrize("kw,code", [
    (dict(head_dim=0, rot_dim=0), B.TPMLP_ERR_SHAPE),
    (dict(head_dim=257, rot_dim=2), B.TPMLP_ERR_SHAPE),
    (dict(rot_dim=66), B.TPMLP_ERR_SHAPE),
    (dict(rot_dim=-2), B.TPMLP_ERR_SHAPE),
    (dict(rot_dim=7), B.TPMLP_ERR_SHAPE),
    (dict(interleaved=2), B.TPMLP_ERR_ARG),
    (dict(scaling=5), B.TPMLP_ERR_ARG),
    (dict(base=0.0), B.TPMLP_ERR_ARG),
    (dict(base=float("nan")), B.TPMLP_ERR_ARG),
    (dict(scaling=1, factor=0.0), B.TPMLP_ERR_ARG),
    (dict(scaling=2, factor=float("inf")), B.TPMLP_ERR_ARG),
    (dict(scaling=3, factor=2.0), B.TPMLP_ERR_ARG),
    (dict(scaling=3, factor=2.0, original_length=10.0, fast_turns=1.0),
     B.TPMLP_ERR_ARG),
    (dict(scaling=4), B.TPMLP_ERR_ARG),
    (dict(amplitude=float("inf")), B.TPMLP_ERR_ARG),
])
def test_create_rejects_bad_configs(lib, kw, code):
    h = ctypes.c_void_p()
    assert lib.tp_rope_create(ctypes.byref(rope_cfg(**kw)),
                              ctypes.byref(h)) == code
    assert h.value is None


def test_create_rejects_a_frequency_that_is_not_finite(lib):
    f = (ctypes.c_double * 32)(*([1.0] * 31 + [float("nan")]))
    h = ctypes.c_void_p()
    cfg = rope_cfg(scaling=4, inv_freq=f)
    assert lib.tp_rope_create(ctypes.byref(cfg),
                              ctypes.byref(h)) == B.TPMLP_ERR_ARG


# --------------------------------------------------------------- views --

def heads(data, H=4, d=64, T=16, group=None, ts=None, gs=0, hs=None):
    hs = d if hs is None else hs
    ts = H * hs if ts is None else ts
    return B.tp_heads(data, ts, gs, hs, H, H if group is None else group)


@pytest.fixture
def handle(lib):
    h = B.tp_rope_create(rope_cfg())
    yield h
    B.tp_rope_destroy(h)


BYTES = 16 * 4 * 64 * 2


def apply(lib, handle, q_in, q_out, k_in=None, k_out=None, pos=None, T=16,
          dtype=B.TPMLP_BF16, inverse=0):
    ref = lambda s: None if s is None else ctypes.byref(s)
    return lib.tp_rope_apply(handle, T, dtype, inverse, ref(q_in), ref(q_out),
                             ref(k_in), ref(k_out), ref(pos), None)


def refused(lib, *args, code, **kw):
    rc = apply(lib, *args, **kw)
    assert rc == code, (rc, B.tp_mlp_last_detail())


def accepted(lib, *args, **kw):
    """Past validation: on a machine without a GPU the device check is what
    refuses."""
    if torch.cuda.is_available():
        pytest.skip("stand-in addresses must not reach a GPU")
    rc = apply(lib, *args, **kw)
    assert rc in (B.TPMLP_ERR_CUDA, B.TPMLP_ERR_ARCH), rc


def test_apply_refuses_bad_arguments(lib, handle):
    a, b = heads(FAKE), heads(2 * FAKE)
    ARG, SHAPE, ALIGN = B.TPMLP_ERR_ARG, B.TPMLP_ERR_SHAPE, B.TPMLP_ERR_ALIGN
    refused(lib, None, a, b, code=ARG)
    refused(lib, handle, a, b, code=ARG, inverse=2)
    refused(lib, handle, a, b, code=ARG, dtype=2)
    refused(lib, handle, a, b, code=SHAPE, T=-1)
    refused(lib, handle, a, b, code=SHAPE, T=(1 << 28) + 1)
    refused(lib, handle, None, None, code=ARG)
    refused(lib, handle, a, None, code=SHAPE)
    refused(lib, handle, a, heads(2 * FAKE, H=3), code=SHAPE)
    refused(lib, handle, a, b, heads(3 * FAKE), None, code=SHAPE)
    refused(lib, handle, heads(None), b, code=ARG)
    refused(lib, handle, heads(FAKE + 1), b, code=ALIGN)
    refused(lib, handle, heads(FAKE + 2), b, code=ALIGN, dtype=B.TPMLP_FP32)
    refused(lib, handle, heads(FAKE, group=3), b, code=SHAPE)
    refused(lib, handle, heads(FAKE, group=0), b, code=SHAPE)
    refused(lib, handle, heads(FAKE, ts=-256), b, code=SHAPE)
    refused(lib, handle, heads(FAKE, ts=1 << 31), b, code=SHAPE)
    refused(lib, handle, heads(FAKE, H=65536), heads(2 * FAKE, H=65536),
            code=SHAPE)


def test_positions_are_checked(lib, handle):
    a, b = heads(FAKE), heads(2 * FAKE)
    P = B.tp_positions
    refused(lib, handle, a, b, pos=P(FAKE, 2, 0, 0), code=B.TPMLP_ERR_ARG)
    refused(lib, handle, a, b, pos=P(None, 0, 0, -1), code=B.TPMLP_ERR_SHAPE)
    refused(lib, handle, a, b, pos=P(FAKE + 4, 1, 0, 0),
            code=B.TPMLP_ERR_ALIGN)


@pytest.mark.parametrize("out", [
    heads(FAKE + 2),                       # the input, one element on
    heads(FAKE + BYTES - 2),               # its last element
    heads(FAKE, hs=128),                   # the same start, another stride
    heads(2 * FAKE, ts=0),                 # all tokens in one place
    heads(2 * FAKE, hs=32),                # heads half over one another
    heads(2 * FAKE, ts=192),               # tokens a head over one another
    heads(2 * FAKE, group=2, gs=64),       # groups over one another
])
def test_outputs_that_overlap_are_refused(lib, handle, out):
    refused(lib, handle, heads(FAKE), out, code=B.TPMLP_ERR_ARG)


def test_q_and_k_of_one_buffer(lib, handle):
    # [T, 3, H, d]: q, k of one projection, in place and into each other
    at = lambda i: heads(FAKE + i * 4 * 64 * 2, ts=3 * 256)
    accepted(lib, handle, at(0), at(0), at(1), at(1))
    accepted(lib, handle, at(0), at(2), at(1), heads(2 * FAKE))
    refused(lib, handle, at(0), at(1), at(1), heads(2 * FAKE),
            code=B.TPMLP_ERR_ARG)
    refused(lib, handle, at(0), at(2), at(1), at(2), code=B.TPMLP_ERR_ARG)
    # heads interleaved in memory, [T, H, 3, d]
    at = lambda i: heads(FAKE + i * 64 * 2, ts=3 * 256, hs=192)
    accepted(lib, handle, at(0), at(0), at(1), at(1))
    refused(lib, handle, at(0), at(0), at(1), heads(FAKE + 32 * 2, ts=3 * 256,
                                                    hs=192),
            code=B.TPMLP_ERR_ARG)
    # shard groups, [T, t, 3, H / t, d]
    at = lambda i: heads(FAKE + i * 128 * 2, ts=768, group=2, gs=384)
    accepted(lib, handle, at(0), at(0), at(1), at(1))
    # head-major, [H, T, d]
    major = lambda p: heads(p, ts=64, hs=16 * 64)
    accepted(lib, handle, major(FAKE), major(2 * FAKE))
    # head-major with q and k side by side, [H, T, 2, d], in place
    both = lambda i: heads(FAKE + i * 64 * 2, ts=128, hs=16 * 128)
    accepted(lib, handle, both(0), both(0), both(1), both(1))
    refused(lib, handle, both(0), both(0), both(1),
            heads(FAKE + 32 * 2, ts=128, hs=16 * 128), code=B.TPMLP_ERR_ARG)
    # more query than key heads in one buffer, [T, Hq + Hk, d]
    few = lambda j, n: heads(FAKE + j * 64 * 2, H=n, ts=6 * 64)
    accepted(lib, handle, few(0, 4), few(0, 4), few(4, 2), few(4, 2))
    refused(lib, handle, few(0, 4), few(0, 4), few(3, 2), few(3, 2),
            code=B.TPMLP_ERR_ARG)
    # the last token's tail reaches into the next token's head
    refused(lib, handle, heads(FAKE, ts=300, hs=70), heads(FAKE + 2 * 290,
            ts=300, hs=70), code=B.TPMLP_ERR_ARG)


def test_views_of_any_alignment_and_broadcast_inputs_pass(lib, handle):
    accepted(lib, handle, heads(FAKE + 2, ts=257), heads(2 * FAKE + 6, ts=259))
    accepted(lib, handle, heads(FAKE, ts=0), heads(2 * FAKE))
    accepted(lib, handle, heads(FAKE, hs=0, ts=64), heads(2 * FAKE))


def test_overlap_against_brute_force(lib, handle):
    """Two outputs of random strides in one buffer: refused exactly when an
    element is written twice, for views with the same strides; never accepted
    wrongly for others."""
    if torch.cuda.is_available():
        pytest.skip("stand-in addresses must not reach a GPU")
    g = np.random.default_rng(0)
    d = 64
    seen = {True: 0, False: 0}
    for n in range(3000):
        T, groups, group = (int(g.integers(1, 4)) for _ in range(3))
        order = g.permutation(3)
        strides, inside = [0, 0, 0], d + int(g.integers(0, 2)) * 64
        for dim in order:                       # nested in a random order
            strides[dim] = inside
            inside = inside * (T, groups, group)[dim] + \
                int(g.integers(0, 3)) * 64
        ts, gs, hs = strides
        shift = int(g.integers(-inside, inside))
        if g.random() < 0.5:
            shift -= shift % 64
        v = lambda at: B.tp_heads(FAKE * 64 + 2 * at, ts, gs, hs,
                                  groups * group, group)
        rows = lambda at: {at + t * ts + i * gs + j * hs for t in range(T)
                           for i in range(groups) for j in range(group)}
        meets = any(abs(x - y) < d for x in rows(0) for y in rows(shift))
        k = heads(FAKE, H=groups * group, T=T)
        rc = apply(lib, handle, k, v(0), k, v(shift), T=T)
        assert (rc == B.TPMLP_ERR_ARG) == meets, (T, strides, shift, rc)
        seen[meets] += 1
    assert min(seen.values()) > 500, seen


def norm_calls(lib, handle, n, grads=None, ws=FAKE * 8, nbytes=None, T=16,
               k=True):
    ref = lambda s: None if s is None else ctypes.byref(s)
    v = [heads(FAKE * (i + 1)) for i in range(6)]
    f = lib.tp_qk_norm_forward(handle, T, B.TPMLP_BF16, ref(n), ref(v[0]),
                               ref(v[1]), ref(v[2]) if k else None,
                               ref(v[3]) if k else None, None, None)
    b = lib.tp_qk_norm_backward(
        handle, T, B.TPMLP_BF16, ref(n), ref(v[0]), ref(v[1]), ref(v[2]),
        *([ref(v[3]), ref(v[4]), ref(v[5])] if k else [None] * 3), None,
        ref(grads), ws,
        B.tp_qk_norm_workspace_bytes(handle) if nbytes is None else nbytes,
        None)
    return f, b


def test_norm_refusals(lib, handle):
    N, G = B.tp_qk_norm, B.tp_qk_norm_grads
    ARG, ALIGN = B.TPMLP_ERR_ARG, B.TPMLP_ERR_ALIGN
    assert norm_calls(lib, handle, None) == (ARG, ARG)
    assert norm_calls(lib, handle, N(3, 1e-6)) == (ARG, ARG)
    assert norm_calls(lib, handle, N(0, 1e-6)) == (ARG, ARG)
    assert norm_calls(lib, handle, N(1, -1.0)) == (ARG, ARG)
    assert norm_calls(lib, handle, N(1, float("nan"))) == (ARG, ARG)
    assert norm_calls(lib, handle, N(1, 0.0, None, FAKE)) == (ARG, ARG)
    assert norm_calls(lib, handle, N(2, 0.0, FAKE + 2)) == (ALIGN, ALIGN)
    ok, g = N(2, 1e-6), G(FAKE * 10)
    assert norm_calls(lib, handle, ok, G(FAKE + 1))[1] == ALIGN
    assert norm_calls(lib, handle, N(1, 1e-6), G(None, FAKE * 10))[1] == ARG
    assert norm_calls(lib, handle, ok, G(None, None, FAKE), k=False)[1] == ARG
    assert norm_calls(lib, handle, ok, G(FAKE * 10, FAKE * 10))[1] == ARG
    assert norm_calls(lib, handle, ok,
                      G(FAKE * 10, None, FAKE * 10 + 252))[1] == ARG
    assert norm_calls(lib, handle, ok, g, ws=None)[1] == ARG
    assert norm_calls(lib, handle, ok, g, ws=FAKE * 8 + 8)[1] == ALIGN
    assert norm_calls(lib, handle, ok, g, nbytes=100)[1] == \
        B.TPMLP_ERR_WORKSPACE
    assert B.tp_qk_norm_workspace_bytes(None) == 0


# ------------------------------------------------------------ gradients --

def grads(*rows):
    return (B.tp_grad_tensor * len(rows))(*rows)


def clip(lib, table, n=None, max_norm=1.0, eps=1e-6, norm=FAKE, ws=FAKE * 8,
         nbytes=1 << 20):
    n = len(table) if n is None else n
    return lib.tp_grad_clip(n, table, max_norm, eps, norm, ws, nbytes, None)


def test_clip_refusals(lib):
    ARG, SHAPE, ALIGN = B.TPMLP_ERR_ARG, B.TPMLP_ERR_SHAPE, B.TPMLP_ERR_ALIGN
    F = B.TPMLP_FP32
    one = grads((FAKE * 2, FAKE * 2, 8, F))
    assert clip(lib, one, max_norm=-1.0) == ARG
    assert clip(lib, one, max_norm=float("nan")) == ARG
    assert clip(lib, one, eps=-1.0) == ARG
    assert clip(lib, one, eps=float("inf")) == ARG
    assert clip(lib, one, n=-1) == SHAPE
    assert clip(lib, None, n=1) == ARG
    assert clip(lib, one, norm=None) == ARG
    assert clip(lib, one, norm=FAKE + 2) == ALIGN
    assert clip(lib, one, ws=None) == ARG
    assert clip(lib, one, ws=FAKE + 8) == ALIGN
    assert clip(lib, one, nbytes=8) == B.TPMLP_ERR_WORKSPACE
    assert clip(lib, grads((None, FAKE, 8, F))) == ARG
    assert clip(lib, grads((FAKE, None, 8, F))) == ARG
    assert clip(lib, grads((FAKE, FAKE, 8, 2))) == ARG
    assert clip(lib, grads((FAKE, FAKE, -1, F))) == SHAPE
    assert clip(lib, grads((FAKE + 2, FAKE + 2, 8, F))) == ALIGN
    assert B.tp_grad_workspace_bytes(-1) == 0
    assert B.tp_grad_workspace_bytes(0) > 0
    assert B.tp_grad_workspace_bytes(10000) > B.tp_grad_workspace_bytes(1)


@pytest.mark.parametrize("rows", [
    [(2, 2, 8), (2, 2, 8)],                # the same tensor twice, in place
    [(2, 2, 8), (2.5, 2.5, 8)],            # half over one another (16 bytes)
    [(2, 4, 8), (4, 5, 8)],                # out on another's gradient
    [(2, 2.5, 8)],                         # out half over its own gradient
    [(2, 4, 8), (3, 4, 8)],                # one out twice
])
def test_clip_refuses_outputs_that_overlap(lib, rows):
    at = lambda x: FAKE + int(x * 32)
    table = grads(*[(at(g), at(o), n, B.TPMLP_FP32) for g, o, n in rows])
    assert clip(lib, table) == B.TPMLP_ERR_ARG


def test_clip_accepts_neighbours_and_shared_inputs(lib):
    if torch.cuda.is_available():
        pytest.skip("stand-in addresses must not reach a GPU")
    at = lambda x: FAKE + int(x * 32)
    F = B.TPMLP_FP32
    for rows in ([(at(2), at(2), 8, F), (at(3), at(3), 8, F)],
                 [(at(2), at(4), 8, F), (at(2), at(5), 8, F)],
                 [(None, None, 0, F), (at(1), at(1), 8, F)]):
        assert clip(lib, grads(*rows)) in (B.TPMLP_ERR_CUDA, B.TPMLP_ERR_ARCH)


# -------------------------------------------------------- python wrappers --

def test_wrappers_refuse_before_the_library(lib):
    with pytest.raises(ValueError):
        R.RotaryEmbedding(64, scaling="cubic")
    with pytest.raises(ValueError):
        R.RotaryEmbedding(64, inv_freq=[1.0])
    with pytest.raises(ValueError):
        R.RotaryEmbedding(4, inv_freq=[1.0, 2.0], scaling="linear")
    with pytest.raises(B.TPMLPError):
        R.RotaryEmbedding(300)
    with pytest.raises(ValueError):
        R.QKNormRotary(64, norm="batch")
    with pytest.raises(ValueError):
        R.QKNormRotary(64, rotary=R.RotaryEmbedding(32))
    with pytest.raises(ValueError):
        C.clip_grad_norm([], 1.0)
    with pytest.raises(ValueError):
        C.clip_grad_norm([torch.zeros(4)], 1.0)
    with pytest.raises(ValueError):
        C.grad_norm({"dX": torch.zeros(4)})


# --------------------------------------------------- in the attention block --

def attn_handle(**kw):
    base = dict(hidden=256, heads=4, shards=2, max_tokens=512, seq_len=256,
                causal=1, use_layernorm=0, ln_eps=1e-5, use_residual=0)
    base.update(kw)
    return B.tp_attn_create(B.tp_attn_config(**base))


def test_attention_settings_are_checked_and_replaceable(lib):
    h = attn_handle()
    try:
        ok, other = rope_cfg(), rope_cfg(head_dim=32, rot_dim=32)
        set_rope = lambda c: lib.tp_attn_set_rope(
            h, None if c is None else ctypes.byref(c))
        assert set_rope(other) == B.TPMLP_ERR_SHAPE
        assert set_rope(rope_cfg(base=-1.0)) == B.TPMLP_ERR_ARG
        for c in (ok, ok, None, ok):
            assert set_rope(c) == B.TPMLP_OK
        assert lib.tp_attn_set_rope(None, None) == B.TPMLP_ERR_ARG
        assert lib.tp_attn_set_qk_norm(h, 3, 1e-6) == B.TPMLP_ERR_ARG
        assert lib.tp_attn_set_qk_norm(h, 1, -1.0) == B.TPMLP_ERR_ARG
        assert lib.tp_attn_set_qk_norm(h, 1, float("nan")) == B.TPMLP_ERR_ARG
        assert lib.tp_attn_set_qk_norm(None, 1, 1e-6) == B.TPMLP_ERR_ARG
        for n in (B.TPQK_RMSNORM, B.TPQK_LAYERNORM, 0):
            assert lib.tp_attn_set_qk_norm(h, n, 1e-6) == B.TPMLP_OK
    finally:
        B.tp_attn_destroy(h)


def test_attention_workspace_holds_q_and_k_twice_with_the_norm(lib):
    h = attn_handle()
    try:
        T = 512
        size = lambda training: B.tp_attn_workspace_bytes(h, T, training)
        off = lambda training, w: B.tp_attn_workspace_offset(h, T, training, w)
        plain = size(0), size(1)
        assert off(1, B.TPATTN_WS_QKR) == off(1, B.TPATTN_WS_QKV)
        B.tp_attn_set_rope(h, rope_cfg())
        assert (size(0), size(1)) == plain
        B.tp_attn_set_qk_norm(h, B.TPQK_RMSNORM, 1e-6)
        assert size(0) == plain[0]
        assert size(1) >= plain[1] + T * 3 * 256 * 2
        assert off(0, B.TPATTN_WS_QKR) == off(0, B.TPATTN_WS_QKV)
        qkr = off(1, B.TPATTN_WS_QKR)
        assert plain[1] <= qkr and qkr + T * 3 * 256 * 2 <= size(1)
        for w in range(4):
            assert off(1, w) < plain[1]
    finally:
        B.tp_attn_destroy(h)


def test_attention_qk_arguments_are_refused_before_any_launch(lib):
    h = attn_handle()
    try:
        def calls(qk=None, grads=None):
            ref = lambda s: None if s is None else ctypes.byref(s)
            n = B.tp_attn_workspace_bytes(h, 256, 1)
            p = [FAKE * (i + 1) for i in range(8)]
            return (lib.tp_attn_forward_qk(
                        h, 256, p[0], p[1], p[2], None, None, None, None, p[3],
                        p[4], n, 1, ref(qk), None),
                    lib.tp_attn_backward_qk(
                        h, 256, p[0], p[1], p[2], p[3], None, p[4], n, p[5],
                        p[6], p[7], None, None, None, None, ref(qk), ref(grads),
                        None))
        Q, G = B.tp_attn_qk, B.tp_qk_norm_grads
        ARG, ALIGN = B.TPMLP_ERR_ARG, B.TPMLP_ERR_ALIGN
        assert calls(Q(FAKE, 0)) == (ARG, ARG)            # no rotation set
        assert calls(Q(None, 0, FAKE)) == (ARG, ARG)      # no norm set
        assert calls(None, G(FAKE))[1] == ARG
        B.tp_attn_set_rope(h, rope_cfg())
        B.tp_attn_set_qk_norm(h, B.TPQK_RMSNORM, 1e-6)
        assert calls(Q(FAKE, 2)) == (ARG, ARG)
        assert calls(Q(FAKE + 4, 1)) == (ALIGN, ALIGN)
        assert calls(Q(None, 0, FAKE + 2)) == (ALIGN, ALIGN)
        assert calls(Q(None, 0, None, FAKE)) == (ARG, ARG)
        assert calls(None, G(None, FAKE))[1] == ARG
        assert calls(None, G(FAKE + 2))[1] == ALIGN
        assert calls(None, G(FAKE, None, FAKE))[1] == ARG
        assert lib.tp_attn_forward_qk(None, *[0] * 14) == ARG
    finally:
        B.tp_attn_destroy(h)


@pytest.mark.parametrize("amp", [1e39, -1e39, float("nan"), -float("inf")])
def test_create_rejects_an_amplitude_beyond_fp32(lib, amp):
    h = ctypes.c_void_p()
    cfg = rope_cfg(amplitude=amp)
    assert lib.tp_rope_create(ctypes.byref(cfg),
                              ctypes.byref(h)) == B.TPMLP_ERR_ARG
    assert h.value is None
    cfg = rope_cfg(amplitude=3e38)
    assert lib.tp_rope_create(ctypes.byref(cfg),
                              ctypes.byref(h)) == B.TPMLP_OK
    assert lib.tp_rope_destroy(h) == B.TPMLP_OK


def test_overlap_of_views_of_different_strides_against_brute_force(lib, handle):
    """Two outputs in one buffer, each with strides, groups and heads of its own
    (their token strides equal in half of the cases): none that share an element
    are accepted."""
    if torch.cuda.is_available():
        pytest.skip("stand-in addresses must not reach a GPU")
    g = np.random.default_rng(5)
    d = 64
    seen = {}
    for n in range(6000):
        T = int(g.integers(1, 5))

        def view():
            groups, group = int(g.integers(1, 4)), int(g.integers(1, 4))
            strides, inside = [0, 0, 0], d + int(g.integers(0, 3)) * 16
            for dim in g.permutation(3):            # nested in a random order
                strides[dim] = inside
                inside = inside * (T, groups, group)[dim] + \
                    int(g.integers(0, 3)) * int(g.choice([16, 64]))
            return strides, groups, group, inside
        a, b = view(), view()
        if g.random() < 0.5:
            b[0][0] = a[0][0]
        span = max(a[3], b[3])
        shift = int(g.integers(-span, span))
        if g.random() < 0.6:
            shift -= shift % 16
        heads_at = lambda v, at: B.tp_heads(FAKE * 64 + 2 * at, *v[0],
                                            v[1] * v[2], v[2])
        rows = lambda v, at: sorted(
            at + t * v[0][0] + i * v[0][1] + j * v[0][2] for t in range(T)
            for i in range(v[1]) for j in range(v[2]))
        ra, rb = rows(a, 0), rows(b, shift)
        own = lambda r: any(y - x < d for x, y in zip(r, r[1:]))
        meets = own(ra) or own(rb) or any(abs(x - y) < d
                                          for x in ra for y in rb)
        rc = apply(lib, handle, heads(FAKE, H=a[1] * a[2], T=T), heads_at(a, 0),
                   heads(2 * FAKE, H=b[1] * b[2], T=T), heads_at(b, shift), T=T)
        refused = rc == B.TPMLP_ERR_ARG
        assert refused or not meets, (T, a, b, shift, rc)
        seen[meets, refused] = seen.get((meets, refused), 0) + 1
    assert seen[True, True] > 1500 and seen[False, False] > 1000, seen
