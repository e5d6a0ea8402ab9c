"""GPU parity of the global gradient norm and of clipping against fp64: many and
few tensors, odd lengths and alignments, mixed types, values whose squares leave
fp32's range, values that are not finite, in place and into other tensors,
repeats, streams and captured graphs."""
import math

import numpy as np
import pytest
import torch

from oracle import qk as O
from tensor_transformer_mlp_tcgen05_gb300 import binding as B
from tensor_transformer_mlp_tcgen05_gb300.clip import clip_grad_norm, grad_norm

pytestmark = pytest.mark.gpu

# The norm: squares are summed over at most 128 elements of a thread in fp32,
# each addition off by at most u = 2^-24 of the sum so far: 128 u of the sum
# of squares at worst, half of that of its root, and one rounding to fp32 (u):
# 65 u.  The factor is rounded once (u) besides: a scaled element is off by
# 66 u of itself and half a step of its type; below the smallest normal number,
# 2^-126, steps no longer shrink: they are 2^-149 in fp32 and 2^-133 in bf16, so
# that half of one, 2^-150 and 2^-134, is the least error to allow for.
U = 2.0 ** -24
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
LEAST = {torch.bfloat16: 2.0 ** -134, torch.float32: 2.0 ** -150}


def close(got, want, dtype):
    tol = (66 * U + HALF_STEP[dtype]) * np.abs(want) * (1 + 1e-6) + LEAST[dtype]
    return (np.abs(f64(got) - want) <= tol).all()


def f64(t):
    return t.detach().cpu().double().numpy()


def randn(n, seed, dtype=torch.float32, scale=1.0):
    g = torch.Generator("cuda").manual_seed(seed)
    return (scale * torch.randn(n, generator=g, device="cuda")).to(dtype)


def check(grads, max_norm, eps=1e-6, out=None):
    before = [f64(g) for g in grads]
    norm, c, want = O.clip(before, max_norm, eps)
    plain = grad_norm(grads)
    got = clip_grad_norm(grads, max_norm, eps=eps, out=out)
    assert torch.equal(plain, got) and got.shape == () and got.is_cuda
    assert abs(float(got) - norm) <= 65 * U * norm
    for g, b, w, o in zip(grads, before, want, grads if out is None else out):
        assert close(o, w, g.dtype)
        if out is not None:
            assert np.array_equal(f64(g), b)
        if c == 1.0:
            assert np.array_equal(f64(o), b)
    return norm


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("sizes", [
    [1], [7], [8], [4097], [16384], [16385], [32768], [32769], [100003],
    [1, 2, 3, 5, 8, 13, 21, 34, 55, 89], [5000000], [1024] * 100,
    [0, 5, 0, 0, 17, 0]])
@pytest.mark.parametrize("inplace", [True, False])
def test_sizes(sizes, dtype, inplace):
    grads = [randn(n, i, dtype) for i, n in enumerate(sizes)]
    out = None if inplace else [torch.full_like(g, 9.0) for g in grads]
    check(grads, 0.37, out=out)


def test_more_tensors_than_one_table():
    grads = [randn(37 + i % 11, i) for i in range(1300)]
    check(grads, 1.0)
    check([g.clone() for g in grads], 1.0,
          out=[torch.empty_like(g) for g in grads])


def test_mixed_types_and_shapes_in_a_dict():
    g = {"dA": randn(300, 1).view(20, 15), "dX": randn(1000, 2) * 1e9,
         "db": randn(33, 3, torch.bfloat16), "dB": randn(5 * 7 * 2, 4).view(5, 7, 2)}
    keep = g["dX"].clone()
    used = [g["dA"], g["db"], g["dB"]]
    norm, c, want = O.clip([f64(t) for t in used], 1.0)
    got = clip_grad_norm(g, 1.0)
    assert abs(float(got) - norm) <= 65 * U * norm
    assert torch.equal(g["dX"], keep)
    for t, w in zip(used, want):
        assert close(t, w, t.dtype)


def test_dicts_are_matched_by_name():
    g = {"a": randn(50, 1), "dX": randn(7, 2), "b": randn(50, 3)}
    out = {"b": torch.empty(50, device="cuda"), "a": torch.empty(50, device="cuda")}
    clip_grad_norm(g, 1.0, out=out)
    n = math.sqrt(float((g["a"].double() ** 2).sum() + (g["b"].double() ** 2).sum()))
    for k in ("a", "b"):
        assert close(out[k], f64(g[k]) * (1 / (n + 1e-6)), torch.float32)
    with pytest.raises(ValueError):
        clip_grad_norm(g, 1.0, out={"a": out["a"]})


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shift", [1, 2, 3, 5])
def test_tensors_off_16_bytes(dtype, shift):
    whole = randn(70001, 3, dtype)
    a, b = whole[shift:40000], whole[40000 + shift:]
    other = torch.full((70001,), 5.0, dtype=dtype, device="cuda")
    check([a, b], 1.0, out=[other[1:1 + a.numel()],
                            other[a.numel() + 2:a.numel() + 2 + b.numel()]])
    assert other[0] == 5.0 and other[a.numel() + 1] == 5.0
    edge = whole[:shift].clone(), whole[40000:40000 + shift].clone()
    check([a, b], 1.0)
    assert torch.equal(whole[:shift], edge[0])
    assert torch.equal(whole[40000:40000 + shift], edge[1])


@pytest.mark.parametrize("scale", [1e-30, 1e-20, 1e-12, 1e12, 1e18, 1e25, 1e36])
def test_squares_beyond_fp32(scale):
    grads = [randn(10007, 1, scale=scale), randn(64, 2, scale=scale * 1e-3),
             randn(5000, 3, torch.bfloat16, scale=scale)]
    norm = check([g.clone() for g in grads], scale, eps=0.0)
    assert math.isfinite(norm) and norm > scale
    # far apart in one tensor
    g = randn(4096, 4)
    g[17] = scale
    check([g], 1.0)


@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan")])
@pytest.mark.parametrize("inplace", [True, False])
def test_a_norm_that_is_not_finite_scales_nothing(bad, inplace):
    grads = [randn(5000, 1), randn(300, 2, torch.bfloat16)]
    grads[1][77] = bad
    keep = [g.clone() for g in grads]
    out = None if inplace else [torch.zeros_like(g) for g in grads]
    n = float(clip_grad_norm(grads, 1.0, out=out))
    assert math.isnan(n) if math.isnan(bad) else n == math.inf
    for k, o in zip(keep, grads if inplace else out):
        same = (o == k) | (o.isnan() & k.isnan())
        assert same.all()


def test_a_norm_beyond_fp32_scales_nothing():
    """3e38 sqrt(5000) is finite in fp64 only: reported as infinity."""
    for g in (torch.full((5000,), 3e38, device="cuda"),
              torch.full((300000,), 3e38, device="cuda")):
        keep, out = g.clone(), torch.zeros_like(g)
        assert float(clip_grad_norm([g], 1.0, out=[out])) == math.inf
        assert torch.equal(out, keep)
        assert float(clip_grad_norm([g], 1.0)) == math.inf
        assert torch.equal(g, keep)


def test_limits_of_max_norm():
    g = randn(1000, 1)
    keep = g.clone()
    check([g], math.inf)
    check([g], 1e30)
    assert torch.equal(g, keep)
    clip_grad_norm([g], 0.0)
    assert (g == 0).all()
    z = torch.zeros(100, device="cuda")
    assert float(clip_grad_norm([z], 1.0)) == 0.0 and (z == 0).all()
    assert float(clip_grad_norm([z], 0.0, eps=0.0)) == 0.0 and (z == 0).all()
    empty = torch.empty(0, device="cuda")
    assert float(grad_norm([empty])) == 0.0


def test_a_tensor_listed_twice_is_refused_in_place_only():
    g = randn(100, 1)
    with pytest.raises(B.TPMLPError):
        clip_grad_norm([g, g], 1.0)
    with pytest.raises(B.TPMLPError):
        clip_grad_norm([g, g[50:]], 1.0)
    want = math.sqrt(2) * float(g.double().norm())
    assert abs(float(grad_norm([g, g])) - want) <= 65 * U * want
    out = [torch.empty_like(g) for _ in range(2)]
    clip_grad_norm([g, g], 1.0, out=out)
    assert torch.equal(out[0], out[1])


def test_refusals():
    g = randn(64, 1)
    for call in (lambda: clip_grad_norm([], 1.0),
                 lambda: clip_grad_norm([g.half()], 1.0),
                 lambda: clip_grad_norm([g[::2]], 1.0),
                 lambda: clip_grad_norm([g, g.cpu()], 1.0),
                 lambda: clip_grad_norm([g], 1.0, out=[]),
                 lambda: clip_grad_norm([g], 1.0, out=[g.bfloat16()]),
                 lambda: clip_grad_norm([g], 1.0, out=[g[:32]])):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: clip_grad_norm([g], -1.0),
                 lambda: clip_grad_norm([g], float("nan")),
                 lambda: clip_grad_norm([g], 1.0, eps=-1.0)):
        with pytest.raises(B.TPMLPError):
            call()


def test_repeats_are_bit_identical():
    grads = [randn(n, n, scale=0.1) for n in (3000001, 777, 50000)]
    a = grad_norm(grads)
    outs = [torch.empty_like(g) for g in grads]
    clip_grad_norm(grads, 1.0, out=outs)
    for _ in range(3):
        again = [torch.empty_like(g) for g in grads]
        assert torch.equal(clip_grad_norm(grads, 1.0, out=again), a)
        for x, y in zip(outs, again):
            assert torch.equal(x, y)


def test_streams_and_graphs():
    sets = [[randn(300000, 10 * i + j) for j in range(3)] for i in range(2)]
    want = [grad_norm(s) for s in sets]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(10):
        for i in range(2):
            outs[i].append(grad_norm(sets[i], stream=streams[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for n in outs[i]:
            assert torch.equal(n, want[i])
    held = [torch.empty_like(g) for g in sets[0]]
    graphs, norms = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            norms.append(clip_grad_norm(sets[0], 1.0, out=held))
        graphs.append(g)
    for step in range(3):
        for g in sets[0]:
            g.mul_(1.5)
        for k, g in enumerate(graphs):
            g.replay()
            ref = [torch.empty_like(x) for x in sets[0]]
            n = clip_grad_norm(sets[0], 1.0, out=ref)
            torch.cuda.synchronize()
            assert torch.equal(n, norms[k])
            for x, y in zip(ref, held):
                assert torch.equal(x, y)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n", [1, 31, 512, 1024, 2048, 5000])
@pytest.mark.parametrize("scale", [2.0 ** 59.5, 2.0 ** 60, 2.0 ** 55])
@pytest.mark.parametrize("off", ["grad", "out", "both"])
def test_large_squares_off_16_bytes(n, dtype, scale, off):
    """Short sets of large values that are read one by one: a warp's total of
    their squares passes 2^128 where each is below 2^120."""
    at = lambda where: 1 if off in (where, "both") else 0
    g = torch.full((n + 1,), scale, dtype=dtype, device="cuda")
    g = g[at("grad"):at("grad") + n]
    out = torch.zeros(n + 1, dtype=dtype, device="cuda")
    out = out[at("out"):at("out") + n]
    assert math.isfinite(check([g], scale, eps=0.0, out=[out]))
    check([g], 1.0)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n", [100, 5003, 70001, 400009])
def test_the_norm_does_not_depend_on_where_the_outputs_are(n, dtype):
    """Outputs off 16 bytes beside gradients that are not: the same norm, bit
    for bit, and nothing written beside them."""
    for seed in range(4):
        g = randn(n, seed, dtype)
        room = torch.full((n + 9,), 7.0, dtype=dtype, device="cuda")
        for shift in (0, 1, 3):
            check([g], 1.0, out=[room[shift:shift + n]])
            assert (room[:shift] == 7.0).all()
            assert (room[shift + n:] == 7.0).all()
            room.fill_(7.0)


def test_a_lazy_copy_as_output_gets_memory_of_its_own():
    g = [randn(3000, 1), randn(3000, 2)]
    keep = [t.clone() for t in g]
    want = [torch.empty_like(t) for t in g]
    n = clip_grad_norm(g, 0.5, out=want)
    lazy = [torch._lazy_clone(t) for t in g]
    assert torch.equal(clip_grad_norm(g, 0.5, out=lazy), n)
    for a, b, c, k in zip(lazy, want, g, keep):
        assert torch.equal(a, b) and torch.equal(c, k)
    lazy = [torch._lazy_clone(t) for t in g]
    clip_grad_norm(lazy, 0.5)
    for a, b, c, k in zip(lazy, want, g, keep):
        assert torch.equal(a, b) and torch.equal(c, k)


def test_activations_gradients_are_left_out_of_the_operators_dict():
    """The dict that the query/key norm's backward returns: dq and dk are the
    activations' gradients, as dX is the blocks'."""
    from tensor_transformer_mlp_tcgen05_gb300.rotary import QKNormRotary
    x = [randn(40 * 3 * 64, i).view(40, 3, 64) for i in range(4)]
    g = QKNormRotary(64, norm="layer").backward(*x)
    keep = {n: t.clone() for n, t in g.items()}
    params = ["dq_gamma", "dk_gamma", "dq_beta", "dk_beta"]
    norm, c, _ = O.clip([f64(keep[n]) for n in params], 1.0)
    assert c < 1.0
    assert abs(float(grad_norm(g)) - norm) <= 65 * U * norm
    out = {n: torch.empty_like(g[n]) for n in params}
    assert abs(float(clip_grad_norm(g, 1.0, out=out)) - norm) <= 65 * U * norm
    assert abs(float(clip_grad_norm(g, 1.0)) - norm) <= 65 * U * norm
    for n in ("dq", "dk"):
        assert torch.equal(g[n], keep[n])
    for n in params:
        assert torch.equal(g[n], out[n])
        assert close(g[n], f64(keep[n]) * c, torch.float32)


def test_the_bindings_of_the_c_abi():
    """The ctypes binding's functions give what the tensor calls give."""
    g = [randn(5000, 1), randn(300, 2, torch.bfloat16)]
    out = [torch.empty_like(t) for t in g]
    want = [torch.empty_like(t) for t in g]
    code = {torch.float32: B.TPMLP_FP32, torch.bfloat16: B.TPMLP_BF16}
    table = (B.tp_grad_tensor * 2)(*[
        (t.data_ptr(), o.data_ptr(), t.numel(), code[t.dtype])
        for t, o in zip(g, out)])
    nbytes = B.tp_grad_workspace_bytes(2)
    ws = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    norm = torch.empty((), device="cuda")
    B.tp_grad_norm(2, table, norm, ws, nbytes)
    assert torch.equal(norm, grad_norm(g))
    norm.zero_()
    B.tp_grad_clip(2, table, 1.0, 1e-6, norm, ws, nbytes)
    assert torch.equal(norm, clip_grad_norm(g, 1.0, out=want))
    for a, b in zip(out, want):
        assert torch.equal(a, b)
    with pytest.raises(B.TPMLPError):
        B.tp_grad_clip(2, table, -1.0, 1e-6, norm, ws, nbytes)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_offsets_past_32_bits(dtype):
    """2^31 + 4099 elements, all zero but a few: the norm is exactly 5."""
    n = (1 << 31) + 4099
    x = torch.zeros(n, dtype=dtype, device="cuda")
    at = [0, 1 << 30, (1 << 31) - 1, 1 << 31, n - 1]
    for i, v in zip(at, (1.0, 2.0, 2.0, 4.0, 0.0)):
        x[i] = v
    assert float(grad_norm([x])) == 5.0
    assert float(clip_grad_norm([x], 2.5, eps=0.0)) == 5.0
    assert [float(x[i]) for i in at] == [0.5, 1.0, 1.0, 2.0, 0.0]
    assert int(torch.count_nonzero(x)) == 4
