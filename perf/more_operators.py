"""The measured cases of the four-bit operators.

Microscaled four-bit floating point (E2M1 codes with one scale for a block of
consecutive elements), as a user's program calls it:

* ``quant``: a matrix quantised along its rows, or along its columns
  (``transpose``: the layout a weight [K, N] is multiplied in), and the values
  that the codes and scales stand for read back;
* ``linear``: activations quantised and multiplied by packed weights, with a
  bias: a projection of many tokens, or of a few;
* ``linear_grad``: that projection's gradients (input, weight and bias), their
  operands quantised as the forward's are;
* ``mlp``: the MLP block's forward on packed weights, GeLU(X A + b1) B + b2.

Two formats.  "nvfp4": blocks of 16, an E4M3 scale s each and a power of two g
for the whole tensor; a value is code * s * g.  s is amax / (6 g) rounded to E4M3
(nearest even, at most 448), a code x / (s g) rounded to E2M1 (nearest even, at
most 6).  g is 1, or ("auto") the smallest power of two with max |x| <= 2688 g.
"mxfp4": blocks of 32, a power of two 2^(floor(log2 amax) - 2) each, g = 1.

With ``own`` false ``run`` computes the plain form in elementary torch
operations; with ``own`` true it calls the package.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
DEV = "cuda"
BLOCK = {"nvfp4": 16, "mxfp4": 32}


def _case(name, op, T, K, N, fmt, dtype="bf16", *, transpose=False,
          scale="one", bias=True, shards=1):
    """T tokens, K inputs, N outputs of a projection (for the MLP block: hidden
    and ffn; for "quant": a [T, K] matrix)."""
    return {"name": name, "op": op, "T": T, "K": K, "N": N, "fmt": fmt,
            "dtype": dtype, "transpose": transpose, "scale": scale,
            "bias": bias, "shards": shards}


def listed():
    return [
        # activations of an odd shape, with the tensor's own power of two
        _case("quant_odd_fp32", "quant", 1003, 1000, 0, "nvfp4", "fp32",
              scale="auto"),
        # activations of a training step on the GPT-3-13B-shaped layer
        _case("quant_rows_13b", "quant", 8192, 5120, 0, "mxfp4"),
        # that layer's first weight, laid out for the product
        _case("quant_weight_13b", "quant", 5120, 20480, 0, "nvfp4",
              transpose=True, scale="auto"),
        # one new token, GPT-2-medium-shaped (h = 1024): the smallest call,
        # latency counts
        _case("linear_one_token", "linear", 1, 1024, 4096, "nvfp4"),
        # one new token for each of 32 requests, the 13B-shaped layer's second
        # weight
        _case("linear_decode_13b", "linear", 32, 20480, 5120, "mxfp4"),
        # a short prompt, sizes that no block or tile divides, fp32 activations
        _case("linear_odd_fp32", "linear", 333, 1003, 1537, "nvfp4", "fp32"),
        # a training step's tokens through the 13B-shaped fused projection
        _case("linear_qkv_13b", "linear", 8192, 5120, 15360, "nvfp4"),
        # gradients of a short, odd batch
        _case("linear_grad_odd", "linear_grad", 777, 1024, 1000, "mxfp4"),
        # gradients of the 13B-shaped output projection
        _case("linear_grad_13b", "linear_grad", 8192, 5120, 5120, "nvfp4"),
        # one new token for each of 8 requests through the 13B-shaped block
        _case("mlp_decode_13b", "mlp", 8, 5120, 20480, "nvfp4", shards=8),
        # the GPT-2-medium-shaped block on one sequence
        _case("mlp_gpt2_medium", "mlp", 1024, 1024, 4096, "mxfp4", shards=4),
        # the 13B-shaped block on 4 x 2048 tokens
        _case("mlp_13b", "mlp", 8192, 5120, 20480, "nvfp4", shards=8),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo),
                                                          math.log(hi)))))))


def draw(rng):
    op = rng.choice(["quant", "quant", "linear", "linear", "linear",
                     "linear_grad", "linear_grad", "mlp", "mlp"])
    fmt = rng.choice(["nvfp4", "mxfp4"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    T = rng.choice([_log(rng, 1, 64), _log(rng, 1, 8192), _log(rng, 256, 8192)])
    K, N = _log(rng, 64, 20480), _log(rng, 64, 20480)
    if rng.random() < 0.5:
        K, N = max(64, K // 64 * 64), max(64, N // 64 * 64)
    scale = rng.choice(["one", "auto"]) if fmt == "nvfp4" else "one"
    if op == "quant":
        K = min(K, 8192 * 12800 // T)
        c = _case("", op, T, K, 0, fmt, dtype, transpose=rng.random() < 0.5,
                  scale=scale)
    elif op == "mlp":
        shards = rng.choice([1, 2, 4, 8])
        h = max(64, min(K, 6144) // 64 * 64)
        f = max(1, N // (64 * shards)) * 64 * shards
        T = min(T, 8192 * 5120 * 20480 // (h * f))
        c = _case("", op, T, h, f, fmt, "bf16", bias=rng.random() < 0.7,
                  shards=shards)
    else:
        most = 8192 * 5120 * (15360 if op == "linear" else 5120)
        T = max(1, min(T, most // (K * N)))
        c = _case("", op, T, K, N, fmt, dtype, bias=rng.random() < 0.7)
    del c["name"]
    return c


# ----------------------------------------------------------------- inputs --

def _inputs(c, seed):
    """Activations, raw weights, biases and the output's gradient."""
    g = torch.Generator(DEV)
    g.manual_seed(seed)
    dt, T, K, N = DT[c["dtype"]], c["T"], c["K"], c["N"]

    def randn(*shape):
        return torch.randn(shape, generator=g, device=DEV)

    # activations: columns of unlike size, as a transformer's channels are
    s = {"x": randn(T, K).mul_(torch.exp(0.5 * randn(K))).to(dt)}
    if c["op"] == "quant":
        return s
    s["weights"] = [randn(K, N).mul_(K ** -0.5).to(dt)]
    if c["op"] == "mlp":
        s["weights"].append(randn(N, K).mul_(N ** -0.5).to(dt))
    s["biases"] = [0.1 * randn(w.shape[1]) if c["bias"] else None
                   for w in s["weights"]]
    if c["op"] == "linear_grad":
        s["dy"] = randn(T, N).mul_(1e-3).to(dt)
    return s


def prepare(case, seed):
    c = case
    s = _inputs(c, seed)
    s["case"] = c
    if c["op"] == "quant":
        return s
    weights = s.pop("weights")
    if own:
        from tensor_transformer_mlp_tcgen05_gb300 import fp4
        from tensor_transformer_mlp_tcgen05_gb300.mlp import TensorParallelMLP
        if c["op"] == "mlp":
            s["block"] = TensorParallelMLP(c["K"], c["N"], c["shards"], c["T"])
            s["packed"] = s["block"].pack_fp4_weights(*weights, format=c["fmt"])
        else:
            s["linear"] = fp4.Fp4Linear(weights[0], s["biases"][0],
                                        format=c["fmt"])
        return s
    # the values that the packed weights stand for
    s["w"] = [_values(w.t(), c["fmt"], "auto") for w in weights]
    if c["op"] == "linear_grad":
        s["w_rows"] = _values(weights[0], c["fmt"], "auto")
    return s


# ------------------------------------------------------------- plain form --

def _blocks(x, size):
    """x [R, C] as [R, blocks, size] in 64 bits, the last block padded with
    zeros (values next to a rounding border are decided exactly)."""
    x = x.double()
    pad = -x.shape[1] % size
    if pad:
        x = torch.cat((x, x.new_zeros(x.shape[0], pad)), 1)
    return x.view(x.shape[0], -1, size)


def _power(x):
    """2^floor(log2 x) of positive x (the quotient is a power of two, so the
    division is exact; library powers need not be)."""
    return x / (2 * torch.frexp(x).mantissa)


def _values(x, fmt, scale):
    """The fp32 values that x's codes and scales along its rows stand for."""
    cols = x.shape[1]
    x = _blocks(x, BLOCK[fmt])
    amax = x.abs().amax(-1, keepdim=True)
    if fmt == "mxfp4":
        s = _power(torch.where(amax > 0, amax, 4.0)) / 4
    else:
        if scale == "auto":
            top = amax.amax()
            p = _power(torch.where(top > 0, top, 2688.0) / 2688)
            x = x / torch.where(top > 2688 * p, 2 * p, p)
            amax = x.abs().amax(-1, keepdim=True)
        v = amax / 6
        step = _power(v.clamp(min=2.0 ** -6)) / 8
        s = (torch.round(v / step) * step).clamp(max=448)
    mag, code = x.abs(), torch.zeros_like(x)
    # half-way points between the codes 0 .5 1 1.5 2 3 4 6; a tie goes to the
    # even code
    for i, b in enumerate((0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)):
        up = mag >= b * s if i % 2 else mag > b * s
        code = code + up * (0.5 if i < 4 else 1.0 if i < 6 else 2.0)
    v = torch.copysign(code, x) * s
    if fmt == "nvfp4" and scale == "auto":
        v = v * torch.where(top > 2688 * p, 2 * p, p)
    return v.view(v.shape[0], -1)[:, :cols].float()


def _gelu(x):
    return 0.5 * x * (1 + torch.erf(x * 0.7071067811865476))


def _plain_linear(x, w, bias, fmt, scale="one"):
    y = _values(x, fmt, scale) @ w.t()
    return y if bias is None else y + bias


def run(state):
    s, c = state, state["case"]
    if own:
        return _run_own(s, c)
    fmt = c["fmt"]
    if c["op"] == "quant":
        x = s["x"].t() if c["transpose"] else s["x"]
        return _values(x, fmt, c["scale"]).bfloat16()
    if c["op"] == "linear":
        return _plain_linear(s["x"], s["w"][0], s["biases"][0],
                             fmt).bfloat16()
    if c["op"] == "mlp":
        y = _gelu(_plain_linear(s["x"], s["w"][0], s["biases"][0], fmt))
        return _plain_linear(y, s["w"][1], s["biases"][1], fmt).bfloat16()
    dx = _values(s["dy"], fmt, "auto") @ s["w_rows"].t()
    dw = _values(s["x"].t(), fmt, "one") @ _values(s["dy"].t(), fmt, "auto").t()
    out = {"dx": dx.bfloat16(), "dw": dw}
    if c["bias"]:
        out["db"] = s["dy"].float().sum(0)
    return out


# -------------------------------------------------------------------- own --

def _run_own(s, c):
    from tensor_transformer_mlp_tcgen05_gb300 import fp4
    if c["op"] == "quant":
        q = fp4.quantize(s["x"], format=c["fmt"], transpose=c["transpose"],
                         scale=None if c["scale"] == "auto" else 1.0)
        return q.dequantize()
    if c["op"] == "linear":
        return s["linear"].forward(s["x"])
    if c["op"] == "mlp":
        return s["block"].forward_fp4(s["x"], s["packed"], *s["biases"])
    g = s["linear"].backward(s["dy"], s["x"])
    return {k: v for k, v in g.items() if v is not None}


def work(case):
    c = case
    T, K, N = c["T"], c["K"], c["N"]
    size = 4 if c["dtype"] == "fp32" else 2
    four = 0.5 + 1 / BLOCK[c["fmt"]]      # bytes of an element with its scale
    if c["op"] == "quant":
        # read, packed (and written so), read back as bf16
        return {"bytes": int(T * K * (size + 2 * four + 2)), "flops": 4 * T * K}
    if c["op"] == "linear":
        return {"bytes": int(T * K * size + N * K * four + 2 * T * N
                             + 4 * N * c["bias"]), "flops": 2 * T * K * N}
    if c["op"] == "mlp":
        return {"bytes": int(4 * T * K + 2 * N * K * four
                             + 4 * (N + K) * c["bias"]),
                "flops": 4 * T * K * N}
    return {"bytes": int(T * (K + N) * size + K * N * four + 2 * T * K
                         + 4 * K * N + 4 * N * c["bias"]),
            "flops": 4 * T * K * N}


# ------------------------------------------------------------------ exact --

def _nearest(y, unit):
    """unit times the E2M1 value nearest to y / unit, found by distance: even
    codes first, so that they keep the ties."""
    best = torch.zeros_like(y)
    gap = y.abs()
    for value in (1.0, 2.0, 4.0, 0.5, 1.5, 3.0, 6.0):
        d = (y.abs() - value * unit).abs()
        closer = d < gap
        best = torch.where(closer, value * unit, best)
        gap = torch.where(closer, d, gap)
    return torch.where(y < 0, -best, best)


def _e4m3(v):
    """v >= 0 rounded to E4M3, by distance to the format's 127 values."""
    table = torch.arange(127, dtype=torch.uint8, device=v.device)
    table = table.view(torch.float8_e4m3fn).double()
    hi = torch.searchsorted(table, v).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    up = table[hi] - v
    down = v - table[lo]
    take = (up < down) | ((up == down) & (hi % 2 == 0))
    return torch.where(take, table[hi], table[lo])


def _exact_values(x, fmt, scale):
    """x [R, C] (64 bits) quantised along its rows."""
    size = BLOCK[fmt]
    R, C = x.shape
    y = torch.zeros((R, -(-C // size) * size), dtype=torch.float64,
                    device=x.device)
    y[:, :C] = x
    y = y.unflatten(1, (-1, size))
    top = y.abs().max(-1, keepdim=True).values
    if fmt == "mxfp4":
        # 2^floor(log2 top) is top without its fraction's bits
        power = torch.where(top > 0, top, 4.0).view(torch.int64)
        unit = (power & (0x7ff << 52)).view(torch.float64) / 4
        return _nearest(y, unit).flatten(1)[:, :C]
    g = 1.0
    if scale == "auto" and float(top.max()) > 0:
        g = 2.0 ** math.ceil(math.log2(float(top.max()) / 2688.0))
    unit = _e4m3(torch.clamp(top / g / 6.0, max=448.0)) * g
    return _nearest(y, unit).flatten(1)[:, :C]


def exact(case, seed):
    """The definitions in 64 bits."""
    c = case
    s = _inputs(c, seed)
    fmt, x = c["fmt"], s["x"].double()
    if c["op"] == "quant":
        return _exact_values(x.t() if c["transpose"] else x, fmt, c["scale"])
    w = [_exact_values(m.double().t(), fmt, "auto") for m in s["weights"]]
    if c["op"] == "linear":
        y = torch.mm(_exact_values(x, fmt, "one"), w[0].t())
        return y + s["biases"][0].double() if c["bias"] else y
    if c["op"] == "mlp":
        h = torch.mm(_exact_values(x, fmt, "one"), w[0].t())
        if c["bias"]:
            h = h + s["biases"][0].double()
        y = h * torch.special.ndtr(h)
        z = torch.mm(_exact_values(y, fmt, "one"), w[1].t())
        return z + s["biases"][1].double() if c["bias"] else z
    dy = s["dy"].double()
    W = s["weights"][0].double()
    out = {"dx": torch.mm(_exact_values(dy, fmt, "auto"),
                          _exact_values(W, fmt, "auto").t()),
           "dw": torch.mm(_exact_values(x.t(), fmt, "one"),
                          _exact_values(dy.t(), fmt, "auto").t())}
    if c["bias"]:
        out["db"] = dy.sum(0)
    return out
