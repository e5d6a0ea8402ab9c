"""The measured cases of the query/key operators and of the gradient norm.

Three operators, each as a user's program calls it:

* ``rope``: rotary positions on the queries and keys of one call (half and
  interleaved layouts, part of the head, frequencies scaled for long
  contexts), and its gradient (``rope_grad``);
* ``qk``: each head of the queries and keys normalised (RMS or LayerNorm,
  with its parameters) and rotated in the same pass, and its gradient
  (``qk_grad``), parameter gradients included;
* ``clip``: the global L2 norm of many gradient tensors, and those tensors
  scaled so that the norm is at most ``max_norm``.

With ``own`` false ``run`` computes the plain form in elementary torch
operations; with ``own`` true it calls the package.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
DEV = "cuda"


def _qk(name, op, T, hq, hk, d, r, dtype, *, shards=0, inter=False, pos="seq",
        max_pos=2048, scaling="none", factor=1.0, base=10000.0, original=0,
        norm="none", eps=1e-6):
    """shards > 0: queries and keys are views of one fused projection
    [T, shards, 3, heads / shards, d] (hq == hk); 0: tensors of their own.
    pos: "seq" = 0 .. max_pos - 1 over and over (no position tensor), "far" =
    one int64 position a token, anywhere below max_pos (single tokens of many
    requests), "ragged" = packed sequences of odd lengths, int32."""
    return {"name": name, "op": op, "T": T, "hq": hq, "hk": hk, "d": d, "r": r,
            "dtype": dtype, "shards": shards, "inter": inter, "pos": pos,
            "max_pos": max_pos, "scaling": scaling, "factor": factor,
            "base": base, "original": original, "norm": norm, "eps": eps}


def _clip(name, sizes, times, dtype, scale, max_norm):
    """`sizes` repeated `times` times: the gradient tensors' lengths."""
    return {"name": name, "op": "clip",
            "sizes": " ".join(str(n) for n in sizes), "times": times,
            "dtype": dtype, "scale": scale, "max_norm": max_norm, "eps": 1e-6}


def listed():
    return [
        # one new token for each of 32 requests, far into their contexts
        # (h = 1024, 16 heads of 64): the smallest call, latency counts
        _qk("rope_decode", "rope", 32, 16, 16, 64, 64, "bf16", pos="far",
            max_pos=1000000, base=1000000.0),
        # packed sequences of odd lengths, fewer key than query heads, half of
        # an 80-wide head rotated, interleaved pairs, fp32
        _qk("rope_packed_fp32", "rope", 1003, 12, 4, 80, 40, "fp32",
            inter=True, pos="ragged", max_pos=4096, scaling="ntk", factor=4.0),
        # the GPT-3-13B-shaped layer's fused projection (4 x 2048 tokens, 40
        # heads of 128 in 8 shards), frequencies stretched band by band
        _qk("rope_gpt3_13b", "rope", 8192, 40, 40, 128, 128, "bf16", shards=8,
            scaling="yarn", factor=4.0, original=512),
        # gradient on the BLOOM-176B-shaped layer (2 x 2048 tokens, 112 heads)
        _qk("rope_grad_bloom", "rope_grad", 4096, 112, 112, 128, 128, "bf16",
            shards=4, inter=True, scaling="linear", factor=2.0),
        # one new token for each of 8 requests on the 13B-shaped layer
        _qk("qk_decode", "qk", 8, 40, 40, 128, 128, "bf16", shards=8,
            pos="far", max_pos=200000, norm="rms"),
        # an odd number of tokens, 96-wide heads, half of each rotated,
        # LayerNorm with a bias (32 heads in 8 shards)
        _qk("qk_odd_layer", "qk", 2047, 32, 32, 96, 48, "bf16", shards=8,
            pos="ragged", max_pos=2048, norm="layer", eps=1e-5),
        # a training step's forward on the 13B-shaped layer
        _qk("qk_gpt3_13b", "qk", 8192, 40, 40, 128, 128, "bf16", shards=8,
            norm="rms"),
        # gradients in fp32, shared key heads, 80-wide heads
        _qk("qk_grad_odd_fp32", "qk_grad", 777, 12, 4, 80, 80, "fp32",
            pos="ragged", max_pos=1024, norm="layer", eps=1e-5),
        # a training step's backward on the 13B-shaped layer
        _qk("qk_grad_gpt3_13b", "qk_grad", 8192, 40, 40, 128, 128, "bf16",
            shards=8, norm="rms"),
        # the bias and LayerNorm gradients of 8 GPT-2-medium-shaped layers:
        # many short tensors
        _clip("clip_vectors", [1024, 1024, 1024, 1024, 4096, 1024], 8, "fp32",
              0.02, 1.0),
        # all gradients of one GPT-2-medium-shaped layer (50 MB: stays in L2)
        _clip("clip_gpt2_medium", [1024 * 4096, 4096 * 1024, 1024 * 3 * 1024,
                                   1024 * 1024, 4096, 1024, 3 * 1024, 1024], 1,
              "fp32", 0.01, 1.0),
        # all gradients of one GPT-3-13B-shaped layer (1.26 GB)
        _clip("clip_gpt3_13b", [5120 * 20480, 20480 * 5120, 5120 * 15360,
                                5120 * 5120, 20480, 5120, 15360, 5120], 1,
              "fp32", 0.001, 1.0),
    ]


def _lengths(c):
    return [int(n) for n in c["sizes"].split()] * c["times"]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo),
                                                          math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "rope_grad", "qk", "qk", "qk_grad", "qk_grad",
                     "clip"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    if op == "clip":
        count = _log(rng, 1, 60)
        total = _log(rng, 1000, 100000000)
        cuts = [rng.random() ** 3 + 1e-6 for _ in range(count)]
        sizes = [max(1, int(total * c / sum(cuts))) for c in cuts]
        scale = rng.choice([1e-4, 0.01, 1.0])
        c = _clip("", sizes, 1, dtype, scale, rng.choice([0.5, 1.0, 5.0]))
    else:
        d = rng.choice([32, 40, 64, 64, 72, 80, 96, 100, 112, 128, 128, 160,
                        192, 256])
        r = rng.choice([d, d, d // 2 // 2 * 2, d // 4 // 2 * 2,
                        2 * rng.randint(1, d // 2)])
        shards = rng.choice([0, 0, 1, 2, 4, 8])
        if shards:
            hq = hk = shards * rng.randint(1, 40 // shards)
        else:
            hk = rng.randint(1, 10)
            hq = hk * rng.randint(1, 4)
        T = _log(rng, 1, 8192)
        T = min(T, 80 * 8192 * 128 // ((hq + hk) * d * (4 if dtype == "fp32"
                                                        else 2) // 2))
        pos = rng.choice(["seq", "far", "ragged"])
        max_pos = (_log(rng, 2048, 4000000) if pos == "far"
                   else _log(rng, 16, 8192))
        scaling = rng.choice(["none", "linear", "ntk", "yarn"])
        norm = ("none" if op.startswith("rope")
                else rng.choice(["rms", "layer"]))
        c = _qk("", op, T, hq, hk, d, r, dtype, shards=shards,
                inter=rng.random() < 0.5, pos=pos, max_pos=max_pos,
                scaling=scaling,
                factor=1.0 if scaling == "none" else rng.choice([1.5, 4.0, 8.0]),
                base=rng.choice([10000.0, 500000.0]),
                original=rng.choice([1024, 4096]) if scaling == "yarn" else 0,
                norm=norm, eps=rng.choice([1e-6, 1e-5]))
    del c["name"]
    return c


# ----------------------------------------------------------------- inputs --

def _frequencies(c):
    """(inverse frequencies [r / 2], amplitude) in double precision: base^
    (-2i/r), then "linear": all divided by factor; "ntk": base times
    factor^(r / (r - 2)); "yarn": pairs that turn fewer than once over the
    original length divided by factor, pairs that turn more than 32 times kept,
    a linear ramp in the number of turns between, and an amplitude of
    0.1 ln(factor) + 1."""
    r, base = c["r"], c["base"]
    if c["scaling"] == "ntk" and r > 2:
        base = base * c["factor"] ** (r / (r - 2))
    f = [base ** (-2.0 * i / r) for i in range(r // 2)]
    amp = 1.0
    if c["scaling"] == "linear":
        f = [x / c["factor"] for x in f]
    if c["scaling"] == "yarn":
        turns = [c["original"] * x / (2 * math.pi) for x in f]
        keep = [min(1.0, max(0.0, (n - 1.0) / 31.0)) for n in turns]
        f = [k * x + (1 - k) * x / c["factor"] for k, x in zip(keep, f)]
        amp = 0.1 * math.log(c["factor"]) + 1.0
    return f, amp


def _pair(c, g, dt):
    """Queries and keys as the program holds them: [T, shards, heads per
    shard, d] views of a fused projection, or [T, heads, d] tensors."""
    T, d = c["T"], c["d"]
    if c["shards"]:
        x = torch.randn((T, c["shards"], 3, c["hq"] // c["shards"], d),
                        generator=g, device=DEV).to(dt)
        return x[:, :, 0], x[:, :, 1]
    return tuple(torch.randn((T, h, d), generator=g, device=DEV).to(dt)
                 for h in (c["hq"], c["hk"]))


def prepare(case, seed):
    c = case
    g = torch.Generator(DEV)
    g.manual_seed(seed)
    dt = DT[c["dtype"]]
    s = {"case": c}
    if c["op"] == "clip":
        s["grads"] = [torch.randn(n, generator=g, device=DEV)
                      .mul_(c["scale"]).to(dt)
                      for n in _lengths(c)]
        s["out"] = [torch.empty_like(x) for x in s["grads"]]
        return s
    s["q"], s["k"] = _pair(c, g, dt)
    f, s["amp"] = _frequencies(c)
    s["inv_freq"] = torch.tensor(f, dtype=torch.float64, device=DEV)
    T = c["T"]
    s["positions"] = None
    if c["pos"] == "far":
        s["positions"] = torch.randint(0, c["max_pos"], (T,), generator=g,
                                       device=DEV)
    if c["pos"] == "ragged":
        start = torch.rand(T, generator=g, device=DEV) < 0.005
        t = torch.arange(T, device=DEV)
        first = torch.where(start, t, torch.zeros_like(t)).cummax(0).values
        s["positions"] = ((t - first) % c["max_pos"]).to(torch.int32)
    if c["norm"] != "none":
        for n in ("q", "k"):
            s[n + "_gamma"] = 1 + 0.2 * torch.randn(c["d"], generator=g,
                                                    device=DEV)
            s[n + "_beta"] = (0.1 * torch.randn(c["d"], generator=g, device=DEV)
                              if c["norm"] == "layer" else None)
    if c["op"].endswith("grad"):
        s["dq"], s["dk"] = _pair(c, g, dt)
    if own:
        from tensor_transformer_mlp_tcgen05_gb300 import rotary
        s["rope"] = rotary.RotaryEmbedding(
            c["d"], rotary_dim=c["r"], base=c["base"], interleaved=c["inter"],
            scaling=c["scaling"], factor=c["factor"],
            original_length=c["original"])
        if c["norm"] != "none":
            s["norm"] = rotary.QKNormRotary(c["d"], norm=c["norm"],
                                            eps=c["eps"], rotary=s["rope"])
    return s


# ------------------------------------------------------------- plain form --

def _cos_sin(s):
    """cos and sin [T, 1.., r / 2] in fp32; the angles themselves in fp64 (a
    far position loses its fraction of a turn in fp32)."""
    c = s["case"]
    if s["positions"] is None:
        pos = torch.arange(c["T"], device=DEV) % c["max_pos"]
    else:
        pos = s["positions"]
    a = pos.to(torch.float64)[:, None] * s["inv_freq"]
    a = a.reshape((c["T"],) + (1,) * (s["q"].dim() - 2) + (-1,))
    return (torch.cos(a) * s["amp"]).float(), (torch.sin(a) * s["amp"]).float()


def _rotate(x, cos, sin, r, inter):
    """The first r elements of every head of x (fp32) rotated pair by pair."""
    if inter:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        y = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
    else:
        a, b = x[..., :r // 2], x[..., r // 2:r]
        y = torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
    return torch.cat((y, x[..., r:]), -1)


def _normal(x, norm, eps):
    """(normalised x, 1 / deviation) over the last axis."""
    if norm == "layer":
        x = x - x.mean(-1, keepdim=True)
    rstd = torch.rsqrt((x * x).mean(-1, keepdim=True) + eps)
    return x * rstd, rstd


def _forward(x, gamma, beta, cos, sin, c):
    x = x.float()
    if c["norm"] != "none":
        x = _normal(x, c["norm"], c["eps"])[0] * gamma
        if beta is not None:
            x = x + beta
    return _rotate(x, cos, sin, c["r"], c["inter"]).to(DT[c["dtype"]])


def _backward(dy, x, gamma, cos, sin, c):
    g = _rotate(dy.float(), cos, -sin, c["r"], c["inter"])
    if c["norm"] == "none":
        return (g.to(DT[c["dtype"]]),)
    xh, rstd = _normal(x.float(), c["norm"], c["eps"])
    rows = tuple(range(x.dim() - 1))
    dgamma, dbeta = (g * xh).sum(rows), g.sum(rows)
    g = g * gamma
    dx = g - xh * (g * xh).mean(-1, keepdim=True)
    if c["norm"] == "layer":
        dx = dx - g.mean(-1, keepdim=True)
    dx = (dx * rstd).to(DT[c["dtype"]])
    return (dx, dgamma, dbeta) if c["norm"] == "layer" else (dx, dgamma)


def _plain_clip(s):
    c = s["case"]
    sq = torch.stack([x.float().square().sum(dtype=torch.float64)
                      for x in s["grads"]])
    norm = sq.sum().sqrt()
    scale = torch.clamp(c["max_norm"] / (norm + c["eps"]), max=1.0).float()
    return {"norm": norm.float(),
            "grads": [o.copy_(x.float() * scale)
                      for x, o in zip(s["grads"], s["out"])]}


# -------------------------------------------------------------------- run --

def run(state):
    s, c = state, state["case"]
    op = c["op"]
    if own:
        return _run_own(s, c, op)
    if op == "clip":
        return _plain_clip(s)
    cos, sin = _cos_sin(s)
    if op in ("rope", "qk"):
        return {n: _forward(s[n], s.get(n + "_gamma"), s.get(n + "_beta"), cos,
                            sin, c) for n in ("q", "k")}
    q = _backward(s["dq"], s["q"], s.get("q_gamma"), cos, sin, c)
    k = _backward(s["dk"], s["k"], s.get("k_gamma"), cos, sin, c)
    return {"q": list(q), "k": list(k)}


def _run_own(s, c, op):
    if op == "clip":
        from tensor_transformer_mlp_tcgen05_gb300 import clip
        norm = clip.clip_grad_norm(s["grads"], c["max_norm"], eps=c["eps"],
                                   out=s["out"])
        return {"norm": norm, "grads": s["out"]}
    where = {"positions": s["positions"], "seq_len": c["max_pos"]}
    if op == "rope":
        q, k = s["rope"].forward(s["q"], s["k"], **where)
        return {"q": q, "k": k}
    if op == "rope_grad":
        q, k = s["rope"].backward(s["dq"], s["dk"], **where)
        return {"q": [q], "k": [k]}
    if op == "qk":
        q, k = s["norm"].forward(s["q"], s["k"], s["q_gamma"], s["k_gamma"],
                                 s["q_beta"], s["k_beta"], **where)
        return {"q": q, "k": k}
    g = s["norm"].backward(s["dq"], s["dk"], s["q"], s["k"], s["q_gamma"],
                           s["k_gamma"], **where)
    names = ("d{0}", "d{0}_gamma", "d{0}_beta")[:3 if c["norm"] == "layer" else 2]
    return {n: [g[m.format(n)] for m in names] for n in ("q", "k")}


def work(case):
    c = case
    if c["op"] == "clip":
        n = sum(_lengths(c))
        return {"bytes": 2 * n * (4 if c["dtype"] == "fp32" else 2),
                "flops": 3 * n}
    n = c["T"] * (c["hq"] + c["hk"]) * c["d"]
    size = 4 if c["dtype"] == "fp32" else 2
    tensors = 3 if c["op"] == "qk_grad" else 2
    extra = c["T"] * {"seq": 0, "far": 8, "ragged": 4}[c["pos"]]
    extra += 0 if c["norm"] == "none" else 8 * c["d"] * (
        (2 if c["norm"] == "layer" else 1) + (1 if tensors == 3 else 0))
    flops = 3 * n * c["r"] // c["d"]
    flops += 0 if c["norm"] == "none" else n * (4 if tensors == 2 else 11)
    return {"bytes": tensors * n * size + extra, "flops": flops}


# ------------------------------------------------------------------ exact --

def _turn(x, z, r, inter):
    """x (fp64) as complex pairs times z."""
    y = x.clone()
    if inter:
        y[..., :r] = torch.view_as_real(
            torch.view_as_complex(x[..., :r].reshape(*x.shape[:-1], r // 2, 2)
                                  .contiguous()) * z).flatten(-2)
    else:
        w = torch.complex(x[..., :r // 2], x[..., r // 2:r]) * z
        y[..., :r // 2], y[..., r // 2:r] = w.real, w.imag
    return y


def exact(case, seed):
    """The definitions in 64 bits: rotations as products of complex numbers,
    gradients by differentiating the forward's definition."""
    c, s = case, prepare(case, seed)
    if c["op"] == "clip":
        norm = torch.linalg.vector_norm(torch.stack(
            [torch.linalg.vector_norm(x.double()) for x in s["grads"]]))
        k = min(1.0, c["max_norm"] / (float(norm) + c["eps"]))
        return {"norm": norm, "grads": [x.double() * k for x in s["grads"]]}
    pos = (s["positions"].double() if s["positions"] is not None else
           torch.arange(c["T"], dtype=torch.float64, device=DEV) % c["max_pos"])
    angle = torch.outer(pos, s["inv_freq"])
    z = torch.polar(torch.full_like(angle, s["amp"]), angle)
    z = z.view(c["T"], *[1] * (s["q"].dim() - 2), -1)

    def forward(x, gamma, beta):
        if c["norm"] == "rms":
            x = x / torch.sqrt(x.pow(2).mean(-1, keepdim=True) + c["eps"])
        if c["norm"] == "layer":
            var, mean = torch.var_mean(x, -1, correction=0, keepdim=True)
            x = (x - mean) / torch.sqrt(var + c["eps"])
        if gamma is not None:
            x = x * gamma
        if beta is not None:
            x = x + beta
        return _turn(x, z, c["r"], c["inter"])

    found = {}
    for n in ("q", "k"):
        leaves = [s[n].double()] + [
            None if s.get(n + m) is None else s[n + m].double()
            for m in ("_gamma", "_beta")]
        if not c["op"].endswith("grad"):
            found[n] = forward(*leaves)
            continue
        held = [v.requires_grad_() for v in leaves if v is not None]
        found[n] = list(torch.autograd.grad(forward(*leaves), held,
                                            s["d" + n].double()))
    return found
