"""What the feed-forward operators on Sherry weights are measured on.

``listed()`` names the measured cases and ``draw()`` makes more of the same
ranges.  ``prepare()`` makes a case's inputs from a seed, ``run()`` is one pass
through the operator and ``exact()`` its definition in 64 bits.  With ``own``
false, ``run`` computes in elementary 32-bit torch operations; with ``own``
true it calls the library.

The operators are the feed-forward half of a decoder layer whose weights are
3:4-sparse ternary (T in {-1,0,+1}, one fp32 scale alpha per output row) and
whose activations are int8 with one fp32 scale s per token:

  gemm_fused            y = act(q T^T s alpha + bias) + residual
  gemm_fused_backward   gradients of q s, alpha and bias
  glu                   h = act(q Tg^T s alpha_g) * (q Tu^T s alpha_u)
  glu_backward          gradients of q s, alpha_g and alpha_u
  layernorm             y = (x - mean) rstd w + b, with mean and rstd
  layernorm_quantize    the same row as int8 with its scale, max|y| / 127
  layernorm_backward    gradients of x, w and b
"""

import math

import torch

own = False

TYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
ACTS = ("none", "relu", "relu2", "silu", "gelu", "gelu_tanh")
EPS = 1e-5


def listed():
    return [
        # one new token through a 7B model's down projection, added to the residual stream
        {"name": "gemm_decode", "op": "gemm_fused", "M": 1, "K": 11008, "N": 4096, "dtype": "bf16",
         "act": "none", "bias": False, "residual": True},
        # a served batch of 16 through a square projection with bias and activation
        {"name": "gemm_batch16", "op": "gemm_fused", "M": 16, "K": 4096, "N": 4096, "dtype": "fp16",
         "act": "gelu", "bias": True, "residual": True},
        # a prompt of 512 tokens through a down projection, added to the residual stream
        {"name": "gemm_prefill", "op": "gemm_fused", "M": 512, "K": 14336, "N": 4096, "dtype": "bf16",
         "act": "none", "bias": False, "residual": True},
        # a training step of a small layer, sizes no tile divides, gradients in 32 bits
        {"name": "gemm_backward_ragged", "op": "gemm_fused_backward", "M": 300, "K": 2064, "N": 1100,
         "dtype": "fp32", "act": "gelu", "bias": True, "residual": False},
        # one new token through a 7B model's gate and up projections
        {"name": "glu_decode", "op": "glu", "M": 1, "K": 4096, "N": 11008, "dtype": "bf16", "act": "silu"},
        # a served batch of 8 through a 70B model's gate and up projections
        {"name": "glu_batch8", "op": "glu", "M": 8, "K": 8192, "N": 28672, "dtype": "fp32", "act": "silu"},
        # a prompt of 512 tokens through gate and up
        {"name": "glu_prefill", "op": "glu", "M": 512, "K": 4096, "N": 14336, "dtype": "bf16", "act": "silu"},
        # a training step's 2048 tokens back through gate and up
        {"name": "glu_backward", "op": "glu_backward", "M": 2048, "K": 4096, "N": 14336, "dtype": "bf16",
         "act": "silu"},
        # a short odd batch back through a small gated block, in 32 bits
        {"name": "glu_backward_ragged", "op": "glu_backward", "M": 77, "K": 1040, "N": 1300, "dtype": "fp32",
         "act": "gelu_tanh"},
        # a served batch of 16 normalized into the int8 tokens the products take
        {"name": "norm_quantize16", "op": "layernorm_quantize", "M": 16, "K": 8192, "dtype": "bf16"},
        # a prompt's or a training step's 2048 tokens normalized
        {"name": "norm_forward", "op": "layernorm", "M": 2048, "K": 4096, "dtype": "bf16"},
        # the same norm's gradients over a training step of 8192 tokens
        {"name": "norm_backward", "op": "layernorm_backward", "M": 8192, "K": 4096, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))


def draw(rng):
    op = rng.choice(("gemm_fused", "gemm_fused", "gemm_fused_backward", "glu", "glu", "glu_backward",
                     "layernorm", "layernorm_quantize", "layernorm_backward"))
    case = {"op": op, "dtype": rng.choice(("fp32", "fp16", "bf16"))}
    if op.startswith("layernorm"):
        case["K"] = 4 * _log(rng, 16, 4096)
        case["M"] = _log(rng, 1, min(8192, (8192 * 4096) // case["K"]))
        return case
    case["K"] = 16 * _log(rng, 16, 896)
    case["N"] = 4 * _log(rng, 64, min(7168, (1 << 26) // (4 * case["K"])))
    case["M"] = _log(rng, 1, min(2048, (2048 * 4096 * 7168) // (case["K"] * case["N"])))
    if op.startswith("glu"):
        case["act"] = rng.choice(ACTS[1:])
    else:
        case["act"] = rng.choice(ACTS)
        case["bias"] = rng.random() < 0.5
        case["residual"] = op == "gemm_fused" and rng.random() < 0.7
    return case


def _ternary(N, K, gen):
    """A 3:4-sparse ternary matrix, dense in 32 bits and in the packed 5-bit
    format (64-row x 128-column tiles, see include/sherry.h)."""
    dev = gen.device
    zero = torch.randint(0, 4, (N, K // 4), generator=gen, device=dev, dtype=torch.int8)
    neg = torch.randint(0, 2, (N, K // 4, 4), generator=gen, device=dev, dtype=torch.int8)
    place = torch.arange(4, device=dev, dtype=torch.int8)
    T = ((1 - 2 * neg) * (place != zero[..., None])).reshape(N, K).float()
    first = torch.where(zero == 0, neg[..., 1], neg[..., 0])
    second = torch.where(zero <= 1, neg[..., 2], neg[..., 1])
    third = torch.where(zero <= 2, neg[..., 3], neg[..., 2])
    code = first + 2 * (first ^ third) + 4 * (first ^ second) + 8 * zero
    rt, kt = -(-N // 64), -(-K // 128)
    codes = torch.zeros((rt * 64, kt * 32), device=dev, dtype=torch.int64)
    codes[:N, :K // 4] = code
    shifts = 5 * torch.arange(8, device=dev)
    groups = (codes.view(rt, 4, 16, kt, 4, 8) << shifts).sum(-1)        # [row tile, t, i, k tile, g]
    groups = groups.permute(0, 3, 4, 2, 1)                              # [row tile, k tile, g, i, t]
    low = (groups[..., None] >> (8 * torch.arange(4, device=dev))) & 255
    packed = torch.cat([low.reshape(rt, kt, 1024), (groups >> 32).reshape(rt, kt, 256)], dim=2)
    return T, packed.to(torch.uint8).flatten()


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dtype, M, K = TYPES[case["dtype"]], case["M"], case["K"]

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    state = {"case": case, "dtype": dtype}
    if case["op"].startswith("layernorm"):
        # a residual stream: tokens of different sizes, a mean, a few large channels
        x = normal(M, K) * (0.5 + 2.0 * torch.rand((M, 1), generator=gen, device="cuda")) + 0.3 * normal(K)
        x = (x * torch.where(torch.rand(K, generator=gen, device="cuda") < 0.005, 20.0, 1.0)).to(dtype)
        state |= {"x": x, "weight": 1.0 + 0.2 * normal(K), "bias": 0.1 * normal(K)}
        if case["op"] == "layernorm_backward":
            state["dy"] = (0.1 * normal(M, K)).to(dtype)
            x64 = x.double()
            mean = x64.mean(1)
            state["mean"] = mean.float()
            state["rstd"] = (x64.var(1, unbiased=False) + EPS).rsqrt().float()
        return state

    N = case["N"]
    x = normal(M, K)
    s = x.abs().amax(1) / 127.0
    state |= {"q": torch.clamp(torch.round(x / s[:, None]), -127, 127).to(torch.int8), "s": s}
    size = (0.75 * K) ** -0.5       # row scales that give outputs of size one

    def weights(key):
        state["T" + key], state["packed" + key] = _ternary(N, K, gen)
        state["alpha" + key] = size * (0.7 + 0.6 * torch.rand(N, generator=gen, device="cuda"))

    weights("")
    if case["op"].startswith("glu"):
        weights("_up")
    else:
        state["bias"] = 0.5 * normal(N) if case["bias"] else None
        state["residual"] = normal(M, N).to(dtype) if case["residual"] else None
    if case["op"].endswith("backward"):
        state["dy"] = (0.05 * normal(M, N)).to(dtype)
    return state


# ---------------------------------------------------------------- plain form
def _act(z, act):
    if act == "none":
        return z
    if act == "relu":
        return torch.where(z > 0, z, 0.0)
    if act == "relu2":
        return torch.where(z > 0, z * z, 0.0)
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * 0.5 ** 0.5))
    return 0.5 * z * (1 + torch.tanh((2 / math.pi) ** 0.5 * (z + 0.044715 * z * z * z)))


def _act_slope(z, act):
    if act == "none":
        return torch.ones_like(z)
    if act == "relu":
        return torch.where(z > 0, 1.0, 0.0)
    if act == "relu2":
        return torch.where(z > 0, 2 * z, 0.0)
    if act == "silu":
        g = 1 / (1 + torch.exp(-z))
        return g * (1 + z * (1 - g))
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * 0.5 ** 0.5)) + z * torch.exp(-0.5 * z * z) * (2 * math.pi) ** -0.5
    c = (2 / math.pi) ** 0.5
    t = torch.tanh(c * (z + 0.044715 * z * z * z))
    return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)


def _plain(st):
    case, dtype = st["case"], st["dtype"]
    op = case["op"]
    if op == "layernorm_quantize":     # in 64 bits: a token's int8 value may lie next to a border
        x = st["x"].double()
        mean = x.mean(1, keepdim=True)
        d = x - mean
        rstd = torch.rsqrt((d * d).mean(1, keepdim=True) + EPS)
        y = d * rstd * st["weight"].double() + st["bias"].double()
        top = y.abs().amax(1, keepdim=True)
        s = torch.where(top > 0, top / 127.0, 1.0).float()
        q = torch.clamp(torch.round(y / s.double()), -127, 127)
        return {"tokens": (q * s.double()).float(), "scale": s[:, 0]}
    if op.startswith("layernorm"):
        x, w = st["x"].float(), st["weight"]
        if op == "layernorm":
            mean = x.mean(1, keepdim=True)
            d = x - mean
            rstd = torch.rsqrt((d * d).mean(1, keepdim=True) + EPS)
            return {"y": (d * rstd * w + st["bias"]).to(dtype), "mean": mean[:, 0], "rstd": rstd[:, 0]}
        dy, rstd = st["dy"].float(), st["rstd"][:, None]
        xh = (x - st["mean"][:, None]) * rstd
        dxh = dy * w
        dx = rstd * (dxh - dxh.mean(1, keepdim=True) - xh * (dxh * xh).mean(1, keepdim=True))
        return {"dx": dx.to(dtype), "dweight": (dy * xh).sum(0), "dbias": dy.sum(0)}
    act, q, s = case["act"], st["q"].float(), st["s"][:, None]
    a = (q @ st["T"].t()) * s          # whole sums below 2^24: exact in 32 bits
    if op.startswith("glu"):
        b = (q @ st["T_up"].t()) * s
        g, u = a * st["alpha"], b * st["alpha_up"]
        if op == "glu":
            return {"h": (_act(g, act) * u).to(dtype)}
        dh = st["dy"].float()
        dg, du = dh * u * _act_slope(g, act), dh * _act(g, act)
        dx = (dg * st["alpha"]) @ st["T"] + (du * st["alpha_up"]) @ st["T_up"]
        return {"dx": dx.to(dtype), "dalpha_gate": (dg * a).sum(0), "dalpha_up": (du * b).sum(0)}
    z = a * st["alpha"]
    if st["bias"] is not None:
        z = z + st["bias"]
    if op == "gemm_fused":
        y = _act(z, act)
        if st["residual"] is not None:
            y = y + st["residual"].float()
        return {"y": y.to(dtype)}
    dz = st["dy"].float() * _act_slope(z, act)
    return {"dx": ((dz * st["alpha"]) @ st["T"]).to(dtype), "dalpha": (dz * a).sum(0), "dbias": dz.sum(0)}


# ------------------------------------------------------------ the library's
def _library(st):
    import bit_weight_amd as bw

    case = st["case"]
    op = case["op"]
    if op == "layernorm":
        y, mean, rstd = bw.layernorm(st["x"], st["weight"], st["bias"], eps=EPS, stats=True)
        return {"y": y, "mean": mean, "rstd": rstd}
    if op == "layernorm_quantize":
        q, s = bw.layernorm_quantize(st["x"], st["weight"], st["bias"], eps=EPS)
        return {"tokens": q * s[:, None], "scale": s}
    if op == "layernorm_backward":
        dx, dw, db = bw.layernorm_backward(st["dy"], st["x"], st["mean"], st["rstd"], st["weight"])
        return {"dx": dx, "dweight": dw, "dbias": db}
    N, K, act = case["N"], case["K"], case["act"]
    if op == "glu":
        return {"h": bw.glu(st["q"], st["s"], st["packed"], st["alpha"], st["packed_up"], st["alpha_up"], N, K,
                            act=act, dtype=st["dtype"])}
    if op == "glu_backward":
        dx, dg, du = bw.glu_backward(st["dy"], st["q"], st["s"], st["packed"], st["alpha"], st["packed_up"],
                                     st["alpha_up"], N, K, act=act)
        return {"dx": dx, "dalpha_gate": dg, "dalpha_up": du}
    if op == "gemm_fused":
        return {"y": bw.gemm_fused(st["q"], st["s"], st["packed"], st["alpha"], N, K, bias=st["bias"], act=act,
                                   residual=st["residual"], dtype=st["dtype"])}
    dx, da, db = bw.gemm_fused_backward(st["dy"], st["q"], st["s"], st["packed"], st["alpha"], N, K,
                                        bias=st["bias"], act=act)
    return {"dx": dx, "dalpha": da, "dbias": db}


def run(state):
    return _library(state) if own else _plain(state)


def work(case):
    M, K, wide = case["M"], case["K"], 4 if case["dtype"] == "fp32" else 2
    op = case["op"]
    if op == "layernorm":
        return {"bytes": 2 * wide * M * K + 8 * K + 8 * M, "flops": 8 * M * K}
    if op == "layernorm_quantize":
        return {"bytes": (wide + 4) * M * K + 8 * K + 4 * M, "flops": 12 * M * K}
    if op == "layernorm_backward":
        return {"bytes": 3 * wide * M * K + 12 * K + 8 * M, "flops": 14 * M * K}
    N = case["N"]
    parts = 2 if op.startswith("glu") else 1
    fixed = M * K + 4 * M + parts * (N * K * 5 // 32 + 4 * N)     # tokens, scales, codes, alpha
    if op.endswith("backward"):
        vectors = 4 * N * (2 if parts == 2 else 2 + bool(case["bias"]))   # dalpha, dbias, bias
        return {"bytes": fixed + wide * M * (N + K) + vectors, "flops": 4 * parts * M * N * K}
    more = 0 if parts == 2 else 4 * N * bool(case["bias"]) + wide * M * N * bool(case["residual"])
    return {"bytes": fixed + more + wide * M * N, "flops": 2 * parts * M * N * K}


# ------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op.startswith("layernorm"):
        x = st["x"].double().requires_grad_(op == "layernorm_backward")
        w = st["weight"].double().requires_grad_(op == "layernorm_backward")
        b = st["bias"].double().requires_grad_(op == "layernorm_backward")
        var, mean = torch.var_mean(x, dim=1, correction=0)
        y = torch.addcmul(b, (x - mean[:, None]) / torch.sqrt(var + EPS)[:, None], w)
        if op == "layernorm":
            return {"y": y, "mean": mean, "rstd": 1 / torch.sqrt(var + EPS)}
        if op == "layernorm_quantize":
            s = (y.abs().max(dim=1).values / 127).float().double()
            s = torch.where(s > 0, s, 1.0)
            return {"tokens": (y / s[:, None]).round().clamp(-127, 127) * s[:, None], "scale": s}
        dx, dw, db = torch.autograd.grad(y, (x, w, b), st["dy"].double())
        return {"dx": dx, "dweight": dw, "dbias": db}

    grad = op.endswith("backward")
    function = {"none": lambda z: z, "relu": torch.nn.functional.relu,
                "relu2": lambda z: torch.nn.functional.relu(z).square(), "silu": torch.nn.functional.silu,
                "gelu": torch.nn.functional.gelu,
                "gelu_tanh": lambda z: torch.nn.functional.gelu(z, approximate="tanh")}[case["act"]]
    xs = (st["q"].double() * st["s"].double()[:, None]).requires_grad_(grad)
    alpha = st["alpha"].double().requires_grad_(grad)
    z = torch.nn.functional.linear(xs, st["T"].double()) * alpha
    if op.startswith("glu"):
        alpha_up = st["alpha_up"].double().requires_grad_(grad)
        h = function(z) * (torch.nn.functional.linear(xs, st["T_up"].double()) * alpha_up)
        if not grad:
            return {"h": h}
        found = torch.autograd.grad(h, (xs, alpha, alpha_up), st["dy"].double())
        return dict(zip(("dx", "dalpha_gate", "dalpha_up"), found))
    bias = torch.zeros_like(st["alpha"]) if st["bias"] is None else st["bias"]
    bias = bias.double().requires_grad_(grad)
    y = function(z + bias)
    if not grad:
        return {"y": y if st["residual"] is None else y + st["residual"].double()}
    return dict(zip(("dx", "dalpha", "dbias"), torch.autograd.grad(y, (xs, alpha, bias), st["dy"].double())))
