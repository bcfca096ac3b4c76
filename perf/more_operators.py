"""What the attention operators of a decoder layer are measured on.

``listed()`` names the measured cases and ``draw()`` makes more of the same
ranges.  ``prepare()`` makes a case's inputs from a seed, ``run()`` is one pass
through the operator and ``exact()`` its definition in 64 bits.  With ``own``
false, ``run`` computes in elementary torch operations; with ``own`` true it
calls the library.

The operators are what lies between the stacked q/k/v projection of a decoder
layer and its output projection, on a paged cache in 8 bits:

  qk_norm_rope           z = R(position) (x / sqrt(mean x^2 + eps) w) for each head of q and k
  qk_norm_rope_backward  gradients of x and of both w
  cache_write            new tokens' k and v into pages, as int8 with one power of two for
                         each block of 16 tokens and head
  cache_read             the values of a range of tokens back
  cache_attention        causal attention of each sequence's newest tokens over its pages,
                         with a sliding window and first tokens that stay visible

The cache: k int8 [pages, heads, page / 16, dim / 16, 16 tokens, 16 features], v the same with
tokens last, scales fp32 [pages, heads, page / 16].  A block's scale is the least 2^e with
max|x| <= 127 2^e over its tokens; it only grows as tokens are added, and the values that are
there are then rounded again.
"""

import math

import torch

own = False

TYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
EPS = 1e-6


def listed():
    return [
        # a served batch of 8, one token each: queries and keys of a stacked projection
        {"name": "norm_rope_decode", "op": "qk_norm_rope", "T": 8, "q_heads": 32, "heads": 8, "dim": 128, "rotary": 128,
         "interleaved": False, "norm": True, "far": 30000, "dtype": "bf16"},
        # a prompt's or a training step's 8192 tokens
        {"name": "norm_rope_prompt", "op": "qk_norm_rope", "T": 8192, "q_heads": 32, "heads": 8, "dim": 128, "rotary": 128,
         "interleaved": False, "norm": True, "far": 8192, "dtype": "bf16"},
        # the same step's gradients
        {"name": "norm_rope_backward", "op": "qk_norm_rope_backward", "T": 8192, "q_heads": 32, "heads": 8, "dim": 128,
         "rotary": 128, "interleaved": False, "norm": True, "far": 8192, "dtype": "bf16"},
        # an odd batch of a small model in 32 bits, heads of 80 features of which 32 turn, at far positions
        {"name": "norm_rope_backward_ragged", "op": "qk_norm_rope_backward", "T": 777, "q_heads": 12, "heads": 4, "dim": 80,
         "rotary": 32, "interleaved": True, "norm": True, "far": 1000000, "dtype": "fp32"},
        # a served batch of 64 writes one token each, into blocks that are partly filled
        {"name": "cache_write_decode", "op": "cache_write", "S": 64, "L": 64, "new": 1, "heads": 8, "dim": 128, "page": 16,
         "dtype": "bf16"},
        # five prompts of odd lengths behind what their sequences hold
        {"name": "cache_write_prompt", "op": "cache_write", "S": 5, "L": 2500, "new": 2100, "heads": 8, "dim": 128,
         "page": 64, "dtype": "bf16"},
        # the keys and values of six sequences read back for a library that takes no pages
        {"name": "cache_read_long", "op": "cache_read", "S": 6, "L": 16000, "new": 16000, "heads": 8, "dim": 128, "page": 64,
         "dtype": "bf16"},
        # the last tokens of an odd batch of a small model, in 32 bits
        {"name": "cache_read_ragged", "op": "cache_read", "S": 7, "L": 900, "new": 300, "heads": 3, "dim": 96, "page": 16,
         "dtype": "fp32"},
        # one new token of one conversation of 1000 tokens
        {"name": "attention_single", "op": "cache_attention", "S": 1, "L": 1000, "new": 1, "q_heads": 32, "heads": 8,
         "dim": 128, "page": 16, "window": 0, "sinks": 0, "dtype": "bf16"},
        # a served batch of 64 conversations of up to 8192 tokens, one new token each
        {"name": "attention_batch64", "op": "cache_attention", "S": 64, "L": 8192, "new": 1, "q_heads": 32, "heads": 8,
         "dim": 128, "page": 64, "window": 0, "sinks": 0, "dtype": "bf16"},
        # sixteen conversations with four drafted tokens each, a window of 4096 and four first tokens, in 32 bits
        {"name": "attention_window_drafts", "op": "cache_attention", "S": 16, "L": 20000, "new": 4, "q_heads": 24, "heads": 8,
         "dim": 64, "page": 32, "window": 4096, "sinks": 4, "dtype": "fp32"},
        # pieces of four prompts, each behind what its sequence holds
        {"name": "attention_prompt", "op": "cache_attention", "S": 4, "L": 6000, "new": 1024, "q_heads": 32, "heads": 8,
         "dim": 128, "page": 64, "window": 0, "sinks": 0, "dtype": "bf16"},
    ]


def _power(e):
    """2^e for whole e between -126 and 127, exactly (a pow may be off in its last bit, which moves ties)."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _log(rng, lo, hi):
    return int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))


def draw(rng):
    op = rng.choice(("qk_norm_rope", "qk_norm_rope_backward", "cache_write", "cache_read", "cache_attention",
                     "cache_attention", "cache_attention"))
    dim, heads = rng.choice((64, 64, 80, 96, 128, 128, 128, 192, 256)), rng.choice((1, 2, 3, 4, 8, 8))
    case = {"op": op, "heads": heads, "dim": dim, "dtype": rng.choice(("fp32", "fp16", "bf16", "bf16"))}
    group = rng.choice((1, 1, 2, 3, 4, 4, 7, 8, 16))
    row = heads * dim
    if op.startswith("qk"):
        case |= {"q_heads": heads * group, "T": _log(rng, 1, min(8192, (8192 * 40 * 128) // (2 * row * (group + 1)))),
                 "rotary": rng.choice((dim, dim, dim // 2)), "interleaved": rng.random() < 0.4, "norm": rng.random() < 0.8,
                 "far": _log(rng, 1000, 1000000)}
        return case
    case |= {"page": rng.choice((16, 16, 32, 64, 128)), "S": _log(rng, 1, 64)}
    if op != "cache_attention":
        case["L"] = _log(rng, 16, max(16, min(16000, (1 << 25) // (row * case["S"]))))
        case["new"] = 1 if rng.random() < 0.3 else _log(rng, 1, case["L"])
        return case
    case |= {"q_heads": heads * group, "window": 0, "sinks": 0}
    if rng.random() < 0.4:
        case |= {"window": _log(rng, 16, 8192), "sinks": rng.choice((0, 1, 4, 16, 100))}
    if rng.random() < 0.6:       # single tokens and drafts
        case["new"] = rng.choice((1, 1, 1, 2, 4, 5))
        case["L"] = _log(rng, 16, max(16, min(32768, (64 * 8192 * 256) // (row * case["S"]))))
    else:                        # prompts and pieces of them
        case["S"] = rng.choice((1, 1, 2, 3, 4))
        case["L"] = _log(rng, 64, 6000)
        case["new"] = _log(rng, 16, min(case["L"], max(16, (4 * 1024 * 6000 * 32 * 32) // (case["S"] * case["L"] * row * group))))
    return case


# ---------------------------------------------------------------- the inputs
def _lengths(case):
    """Tokens and new tokens of each sequence: spread between a quarter of L and L."""
    part = [1.0 if i == 0 else 0.25 + 0.75 * ((0.618034 * (i + 1)) % 1.0) for i in range(case["S"])]
    lens = [max(1, round(p * case["L"])) for p in part]
    new = [case["new"] if case["new"] <= 8 else max(1, round(p * case["new"])) for p in part]
    return lens, [min(a, b) for a, b in zip(lens, new)]


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dtype, H, D = TYPES[case["dtype"]], case["heads"], case["dim"]

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    def whole(values):
        return torch.tensor(values, dtype=torch.int32, device="cuda")

    state = {"case": case, "dtype": dtype}
    if case["op"].startswith("qk"):
        T, Hq, R = case["T"], case["q_heads"], case["rotary"]
        # the stacked projection's row: queries, keys, values; some features far larger than the rest
        x = normal(T, (Hq + 2 * H) * D) * torch.where(torch.rand((Hq + 2 * H) * D, generator=gen, device="cuda") < 0.01, 8.0, 1.0)
        state |= {"x": x.to(dtype), "freqs": 10000.0 ** (-torch.arange(0, R, 2, device="cuda", dtype=torch.float64) / R),
                  "positions": torch.randint(0, case["far"], (T,), generator=gen, device="cuda", dtype=torch.int32),
                  "q_weight": None, "k_weight": None}
        if case["norm"]:
            state |= {"q_weight": 1.0 + 0.3 * normal(D), "k_weight": 1.0 + 0.3 * normal(D)}
        if case["op"].endswith("backward"):
            state |= {"dq": (0.05 * normal(T, Hq, D)).to(dtype), "dk": (0.05 * normal(T, H, D)).to(dtype)}
        return state

    lens, new = _lengths(case)
    S, page = case["S"], case["page"]
    each = [-(-n // page) for n in lens]
    pages, wide = sum(each) + 3, max(each)
    order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    first = [sum(each[:i]) for i in range(S)]
    place = torch.arange(wide, device="cuda")[None, :]
    used = place < whole(each)[:, None]
    table = torch.where(used, order[torch.clamp(whole(first)[:, None] + place, max=pages - 1)], 0)
    starts = [sum(new[:i]) for i in range(S + 1)]
    T = starts[-1]
    shape = (pages, H, page // 16, D // 16, 16, 16)

    def held():      # what earlier writes left: values up to about 100 steps
        return torch.clamp(torch.round(33.0 * torch.randn(shape, generator=gen, device="cuda", dtype=torch.float16)),
                           -127, 127).to(torch.int8)

    def steps():     # and their powers of two, which differ a little from block to block
        return _power(torch.randint(-6, -4, shape[:3], generator=gen, device="cuda"))

    state |= {"k_cache": held(), "v_cache": held(), "k_scale": steps(), "v_scale": steps(), "table": table.contiguous(),
              "starts": whole(starts), "lens": whole(lens), "T": T, "most": max(new), "longest": max(lens),
              "all_starts": whole([sum(lens[:i]) for i in range(S + 1)]), "all_T": sum(lens)}
    if case["op"] == "cache_write":
        # keys and values as slices of one projection's rows, tokens of different sizes
        kv = (normal(T, 2 * H * D) * (0.4 + 1.2 * torch.rand((T, 1), generator=gen, device="cuda"))).to(dtype)
        state |= {"k": kv[:, :H * D].view(T, H, D), "v": kv[:, H * D:].view(T, H, D)}
    if case["op"] == "cache_attention":
        state["q"] = (1.5 * normal(T, case["q_heads"], D)).to(dtype)
    return state


# ---------------------------------------------------------------- plain forms
def _turn(x, cos, sin, interleaved):
    """The first 2 n features of each head turned by n angles; cos, sin [T, 1, n]."""
    n = cos.shape[-1]
    a, b = (x[..., 0:2 * n:2], x[..., 1:2 * n:2]) if interleaved else (x[..., :n], x[..., n:2 * n])
    a, b = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack((a, b), -1).flatten(-2) if interleaved else torch.cat((a, b), -1)
    return torch.cat((turned, x[..., 2 * n:]), -1)


def _plain_rope(st):
    case, dtype = st["case"], st["dtype"]
    T, D, Hq, H = case["T"], case["dim"], case["q_heads"], case["heads"]
    angle = (st["positions"].double()[:, None] * st["freqs"])[:, None, :]
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    x = st["x"][:, :(Hq + H) * D].float().view(T, Hq + H, D)
    back = case["op"].endswith("backward")
    if case["norm"]:
        w = torch.cat((st["q_weight"].expand(Hq, D), st["k_weight"].expand(H, D)))
        r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
        xr = x * r
    if not back:
        z = _turn(xr * w if case["norm"] else x, cos, sin, case["interleaved"]).to(dtype)
        return {"q": z[:, :Hq].contiguous(), "k": z[:, Hq:].contiguous()}
    dy = _turn(torch.cat((st["dq"], st["dk"]), 1).float(), cos, -sin, case["interleaved"])
    if not case["norm"]:
        return {"dx": dy.to(dtype).view(T, -1)}
    dw = (dy * xr).sum(0)
    g = dy * w
    dx = r * (g - xr * (g * xr).mean(-1, keepdim=True))
    return {"dx": dx.to(dtype).view(T, -1), "dq_weight": dw[:Hq].sum(0), "dk_weight": dw[Hq:].sum(0)}


def _token_places(st, starts, lens, T):
    """Sequence and position of each of T tokens: the last ones of each sequence."""
    t = torch.arange(T, device="cuda")
    s = torch.searchsorted(starts[1:].long(), t, right=True)
    return s, t - starts[s + 1] + lens[s]


def _plain_read(st, starts, T, dtype):
    """Keys and values of the tokens that starts asks for, [T, heads, dim]."""
    page = st["case"]["page"]
    s, at = _token_places(st, starts, st["lens"], T)
    p, b, i = st["table"][s, at // page].long(), (at % page) // 16, at % 16
    k = st["k_cache"][p, :, b, :, i].flatten(2).float() * st["k_scale"][p, :, b][..., None]
    v = st["v_cache"][p, :, b, :, :, i].flatten(2).float() * st["v_scale"][p, :, b][..., None]
    return k.to(dtype), v.to(dtype)


def _least_scale(top):
    m, e = torch.frexp(top)
    return _power(torch.where(top > 0, torch.clamp(e - 7 + (m > 127 / 128), min=-126), -126))


def _plain_write_one(st, x, cache, scale, tokens_last):
    """New tokens x [T, heads, dim] into the blocks that they touch."""
    case, S, page, H, D = st["case"], st["case"]["S"], st["case"]["page"], st["case"]["heads"], st["case"]["dim"]
    new = st["starts"][1:] - st["starts"][:-1]
    begin = st["lens"] - new                                            # tokens that are there
    n = (st["most"] + 14) // 16 + 1                                     # blocks that a sequence may touch
    block = begin[:, None] // 16 + torch.arange(n, device="cuda")       # [S, n]
    at = block[..., None] * 16 + torch.arange(16, device="cuda")        # [S, n, 16] positions
    there, fresh = at < begin[:, None, None], (at >= begin[:, None, None]) & (at < st["lens"][:, None, None])
    touched = fresh.any(-1)
    row = torch.clamp(st["starts"][:-1, None, None] + at - begin[:, None, None], 0, st["T"] - 1)
    values = torch.where(fresh[..., None, None], x[row].float(), 0.0)   # [S, n, 16, heads, dim]
    p = st["table"][torch.arange(S, device="cuda")[:, None], torch.clamp(block * 16 // page, max=st["table"].shape[1] - 1)]
    p, b = p.long(), block % (page // 16)
    old_scale = torch.where(there.any(-1)[..., None], scale[p, :, b], 0.0)                  # [S, n, heads]
    both = torch.maximum(old_scale, _least_scale(values.abs().amax((2, 4))))
    old = cache[p, :, b].float()                                        # [S, n, heads, dim / 16, 16, 16]
    old = (old.permute(0, 1, 5, 2, 3, 4) if tokens_last else old.permute(0, 1, 4, 2, 3, 5)).reshape(S, n, 16, H, D)
    old = torch.round(old * (old_scale / both)[:, :, None, :, None])
    q = torch.where(fresh[..., None, None], torch.round(values / both[:, :, None, :, None]), old)
    q = q.view(S, n, 16, H, D // 16, 16)
    q = (q.permute(0, 1, 3, 4, 5, 2) if tokens_last else q.permute(0, 1, 3, 4, 2, 5)).to(torch.int8)
    # (a sequence's first block is always touched: the places of untouched ones write it again)
    row, take = torch.arange(S, device="cuda")[:, None], torch.where(touched, torch.arange(n, device="cuda"), 0)
    p, b = p[row, take], b[row, take]
    cache[p, :, b] = q[row, take]
    scale[p, :, b] = both[row, take]


def _plain_attention(st):
    case, dtype = st["case"], st["dtype"]
    S, H, Hq, D, page = case["S"], case["heads"], case["q_heads"], case["dim"], case["page"]
    n, L, T = st["most"], st["table"].shape[1] * page, st["T"]
    p = st["table"].long()                                              # [S, pages of a sequence]
    k = st["k_cache"][p].float() * st["k_scale"][p][..., None, None, None]
    k = k.permute(0, 2, 1, 3, 5, 4, 6).reshape(S, H, L, D)
    v = st["v_cache"][p].float() * st["v_scale"][p][..., None, None, None]
    v = v.permute(0, 2, 1, 3, 6, 4, 5).reshape(S, H, L, D)
    new = st["starts"][1:] - st["starts"][:-1]
    j = torch.arange(n, device="cuda")
    row = torch.clamp(st["starts"][:-1, None] + j, max=T - 1)
    q = st["q"][row].float().view(S, n, H, Hq // H, D).permute(0, 2, 3, 1, 4).reshape(S, H, Hq // H * n, D)
    score = ((q * D ** -0.5) @ k.transpose(2, 3)).view(S, H, Hq // H, n, L)
    at = (st["lens"] - new)[:, None] + j                                # [S, n]
    key = torch.arange(L, device="cuda")
    seen = key <= at[..., None]
    if case["window"]:
        seen = seen & ((at[..., None] - key < case["window"]) | (key < case["sinks"]))
    score = torch.where(seen[:, None, None], score, -math.inf)
    top = score.amax(-1, keepdim=True)
    e = torch.exp(score - top)
    total = e.sum(-1, keepdim=True)
    y = (e.view(S, H, -1, L) @ v).view(S, H, Hq // H, n, D) / total
    lse = (top + torch.log(total))[..., 0]
    s, at = _token_places(st, st["starts"], new, T)
    return {"y": y.permute(0, 3, 1, 2, 4).reshape(S, n, Hq, D)[s, at].to(dtype),
            "lse": lse.permute(0, 3, 1, 2).reshape(S, n, Hq)[s, at].contiguous()}


def _plain(st):
    op = st["case"]["op"]
    if op.startswith("qk"):
        return _plain_rope(st)
    if op == "cache_attention":
        return _plain_attention(st)
    if op == "cache_write":
        _plain_write_one(st, st["k"], st["k_cache"], st["k_scale"], False)
        _plain_write_one(st, st["v"], st["v_cache"], st["v_scale"], True)
        k, v = _plain_read(st, st["all_starts"], st["all_T"], st["dtype"])
        return {"k": k, "v": v, "k_scale": st["k_scale"], "v_scale": st["v_scale"]}
    k, v = _plain_read(st, st["starts"], st["T"], st["dtype"])
    return {"k": k, "v": v}


# ------------------------------------------------------------- the library's
def _library(st):
    import bit_weight_amd as bw

    case = st["case"]
    op = case["op"]
    if op == "qk_norm_rope":
        q, k = bw.qk_norm_rope(st["x"], st["positions"], st["freqs"], case["q_heads"], case["heads"], case["dim"],
                               q_weight=st["q_weight"], k_weight=st["k_weight"], eps=EPS, norm=case["norm"],
                               interleaved=case["interleaved"])
        return {"q": q, "k": k}
    if op == "qk_norm_rope_backward":
        dx, dqw, dkw = bw.qk_norm_rope_backward(st["dq"], st["dk"], st["x"], st["positions"], st["freqs"],
                                                q_weight=st["q_weight"], k_weight=st["k_weight"], eps=EPS,
                                                norm=case["norm"], interleaved=case["interleaved"])
        return {"dx": dx, "dq_weight": dqw, "dk_weight": dkw} if case["norm"] else {"dx": dx}
    cache = bw.KVCache(st["k_cache"], st["v_cache"], st["k_scale"], st["v_scale"])
    if op == "cache_attention":
        y, lse = bw.cache_attention(st["q"], cache, st["table"], st["starts"], st["lens"],
                                    window=case["window"] or None, sinks=case["sinks"], lse=True)
        return {"y": y, "lse": lse}
    if op == "cache_write":
        bw.cache_write(cache, st["k"], st["v"], st["table"], st["starts"], st["lens"])
        k, v = bw.cache_read(cache, st["table"], st["all_starts"], st["lens"], st["all_T"], dtype=st["dtype"])
        return {"k": k, "v": v, "k_scale": cache.k_scale, "v_scale": cache.v_scale}
    k, v = bw.cache_read(cache, st["table"], st["starts"], st["lens"], st["T"], dtype=st["dtype"])
    return {"k": k, "v": v}


def run(state):
    return _library(state) if own else _plain(state)


def work(case):
    wide, H, D = 4 if case["dtype"] == "fp32" else 2, case["heads"], case["dim"]
    if case["op"].startswith("qk"):
        row = (case["q_heads"] + H) * D
        if case["op"].endswith("backward"):
            return {"bytes": case["T"] * ((3 if case["norm"] else 2) * wide * row + 4) + 16 * D, "flops": 14 * case["T"] * row}
        return {"bytes": case["T"] * (2 * wide * row + 4) + 8 * D, "flops": 8 * case["T"] * row}
    lens, new = _lengths(case)
    row = 2 * H * D                      # a token's keys and values
    if case["op"] == "cache_write":      # new tokens in and quantized, then every token of the sequences read back
        return {"bytes": sum(new) * row * (wide + 1) + sum(lens) * row * (1 + wide), "flops": 2 * (sum(new) + sum(lens)) * row}
    if case["op"] == "cache_read":
        return {"bytes": sum(new) * row * (1 + wide), "flops": sum(new) * row}
    Hq, W, Z = case["q_heads"], case["window"], case["sinks"]
    pairs = held = 0
    for a, b in zip(lens, new):
        first = a - b                    # the first query's position; what the window of any query holds is read once
        seen = [p + 1 if not W else min(p + 1, W) + max(0, min(Z, p + 1 - W)) for p in range(first, a)]
        pairs += sum(seen)
        held += a if not W else min(a, W + b - 1) + max(0, min(Z, first + 1 - W))
    return {"bytes": 2 * wide * sum(new) * Hq * D + held * row + 4 * sum(new) * Hq, "flops": 4 * D * Hq * pairs}


# ------------------------------------------------- the definition in 64 bits
def _rotation(x, angle, interleaved):
    """Complex numbers made of the turning features, times e^(i angle)."""
    n = angle.shape[-1]
    head, rest = x[..., :2 * n], x[..., 2 * n:]
    pair = head.unflatten(-1, (n, 2)) if interleaved else head.unflatten(-1, (2, n)).transpose(-1, -2)
    z = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * torch.polar(torch.ones_like(angle), angle))
    return torch.cat(((z if interleaved else z.transpose(-1, -2)).flatten(-2), rest), -1)


def _exact_rope(st):
    case = st["case"]
    back = case["op"].endswith("backward")
    T, D, Hq, H = case["T"], case["dim"], case["q_heads"], case["heads"]
    angle = torch.outer(st["positions"].double(), st["freqs"])[:, None]
    x = st["x"][:, :(Hq + H) * D].double().requires_grad_(back)
    found, weights = [], []
    for part, w in ((x[:, :Hq * D].unflatten(1, (Hq, D)), st["q_weight"]), (x[:, Hq * D:].unflatten(1, (H, D)), st["k_weight"])):
        if case["norm"]:
            weights.append(w.double().requires_grad_(back))
            part = part / torch.sqrt(part.square().mean(2, keepdim=True) + EPS) * weights[-1]
        found.append(_rotation(part, angle, case["interleaved"]))
    if not back:
        return {"q": found[0], "k": found[1]}
    grads = torch.autograd.grad(found, [x, *weights], [st["dq"].double(), st["dk"].double()])
    return dict(zip(("dx", "dq_weight", "dk_weight"), grads))


def _exact_tokens(st, which, sequence, lens):
    """All keys or values of one sequence, [tokens, heads, dim]."""
    page = st["case"]["page"]
    blocks = torch.arange(-(-lens // 16), device="cuda")
    p = st["table"][sequence].long()[blocks * 16 // page]
    b = blocks % (page // 16)
    q = st[which + "_cache"][p, :, b].double() * st[which + "_scale"][p, :, b].double()[..., None, None, None]
    q = q.movedim(3 if which == "k" else 4, 1)       # [blocks, 16 tokens, heads, dim / 16, 16]
    return q.flatten(3).flatten(0, 1)[:lens]


def _exact_write(st, which, lens, new, starts):
    """Every token after the write, sequence by sequence, [all tokens, heads, dim], and the scales."""
    x, page, scale, out = st[which].double(), st["case"]["page"], st[which + "_scale"].clone(), []
    table = st["table"].tolist()
    for i, (a, b) in enumerate(zip(lens, new)):
        first = a - b
        held = _exact_tokens(st, which, i, a)
        lo = first // 16
        parts = -(-a // 16) - lo
        at = torch.arange(lo * 16, (lo + parts) * 16, device="cuda")
        fresh = (at >= first) & (at < a)
        values = torch.zeros((parts * 16, *x.shape[1:]), device="cuda", dtype=torch.float64)
        values[fresh] = x[starts[i]:starts[i] + b]
        top = values.unflatten(0, (parts, 16)).abs().amax((1, 3))
        e = torch.clamp(torch.ceil(torch.log2(torch.clamp(top / 127, min=2.0 ** -126))).int(), -124, 126)
        e = torch.where(127 * _power(e - 1).double() >= top, e - 1, e)
        unit = _power(torch.where(127 * _power(e).double() < top, e + 1, e)).double()
        block = torch.arange(lo, lo + parts, device="cuda")
        p = torch.tensor(table[i], device="cuda")[block * 16 // page]
        if first % 16:
            unit[0] = torch.maximum(unit[0], scale[p[0], :, block[0] % (page // 16)].double())
        scale[p, :, block % (page // 16)] = unit.float()
        each = unit.repeat_interleave(16, 0)[..., None]
        whole = torch.where(fresh[:, None, None], values, 0.0)
        old = min(first - lo * 16, 16)
        whole[:old] = held[lo * 16:first]
        out.append(torch.cat((held[:lo * 16], (torch.round(whole / each) * each)[:a - lo * 16])))
    return torch.cat(out), scale


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op.startswith("qk"):
        return _exact_rope(st)
    lens, new = _lengths(case)
    starts = st["starts"].tolist()
    if op == "cache_write":
        k, k_scale = _exact_write(st, "k", lens, new, starts)
        v, v_scale = _exact_write(st, "v", lens, new, starts)
        return {"k": k, "v": v, "k_scale": k_scale, "v_scale": v_scale}
    if op == "cache_read":
        return {w: torch.cat([_exact_tokens(st, w, i, a)[a - b:] for i, (a, b) in enumerate(zip(lens, new))]) for w in "kv"}
    ys, ls = [], []
    for i, (a, b) in enumerate(zip(lens, new)):
        k, v = _exact_tokens(st, "k", i, a), _exact_tokens(st, "v", i, a)
        q = st["q"][starts[i]:starts[i] + b].double()
        group = case["q_heads"] // case["heads"]
        distance = torch.arange(a - b, a, device="cuda")[:, None] - torch.arange(a, device="cuda")
        hidden = distance < 0
        if case["window"]:
            hidden |= (distance >= case["window"]) & (torch.arange(a, device="cuda") >= case["sinks"])
        heads = []
        for h in range(case["q_heads"]):
            s = (q[:, h] @ k[:, h // group].t() / math.sqrt(case["dim"])).masked_fill(hidden, -math.inf)
            l = torch.logsumexp(s, 1)
            heads.append((torch.exp(s - l[:, None]) @ v[:, h // group], l))
        ys.append(torch.stack([y for y, _ in heads], 1))
        ls.append(torch.stack([l for _, l in heads], 1))
    return {"y": torch.cat(ys), "lse": torch.cat(ls)}
