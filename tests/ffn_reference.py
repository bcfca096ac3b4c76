"""Plain 64-bit forms of the feed-forward operators and bounds on what fp32
arithmetic may add to them.

Bounds count roundings: u = 2^-24 is the most one fp32 operation is off by,
relative to its result, and half of torch.finfo(t).eps the most the final
rounding to t is.  Library functions (exp, erf, tanh) are taken to be within
4 u.  Every bound is first order with a factor of 1.01 for the rest.
"""

import math

import torch

U = 2.0 ** -24
ACTS = ("none", "relu", "relu2", "silu", "gelu", "gelu_tanh")
TYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
C = math.sqrt(2 / math.pi)


def act(z, name):
    if name == "relu":
        return z.clamp(min=0)
    if name == "relu2":
        return z.clamp(min=0) ** 2
    if name == "silu":
        return z * torch.sigmoid(z)
    if name == "gelu":
        return z * 0.5 * torch.erfc(-z / math.sqrt(2))
    if name == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(C * (z + 0.044715 * z ** 3)))
    return z


def slope(z, name):
    if name == "relu":
        return (z > 0).double()
    if name == "relu2":
        return 2 * z.clamp(min=0)
    if name == "silu":
        s = torch.sigmoid(z)
        return s + z * s * (1 - s)
    if name == "gelu":
        return 0.5 * torch.erfc(-z / math.sqrt(2)) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        t = torch.tanh(C * (z + 0.044715 * z ** 3))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * C * (1 + 3 * 0.044715 * z * z)
    return torch.ones_like(z)


def act_error(z, dz, name):
    """Bound on |act(z') - act(z)| for |z' - z| <= dz, act in fp32: none and
    relu pass dz on; relu2 doubles it times |z| and rounds once; the others
    have |slope| <= 1.13 and take at most 12 roundings of values up to |z|
    (a function's 4 u, the sums 1 + .. below 2, products; tanh's argument is
    off by 6 u of itself, and |x tanh'(x)| < 0.45)."""
    if name in ("none", "relu"):
        return dz
    if name == "relu2":
        return 2 * z.abs() * dz + dz ** 2 + U * z ** 2
    return 1.13 * dz + 12 * U * z.abs()


def slope_error(z, dz, name):
    """The same for act'.  relu's slope jumps at 0: inputs next to it are left
    to the caller.  |act''| <= 1 for the smooth ones (relu2: 2), whose
    slopes take at most 24 roundings of values up to 1 + |z| (exp(-z^2 / 2)
    is off by z^2 u more, and z^3 exp(-z^2 / 2) < 1.2)."""
    if name in ("none", "relu"):
        return torch.zeros_like(z)
    if name == "relu2":
        return 2 * dz + U * z.abs()
    return dz + 24 * U * (1 + z.abs().clamp(max=8))


def rounded(y, err, dtype):
    """The bound after the one rounding to dtype: half a step of a value that
    is itself off by err, and half a subnormal step."""
    info = torch.finfo(dtype)
    return 1.01 * (err + (y.abs() + err) * info.eps / 2) + info.smallest_normal * info.eps


def product(q, s, T, alpha):
    """(p, z) = (acc s, acc s alpha) in 64 bits, acc exact.  In fp32 p is off
    by 2 u of itself (acc to float, times s) and z by 3 u."""
    p = (q.double() @ T.double().t()) * s.double()[:, None]
    return p, p * alpha.double()


def gemm_fused(q, s, T, alpha, bias, name, residual, dtype):
    _, z = product(q, s, T, alpha)
    dz = 3 * U * z.abs()
    if bias is not None:
        z = z + bias.double()
        dz = dz + U * z.abs()
    y = act(z, name)
    err = act_error(z, dz, name)
    if residual is not None:
        y = y + residual.double()
        err = err + U * y.abs()
    return y, rounded(y, err, dtype)


def glu(q, s, Tg, ag, Tu, au, name, dtype):
    _, g = product(q, s, Tg, ag)
    _, u = product(q, s, Tu, au)
    a = act(g, name)
    h = a * u
    err = act_error(g, 3 * U * g.abs(), name) * u.abs() + 4 * U * h.abs()
    return h, rounded(h, err, dtype)


def layernorm(x, w, b, eps, dtype):
    """(y, bound, mean, its bound, rstd, its bound).  A sum over K features
    takes at most `adds` additions on its way: those of one lane (up to 64
    values, or K / 4096 x 4 in loops) and of the joins."""
    K = x.shape[1]
    x = x.double()
    adds = max(64, K // 1024) + 32
    mean = x.mean(1, keepdim=True)
    dmean = (adds + 1) * U * x.abs().mean(1, keepdim=True)
    d = x - mean
    dd = dmean + U * d.abs()
    var = (d * d).mean(1, keepdim=True)
    dvar = (adds + 3) * U * var + 2 * (d.abs() * dd).mean(1, keepdim=True) + dmean ** 2
    rstd = 1 / torch.sqrt(var + eps)
    rel = dvar / (2 * (var + eps)) + 3 * U
    w = torch.ones(K) if w is None else w
    b = torch.zeros(K) if b is None else b
    t = d * rstd * w.double()
    y = t + b.double()
    err = (dd * rstd * w.double().abs()) + t.abs() * (rel + 2 * U) + U * y.abs()
    return (y, rounded(y, err, dtype), mean[:, 0], 1.01 * dmean[:, 0], rstd[:, 0],
            1.01 * (rel * rstd)[:, 0])


def layernorm_quantize(x, w, b, eps):
    """(v / s, s): what rounds to q, and the scale, in 64 bits."""
    x = x.double()
    d = x - x.mean(1, keepdim=True)
    v = d / torch.sqrt((d * d).mean(1, keepdim=True) + eps)
    if w is not None:
        v = v * w.double()
    if b is not None:
        v = v + b.double()
    s = (v.abs().amax(1) / 127).float()
    s = torch.where(s > 0, s, torch.ones_like(s))
    return v / s.double()[:, None], s


def layernorm_backward(dy, x, mean, rstd, w, dtype):
    """((dx, bound), (dw, bound), (db, bound)); dw and db are sums over M
    tokens in some order: at most M + 2 roundings each."""
    M, K = x.shape
    adds = max(64, K // 1024) + 32
    dy, x, mean, rstd = dy.double(), x.double(), mean.double()[:, None], rstd.double()[:, None]
    w = torch.ones(K, dtype=torch.float64) if w is None else w.double()
    xh = (x - mean) * rstd
    g = dy * w
    m1, m2 = g.mean(1, keepdim=True), (g * xh).mean(1, keepdim=True)
    e1 = (adds + 2) * U * g.abs().mean(1, keepdim=True)
    e2 = (adds + 5) * U * (g * xh).abs().mean(1, keepdim=True)
    dx = rstd * (g - m1 - xh * m2)
    err = rstd * (e1 + xh.abs() * e2 + 3 * U * (g.abs() + m1.abs() + 2 * (xh * m2).abs())) + U * dx.abs()
    dw, db = (dy * xh).sum(0), dy.sum(0)
    return ((dx, rounded(dx, err, dtype)), (dw, (M + 5) * 1.01 * U * (dy * xh).abs().sum(0) + 1e-37),
            (db, (M + 2) * 1.01 * U * dy.abs().sum(0) + 1e-37))
