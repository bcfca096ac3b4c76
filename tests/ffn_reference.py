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


def input_gradient(parts, top, dtype):
    """dx = sum over parts of c @ T and its bound; parts are (c, error of c, T)
    with c = dz alpha, top [M] bounds |c| as the library does.  A power of two
    takes top to (2^14, 2^15]; there one fp16 term is off by 2^-11 of c (two:
    2^-22) or half a subnormal step, 2^-25, which is 2^-39 of top.  n terms
    added in fp32 in any order take n roundings of at most sum |c|."""
    two = dtype != torch.bfloat16
    term = 2.0 ** -22 if two else 2.0 ** -11
    dx = sum(c @ T.double() for c, _, T in parts)
    n = sum(T.shape[0] for _, _, T in parts) * (2 if two else 1)
    err = sum((e + term * c.abs() + 2.0 ** -39 * top[:, None] + (n + 4) * U * c.abs()) @ T.double().abs()
              for c, e, T in parts)
    return dx, rounded(dx, err, dtype)


def top_of(dy, q, s, alpha, alpha2, bias, name):
    """The library's bound on a token's |dz alpha|, from max|dy|, sum|q| s and
    the largest scales; |act'| <= 1.25, or 2 |z| for relu2."""
    total = q.double().abs().sum(1) * s.double()
    a = alpha.abs().max().double()
    pre = total * a + (0 if bias is None else bias.abs().max().double())
    top = dy.double().abs().amax(1) * (2 * pre if name == "relu2" else 1.25) * a
    return top if alpha2 is None else top * total * alpha2.abs().max().double()


def gemm_fused_backward(dy, q, s, T, alpha, bias, name, dtype):
    """((dx, bound), (dalpha, bound), (dbias, bound))."""
    p, z = product(q, s, T, alpha)
    ez = 3 * U * z.abs()
    if bias is not None:
        z = z + bias.double()
        ez = ez + U * z.abs()
    dy = dy.double()
    dz = dy * slope(z, name)
    edz = dy.abs() * slope_error(z, ez, name) + U * dz.abs()
    a = alpha.double()
    top = top_of(dy, q, s, alpha, None, bias, name)
    dx = input_gradient([(dz * a, edz * a.abs() + 2 * U * (dz * a).abs(), T)], top, dtype)
    M = dy.shape[0]
    da = (dz * p).sum(0)
    eda = (edz * p.abs()).sum(0) + (M + 6) * U * (dz * p).abs().sum(0)
    db = dz.sum(0)
    edb = edz.sum(0) + (M + 2) * U * dz.abs().sum(0)
    return dx, (da, 1.01 * eda + 1e-37), (db, 1.01 * edb + 1e-37)


def glu_backward(dh, q, s, Tg, ag, Tu, au, name, dtype):
    """((dx, bound), (dalpha_gate, bound), (dalpha_up, bound))."""
    pg, g = product(q, s, Tg, ag)
    pu, u = product(q, s, Tu, au)
    dh, ag, au = dh.double(), ag.double(), au.double()
    eg, eu = 3 * U * g.abs(), 3 * U * u.abs()
    sl, a = slope(g, name), act(g, name)
    dg, du = dh * u * sl, dh * a
    edg = (dh * u).abs() * slope_error(g, eg, name) + 6 * U * dg.abs()
    edu = dh.abs() * act_error(g, eg, name) + U * du.abs()
    top = top_of(dh, q, s, ag, au, None, name)
    dx = input_gradient([(dg * ag, edg * ag.abs() + 2 * U * (dg * ag).abs(), Tg),
                         (du * au, edu * au.abs() + 2 * U * (du * au).abs(), Tu)], top, dtype)
    M = dh.shape[0]
    found = [dx]
    for d, e, p in ((dg, edg, pg), (du, edu, pu)):
        err = (e * p.abs()).sum(0) + (M + 6) * U * (d * p).abs().sum(0)
        found.append(((d * p).sum(0), 1.01 * err + 1e-37))
    return found


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
