"""The attention operators' definitions in 64 bits on the CPU, each with a bound
on its error that counts roundings (U: half a step of fp32, relative)."""

import math

import torch

TYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
U = 2.0 ** -24


def rounding(z, dtype):
    """Half a step of dtype at z: eps / 2 relative, and among subnormal numbers,
    whose step is tiny * eps whatever their size, half of that (fp16: 2^-25)."""
    info = torch.finfo(dtype)
    return torch.clamp(z.abs() * (info.eps / 2), min=info.tiny * info.eps / 2)


def gen(seed):
    return torch.Generator().manual_seed(seed)


# ------------------------------------------------------------ norm and rotation
def turn(x, positions, freqs, interleaved, back=False):
    """x [T, H, D] in 64 bits, its first 2 len(freqs) features turned."""
    n = freqs.numel()
    t = positions.double()[:, None, None] * freqs.double() * (-1 if back else 1)
    c, s = torch.cos(t), torch.sin(t)
    z = x.clone()
    ia, ib = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if interleaved else (slice(0, n), slice(n, 2 * n))
    z[..., ia] = x[..., ia] * c - x[..., ib] * s
    z[..., ib] = x[..., ib] * c + x[..., ia] * s
    return z


def both(x, n, interleaved):
    """|a| + |b| of each feature's pair, |x| of those that do not turn."""
    x = x.abs()
    s = x.clone()
    ia, ib = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if interleaved else (slice(0, n), slice(n, 2 * n))
    s[..., ia] = s[..., ib] = x[..., ia] + x[..., ib]
    return s


def inverse_rms(x, eps):
    return 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)


def norm_rope(x, positions, freqs, w, eps, norm, interleaved, dtype):
    """x [T, H, D] -> z and its bound.  r: 13 roundings under the root and 2 of
    its own, 9 U; y: 2 more; cosines: the turn's fraction to fp32 and 2 of the
    function, 4 U; two for the sum of products: 17, and the last to dtype."""
    x = x.double()
    y = x * inverse_rms(x, eps) * (1 if w is None else w.double()) if norm else x
    z = turn(y, positions, freqs, interleaved)
    return z, 20 * U * both(y, freqs.numel(), interleaved) + rounding(z, dtype)


def norm_rope_backward(dz, x, positions, freqs, w, eps, norm, interleaved, dtype):
    """-> (dx, bound), (dw, bound) of one kind of heads (dw None without the norm)."""
    dz, x = dz.double(), x.double()
    dy = turn(dz, positions, freqs, interleaved, back=True)
    ey = 6 * U * both(dz, freqs.numel(), interleaved)
    if not norm:
        return (dy, ey + rounding(dy, dtype)), None
    w = torch.ones(x.shape[-1]).double() if w is None else w.double()
    r = inverse_rms(x, eps)
    xr, g, eg = x * r, dy * w, ey * w.abs() + U * (dy * w).abs()
    mean = (g * xr).mean(-1, keepdim=True)
    dx = r * (g - xr * mean)
    e = r * (eg + xr.abs() * ((eg * xr.abs()).mean(-1, keepdim=True) + 30 * U * (g * xr).abs().mean(-1, keepdim=True))
             + 14 * U * (g.abs() + xr.abs() * mean.abs()))
    dw = (dy * xr).sum((0, 1))
    n = x.shape[0] * x.shape[1]
    ew = (ey * xr.abs() + (12 + n) * U * (dy * xr).abs()).sum((0, 1))
    return (dx, e + rounding(dx, dtype)), (dw, ew + 1e-45)


# --------------------------------------------------------------------- the cache
def least_scale(top):
    """The least 2^e, e >= -126, with top <= 127 2^e."""
    e = -126
    while 127 * 2.0 ** e < top:
        e += 1
    return 2.0 ** e


class Blocks:
    """One sequence's keys or values, block by block: what the cache should hold."""

    def __init__(self, H, D):
        self.H, self.D, self.blocks = H, D, {}      # (block, head) -> [scale, values of its tokens]

    def write(self, first, x):
        """Tokens x [n, H, D] (64 bits) at positions first, first + 1, ..."""
        n = x.shape[0]
        for b in range(max(first, 0) // 16, (first + n + 15) // 16):
            lo, hi = max(first, 16 * b, 0), min(first + n, 16 * b + 16)
            if lo >= hi:
                continue
            for h in range(self.H):
                new = x[lo - first:hi - first, h]
                scale = least_scale(new.abs().max().item()) if torch.isfinite(new).all() else math.nan
                q = torch.zeros(16, self.D, dtype=torch.float64)
                if lo > 16 * b:
                    old_scale, old = self.blocks.get((b, h), (0.0, q))
                    if math.isnan(old_scale) or old_scale > scale:
                        scale = old_scale
                    if scale == scale:
                        q[:lo - 16 * b] = torch.round(old[:lo - 16 * b] * (old_scale / scale))
                if scale == scale:
                    q[lo - 16 * b:hi - 16 * b] = torch.round(new / scale)
                self.blocks[b, h] = (scale, q)

    def read(self, n):
        out = torch.zeros(n, self.H, self.D, dtype=torch.float64)
        for (b, h), (scale, q) in self.blocks.items():
            m = min(16, n - 16 * b)
            if m > 0:
                out[16 * b:16 * b + m, h] = q[:m] * scale
        return out


# --------------------------------------------------------------------- attention
def attention(q, k, v, scale, window, sinks, dtype, units):
    """Queries q [n, Hq, D] at the end of tokens k, v [L, H, D] -> (y, bound), (lse,
    bound).  units [L, H]: the values' scales.  Scores: D products with fp32
    sums, twice U each; q to 22 bits where it is fp32.  Weights: the rounding to
    fp16, or to two terms and 2^-32 of the largest times the largest scale; what
    the score's error and fp32's exponent (2 U (|t| + |m|)) make of them; the sum's."""
    n, Hq, D = q.shape
    L, H, _ = k.shape
    q, k, v = q.double(), k.double(), v.double()
    two = dtype == torch.float32
    group = Hq // H
    y, ey = torch.zeros(n, Hq, D).double(), torch.zeros(n, Hq, D).double()
    lse, el = torch.full((n, Hq), -math.inf).double(), torch.zeros(n, Hq).double()
    for h in range(Hq):
        kh, vh, uh = k[:, h // group], v[:, h // group], units[:, h // group].double()
        for j in range(n):
            p = L - n + j
            t = torch.arange(L)
            seen = t <= p
            if window:
                seen &= (p - t < window) | (t < sinks)
            if not seen.any():
                continue
            s = scale * (kh[seen] @ q[j, h])
            size = abs(scale) * (kh[seen].abs() @ q[j, h].abs())
            es = (2 * D + 6) * U * size + 2.0 ** -22 * size * two
            m = s.max()
            e = torch.exp(s - m)
            w = e / e.sum()
            lse[j, h] = m + torch.log(e.sum())
            y[j, h] = w @ vh[seen]
            count = int(seen.sum())
            ew = es + 2 * U * (s.abs() + m.abs()) + 4 * U        # relative, of each weight
            total = float((w * ew).sum()) + 2 * count * U
            el[j, h] = total + 4 * U * (lse[j, h].abs() + 1)
            av = vh[seen].abs()
            term = 2.0 ** -22 if two else 2.0 ** -11
            ey[j, h] = (w * ew) @ av + (term + total + 2 * (count + 16) * U) * (w @ av) \
                + count * 2.0 ** -32 * 256 / e.sum() * 127 * uh[seen].max()
    return (y, ey + rounding(y, dtype)), (lse, el)
