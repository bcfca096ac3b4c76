"""The feed-forward operators on the GPU against their 64-bit definitions
(ffn_reference.py), whose bounds count the roundings fp32 arithmetic and the
output type may add."""

import numpy as np
import pytest
import torch

import bit_weight_amd as bw
import ffn_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)


def _say(*a):
    print(*a, flush=True)


def _gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def tokens(M, K, seed):
    g = _gen(seed)
    q = torch.randint(-128, 128, (M, K), generator=g, dtype=torch.int16).to(torch.int8)
    return q, (0.5 + torch.rand(M, generator=g)) / 60


def weights(orc, N, K, seed):
    """(T, packed on the GPU, alpha) of a random 3:4-sparse ternary matrix."""
    W = torch.randn((N, K), generator=_gen(seed))
    T, alpha = orc.quantize(W.numpy())
    packed, galpha = bw.quantize_pack(W.cuda())
    alpha = torch.from_numpy(alpha) * (0.75 * K) ** -0.5
    return torch.from_numpy(T), packed, alpha


def check(name, got, want, bound):
    got = got.double().cpu()
    assert got.shape == want.shape, (name, got.shape, want.shape)
    off = (got - want).abs()
    bad = ~(off <= bound)
    worst = (off / bound.clamp(min=1e-300)).max().item()
    assert not bad.any(), f"{name}: {int(bad.sum())} of {bad.numel()} outside, worst {worst:.3g} of the bound"


# (M, N, K): one token to several tiles; N and K off the 64 x 128 tiles; K split
# and not; every path and tile shape of the product
SHAPES = [(1, 4, 16), (1, 4096, 4096), (2, 1100, 2064), (3, 68, 11008), (7, 8192, 1024), (8, 260, 272),
          (16, 1300, 1040), (17, 4096, 512), (33, 132, 4096), (64, 2052, 784), (65, 300, 8192), (100, 516, 2048),
          (129, 1028, 400), (300, 640, 1296), (260, 16644, 256), (513, 4100, 144),
          (300, 24580, 144), (513, 8196, 272), (256, 16388, 1040)]


@pytest.mark.parametrize("i,shape", list(enumerate(SHAPES)))
def test_gemm_fused(orc, i, shape):
    M, N, K = shape
    name = ref.ACTS[i % 6]
    dtype = list(ref.TYPES.values())[i % 3]
    _say(f"gemm_fused {shape} {name} {dtype} {bw.plan(M, N, K)}")
    q, s = tokens(M, K, 10 + i)
    T, packed, alpha = weights(orc, N, K, 20 + i)
    bias = torch.randn(N, generator=_gen(30 + i)) if i % 4 != 1 else None
    res = torch.randn((M, N), generator=_gen(40 + i)).to(dtype) if i % 4 != 2 else None
    y = bw.gemm_fused(q.cuda(), s.cuda(), packed, alpha.cuda(), N, K, act=name, dtype=dtype,
                      bias=None if bias is None else bias.cuda(), residual=None if res is None else res.cuda())
    torch.cuda.synchronize()
    assert y.dtype == dtype
    check("y", y, *ref.gemm_fused(q, s, T, alpha, bias, name, res, dtype))


@pytest.mark.parametrize("name", ref.ACTS)
@pytest.mark.parametrize("t", list(ref.TYPES))
@pytest.mark.parametrize("M", [3, 140])
def test_gemm_fused_every_activation_and_type(orc, name, t, M):
    N, K, dtype = 192, 272, ref.TYPES[t]
    q, s = tokens(M, K, 1)
    T, packed, alpha = weights(orc, N, K, 2)
    alpha = alpha * 3
    bias = torch.randn(N, generator=_gen(3))
    res = torch.randn((M, N), generator=_gen(4)).to(dtype)
    out = res.cuda()
    y = bw.gemm_fused(q.cuda(), s.cuda(), packed, alpha.cuda(), N, K, bias=bias.cuda(), act=name, residual=out,
                      dtype=dtype, out=out)      # in place on the residual
    torch.cuda.synchronize()
    assert y.data_ptr() == out.data_ptr()
    check("y", y, *ref.gemm_fused(q, s, T, alpha, bias, name, res, dtype))


@pytest.mark.parametrize("i,shape", list(enumerate(SHAPES)))
def test_glu(orc, i, shape):
    M, N, K = shape
    name = ref.ACTS[(i + 3) % 6]
    dtype = list(ref.TYPES.values())[(i + 1) % 3]
    _say(f"glu {shape} {name} {dtype}")
    q, s = tokens(M, K, 110 + i)
    Tg, pg, ag = weights(orc, N, K, 120 + i)
    Tu, pu, au = weights(orc, N, K, 130 + i)
    h = bw.glu(q.cuda(), s.cuda(), pg, ag.cuda(), pu, au.cuda(), N, K, act=name, dtype=dtype)
    torch.cuda.synchronize()
    assert h.dtype == dtype
    check("h", h, *ref.glu(q, s, Tg, ag, Tu, au, name, dtype))


def test_glu_cells_hold_the_largest_sums(orc):
    """Split along K with every sum at its largest magnitude and both signs:
    the shared 64-bit cells hold the two sums and the arrivals apart."""
    M, N, K = 2, 64, 65536
    block = torch.tensor([1, 1, 1, 0], dtype=torch.int8).repeat(K // 4)
    Tg = torch.stack([block if n % 2 else -block for n in range(N)])
    Tu = torch.stack([block if n % 3 else -block for n in range(N)])
    pack = [torch.from_numpy(orc.pack(t.numpy())).cuda() for t in (Tg, Tu)]
    q = torch.full((M, K), -128, dtype=torch.int8)
    q[1] = 127
    s, one = torch.full((M,), 2.0 ** -10), torch.ones(N)
    assert int(bw.lib().sherry_glu_workspace_bytes(M, N, K)) > 0
    for _ in range(2):      # the cells are zero again after each call
        h = bw.glu(q.cuda(), s.cuda(), pack[0], one.cuda(), pack[1], one.cuda(), N, K, act="none")
        torch.cuda.synchronize()
        check("h", h, *ref.glu(q, s, Tg, one, Tu, one, "none", torch.float32))


def test_rows_and_columns_around_the_output_stay(orc):
    """Outputs inside a larger buffer: nothing before or behind is written."""
    for M, N, K in [(5, 68, 272), (200, 132, 144)]:
        q, s = tokens(M, K, 5)
        Tg, pg, ag = weights(orc, N, K, 6)
        for dtype in (torch.float32, torch.bfloat16):
            buf = torch.full((M + 2, N), 7.0, dtype=dtype, device="cuda")
            bw.gemm_fused(q.cuda(), s.cuda(), pg, ag.cuda(), N, K, dtype=dtype, out=buf.view(-1)[8:8 + M * N].view(M, N))
            torch.cuda.synchronize()
            flat = buf.view(-1)
            assert bool((flat[:8] == 7).all()) and bool((flat[8 + M * N:] == 7).all())


# ---------------------------------------------------------- backward passes
# (M, N, K): token tiles of 32 to 256 (one, several, ragged), sums over 1 to
# many row tiles, split and not, columns past the last half tile
BACK = [(1, 4, 16), (1, 640, 272), (31, 68, 144), (33, 132, 1040), (64, 1100, 528), (77, 1300, 1040),
        (130, 516, 2064), (300, 1100, 528), (385, 64, 272), (520, 260, 784), (700, 2112, 336), (140, 4160, 512), (300, 12292, 272), (260, 24580, 144)]


@pytest.mark.parametrize("i,shape", list(enumerate(BACK)))
@pytest.mark.parametrize("t", list(ref.TYPES))
def test_gemm_fused_backward(orc, i, shape, t):
    M, N, K = shape
    name, dtype = ref.ACTS[(i + 2) % 6], ref.TYPES[t]
    _say(f"gemm_fused_backward {shape} {name} {dtype}")
    q, s = tokens(M, K, 210 + i)
    T, packed, alpha = weights(orc, N, K, 220 + i)
    bias = torch.randn(N, generator=_gen(230 + i)) if i % 3 else None
    dy = (torch.randn((M, N), generator=_gen(240 + i)) * 0.01).to(dtype)
    args = [v.cuda() for v in (dy, q, s)] + [packed, alpha.cuda(), N, K]
    kw = dict(bias=None if bias is None else bias.cuda(), act=name)
    got = bw.gemm_fused_backward(*args, **kw)
    torch.cuda.synchronize()
    assert got[0].dtype == dtype
    for what, v, want in zip(("dx", "dalpha", "dbias"), got, ref.gemm_fused_backward(dy, q, s, T, alpha, bias, name, dtype)):
        check(what, v, *want)
    assert all(torch.equal(u, v) for u, v in zip(got, bw.gemm_fused_backward(*args, **kw)))   # equal bits


@pytest.mark.parametrize("i,shape", list(enumerate(BACK)))
@pytest.mark.parametrize("t", list(ref.TYPES))
def test_glu_backward(orc, i, shape, t):
    M, N, K = shape
    name, dtype = ref.ACTS[(i + 3) % 6], ref.TYPES[t]
    _say(f"glu_backward {shape} {name} {dtype}")
    q, s = tokens(M, K, 310 + i)
    Tg, pg, ag = weights(orc, N, K, 320 + i)
    Tu, pu, au = weights(orc, N, K, 330 + i)
    dh = (torch.randn((M, N), generator=_gen(340 + i)) * 0.01).to(dtype)
    args = [v.cuda() for v in (dh, q, s)] + [pg, ag.cuda(), pu, au.cuda(), N, K]
    got = bw.glu_backward(*args, act=name)
    torch.cuda.synchronize()
    assert got[0].dtype == dtype
    want = ref.glu_backward(dh, q, s, Tg, ag, Tu, au, name, dtype)
    for what, v, w in zip(("dx", "dalpha_gate", "dalpha_up"), got, want):
        check(what, v, *w)
    assert all(torch.equal(u, v) for u, v in zip(got, bw.glu_backward(*args, act=name)))      # equal bits


@pytest.mark.parametrize("scale", [1e-30, 1e-12, 1.0, 1e12, 1e25])
def test_backward_gradients_of_any_size(orc, scale):
    """fp16 terms under a scale per token: gradients far outside fp16's range,
    tokens of very different sizes, a token without any gradient."""
    M, N, K = 70, 192, 272
    q, s = tokens(M, K, 1)
    T, packed, alpha = weights(orc, N, K, 2)
    dy = torch.randn((M, N), generator=_gen(3)) * scale * 10.0 ** torch.linspace(-6, 6, M)[:, None]
    dy[5] = 0
    q[9] = 0
    got = bw.gemm_fused_backward(dy.cuda(), q.cuda(), s.cuda(), packed, alpha.cuda(), N, K, act="silu")
    torch.cuda.synchronize()
    want = ref.gemm_fused_backward(dy, q, s, T, alpha, None, "silu", torch.float32)
    for what, v, w in zip(("dx", "dalpha", "dbias"), got, want):
        check(what, v, *w)
    assert bool((got[0][5] == 0).all())


def test_backward_reads_the_gradients_up_to_two_gibibytes():
    """The widest outputs, gated, in two fp16 terms: a tile of 256 tokens whose
    last term ends 2^31 bytes behind its first.  Only the last token's last 64
    outputs have a gradient, so dx is the sum over them alone (the zeros add
    without rounding); code 0 is the block (0, 1, 1, 1)."""
    M, N, K, n = 256, 1 << 20, 1024, 64
    q, s = tokens(M, K, 1)
    packed = torch.zeros(N // 64 * (K // 128) * 1280, dtype=torch.uint8, device="cuda")
    T = torch.tensor([0.0, 1.0, 1.0, 1.0]).repeat(n, K // 4)
    alpha = (0.5 + torch.rand((2, n), generator=_gen(2))) * (0.75 * K) ** -0.5
    dh = torch.randn((1, n), generator=_gen(3))
    wide = torch.zeros((2, N), device="cuda")
    wide[:, -n:] = alpha
    grad = torch.zeros((M, N), device="cuda")
    grad[-1, -n:] = dh[0]
    got = bw.glu_backward(grad, q.cuda(), s.cuda(), packed, wide[0], packed, wide[1], N, K, act="silu")
    torch.cuda.synchronize()
    want = ref.glu_backward(dh, q[-1:], s[-1:], T, alpha[0], T, alpha[1], "silu", torch.float32)
    check("dx", got[0][-1:], *want[0])
    assert not got[0][:-1].any()
    for v, w in zip(got[1:], want[1:]):
        check("dalpha", v[-n:], *w)
        assert not v[:-n].any()


def test_backward_infinite_and_nan_gradients_stay_in_their_token(orc):
    M, N, K = 40, 132, 272
    q, s = tokens(M, K, 1)
    T, packed, alpha = weights(orc, N, K, 2)
    dy = torch.randn((M, N), generator=_gen(3))
    clean = ref.gemm_fused_backward(dy, q, s, T, alpha, None, "none", torch.float32)[0]
    dy[3, 7], dy[11, 130] = float("inf"), float("nan")
    dx = bw.gemm_fused_backward(dy.cuda(), q.cuda(), s.cuda(), packed, alpha.cuda(), N, K)[0].cpu()
    keep = [m for m in range(M) if m not in (3, 11)]
    check("dx", dx[keep], clean[0][keep], clean[1][keep])
    # inf x (+-1) keeps its sign, inf x 0 and NaN are NaN
    want = torch.where(T[7] == 0, float("nan"), float("inf") * T[7].float())
    assert torch.equal(dx[3].isnan(), want.isnan()) and torch.equal(dx[3][T[7] != 0], want[T[7] != 0])
    assert bool(dx[11].isnan().all())


def test_backward_with_outputs_masked_by_their_bias(orc):
    """A bias of -inf closes an output under relu and relu2: its gradients are
    0 and the others' are as without it."""
    M, N, K = 35, 132, 272
    q, s = tokens(M, K, 1)
    T, packed, alpha = weights(orc, N, K, 2)
    bias = torch.randn(N, generator=_gen(5))
    dy = torch.randn((M, N), generator=_gen(6))
    open_ = torch.arange(N) % 5 != 2
    for name in ("relu", "relu2"):
        masked = torch.where(open_, bias, float("-inf"))
        got = bw.gemm_fused_backward(dy.cuda(), q.cuda(), s.cuda(), packed, alpha.cuda(), N, K, bias=masked.cuda(), act=name)
        torch.cuda.synchronize()
        want = ref.gemm_fused_backward(torch.where(open_, dy, 0.0), q, s, T, alpha, bias, name, torch.float32)
        for what, v, w in zip(("dx", "dalpha", "dbias"), got, want):
            check(what, v, *w)


@pytest.mark.parametrize("name", ref.ACTS[3:])
def test_backward_against_differences(orc, name):
    """dalpha and dbias against central differences of the forward in fp32:
    steps of 2^-7 leave 2^-14 / 6 times the third derivative, below 2 times
    the value's size here, and the forward's rounding over the step."""
    M, N, K = 24, 64, 272
    q, s = tokens(M, K, 1)
    T, packed, alpha = weights(orc, N, K, 2)
    bias = torch.randn(N, generator=_gen(3))
    dy = torch.randn((M, N), generator=_gen(4))
    d = [v.cuda() for v in (q, s)] + [packed]
    _, da, db = bw.gemm_fused_backward(dy.cuda(), *d, alpha.cuda(), N, K, bias=bias.cuda(), act=name)
    forward = lambda a, b: bw.gemm_fused(*d, a.cuda(), N, K, bias=b.cuda(), act=name).double().cpu()
    h = 2.0 ** -7
    fd_b = ((forward(alpha, bias + h) - forward(alpha, bias - h)) * dy).sum(0) / (2 * h)
    size = dy.abs().double().sum(0)
    tol = size * (2 * h ** 2 / 6 + 64 * ref.U * (2 + bias.abs().max().double()) * 8 / h)
    check("dbias", db, fd_b, tol)
    p = (q.double() @ T.double().t()) * s.double()[:, None]
    step = h / p.abs().max().item()
    fd_a = ((forward(alpha + step, bias) - forward(alpha - step, bias)) * dy).sum(0) / (2 * step)
    check("dalpha", da, fd_a, tol * p.abs().max())


@pytest.mark.parametrize("name", ref.ACTS[3:])
@pytest.mark.parametrize("M", [9, 70])
def test_gated_backward_against_differences(orc, name, M):
    """Along t, at 1, with h(t) = act(t g) t u (the token's scale), act(t g) u
    (alpha_gate) and act(g) t u (alpha_up): central differences of the
    forward in fp32 against the gradients.  A step of d leaves d^2 / 6 times
    the third derivative, with |act''|, |act'''| <= 1.2 at most 1.2 |u| (3 g^2
    + |g|^3), and the forward's bound over d."""
    N, K, d = 132, 272, 2.0 ** -6
    q, s = tokens(M, K, 1)
    Tg, pg, ag = weights(orc, N, K, 2)
    Tu, pu, au = weights(orc, N, K, 3)
    dh = torch.randn((M, N), generator=_gen(4))
    dx, dg, du = (t.double().cpu() for t in bw.glu_backward(
        dh.cuda(), q.cuda(), s.cuda(), pg, ag.cuda(), pu, au.cuda(), N, K, act=name))
    bounds = ref.glu_backward(dh, q, s, Tg, ag, Tu, au, name, torch.float32)

    def forward(s_, ag_, au_):
        return bw.glu(q.cuda(), s_.cuda(), pg, ag_.cuda(), pu, au_.cuda(), N, K, act=name).double().cpu()

    _, g = ref.product(q, s, Tg, ag)
    _, u = ref.product(q, s, Tu, au)
    _, err = ref.glu(q, s, Tg, ag, Tu, au, name, torch.float32)
    cut = d ** 2 / 6 * 1.2 * u.abs() * (3 * g ** 2 + g.abs() ** 3) + 1.1 * err / d + 8 * ref.U / d * (g * u).abs()
    a = dh.double().abs()
    for along, dim, mine, bound in (
            ((1, 0, 0), 1, (dx * q.double()).sum(1) * s.double(), (bounds[0][1] * q.double().abs()).sum(1) * s.double()),
            ((0, 1, 0), 0, dg * ag.double(), bounds[1][1] * ag.double()),
            ((0, 0, 1), 0, du * au.double(), bounds[2][1] * au.double())):
        up = forward(*(v * (1 + d * on) for v, on in zip((s, ag, au), along)))
        down = forward(*(v * (1 - d * on) for v, on in zip((s, ag, au), along)))
        check(str(along), mine, (dh.double() * (up - down)).sum(dim) / (2 * d), (a * cut).sum(dim) + bound)


def test_layernorm_backward_against_differences():
    """Along random directions of x, w and b: central differences of the
    definition in 64 bits.  mean and rstd are its own, rounded to fp32 (off by
    U of themselves), so that only the steps and the gradients' bounds count:
    steps of 2^-12 leave 2^-24 / 6 times the third derivative in x, which for
    spreads of 0.5 and more and directions of size one is below 2^6 of the
    terms' size."""
    M, K, h = 12, 516, 2.0 ** -12
    x, w, b = norm_inputs(M, K, torch.float32, 3)
    g = _gen(5)
    dy, vx, vw, vb = (torch.randn(sh, generator=g) for sh in ((M, K), (M, K), (K,), (K,)))
    x64 = x.double()
    mean = x64.mean(1).float()
    rstd = (x64.var(1, unbiased=False) + 1e-5).rsqrt().float()
    dx, dw, db = (t.double().cpu() for t in bw.layernorm_backward(dy.cuda(), x.cuda(), mean.cuda(), rstd.cuda(), w.cuda()))
    bounds = ref.layernorm_backward(dy, x, mean, rstd, w, torch.float32)

    def loss(t, along):      # per token
        xx, ww, bb = (p.double() + t * on * v.double() for p, v, on in zip((x, w, b), (vx, vw, vb), along))
        d = xx - xx.mean(1, keepdim=True)
        return (dy.double() * (d / torch.sqrt((d * d).mean(1, keepdim=True) + 1e-5) * ww + bb)).sum(1)

    difference = lambda along: (loss(h, along) - loss(-h, along)) / (2 * h)
    r = rstd.double()[:, None]
    xh = (x64 - mean.double()[:, None]).abs() * r
    gw = (dy.double() * w.double()).abs()
    # what rounding mean and rstd changes of dx . v: each of its three terms by
    # a few U of rstd and of |mean| rstd in xh
    terms = r * (gw + gw.mean(1, keepdim=True) + (1 + xh) * (gw * (1 + xh)).mean(1, keepdim=True))
    moved = 8 * ref.U * (1 + (mean.double().abs()[:, None] * r)) * (terms * vx.double().abs())
    check("dx", (dx * vx).sum(1), difference((1, 0, 0)),
          (bounds[0][1] * vx.abs() + moved + 2.0 ** -24 / 6 * 64 * terms * (1 + vx.double().abs())).sum(1))
    stat = 4 * ref.U * ((xh + mean.double().abs()[:, None] * r) * dy.double().abs() * vw.double().abs()).sum()
    check("dw", (dw * vw).sum(), difference((0, 1, 0)).sum(), (bounds[1][1] * vw.abs()).sum() + stat + 1e-9 * (xh * dy.abs()).sum())
    check("db", (db * vb).sum(), difference((0, 0, 1)).sum(), (bounds[2][1] * vb.abs()).sum() + 1e-9 * dy.double().abs().sum())


# ------------------------------------------------------------------ layer norm
def norm_inputs(M, K, dtype, seed):
    g = _gen(seed)
    x = torch.randn((M, K), generator=g) * (0.5 + 3 * torch.rand((M, 1), generator=g)) + torch.randn((M, 1), generator=g)
    return x.to(dtype), 1 + 0.3 * torch.randn(K, generator=g), 0.2 * torch.randn(K, generator=g)


NORMS = [(1, 4), (5, 252), (300, 2052), (700, 1032), (1500, 8200), (260, 16376), (257, 6000), (2, 512), (3, 1032), (3, 260), (9, 1020), (2, 1028), (6, 2048), (1, 4096), (33, 4100), (3, 8196), (2, 16384),
         (3, 16388), (1, 40000), (600, 64)]


@pytest.mark.parametrize("i,shape", list(enumerate(NORMS)))
@pytest.mark.parametrize("t", list(ref.TYPES))
def test_layernorm(i, shape, t):
    M, K = shape
    dtype = ref.TYPES[t]
    x, w, b = norm_inputs(M, K, dtype, i)
    if i % 3 == 1:
        w = None
    if i % 3 == 2:
        b = None
    gw, gb = (None if v is None else v.cuda() for v in (w, b))
    y, mean, rstd = bw.layernorm(x.cuda(), gw, gb, eps=1e-5, stats=True)
    torch.cuda.synchronize()
    ry, ty, rm, tm, rr, tr = ref.layernorm(x, w, b, 1e-5, dtype)
    check("y", y, ry, ty)
    check("mean", mean, rm, tm + 1e-37)
    check("rstd", rstd, rr, tr)
    buf = x.cuda()
    assert torch.equal(bw.layernorm(buf, gw, gb, eps=1e-5, out=buf), y)      # in place
    # the int8 form: a step may differ only where 64-bit arithmetic is undecided
    qv, s = bw.layernorm_quantize(x.cuda(), gw, gb, eps=1e-5)
    torch.cuda.synchronize()
    rv, rs = ref.layernorm_quantize(x, w, b, 1e-5)
    assert torch.equal(s.cpu(), rs)
    border = (rv - rv.floor() - 0.5).abs() < 1e-9
    assert bool(((qv.cpu().double() == rv.round().clamp(-127, 127)) | border).all())


@pytest.mark.parametrize("i,shape", list(enumerate(NORMS)) + [(20, (3000, 256)), (21, (1100, 1536))])
@pytest.mark.parametrize("t", list(ref.TYPES))
def test_layernorm_backward(i, shape, t):
    M, K = shape
    dtype = ref.TYPES[t]
    x, w, _ = norm_inputs(M, K, dtype, i)
    dy = torch.randn((M, K), generator=_gen(50 + i)).to(dtype)
    w = None if i % 3 == 1 else w
    _, mean, rstd = bw.layernorm(x.cuda(), eps=1e-5, stats=True)
    grads = bw.layernorm_backward(dy.cuda(), x.cuda(), mean, rstd, None if w is None else w.cuda())
    torch.cuda.synchronize()
    for name, got, want in zip(("dx", "dw", "db"), grads, ref.layernorm_backward(dy, x, mean.cpu(), rstd.cpu(), w, dtype)):
        check(name, got, *want)
    again = bw.layernorm_backward(dy.cuda(), x.cuda(), mean, rstd, None if w is None else w.cuda())
    assert all(torch.equal(p, q) for p, q in zip(grads, again))
    buf = dy.cuda()
    inplace = bw.layernorm_backward(buf, x.cuda(), mean, rstd, None if w is None else w.cuda(), out=buf)
    assert inplace[0].data_ptr() == buf.data_ptr() and all(torch.equal(p, q) for p, q in zip(inplace, grads))


@pytest.mark.parametrize("t", list(ref.TYPES))
@pytest.mark.parametrize("M,K", [(1, 4), (5, 260), (7, 1028), (9, 2052), (300, 2056), (3, 4100), (2, 8196), (2, 12300), (2, 16388)])
def test_layernorm_leaves_what_surrounds_its_output(M, K, t):
    dtype = ref.TYPES[t]
    x, w, b = norm_inputs(M, K, dtype, 9)
    x, w, b = x.cuda(), w.cuda(), b.cuda()
    pad = 1 << 16
    whole = torch.full((M * K + 2 * pad,), 7.0, dtype=dtype, device="cuda")
    out = whole[pad:pad + M * K].view(M, K)
    y, mean, rstd = bw.layernorm(x, w, b, stats=True)
    grads = bw.layernorm_backward(y, x, mean, rstd, w)
    for want, call in ((y, lambda: bw.layernorm(x, w, b, out=out)),
                       (grads[0], lambda: bw.layernorm_backward(y, x, mean, rstd, w, out=out)[0])):
        assert torch.equal(call(), want)
        assert (whole[:pad] == 7).all() and (whole[pad + M * K:] == 7).all()


def test_layernorm_rows_without_spread_and_a_far_mean():
    """Equal features (variance 0), zeros, and a mean far above the spread:
    rstd = eps^-1/2 of the first two; an all-zero token quantizes to s = 1."""
    K = 512
    x = torch.zeros((3, K))
    x[0] = 3.25
    x[2] = 1000 + torch.randn(K, generator=_gen(1))
    y, mean, rstd = bw.layernorm(x.cuda(), eps=1e-5, stats=True)
    q, s = bw.layernorm_quantize(x.cuda(), eps=1e-5)
    torch.cuda.synchronize()
    assert bool((y[:2] == 0).all()) and bool((q[:2] == 0).all()) and bool((s[:2] == 1).all())
    ry, ty, *_ = ref.layernorm(x, None, None, 1e-5, torch.float32)
    check("y", y, ry, ty)
    rv, rs = ref.layernorm_quantize(x, None, None, 1e-5)
    assert torch.equal(s.cpu(), rs) and torch.equal(q.cpu().double(), rv.round().clamp(-127, 127))


@pytest.mark.parametrize("K", [512, 4096, 8192, 16384, 16388])
@pytest.mark.parametrize("size,weight", [(1e-30, 1.0), (1e30, 1.0), (1.0, 1e-43), (1.0, 1e30), (1e-3, 1e-40)])
def test_layernorm_quantize_of_any_size(K, size, weight):
    """Values and scales far from 1, scales among the subnormal numbers (a
    rounded one may leave more than 127 steps: clamped)."""
    x, w, b = norm_inputs(6, K, torch.float32, 5)
    x, w = x * size, w * weight
    q, s = bw.layernorm_quantize(x.cuda(), w.cuda(), eps=1e-5)
    torch.cuda.synchronize()
    rv, rs = ref.layernorm_quantize(x, w, None, float(np.float32(1e-5)))
    assert torch.equal(s.cpu(), rs)
    border = (rv - rv.floor() - 0.5).abs() < 1e-9
    assert bool(((q.cpu().double() == rv.round().clamp(-127, 127)) | border).all())


def test_layernorm_nan_stays_in_its_row():
    x = torch.randn((4, 300), generator=_gen(2))
    x[1, 7] = float("nan")
    x[2, 3] = float("inf")
    y = bw.layernorm(x.cuda())
    torch.cuda.synchronize()
    assert bool(y[1].isnan().all()) and bool(y[2].isnan().any())
    ry, ty, *_ = ref.layernorm(x[[0, 3]], None, None, 1e-5, torch.float32)
    check("y", y[[0, 3]], ry, ty)


# ------------------------------------------------- the operators as they are used
class Block:
    """The feed-forward half of a decoder layer: norm, int8 tokens, gated
    block, int8 tokens, down projection added to the residual stream."""

    def __init__(self, orc, D, F, seed):
        self.D, self.F = D, F
        self.T, self.packed, self.alpha = {}, {}, {}
        for i, (name, n, k) in enumerate((("gate", F, D), ("up", F, D), ("down", D, F))):
            self.T[name], self.packed[name], alpha = weights(orc, n, k, seed + i)
            self.alpha[name] = alpha.cuda()
        g = _gen(seed + 9)
        self.w, self.b = (1 + 0.2 * torch.randn(D, generator=g)).cuda(), (0.1 * torch.randn(D, generator=g)).cuda()

    def forward(self, x):
        q, s = bw.layernorm_quantize(x, self.w, self.b)
        h = bw.glu(q, s, self.packed["gate"], self.alpha["gate"], self.packed["up"], self.alpha["up"], self.F, self.D)
        hq, hs = bw.quantize_act(h)
        y = bw.gemm_fused(hq, hs, self.packed["down"], self.alpha["down"], self.D, self.F, residual=x, dtype=x.dtype)
        return y, q, s, h, hq, hs

    def backward(self, dy, x, q, s, hq, hs):
        dh, da, db = bw.gemm_fused_backward(dy, hq, hs, self.packed["down"], self.alpha["down"], self.D, self.F)
        dxn, dg, du = bw.glu_backward(dh, q, s, self.packed["gate"], self.alpha["gate"], self.packed["up"],
                                      self.alpha["up"], self.F, self.D)
        _, mean, rstd = bw.layernorm(x, self.w, self.b, stats=True)
        dx, dw, dbias = bw.layernorm_backward(dxn, x, mean, rstd, self.w)
        return dx, da, dg, du, dw, dbias, dh, dxn


@pytest.mark.parametrize("M", [1, 5, 16, 40, 100, 200])
@pytest.mark.parametrize("t", list(ref.TYPES))
def test_feed_forward_block(orc, M, t):
    """Each step against its definition on what the step before it gave."""
    D, F, dtype = 512, 1424, ref.TYPES[t]
    blk = Block(orc, D, F, 700)
    x = (2 * torch.randn((M, D), generator=_gen(M))).to(dtype)
    y, q, s, h, hq, hs = blk.forward(x.cuda())
    torch.cuda.synchronize()
    rv, rs = ref.layernorm_quantize(x, blk.w.cpu(), blk.b.cpu(), 1e-5)
    assert torch.equal(s.cpu(), rs)
    assert bool(((q.cpu().double() == rv.round()) | ((rv - rv.floor() - 0.5).abs() < 1e-9)).all())
    a = {k: v.cpu() for k, v in blk.alpha.items()}
    check("h", h, *ref.glu(q.cpu(), s.cpu(), blk.T["gate"], a["gate"], blk.T["up"], a["up"], "silu", torch.float32))
    check("y", y, *ref.gemm_fused(hq.cpu(), hs.cpu(), blk.T["down"], a["down"], None, "none", x, dtype))
    dy = torch.randn((M, D), generator=_gen(M + 1)).to(dtype)
    dx, da, dg, du, dw, db, dh, dxn = blk.backward(dy.cuda(), x.cuda(), q, s, hq, hs)
    torch.cuda.synchronize()
    want = ref.gemm_fused_backward(dy, hq.cpu(), hs.cpu(), blk.T["down"], a["down"], None, "none", dtype)
    check("dh", dh, *want[0])
    check("dalpha", da, *want[1])
    want = ref.glu_backward(dh.cpu(), q.cpu(), s.cpu(), blk.T["gate"], a["gate"], blk.T["up"], a["up"], "silu", dtype)
    for name, v, w in zip(("dxn", "dgate", "dup"), (dxn, dg, du), want):
        check(name, v, *w)


@pytest.mark.parametrize("M", [1, 7, 200])
def test_captured_block_replays(orc, M):
    """Forward and backward in one graph; replayed with new inputs, eager work
    and synchronizations between the replays."""
    blk = Block(orc, 256, 2048, 800)      # K = 2048 is split in the down projection at small M
    x = torch.randn((M, 256), generator=_gen(1)).cuda()
    dy = torch.randn((M, 256), generator=_gen(2)).cuda()

    def work():
        y, q, s, h, hq, hs = blk.forward(x)
        return (y, h, *blk.backward(dy, x, q, s, hq, hs))

    work()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = work()
    for i in range(4):
        x.copy_(torch.randn((M, 256), generator=_gen(10 + i)))
        dy.copy_(torch.randn((M, 256), generator=_gen(20 + i)))
        eager = [v.clone() for v in work()]
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(eager, held):
            assert torch.equal(a, b)


def test_two_graphs_and_eager_calls_side_by_side(orc):
    """Split-K products captured into two graphs on one stream, replayed on
    two streams at once beside eager calls on a third: each has cells of its
    own, zeroed by itself, whichever is replayed first."""
    N, K = 1024, 8192
    T, packed, alpha = weights(orc, N, K, 1)
    Tu, pu, au = weights(orc, N, K, 2)
    alpha, au = alpha.cuda(), au.cuda()
    data = [tokens(4, K, 50 + i) for i in range(3)]
    dev = [(q.cuda(), s.cuda()) for q, s in data]
    assert bw.lib().sherry_glu_workspace_bytes(4, N, K) > 0
    run = lambda i: bw.glu(*dev[i], packed, alpha, pu, au, N, K)
    want = [run(i).clone() for i in range(3)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    graphs, held = [], []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            held.append(run(i))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in range(3)]
    for order in ((1, 0), (0, 1), (1, 0)):
        for h in held:
            h.zero_()
        torch.cuda.synchronize()
        for _ in range(5):
            for i in order:
                with torch.cuda.stream(streams[i]):
                    graphs[i].replay()
            with torch.cuda.stream(streams[2]):
                eager = run(2)
        torch.cuda.synchronize()
        assert torch.equal(held[0], want[0]) and torch.equal(held[1], want[1]) and torch.equal(eager, want[2])
    check("h", want[0], *ref.glu(*data[0], T, alpha.cpu(), Tu, au.cpu(), "silu", torch.float32))


def test_calls_follow_the_current_stream(orc):
    """Inputs written on a side stream, the operators called on it."""
    blk = Block(orc, 512, 1024, 900)
    x = torch.randn((9, 512), generator=_gen(3))
    want = [v.clone() for v in blk.forward(x.cuda())]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        busy = torch.randn((4096, 4096), device="cuda")
        for _ in range(4):
            busy = busy @ busy * 1e-3
        got = blk.forward(x.cuda() + 0 * busy[:9, :512].nan_to_num(0, 0, 0))
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_refusals_of_device_tensors(orc):
    N, K = 64, 128
    q, s = (v.cuda() for v in tokens(3, K, 1))
    _, packed, alpha = weights(orc, N, K, 1)
    alpha = alpha.cuda()
    ok = dict(x=q, s_x=s, packed=packed, alpha=alpha, N=N, K=K)
    bw.gemm_fused(**ok)
    for kw in (dict(x=q.float()), dict(x=q[:, ::2]), dict(x=q.t()), dict(s_x=s[:2]), dict(s_x=s.double()),
               dict(packed=packed[:-1]), dict(packed=packed.cpu()), dict(alpha=alpha[:32]), dict(alpha=alpha.half()),
               dict(bias=alpha[:32]), dict(bias=alpha.cpu()), dict(residual=torch.zeros(3, N, device="cuda").half()),
               dict(residual=torch.zeros(N, 3, device="cuda").t()), dict(residual=torch.zeros(2, N, device="cuda")),
               dict(out=torch.zeros(3, N, device="cuda", dtype=torch.bfloat16)), dict(out=torch.zeros(3, N)),
               dict(dtype=torch.int8), dict(workspace=torch.zeros(8, device="cuda")), dict(N=128), dict(K=256)):
        with pytest.raises(RuntimeError):
            bw.gemm_fused(**(ok | kw))
    with pytest.raises(ValueError):
        bw.gemm_fused(**ok, act="swish")
    with pytest.raises(bw.SherryError):      # an output that is not 16-byte aligned
        bw.gemm_fused(**ok, out=torch.zeros(3 * N + 1, device="cuda")[1:].view(3, N))
    with pytest.raises(bw.SherryError):
        bw.gemm_fused(q[:0], s[:0], packed, alpha, N, K)
    with pytest.raises(bw.SherryError):      # a workspace of the caller's that is too small
        T2, p2, a2 = weights(orc, 1024, 8192, 2)
        bw.gemm_fused(*(v.cuda() for v in tokens(2, 8192, 2)), p2, a2.cuda(), 1024, 8192,
                      workspace=torch.zeros(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(RuntimeError):
        bw.glu_backward(torch.zeros(3, N, device="cuda", dtype=torch.float64), q, s, packed, alpha, packed, alpha, N, K)
    x = torch.zeros((2, 130), device="cuda")
    with pytest.raises(bw.SherryError):      # K % 4
        bw.layernorm(x)
    with pytest.raises(bw.SherryError):
        bw.layernorm(x[:, :128].contiguous(), eps=0.0)
    with pytest.raises(RuntimeError):
        bw.layernorm(x[:, :128])
    torch.cuda.synchronize()
