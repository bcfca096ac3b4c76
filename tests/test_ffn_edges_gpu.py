"""Edges of the feed-forward operators on the GPU: inputs whose sizes differ by
many powers of two, non-finite ones, and calls around autograd and graphs."""

import pytest
import torch

import bit_weight_amd as bw
import ffn_reference as ref
from test_ffn_gpu import _gen, check, tokens, weights

pytestmark = pytest.mark.gpu
LOWEST = torch.finfo(torch.float32).min


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)


def closed_by_bias(orc, name, t, closing):
    """The gradients with every fifth output closed by a bias, and what they
    are with that output's gradient 0 instead: the slope there is exactly 0
    (|p alpha| < 16, so z < -1e5)."""
    M, N, K, dtype = 35, 132, 272, ref.TYPES[t]
    q, s = tokens(M, K, 1)
    T, packed, alpha = weights(orc, N, K, 2)
    bias = torch.randn(N, generator=_gen(5))
    dy = torch.randn((M, N), generator=_gen(6)).to(dtype)
    open_ = torch.arange(N) % 5 != 2
    masked = torch.where(open_, bias, closing)
    got = bw.gemm_fused_backward(dy.cuda(), q.cuda(), s.cuda(), packed, alpha.cuda(), N, K, bias=masked.cuda(), act=name)
    torch.cuda.synchronize()
    want = ref.gemm_fused_backward(torch.where(open_, dy, 0.0), q, s, T, alpha, bias, name, dtype)
    for what, v, w in zip(("dx", "dalpha", "dbias"), got, want):
        check(what, v, *w)


@pytest.mark.parametrize("t", list(ref.TYPES))
@pytest.mark.parametrize("closing", [-1e6, -1e12, LOWEST])
@pytest.mark.parametrize("name", ["relu", "relu2"])
def test_backward_with_outputs_closed_by_a_finite_bias(orc, name, t, closing):
    closed_by_bias(orc, name, t, closing)


# dx's terms are off by 2^-11 (one fp16 term, bf16 results) or 2^-22 (two) of
# themselves and by FLOOR of the largest |dz alpha| of their token, however
# large the factors are that no gradient passes.
TERM = {torch.bfloat16: 2.0 ** -11, torch.float16: 2.0 ** -22, torch.float32: 2.0 ** -22}
FLOOR = {torch.bfloat16: 2.0 ** -16, torch.float16: 2.0 ** -24, torch.float32: 2.0 ** -24}


def dx_and_bound(parts, dtype):
    """As ffn_reference.input_gradient, with the floor from the exact terms."""
    top = torch.stack([c.abs().amax(1) for c, _, _ in parts]).amax(0)
    return ref.input_gradient(parts, top * FLOOR[dtype] * 2.0 ** 39, dtype)


def gated_terms(dh, q, s, Tg, ag, Tu, au, name):
    """[(dz alpha, its error in fp32, T)] of both matrices, as in
    ffn_reference.glu_backward."""
    _, g = ref.product(q, s, Tg, ag)
    _, u = ref.product(q, s, Tu, au)
    dh, ag, au = dh.double(), ag.double(), au.double()
    sl, a = ref.slope(g, name), ref.act(g, name)
    dg, du = dh * u * sl, dh * a
    eg = 3 * ref.U * g.abs()
    edg = (dh * u).abs() * ref.slope_error(g, eg, name) + 6 * ref.U * dg.abs()
    edu = dh.abs() * ref.act_error(g, eg, name) + ref.U * du.abs()
    if name in ("relu", "relu2"):       # (a negative gate's sign is exact, and so are its zeros)
        edg, edu = (torch.where(g < 0, 0.0, e) for e in (edg, edu))
    return [(dg * ag, edg * ag.abs() + 2 * ref.U * (dg * ag).abs(), Tg),
            (du * au, edu * au.abs() + 2 * ref.U * (du * au).abs(), Tu)]


def closed_outlier(orc, M, N, K, factor, seed):
    """A gated block whose output 7 has scales `factor` times the others' and,
    in two tokens of three, a gradient `factor` times the others', but a gate
    that is closed (negative) for every token."""
    q, s = tokens(M, K, seed)
    q = q.clamp(min=-127)
    Tg, pg, ag = weights(orc, N, K, seed + 1)
    Tu, pu, au = weights(orc, N, K, seed + 2)
    acc = q.double() @ Tg[7].double()
    q = torch.where(acc[:, None] > 0, -q, q)
    q[acc == 0] = 0
    dh = torch.randn((M, N), generator=_gen(seed + 3)) * 0.01
    dh[:, 7] *= torch.where(torch.arange(M) % 3 < 2, factor, 1.0)
    ag[7] *= factor
    au[7] *= factor
    return q, s, Tg, pg, ag, Tu, pu, au, dh


@pytest.mark.parametrize("t", list(ref.TYPES))
@pytest.mark.parametrize("factor", [2.0 ** 3, 2.0 ** 5, 2.0 ** 12])
@pytest.mark.parametrize("M,N", [(1, 132), (40, 132), (77, 1300), (140, 4160), (300, 24580)])
def test_gated_backward_beside_a_closed_outlier(orc, M, N, factor, t):
    dtype = ref.TYPES[t]
    q, s, Tg, pg, ag, Tu, pu, au, dh = closed_outlier(orc, M, N, 272, factor, 41)
    dh = dh.to(dtype)
    args = [v.cuda() for v in (dh, q, s)] + [pg, ag.cuda(), pu, au.cuda(), N, 272]
    got = bw.glu_backward(*args, act="relu2")
    torch.cuda.synchronize()
    check("dx", got[0], *dx_and_bound(gated_terms(dh, q, s, Tg, ag, Tu, au, "relu2"), dtype))
    for v, w in zip(got[1:], ref.glu_backward(dh, q, s, Tg, ag, Tu, au, "relu2", dtype)[1:]):
        check("dalpha", v, *w)
    assert all(torch.equal(u, v) for u, v in zip(got, bw.glu_backward(*args, act="relu2")))      # equal bits


@pytest.mark.parametrize("t", ["fp32", "fp16"])
@pytest.mark.parametrize("name", ["relu", "relu2"])
@pytest.mark.parametrize("factor", [1.0, 2.0 ** 4, 2.0 ** 8, 2.0 ** 15])
def test_gated_backward_keeps_the_digits_of_one_open_output(orc, name, factor, t):
    """Gradients at the closed outlier and one other output only: dx is one
    term of each matrix, so no sum's rounding hides its digits (the high and
    low parts and the two matrices' terms: 4 additions)."""
    M, N, K, dtype = 60, 132, 1040, ref.TYPES[t]
    q, s, Tg, pg, ag, Tu, pu, au, dh = closed_outlier(orc, M, N, K, factor, 51)
    dh = torch.where((torch.arange(N) == 7) | (torch.arange(N) == 20), dh, 0.0)
    if t == "fp16":
        dh = dh.clamp(-60000, 60000)
    dh = dh.to(dtype)
    got = bw.glu_backward(*[v.cuda() for v in (dh, q, s)], pg, ag.cuda(), pu, au.cuda(), N, K, act=name)[0]
    torch.cuda.synchronize()
    parts = gated_terms(dh, q, s, Tg, ag, Tu, au, name)
    dx = sum(c @ T.double() for c, _, T in parts)
    top = torch.stack([c.abs().amax(1) for c, _, _ in parts]).amax(0)
    size = sum(c.abs().sum(1) for c, _, _ in parts)
    err = sum(e.sum(1) for _, e, _ in parts) + (TERM[dtype] + 5 * ref.U) * size + 2 * FLOOR[dtype] * top
    check("dx", got, dx, ref.rounded(dx, err[:, None].expand_as(dx), dtype))


@pytest.mark.parametrize("t", list(ref.TYPES))
@pytest.mark.parametrize("name", ["relu", "relu2", "silu"])
def test_product_backward_beside_a_closed_outlier(orc, name, t):
    """Ungated: a row scale and a gradient column far above the others', closed
    by the sign of its sums (relu, relu2) or far in silu's tail."""
    M, N, K, dtype = 70, 196, 528, ref.TYPES[t]
    q, s, T, packed, alpha, _, _, _, dy = closed_outlier(orc, M, N, K, 2.0 ** 14, 61)
    if name == "silu":
        q[(q.double() @ T[7].double()).abs() < 64] = 0
    dy = dy.to(dtype)
    got = bw.gemm_fused_backward(dy.cuda(), q.cuda(), s.cuda(), packed, alpha.cuda(), N, K, act=name)
    torch.cuda.synchronize()
    _, z = ref.product(q, s, T, alpha)
    dyd, a = dy.double(), alpha.double()
    dz = dyd * ref.slope(z, name)
    e = dyd.abs() * torch.where(dz == 0, 0.0, ref.slope_error(z, 3 * ref.U * z.abs(), name)) + ref.U * dz.abs()
    e = torch.where(z < -100, dz.abs(), e)        # (silu's tail: the slope may as well be 0)
    dx, bound = dx_and_bound([(dz * a, e * a.abs() + 2 * ref.U * (dz * a).abs(), T)], dtype)
    # where the outlier is open (silu, all sums 0) its gradients pass 65520,
    # from where on fp16 rounds to infinity
    most = 65520.0 if dtype == torch.float16 else float("inf")
    over, near = dx.abs() - bound >= most, dx.abs() + bound >= most
    v = got[0].cpu().double()
    assert torch.equal(v[over], dx[over].sign() * float("inf"))
    check("dx", torch.where(near, dx, v), dx, bound)


def test_captured_backward_beside_outliers_that_come_and_go(orc):
    """One graph replayed with tokens that need another scale and with tokens
    that do not, eager work between the replays."""
    M, N, K = 77, 1300, 272
    sets = [closed_outlier(orc, M, N, K, f, 41) for f in (2.0 ** 12, 1.0, 2.0 ** 30, 1.0, 2.0 ** 5)]
    _, s, _, pg, _, _, pu, _, _ = sets[0]
    live = [v.cuda().clone() for v in (sets[0][8], sets[0][0], s, sets[0][4], sets[0][7])]

    def work():
        dh, q, sx, ag, au = live
        return bw.glu_backward(dh, q, sx, pg, ag, pu, au, N, K, act="relu2")

    work()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = work()
    for q, sx, _, _, ag, _, _, au, dh in sets:
        for v, new in zip(live, (dh, q, sx, ag, au)):
            v.copy_(new)
        eager = [v.clone() for v in work()]
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(eager, held))


def aligned_tokens(M, K, T, rows, seed):
    """Tokens of which every third takes the signs of a row of T, so that its
    sum there is sqrt(K) / 8 times what tokens of their size reach elsewhere."""
    q, s = tokens(M, K, seed)
    for i, m in enumerate(range(0, M, 3)):
        q[m] = 127 * T[rows[i % len(rows)]]
    return q, s


@pytest.mark.parametrize("t", list(ref.TYPES))
@pytest.mark.parametrize("name", ["relu2", "silu", "gelu"])
@pytest.mark.parametrize("M,N,K", [(1, 132, 4096), (70, 196, 4096), (300, 1100, 1040), (5, 68, 65536)])
def test_backward_of_tokens_aligned_with_a_row(orc, M, N, K, name, t):
    """Gradients above what the first scale allows for, gated (both matrices
    alike) and not."""
    dtype = ref.TYPES[t]
    T, packed, alpha = weights(orc, N, K, 91)
    q, s = aligned_tokens(M, K, T, (20, 3, 64), 92)
    dh = (torch.randn((M, N), generator=_gen(93)) * 1e-4).to(dtype)
    d = [v.cuda() for v in (dh, q, s)] + [packed, alpha.cuda()]
    got = bw.glu_backward(*d, packed, alpha.cuda(), N, K, act=name)
    torch.cuda.synchronize()
    check("dx", got[0], *dx_and_bound(gated_terms(dh, q, s, T, alpha, T, alpha, name), dtype))
    for v, w in zip(got[1:], ref.glu_backward(dh, q, s, T, alpha, T, alpha, name, dtype)[1:]):
        check("dalpha", v, *w)
    got = bw.gemm_fused_backward(*d, N, K, act=name)
    torch.cuda.synchronize()
    _, z = ref.product(q, s, T, alpha)
    a, dz = alpha.double(), dh.double() * ref.slope(z, name)
    e = dh.double().abs() * ref.slope_error(z, 3 * ref.U * z.abs(), name) + ref.U * dz.abs()
    check("dx", got[0], *dx_and_bound([(dz * a, e * a.abs() + 2 * ref.U * (dz * a).abs(), T)], dtype))
    for v, w in zip(got[1:], ref.gemm_fused_backward(dh, q, s, T, alpha, None, name, dtype)[1:]):
        check("dalpha", v, *w)


def test_infinite_gradient_beside_one_above_its_scale(orc):
    """An infinite gradient at one output and a finite one at another that the
    first scale would make infinite: only the first is."""
    M, N, K = 6, 132, 4096
    T, packed, alpha = weights(orc, N, K, 91)
    q, s = aligned_tokens(M, K, T, (20,), 92)
    acc = q[3].double() @ T.double().t()
    acc[20] = 0
    n = int(acc.argmax())
    dy = torch.randn((M, N), generator=_gen(94))
    dy[3, n], dy[3, 20] = float("inf"), -1e3
    dx = bw.gemm_fused_backward(dy.cuda(), q.cuda(), s.cuda(), packed, alpha.cuda(), N, K, act="relu2")[0].cpu()
    want = torch.where(T[n] == 0, float("nan"), float("inf") * T[n].float())
    assert torch.equal(dx[3].isnan(), want.isnan()) and torch.equal(dx[3][T[n] != 0], want[T[n] != 0])
    assert bool(dx[[0, 1, 2, 4, 5]].isfinite().all())


@pytest.mark.parametrize("t", list(ref.TYPES))
@pytest.mark.parametrize("closing", [-1e6, -1e12, LOWEST])
@pytest.mark.parametrize("name", ["silu", "gelu", "gelu_tanh"])
def test_backward_of_the_smooth_activations_far_below_zero(orc, name, t, closing):
    closed_by_bias(orc, name, t, closing)


@pytest.mark.parametrize("name", ref.ACTS[1:])
@pytest.mark.parametrize("M", [3, 140])
def test_activations_far_above_zero(orc, name, M):
    """Biases up to 1e30: act(z) = z (z^2), off by at most 4 roundings of z and 12 of
    the activation, and slope 1 (2 z, times a gradient
    that keeps the product finite)."""
    N, K = 132, 272
    q, s = tokens(M, K, 1)
    T, packed, alpha = weights(orc, N, K, 2)
    bias = 10.0 ** torch.linspace(3, 15 if name == "relu2" else 30, N)
    dy = torch.randn((M, N), generator=_gen(6)) / bias
    d = [v.cuda() for v in (q, s)] + [packed, alpha.cuda(), N, K]
    y = bw.gemm_fused(*d, bias=bias.cuda(), act=name)
    _, _, db = bw.gemm_fused_backward(dy.cuda(), *d, bias=bias.cuda(), act=name)
    torch.cuda.synchronize()
    _, z = ref.product(q, s, T, alpha)
    z = z + bias.double()
    want = z * z if name == "relu2" else z
    check("y", y, want, 16 * ref.U * want.abs())
    dz = dy.double() * (2 * z if name == "relu2" else 1.0)
    check("dbias", db, dz.sum(0), (M + 40) * ref.U * dz.abs().sum(0))


@pytest.mark.parametrize("t", list(ref.TYPES))
@pytest.mark.parametrize("K", [12, 196, 300, 308, 364, 396, 1100, 3136, 4900, 9900, 16380, 16388, 19600])
def test_int8_norm_of_equal_features(K, t):
    """No spread, so v = 0 whatever the features' value: s = 1 and q = 0.  (In
    64 bits the sum of K equal fp32 values is exact, and so is its K-th.)"""
    x = torch.tensor([1.0, -3.25, 0.1, 1000.7, 1e-30, 60000.0, 0.0])[:, None].expand(-1, K).contiguous().to(ref.TYPES[t])
    for M in (1, 7, 700):       # 16 and 4 waves a token
        q, s = bw.layernorm_quantize(x.repeat(M // 7 + 1, 1)[:M].cuda())
        torch.cuda.synchronize()
        assert bool((s == 1).all()) and not q.any()


@pytest.mark.parametrize("t", list(ref.TYPES))
@pytest.mark.parametrize("K", [64, 1028, 2048, 8192, 8200, 16384, 16388])
@pytest.mark.parametrize("M", [5, 300])
def test_int8_norm_passes_on_what_is_not_finite(M, K, t):
    """A NaN or an infinity in a token: no scale (NaN), so every product of the
    token is NaN; the other tokens are as without it."""
    x = torch.randn((M, K), generator=_gen(M + K)).to(ref.TYPES[t])
    clean = bw.layernorm_quantize(x.cuda())
    bad = {1: float("nan"), 2: float("inf"), 4: -float("inf"), M - 2: float("nan")}
    for i, (m, v) in enumerate(bad.items()):
        x[m, (K - 1) * i // 3] = v
    q, s = bw.layernorm_quantize(x.cuda())
    torch.cuda.synchronize()
    lost = torch.zeros(M, dtype=torch.bool)
    lost[list(bad)] = True
    assert torch.equal(s.isnan().cpu(), lost)
    assert torch.equal(s.cpu()[~lost], clean[1].cpu()[~lost]) and torch.equal(q.cpu()[~lost], clean[0].cpu()[~lost])


@pytest.mark.parametrize("which", ["weight", "bias"])
@pytest.mark.parametrize("K", [64, 1028, 8192, 16384, 16388])
@pytest.mark.parametrize("M", [5, 300])
def test_int8_norm_passes_on_a_weight_that_is_not_finite(M, K, which):
    x = torch.randn((M, K), generator=_gen(K)).cuda()
    for v in (float("nan"), float("inf")):
        for k in (0, K // 2 + 1, K - 1):
            w = torch.ones(K, device="cuda")
            w[k] = v
            q, s = bw.layernorm_quantize(x, **{which: w})
            torch.cuda.synchronize()
            assert bool(s.isnan().all())


def test_gated_cells_hold_the_largest_sums_and_the_most_splits(orc):
    """K = 2^20, where the shared 64-bit cells are fullest: |sum| = 128 * 3/4 *
    2^20, between 2^26 and 2^27, in both 28-bit fields and with both signs,
    and as many splits as 8 bits count (of the 256 that the CUs ask for at
    most 255: 249 of 33 k tiles)."""
    M, N, K = 2, 64, 1 << 20
    assert int(bw.lib().sherry_glu_workspace_bytes(M, N, K)) > 0
    block = torch.tensor([1, 1, 1, 0], dtype=torch.int8).repeat(K // 4)
    flip = torch.arange(N)
    Tg = torch.where(flip % 2 == 0, -1, 1)[:, None].to(torch.int8) * block
    Tu = torch.where(flip % 3 == 0, -1, 1)[:, None].to(torch.int8) * block
    pack = [torch.from_numpy(orc.pack(t.numpy())).cuda() for t in (Tg, Tu)]
    q = torch.full((M, K), -128, dtype=torch.int8)
    q[1] = 127
    s, one = torch.full((M,), 2.0 ** -14), torch.ones(N)
    top = 0.75 * K * q[:, 0].double()[:, None] * 2.0 ** -14
    want = top * torch.where(flip % 2 == 0, -1.0, 1.0) * top * torch.where(flip % 3 == 0, -1.0, 1.0)
    for _ in range(2):      # the cells are zero again after each call
        h = bw.glu(q.cuda(), s.cuda(), pack[0], one.cuda(), pack[1], one.cuda(), N, K, act="none")
        torch.cuda.synchronize()
        check("h", h, want, 8 * ref.U * want.abs())


def test_capture_leaves_the_eager_workspaces_alone(orc):
    """Split-K products first called under capture: what they take belongs to
    the graph, so eager calls on that stream, before the first replay and
    beside later ones, find cells of their own."""
    N, K, M = 1024, 8192, 4
    T, packed, alpha = weights(orc, N, K, 1)
    alpha = alpha.cuda()
    q, s = tokens(M, K, 50)
    dq, ds = q.cuda(), s.cuda()
    x = (q.float() * s[:, None]).cuda()
    p2, a2 = bw.quantize_pack2(torch.randn((N, K), generator=_gen(2)).cuda())
    assert bw.workspace_bytes(M, N, K) > 0 and bw.linear_scratch_bytes(M, N, K) > 0
    calls = [lambda: bw.gemm(dq, ds, packed, alpha, N, K), lambda: bw.gemm_i32(dq, packed, N, K),
             lambda: bw.linear(x, packed, alpha, N, K), lambda: bw.gemm2(dq, ds, p2, a2, N, K),
             lambda: bw.gemm_fused(dq, ds, packed, alpha, N, K)]
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        warm = [c() for c in calls]
    torch.cuda.synchronize()
    for i, call in enumerate(calls):
        for known in (False, True):        # the stream has no workspace yet, or one
            fresh = torch.cuda.Stream()
            with torch.cuda.stream(fresh):
                if known:
                    call()
            torch.cuda.synchronize()
            before = {k: v.data_ptr() for d in (bw._workspaces._bufs, bw._scratch) for k, v in d.items()}
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=fresh):
                held = call()
            after = {k: v.data_ptr() for d in (bw._workspaces._bufs, bw._scratch) for k, v in d.items()}
            assert before == after
            for _ in range(3):
                with torch.cuda.stream(side):
                    graph.replay()
                with torch.cuda.stream(fresh):
                    eager = call()
                torch.cuda.synchronize()
                assert torch.equal(held, warm[i]) and torch.equal(eager, warm[i])


def test_outputs_do_not_lose_gradients_silently(orc):
    """With a tensor that requires a gradient the output says so, and a
    backward pass through it fails by the operator's name; without grad mode,
    or without such a tensor, outputs are plain."""
    M, N, K = 3, 64, 128
    q, s = (v.cuda() for v in tokens(M, K, 1))
    _, packed, alpha = weights(orc, N, K, 2)
    alpha = alpha.cuda()
    x, w = torch.randn((M, K), device="cuda"), torch.ones(K, device="cuda")
    dy = torch.randn((M, N), device="cuda")
    res = torch.randn((M, N), device="cuda")
    on = lambda t: t.clone().requires_grad_()
    mean, rstd = bw.layernorm(x, stats=True)[1:]
    cases = {
        "gemm_fused": [lambda f: bw.gemm_fused(q, s, packed, f(alpha), N, K),
                       lambda f: bw.gemm_fused(q, f(s), packed, alpha, N, K),
                       lambda f: bw.gemm_fused(q, s, packed, alpha, N, K, bias=f(alpha)),
                       lambda f: bw.gemm_fused(q, s, packed, alpha, N, K, residual=f(res))],
        "glu": [lambda f: bw.glu(q, s, packed, f(alpha), packed, alpha, N, K),
                lambda f: bw.glu(q, s, packed, alpha, packed, f(alpha), N, K)],
        "layernorm": [lambda f: bw.layernorm(f(x), w), lambda f: bw.layernorm(x, f(w)),
                      lambda f: bw.layernorm(x, w, f(w)), lambda f: bw.layernorm(x, f(w), stats=True)],
        "layernorm_quantize": [lambda f: bw.layernorm_quantize(f(x), w), lambda f: bw.layernorm_quantize(x, w, f(w))],
        "gemm_fused_backward": [lambda f: bw.gemm_fused_backward(f(dy), q, s, packed, alpha, N, K)],
        "glu_backward": [lambda f: bw.glu_backward(dy, q, s, packed, f(alpha), packed, alpha, N, K)],
        "layernorm_backward": [lambda f: bw.layernorm_backward(f(x), x, mean, rstd, w)],
    }
    for name, calls in cases.items():
        for call in calls:
            plain, tracked = call(lambda t: t), call(on)
            with torch.no_grad():
                without = call(on)
            plain, tracked, without = (v if isinstance(v, tuple) else (v,) for v in (plain, tracked, without))
            for a, b, c in zip(plain, tracked, without):
                assert torch.equal(a, b) and torch.equal(a, c) and not a.requires_grad and not c.requires_grad
                assert b.requires_grad == b.is_floating_point()
                if b.requires_grad:
                    with pytest.raises(RuntimeError, match=f"bit_weight_amd.{name} .*not implemented"):
                        b.sum().backward()
    # a given output cannot carry it: refused, as torch's own functions do
    out = torch.empty((M, N), device="cuda")
    for call in (lambda: bw.gemm_fused(q, s, packed, on(alpha), N, K, out=out),
                 lambda: bw.glu(q, s, packed, on(alpha), packed, alpha, N, K, out=out),
                 lambda: bw.gemm_fused(q, s, packed, alpha, N, K, out=on(out)),
                 lambda: bw.layernorm(on(x), out=torch.empty_like(x)),
                 lambda: bw.layernorm_backward(x, x, mean, rstd, on(w), out=torch.empty_like(x))):
        with pytest.raises(RuntimeError, match="out="):
            call()
        with torch.no_grad():
            call()


def test_a_hand_written_autograd_function(orc):
    """The way to train through the operators: a torch.autograd.Function of
    their forward and backward."""
    M, N, K = 5, 64, 128
    q, s = (v.cuda() for v in tokens(M, K, 1))
    _, pg, ag = weights(orc, N, K, 2)
    _, pu, au = weights(orc, N, K, 3)
    ag, au = ag.cuda().requires_grad_(), au.cuda().requires_grad_()

    class Glu(torch.autograd.Function):
        @staticmethod
        def forward(ctx, ag, au):
            ctx.save_for_backward(ag, au)
            return bw.glu(q, s, pg, ag, pu, au, N, K)

        @staticmethod
        def backward(ctx, dh):
            ag, au = ctx.saved_tensors
            return bw.glu_backward(dh, q, s, pg, ag, pu, au, N, K)[1:]

    h = Glu.apply(ag, au)
    dh = torch.randn_like(h)
    h.backward(dh)
    with torch.no_grad():
        _, dg, du = bw.glu_backward(dh, q, s, pg, ag, pu, au, N, K)
    assert torch.equal(ag.grad, dg) and torch.equal(au.grad, du)


def test_stats_that_have_no_truth_value_are_refused():
    x = torch.randn((2, 128), device="cuda")
    for call in (bw.layernorm, bw.layernorm_quantize):
        with pytest.raises(RuntimeError, match="ambiguous"):
            call(x, stats=torch.ones(2))


# The ends of the ranges: 2^20 tokens, outputs or inputs, one block of the others
@pytest.mark.parametrize("t", list(ref.TYPES))
@pytest.mark.parametrize("M,N,K", [(1 << 20, 4, 16), (1, 1 << 20, 16), (70, 1 << 18, 16), (3, 4, 1 << 20), (140, 4, 1 << 18)])
def test_products_at_the_ends_of_their_range(orc, M, N, K, t):
    dtype = ref.TYPES[t]
    q, s = tokens(M, K, 71)
    Tg, pg, ag = weights(orc, N, K, 72)
    Tu, pu, au = weights(orc, N, K, 73)
    bias, res = torch.randn(N, generator=_gen(74)), torch.randn((M, N), generator=_gen(75)).to(dtype)
    dy = (torch.randn((M, N), generator=_gen(76)) * 0.01).to(dtype)
    d = [v.cuda() for v in (q, s)]
    y = bw.gemm_fused(*d, pg, ag.cuda(), N, K, bias=bias.cuda(), act="gelu", residual=res.cuda(), dtype=dtype)
    check("y", y, *ref.gemm_fused(q, s, Tg, ag, bias, "gelu", res, dtype))
    h = bw.glu(*d, pg, ag.cuda(), pu, au.cuda(), N, K, dtype=dtype)
    check("h", h, *ref.glu(q, s, Tg, ag, Tu, au, "silu", dtype))
    for name, v, w in zip(("dx", "dalpha", "dbias"),
                          bw.gemm_fused_backward(dy.cuda(), *d, pg, ag.cuda(), N, K, bias=bias.cuda(), act="gelu"),
                          ref.gemm_fused_backward(dy, q, s, Tg, ag, bias, "gelu", dtype)):
        check(name, v, *w)
    for name, v, w in zip(("dx", "dgate", "dup"), bw.glu_backward(dy.cuda(), *d, pg, ag.cuda(), pu, au.cuda(), N, K),
                          ref.glu_backward(dy, q, s, Tg, ag, Tu, au, "silu", dtype)):
        check(name, v, *w)


EPS = torch.tensor(1e-5).item()     # the default, as fp32 holds it


@pytest.mark.parametrize("t", list(ref.TYPES))
@pytest.mark.parametrize("M,K", [(1 << 20, 4), (2, 1 << 20)])
def test_norms_at_the_ends_of_their_range(M, K, t):
    dtype = ref.TYPES[t]
    g = _gen(81)
    x, w, b = torch.randn((M, K), generator=g).to(dtype), 1 + 0.3 * torch.randn(K, generator=g), 0.2 * torch.randn(K, generator=g)
    dy = torch.randn((M, K), generator=g).to(dtype)
    y, mean, rstd = bw.layernorm(x.cuda(), w.cuda(), b.cuda(), stats=True)
    check("y", y, *ref.layernorm(x, w, b, EPS, dtype)[:2])
    q, s = bw.layernorm_quantize(x.cuda(), w.cuda(), b.cuda())
    rv, rs = ref.layernorm_quantize(x, w, b, EPS)
    # equal but where 64-bit arithmetic (within 1e-12 here) does not decide a
    # rounding: of the scale to fp32, of a value between two steps
    d = x.double() - x.double().mean(1, keepdim=True)
    s64 = (d / torch.sqrt((d * d).mean(1, keepdim=True) + EPS) * w.double() + b.double()).abs().amax(1) / 127
    open_ = (s64 * (1 + 1e-12)).float() != (s64 * (1 - 1e-12)).float()
    # (undecided: 2e-12 of steps of 2^-24 to 2^-23, so up to M 2^-14.8 on average)
    assert bool(((s.cpu() == rs) | open_).all()) and int(open_.sum()) <= 2 + M * 2.0 ** -13
    border = (rv - rv.floor() - 0.5).abs() < 1e-9
    assert bool(((q.cpu().double() == rv.round().clamp(-127, 127)) | border | open_[:, None]).all())
    for name, v, want in zip(("dx", "dw", "db"), bw.layernorm_backward(dy.cuda(), x.cuda(), mean, rstd, w.cuda()),
                             ref.layernorm_backward(dy, x, mean.cpu(), rstd.cpu(), w, dtype)):
        check(name, v, *want)
