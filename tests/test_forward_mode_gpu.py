"""Forward-mode tangents are refused by name, not left out, as gradients are; where
forward mode is off (inside a torch.autograd.Function) the operators run."""

import pytest
import torch
import torch.autograd.forward_ad as fwd

import bit_weight_amd as bw
from test_attention_edges_gpu import i32
from test_attention_gpu import filled, freqs_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)


def calls():
    """Of each operator, a call with one of its tensors at a time handed to f."""
    T, Hq, H, D, K, N = 3, 4, 2, 32, 256, 64
    rand = lambda *shape: torch.randn(*shape, device="cuda")
    x, wq, wk, pos, fr = rand(T, (Hq + H) * D), rand(D), rand(D), i32(0, 1, 2), freqs_of(D).cuda()
    cache, table, tl, _ = filled([20], 16, H, D, 3)
    starts = i32(0, T)
    q, k = bw.qk_norm_rope(x, pos, fr, Hq, H, D, wq, wk)
    ks, vs = cache.k_scale, cache.v_scale
    yield from (
        ("qk_norm_rope", lambda f: bw.qk_norm_rope(f(x), pos, fr, Hq, H, D, wq, wk)),
        ("qk_norm_rope", lambda f: bw.qk_norm_rope(x, pos, f(fr), Hq, H, D, wq, wk)),
        ("qk_norm_rope", lambda f: bw.qk_norm_rope(x, pos, fr, Hq, H, D, f(wq), wk)),
        ("qk_norm_rope", lambda f: bw.qk_norm_rope(x, pos, fr, Hq, H, D, wq, f(wk))),
        ("qk_norm_rope_backward", lambda f: bw.qk_norm_rope_backward(f(q), k, x, pos, fr, wq, wk)),
        ("qk_norm_rope_backward", lambda f: bw.qk_norm_rope_backward(q, f(k), x, pos, fr, wq, wk)),
        ("qk_norm_rope_backward", lambda f: bw.qk_norm_rope_backward(q, k, f(x), pos, fr, wq, wk)),
        ("qk_norm_rope_backward", lambda f: bw.qk_norm_rope_backward(q, k, x, pos, fr, wq, wk, out=f(torch.empty_like(x)))),
        ("cache_write", lambda f: bw.cache_write(cache, f(k), k, table, starts, tl)),
        ("cache_write", lambda f: bw.cache_write(cache, k, f(k), table, starts, tl)),
        ("cache_write", lambda f: bw.cache_write(cache._replace(k_scale=f(ks)), k, k, table, starts, tl)),
        ("cache_read", lambda f: bw.cache_read(cache._replace(v_scale=f(vs)), table, starts, tl, T)),
        ("cache_attention", lambda f: bw.cache_attention(f(q), cache, table, starts, tl)),
        ("cache_attention", lambda f: bw.cache_attention(q, cache._replace(k_scale=f(ks)), table, starts, tl)),
        ("cache_attention", lambda f: bw.cache_attention(q, cache, table, starts, tl, out=f(torch.empty_like(q)))),
    )
    packed, alpha = bw.quantize_pack(rand(N, K))
    x8, s = bw.quantize_act(rand(T, K))
    z, bias, w = rand(T, N), rand(N), rand(K)
    y, mean, rstd = bw.layernorm(rand(T, K), w, w, stats=True)
    yield from (
        ("gemm_fused", lambda f: bw.gemm_fused(x8, f(s), packed, alpha, N, K)),
        ("gemm_fused", lambda f: bw.gemm_fused(x8, s, packed, f(alpha), N, K)),
        ("gemm_fused", lambda f: bw.gemm_fused(x8, s, packed, alpha, N, K, bias=f(bias))),
        ("gemm_fused", lambda f: bw.gemm_fused(x8, s, packed, alpha, N, K, residual=f(z))),
        ("layernorm", lambda f: bw.layernorm(f(y), w, w)),
        ("layernorm_quantize", lambda f: bw.layernorm_quantize(y, f(w), w)),
        ("layernorm_backward", lambda f: bw.layernorm_backward(f(y), y, mean, rstd, w)),
    )


def test_tangents_are_not_lost_silently():
    for name, call in calls():
        call(lambda t: t)
        with fwd.dual_level():
            dual = lambda t: fwd.make_dual(t, torch.ones_like(t))
            for context in (torch.enable_grad, torch.no_grad):      # (forward mode does not go by the grad mode)
                with context(), pytest.raises(NotImplementedError, match=f"{name} .*forward"):
                    call(dual)
            call(lambda t: t)
            call(lambda t: fwd.unpack_dual(dual(t)).primal)
    torch.cuda.synchronize()


def test_a_function_with_a_tangent_of_its_own():
    """A torch.autograd.Function with a jvp runs the operator with forward mode off."""
    T, Hq, H, D = 3, 4, 2, 32
    pos, fr = i32(0, 1, 2), freqs_of(D).cuda()
    turn = lambda x: bw.qk_norm_rope(x, pos, fr, Hq, H, D, norm=False)[0]

    class Turn(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x):
            return turn(x)

        @staticmethod
        def jvp(ctx, dx):
            return turn(dx)       # (the rotation is linear)

    x, dx = (torch.randn(T, (Hq + H) * D, device="cuda") for _ in range(2))
    with fwd.dual_level():
        y, dy = fwd.unpack_dual(Turn.apply(fwd.make_dual(x, dx)))
    assert torch.equal(y, turn(x)) and torch.equal(dy, turn(dx))
