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
