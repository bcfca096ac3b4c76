"""Gradients of the head norms over x itself, beside x in the columns of a wider
matrix, and refused in between."""

import pytest
import torch

import bit_weight_amd as bw

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)


@pytest.mark.parametrize("t", [torch.float32, torch.bfloat16])
def test_in_place_and_beside(t):
    T, Hq, Hk, D = 70, 3, 2, 64
    width = (Hq + Hk) * D
    g = torch.Generator().manual_seed(7)
    rand = lambda *shape: torch.randn(*shape, generator=g).to(t).cuda()
    big = rand(T, 3 * width)
    x, beside = big[:, :width], big[:, width:2 * width]
    dq, dk = rand(T, Hq, D), rand(T, Hk, D)
    pos = torch.arange(T, dtype=torch.int32).cuda()
    fr = 100.0 ** (-torch.arange(0, D, 2, dtype=torch.float64) / D).cuda()
    want, rest = bw.qk_norm_rope_backward(dq, dk, x, pos, fr), big[:, 2 * width:].clone()
    for refused in (big[:, 8:width + 8], big[:, width - 8:2 * width - 8], big[1:, 2 * width:]):
        with pytest.raises((bw.SherryError, RuntimeError)):
            bw.qk_norm_rope_backward(dq, dk, x, pos, fr, out=refused)
    with pytest.raises(bw.SherryError):      # the rows before x's
        bw.qk_norm_rope_backward(dq[1:], dk[1:], x[1:], pos[1:], fr, out=x[:-1])
    for out in (beside, x):
        before = x.clone()
        got = bw.qk_norm_rope_backward(dq, dk, x, pos, fr, out=out)
        assert all(torch.equal(a, b) for a, b in zip(got, want)) and got[0].data_ptr() == out.data_ptr()
        assert out is x or torch.equal(x, before)
    assert torch.equal(big[:, 2 * width:], rest)
