"""How far the attention's results are from the definition in 64 bits, beside the
one rounding that their type makes necessary."""

import pytest
import torch

import attention_reference as ref
import bit_weight_amd as bw
from test_attention_edges_gpu import held_rows, i32
from test_attention_gpu import filled
from test_attention_tiles_gpu import wide  # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)


def exact(q, k, v, scale):
    """All queries at once, in 64 bits."""
    n, group = q.shape[0], q.shape[1] // k.shape[1]
    k, v = (x.double().repeat_interleave(group, 1).transpose(0, 1) for x in (k, v))      # [Hq, L, D]
    s = scale * (q.double().transpose(0, 1) @ k.transpose(1, 2).contiguous())
    L = k.shape[1]
    hidden = torch.arange(L)[None, :] > L - n + torch.arange(n)[:, None]
    return (torch.softmax(s.masked_fill(hidden, -torch.inf), -1) @ v).transpose(0, 1)


@pytest.mark.parametrize("tiles", [False, True])
@pytest.mark.parametrize("n,D", [(100, 64), (900, 128), (3000, 96)])
def test_rounding_of_fp16(wide, n, D, tiles):  # noqa: F811
    """The error's root mean square is the last rounding's, for fp16 as for a result in
    64 bits that is rounded once.  What may come to it: weights of 22 bits and scores in
    fp32 (D products, 2^-24 each at most: in the mean square sqrt(2 D) 2^-24, 2^-20, of
    sums of D terms) against 2^-12: less than a hundredth; twentieths are allowed.
    Weights of 11 bits alone, whose errors average out over the tokens as the values
    do, would bring as much again as half of the rounding's square."""
    H, Hq, page = 2, 8, 16
    cache, table, tl, held = filled([n], page, H, D, 131)
    new = min(n, 200) if tiles else 8
    q = torch.randn(new, Hq, D, generator=ref.gen(977)).half()
    k, v = held_rows(held, [n])[0]
    want = exact(q, k, v, D ** -0.5)
    got = bw.cache_attention(q.cuda(), cache, table, i32(0, new), tl).cpu()
    assert bool(wide) == tiles
    error = (got.double() - want).square().mean().sqrt()
    rounding = (want.half().double() - want).square().mean().sqrt()
    assert rounding <= error * 1.0000001 and error <= 1.05 * rounding, float(error / rounding)
