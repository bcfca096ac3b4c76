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


@pytest.mark.parametrize("tiles", [False, True])
@pytest.mark.parametrize("seed", range(4))
def test_two_terms_of_fp32(wide, seed, tiles):  # noqa: F811
    """A few tokens of weights near the largest above thousands of small ones, in fp32.
    Queries have one feature that is not 0, of few bits, so that a score is one exact
    product: times the scale's factor, and less the maximum, 4 U of |s| + |m|, U = 2^-24.
    Weights: 2^-22 and 4 U; the sums (the weights' and the products') 2 U for each of up
    to n terms would be the worst order's: lanes and steps of 64 make it 2 (n / 64 + 64) U;
    fp16's last step: half of 2^-24 under weights that are 2^7 as large as the maximum's
    at least: 2^-32 a token, times the largest value.  The join's: 16 U.  (One term alone
    would miss this bound by three to six times.)"""
    n, D, H, Hq, page = 4000, 64, 1, 4, 16
    new = 64 if tiles else 4
    g = ref.gen(140 + seed)
    cache, table, tl, _ = filled([n], page, H, D, 141)
    k = torch.zeros(n, H, D)
    k[:, 0, 0] = 0.25 * torch.randint(-16, 16, (n,), generator=g)      # in 8 bits without a rounding
    peaks = torch.randperm(n - new, generator=g)[:6]
    k[:, 0, 1] = -8.0
    k[peaks, 0, 1] = 0.0
    v = torch.randint(64, 128, (n, H, D), generator=g) * (2.0 * torch.randint(0, 2, (n, H, D), generator=g) - 1)
    bw.cache_write(cache, k.cuda(), v.cuda(), table, i32(0, n), tl)
    rk, rv = bw.cache_read(cache, table, i32(0, n), tl, n)
    assert torch.equal(rk.cpu(), k) and torch.equal(rv.cpu(), v)
    q = torch.zeros(new, Hq, D)
    q[:, :, 0] = 0.125 * torch.randint(-3, 4, (new, Hq), generator=g)
    q[:, :, 1] = 2.0      # 16 of e lower where it is no peak
    got = bw.cache_attention(q.cuda(), cache, table, i32(0, new), tl, scale=1.0).double().cpu()
    assert bool(wide) == tiles
    s = torch.einsum("thd,lgd->thl", q.double(), k.double())      # exact, and so is the difference below
    hidden = torch.arange(n)[None, :] > n - new + torch.arange(new)[:, None]
    s = s.masked_fill(hidden[:, None], -torch.inf)
    m = s.amax(-1, keepdim=True)
    e = torch.exp(s - m)
    total = e.sum(-1, keepdim=True)
    w, av = e / total, v[:, 0].double()
    want = w @ av
    U = ref.U
    each = torch.where(w > 0, 2.0 ** -22 + (4 + 4 * (s.abs() + m.abs()).nan_to_num(0.0, 0.0, 0.0)) * U, 0.0)      # relative, of a weight
    sums = (2 * (n / 64 + 64) + 16) * U
    bound = (w * each) @ av.abs() + ((w * each).sum(-1, keepdim=True) + 2 * sums) * (w @ av.abs()) \
        + n * 2.0 ** -32 * 127 / total + want.abs() * U
    off = (got - want).abs()
    assert float((off / bound).max()) <= 1, float((off / bound).max())
