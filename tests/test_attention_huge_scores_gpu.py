"""Scores so large that fp32's steps at them are wider than the exponential's range:
the token of the largest score has all of the weight, in both kernels."""

import pytest
import torch

import attention_reference as ref
import bit_weight_amd as bw
from test_attention_edges_gpu import i32
from test_attention_gpu import sequences
from test_attention_tiles_gpu import wide  # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)


@pytest.mark.parametrize("t", list(ref.TYPES))
@pytest.mark.parametrize("tiles", [False, True])
@pytest.mark.parametrize("size", [2.0 ** 26, 2.0 ** 30, 2.0 ** 40, 2.0 ** 100])
@pytest.mark.parametrize("by", ["keys", "scale", "a negative scale"])
def test_the_largest_score_takes_all(wide, by, size, tiles, t):  # noqa: F811
    """Keys of random integers times `size`, or the scale as large.  Scores are integers
    times 0.3 (so that no product with log2 e is exact); queries whose two largest differ
    by 2^-10 of them or more (fp32 queries have 2^-22 in their terms, scores 2^-17) are
    compared: y is the value of that token, lse its score to fp32's rounding of a product
    and a sum of 64, 2^-17."""
    dtype, n, D, Hq, page = ref.TYPES[t], 200, 64, 4, 16
    new = 200 if tiles else 8
    g = ref.gen(161)
    cache, table, starts, tl = sequences([n], [n], page, 1, D, 162)
    k = torch.randint(-100, 101, (n, 1, D), generator=g).float()
    k[:, :, 0] = 127.0 - 254.0 * torch.randint(0, 2, (n, 1), generator=g)      # (all blocks' scales are 1)
    v = torch.randint(-127, 128, (n, 1, D), generator=g).float()
    v[:, :, 1] = 127.0
    bw.cache_write(cache, (k * (size if by == "keys" else 1.0)).cuda(), v.cuda(), table, starts, tl)
    q = torch.randint(-8, 9, (new, Hq, D), generator=g).to(dtype)
    scale = torch.tensor(0.3 * (1.0 if by == "keys" else size) * (-1.0 if by == "a negative scale" else 1.0)).item()
    y, lse = bw.cache_attention(q.cuda(), cache, table, i32(0, new), tl, scale=scale, lse=True)
    assert bool(wide) == tiles
    s = torch.einsum("thd,ld->thl", q.double(), k[:, 0].double()) * scale * (size if by == "keys" else 1.0)
    hidden = torch.arange(n)[None, :] > n - new + torch.arange(new)[:, None]
    s = s.masked_fill(hidden[:, None], -torch.inf)
    two = s.topk(2, -1)
    largest, next_one = two.values.unbind(-1)
    clear = (largest - next_one >= 2.0 ** -10 * torch.maximum(largest.abs(), next_one.abs().nan_to_num(posinf=0.0))) & (largest != 0)
    assert clear.double().mean() > 0.7
    want = v[two.indices[..., 0], 0]
    y, lse = y.cpu(), lse.cpu().double()
    assert torch.isfinite(y).all() and torch.isfinite(lse).all()
    assert torch.equal(y[clear].float(), want[clear])
    assert bool(((lse - largest).abs() <= 2.0 ** -17 * largest.abs())[clear].all())
