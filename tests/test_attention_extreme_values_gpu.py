"""Values near the ends of fp32's range: a mean of values is no larger than they are,
and no less exact where they are tiny."""

import pytest
import torch

import attention_reference as ref
import bit_weight_amd as bw
from test_attention_edges_gpu import i32
from test_attention_gpu import check, scales_of, sequences
from test_attention_hidden_gpu import check_rows
from test_attention_tiles_gpu import wide  # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)


# queries, tokens: a unit in one workgroup, a unit in parts, tiles, tiles in parts
SIZES = {"unit": (3, 40), "parts": (2, 6000), "tiles": (100, 100), "tiles in parts": (260, 3000)}


@pytest.mark.parametrize("t", ["fp32", "bf16"])
@pytest.mark.parametrize("D,Hq", [(64, 2), (128, 1), (256, 1)])
@pytest.mark.parametrize("kind", list(SIZES))
@pytest.mark.parametrize("size", [2.0 ** 127, 2.0 ** 118, 2.0 ** -115, 2.0 ** -120, 2.0 ** -130])
def test_ends_of_the_range(wide, size, kind, D, Hq, t):  # noqa: F811
    """Values of one sign from `size` to 1.9 times that: their scales are 2^121 down to
    2^-126, the smallest."""
    new, n = SIZES[kind]
    dtype, page, g = ref.TYPES[t], 64, ref.gen(171)
    cache, table, starts, tl = sequences([n], [n], page, 1, D, 172)
    k = torch.randn(n, 1, D, generator=g)
    v = size * (1 + 0.9 * torch.rand(n, 1, D, generator=g))
    bw.cache_write(cache, k.cuda(), v.cuda(), table, starts, tl)
    held = []
    for x in (k, v):
        held.append(ref.Blocks(1, D))
        held[-1].write(0, x.double())
    k, v = (b.read(n) for b in held)
    units = scales_of(cache, table, 0, n, page)
    q = torch.randn(new, Hq, D, generator=ref.gen(273)).to(dtype)
    y, lse = bw.cache_attention(q.cuda(), cache, table, i32(0, new), tl, lse=True)
    assert bool(wide) == ("tiles" in kind)
    if n < 1000:
        want, want_lse = ref.attention(q, k, v, D ** -0.5, None, 0, dtype, units)
        check("y", y, *want)
        check("lse", lse, *want_lse)
    else:
        check_rows(q, y, lse, k, v, units, None, 0, sorted({0, 1, new // 2, new - 1}), Hq - 1)


@pytest.mark.parametrize("kind", list(SIZES))
def test_parts_of_both_ends(wide, kind):  # noqa: F811
    """Largest values of either sign in neighbouring blocks, and the smallest beside them."""
    new, n = SIZES[kind]
    D, page, g = 64, 16, ref.gen(181)
    cache, table, starts, tl = sequences([n], [n], page, 1, D, 182)
    block = torch.arange(n) // 16 % 3
    k = torch.randn(n, 1, D, generator=g)
    v = (1 + 0.9 * torch.rand(n, 1, D, generator=g)) * torch.tensor([2.0 ** 127, -2.0 ** 127, 2.0 ** -120])[block][:, None, None]
    bw.cache_write(cache, k.cuda(), v.cuda(), table, starts, tl)
    held = []
    for x in (k, v):
        held.append(ref.Blocks(1, D))
        held[-1].write(0, x.double())
    q = torch.randn(new, 1, D, generator=ref.gen(283)).cuda()
    y, lse = bw.cache_attention(q, cache, table, i32(0, new), tl, lse=True)
    assert bool(wide) == ("tiles" in kind)
    check_rows(q.cpu(), y, lse, *(b.read(n) for b in held), scales_of(cache, table, 0, n, page), None, 0, sorted({0, 1, new // 2, new - 1}), 0)
