"""Attention of sequences that are longer than their table, where a window hides
everything that the table has room for: NaN, in both kernels, not the zeros of a
query that sees nothing."""

import math

import pytest
import torch

import attention_reference as ref
import bit_weight_amd as bw
from test_attention_edges_gpu import i32
from test_attention_gpu import check, filled, scales_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)


# Rows of 16 take few queries; tiles of 128 where queries times heads, over 16, times
# the window's steps are 32000 or more.
SIZES = {"rows": (3, 4, 2), "tiles": (520, 1024, 8)}      # queries, heads, key heads


@pytest.mark.parametrize("t", list(ref.TYPES))
@pytest.mark.parametrize("kernel", list(SIZES))
@pytest.mark.parametrize("window,sinks", [(64, 0), (1, 0), (40, 5), (None, 0)])
def test_longer_than_the_table(kernel, window, sinks, t):
    """The table has room for 160 tokens of a sequence of 600; the sequence after it
    has what it needs and is not touched."""
    new, Hq, H = SIZES[kernel]
    dtype, page, D = ref.TYPES[t], 16, 16
    cache, table, _, held = filled([160, 160], page, H, D, 21)
    assert table.shape[1] == 10
    q = torch.randn(new + 2, Hq, D, generator=ref.gen(22)).to(dtype)
    tl = i32(600, 160)
    y, lse = bw.cache_attention(q.cuda(), cache, table, i32(0, new, new + 2), tl, window=window, sinks=sinks, lse=True)
    assert y[:new].isnan().all() and lse[:new].isnan().all()
    few, each = 8, Hq // H      # (heads to check)
    heads = slice(0, few // each) if each < few else slice(0, 1)
    few = (heads.stop - heads.start) * each
    want, want_lse = ref.attention(q[new:, :few], held[1][0].read(160)[:, heads], held[1][1].read(160)[:, heads], D ** -0.5,
                                   window, sinks, dtype, scales_of(cache, table, 1, 160, page)[:, heads])
    check("y", y[new:, :few], *want)
    check("lse", lse[new:, :few], *want_lse)


@pytest.mark.parametrize("t", ["bf16", "fp32"])
def test_longer_than_the_table_in_parts(t):
    """A window of many steps, so that a query's are cut into parts: some of them, or all,
    lie behind the table's room."""
    dtype, page, H, D, n = ref.TYPES[t], 16, 1, 64, 4000
    cache, table, _, _ = filled([n], page, H, D, 31)
    q = torch.randn(2, 4, D, generator=ref.gen(32)).to(dtype).cuda()
    for length in (n + 1, n + 2999, n + 3000, n + 3001, 2 * n, 1 << 30):
        for sinks in (0, 2000):
            y, lse = bw.cache_attention(q, cache, table, i32(0, 2), i32(length), window=3000, sinks=sinks, lse=True)
            assert y.isnan().all() and lse.isnan().all(), (length, sinks)
    y, lse = bw.cache_attention(q, cache, table, i32(0, 2), i32(n), window=3000, lse=True)
    assert torch.isfinite(y).all() and torch.isfinite(lse).all()
    # in positions that nobody sees nothing is wrong with such a sequence's neighbours or a shorter one
    y, lse = bw.cache_attention(q, cache, table, i32(0, 2), i32(0), window=3000, lse=True)
    assert bool((y == 0).all()) and bool((lse == -math.inf).all())
