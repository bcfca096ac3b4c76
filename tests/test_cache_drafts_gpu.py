"""Drafts that were refused: earlier positions written again. The block keeps the
scale it has come to, as the header says, until its first position is written."""

import math

import pytest
import torch

import attention_reference as ref
import bit_weight_amd as bw
from test_attention_edges_gpu import i32
from test_attention_gpu import sequences

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)


@pytest.mark.parametrize("t", list(ref.TYPES))
@pytest.mark.parametrize("draft", [1.0, 300.0, math.inf, math.nan])
def test_refused_drafts(draft, t):
    """19 tokens, a draft of four behind them refused after two, two others in the place
    of the rest; the blocks are the definition's to the last bit at every step, and the
    first block, which the drafts do not reach, is untouched."""
    dtype, H, D, page = ref.TYPES[t], 2, 48, 16
    cache, table, _, _ = sequences([48], [48], page, H, D, 5)
    held = [ref.Blocks(H, D), ref.Blocks(H, D)]
    g = ref.gen(6)

    def write(first, *rows):
        n = rows[0].shape[0]
        bw.cache_write(cache, *(r.cuda() for r in rows), table, i32(0, n), i32(first + n))
        for b, r in zip(held, rows):
            b.write(first, r.double())
        end = first + n
        got = bw.cache_read(cache, table, i32(0, end), i32(end), end)
        for b, x in zip(held, got):
            want = b.read(end).float()
            assert torch.equal(x.cpu().nan_to_num(9.0), want.nan_to_num(9.0)) and torch.equal(x.cpu().isnan(), want.isnan())
        return [x.cpu() for x in got]

    rand = lambda n: [torch.randn(n, H, D, generator=g).to(dtype) for _ in range(2)]
    write(0, *rand(19))
    drafted = rand(4)
    for d in drafted:
        d[3, 1, 7] *= draft
    write(19, *drafted)
    fresh = rand(2)
    after = write(21, *fresh)
    for x, r, d in zip(after, fresh, drafted):
        assert torch.isfinite(x[:16]).all() and torch.isfinite(x[:, 0]).all()       # other blocks, other heads
        if not math.isfinite(draft):
            assert x[16:, 1].isnan().all()        # a block that was not finite stays so
        elif draft > 100:        # coarser than the tokens that are left would make it
            scale = ref.least_scale(float(d[3, 1].double().abs().max()))
            assert scale > ref.least_scale(float(x[16:, 1].abs().max()))
            assert torch.equal(x[21:, 1].double(), torch.round(r[:, 1].double() / scale) * scale)
    # the block's first position written again makes it the new tokens' alone
    again = rand(7)
    back = write(16, *again)
    assert all(torch.isfinite(x).all() for x in back)
    alone = [ref.Blocks(H, D), ref.Blocks(H, D)]
    for b, a, x in zip(alone, again, back):
        b.write(16, a.double())
        assert torch.equal(x[16:], b.read(23)[16:].float())
