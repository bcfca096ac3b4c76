"""A prompt and many single tokens in one call, as a server makes it.  One kernel takes
all sequences of a call, by the average of rows a sequence: 16-row units where the
single tokens are many, 128-row tiles where the prompt outweighs them."""

import pytest
import torch

import attention_reference as ref
import bit_weight_amd as bw
from test_attention_edges_gpu import check_attention, held_rows, running
from test_attention_gpu import filled
from test_attention_tiles_gpu import wide  # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)


@pytest.mark.parametrize("t", list(ref.TYPES))
@pytest.mark.parametrize("singles,at,window,sinks", [(70, 0, None, 0), (40, 40, None, 0), (9, 4, None, 0), (9, 0, None, 0), (9, 9, 100, 20)])
def test_a_prompt_among_single_tokens(wide, singles, at, window, sinks, t):  # noqa: F811
    dtype, H, Hq, D, page = ref.TYPES[t], 2, 6, 64, 16
    lens = [20 + (37 * i) % 211 for i in range(singles)]
    new = [1] * singles
    lens.insert(at, 430)
    new.insert(at, 300)
    lens[-1 if at == 0 else 0] = 900
    cache, table, tl, held = filled(lens, page, H, D, 151)
    q = torch.randn(sum(new), Hq, D, generator=ref.gen(251)).to(dtype).cuda()
    y, lse = bw.cache_attention(q, cache, table, running(new), tl, window=window, sinks=sinks, lse=True)
    assert bool(wide) == (window is None and sum(new) * 3 >= 64 * len(new))
    only = {at, at - 1, at + 1, 0, singles} & set(range(singles + 1))
    check_attention(q, y, lse, cache, table, lens, new, held_rows(held, lens), D ** -0.5, window, sinks, page, only)
