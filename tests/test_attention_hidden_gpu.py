"""What a query does not see leaves its result alone, whatever scale the values
there have: tokens after it, before its window, in pages that are no more."""

import pytest
import torch

import attention_reference as ref
import bit_weight_amd as bw
from test_attention_edges_gpu import i32
from test_attention_gpu import check, scales_of, sequences
from test_attention_tiles_gpu import STEPS, wide  # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)


# Powers of two that small and large values have: as far apart as the type of y allows.
FAR = {"fp32": (-100, 20), "bf16": (-100, 20), "fp16": (-14, 13)}


def written(sizes, H, D, seed, scale_of_keys=1.0):
    """A cache of pages of 16 with one sequence, its values' block b about 2^sizes[b],
    and what it holds."""
    n = 16 * len(sizes)
    cache, table, starts, tl = sequences([n], [n], 16, H, D, seed)
    g = ref.gen(seed + 1)
    size = 2.0 ** torch.tensor(sizes, dtype=torch.float32).repeat_interleave(16)[:, None, None]
    k, v = scale_of_keys * torch.randn(n, H, D, generator=g), torch.randn(n, H, D, generator=g) * size
    bw.cache_write(cache, k.cuda(), v.cuda(), table, starts, tl)
    held = []
    for x in (k, v):
        held.append(ref.Blocks(H, D))
        held[-1].write(0, x.double())
    return cache, table, tl, [b.read(n) for b in held]


def check_rows(q, y, lse, k, v, units, window, sinks, rows, head):
    """Rows `rows` of query head `head`, each as the last of its tokens."""
    n, new, group = k.shape[0], q.shape[0], q.shape[1] // k.shape[1]
    kv = slice(head // group, head // group + 1)
    for j in rows:
        end = n - new + j + 1
        want, want_lse = ref.attention(q[j:j + 1, head:head + 1], k[:end, kv], v[:end, kv], q.shape[2] ** -0.5, window, sinks,
                                       q.dtype, units[:end, kv])
        check(f"y of row {j}", y[j:j + 1, head:head + 1], *want)
        check(f"lse of row {j}", lse[j:j + 1, head:head + 1], *want_lse)


def released(kernel, t, group_rows):
    """A sequence whose pages before the windows are gone (-1, or past the cache),
    while page 0 is another sequence's and holds values 2^120 as large."""
    low, high = FAR[t]
    new, Hq, H, D, window = group_rows
    dtype, n = ref.TYPES[t], 64 * 16
    cache, table, tl, (k, v) = written([low] * 64, H, D, 41)
    if kernel == "tiles":
        assert new * Hq // 16 * (window // 64 + 1) >= STEPS
    # page 0 moves to a spare one, if this sequence has it
    spare = next(p for p in range(cache.k.shape[0]) if p not in table.tolist()[0] and p)
    for c in cache:
        c[spare] = c[0]
    table[table == 0] = spare
    cache.v_scale[0] = 2.0 ** high
    cache.k_scale[0] = 1.0
    units = scales_of(cache, table, 0, n, 16)
    seen = n - new - window + 1      # the first token that anyone sees
    table[0, :seen // 16] = -1
    table[0, :seen // 16:2] = cache.k.shape[0] + 5
    q = torch.randn(new, Hq, D, generator=ref.gen(43)).to(dtype)
    y, lse = bw.cache_attention(q.cuda(), cache, table, i32(0, new), tl, window=window, lse=True)
    for head in (0, Hq - 1):
        check_rows(q, y, lse, k, v, units, window, 0, sorted({0, 1, 7, new // 2, new - 1} & set(range(new))), head)


@pytest.mark.parametrize("t", list(ref.TYPES))
@pytest.mark.parametrize("kernel,sizes", [("rows", (3, 8, 2, 64, 40)), ("tiles", (520, 1024, 4, 32, 40)), ("tiles", (512, 1024, 64, 16, 9))])
def test_pages_released_before_the_window(kernel, sizes, t):
    released(kernel, t, sizes)


@pytest.mark.parametrize("t", list(ref.TYPES))
@pytest.mark.parametrize("kernel,new,Hq,H", [("rows", 3, 4, 2), ("tiles", 520, 1024, 4)])
def test_blocks_before_every_window(kernel, new, Hq, H, t):
    """Blocks of the same 64 tokens that lie before the windows: every fourth is small,
    and the windows of a token's tile see that alone."""
    low, high = FAR[t]
    dtype, D, window = ref.TYPES[t], 32, 5
    cache, table, tl, (k, v) = written([high, high, high, low] * 16, H, D, 51)
    n = 64 * 16
    if kernel == "tiles":
        assert new * Hq // 16 >= STEPS
    q = torch.randn(new, Hq, D, generator=ref.gen(53)).to(dtype)
    y, lse = bw.cache_attention(q.cuda(), cache, table, i32(0, new), tl, window=window, lse=True)
    small = [j for j in range(new) if (n - new + j) % 64 >= 48 + window][-12:]
    check_rows(q, y, lse, k, v, scales_of(cache, table, 0, n, 16), window, 0, [*small, new - 1], Hq - 1)


@pytest.mark.parametrize("t", list(ref.TYPES))
@pytest.mark.parametrize("blocks", [[0, 1, 0, 0], [0, 0, 0, 1], [1, 0, 1, 0], [0, 0, 0, 0, 1, 0, 0, 1, 0]])
@pytest.mark.parametrize("D,Hq,H", [(64, 4, 1), (128, 2, 2), (256, 3, 1)])
def test_tokens_after_the_query(wide, D, Hq, H, blocks, t):  # noqa: F811
    """Prompts without history whose blocks are small or large: no query depends on
    the scale of tokens after it, in the tiles and in the 16-row kernel."""
    dtype, far = ref.TYPES[t], FAR[t]
    cache, table, tl, (k, v) = written([far[b] for b in blocks], H, D, 61)
    n = 16 * len(blocks)
    units = scales_of(cache, table, 0, n, 16)
    q = torch.randn(n, Hq, D, generator=ref.gen(63)).to(dtype)
    want, want_lse = ref.attention(q, k, v, D ** -0.5, None, 0, dtype, units)
    y, lse = bw.cache_attention(q.cuda(), cache, table, i32(0, n), tl, lse=True)
    assert wide
    check("y", y, *want)
    check("lse", lse, *want_lse)
    few = 16 * H // Hq      # queries of a unit of 16 rows
    for at in (0, 16, n - few):
        y, lse = bw.cache_attention(q[at:at + few].cuda(), cache, table, i32(0, few), i32(at + few), lse=True)
        check("y", y, want[0][at:at + few], want[1][at:at + few])
        check("lse", lse, want_lse[0][at:at + few], want_lse[1][at:at + few])


@pytest.mark.parametrize("t", list(ref.TYPES))
@pytest.mark.parametrize("sinks", [0, 3, 16, 21])
def test_windows_of_a_tile(sinks, t):
    """Tiles of eight tokens: some of their windows see a large block, the others only
    a small one; first tokens are small."""
    low, high = FAR[t]
    dtype, Hq, H, D, window, new = ref.TYPES[t], 1024, 64, 16, 5, 1000
    assert new * Hq // 16 * ((window + sinks) // 64 + 1) >= STEPS
    cache, table, tl, (k, v) = written([low, low] + [high, low] * 31, H, D, 71)
    n = 64 * 16
    q = torch.randn(new, Hq, D, generator=ref.gen(73)).to(dtype)
    y, lse = bw.cache_attention(q.cuda(), cache, table, i32(0, new), tl, window=window, sinks=sinks, lse=True)
    units = scales_of(cache, table, 0, n, 16)
    for head in (0, 700):
        check_rows(q, y, lse, k, v, units, window, sinks, list(range(0, 40)) + list(range(500, 540)) + [new - 1], head)


@pytest.mark.parametrize("t", ["bf16", "fp32"])
@pytest.mark.parametrize("blocks", [[0, 1, 0, 0] * 16, [0] * 40 + [1] + [0] * 23])
def test_tokens_after_the_query_in_parts(wide, blocks, t):  # noqa: F811
    """Queries of a longer prompt, whose steps several workgroups share."""
    dtype, far, D, Hq = ref.TYPES[t], FAR[t], 64, 2
    cache, table, tl, (k, v) = written([far[b] for b in blocks], 1, D, 81)
    n = 16 * len(blocks)
    q = torch.randn(n, Hq, D, generator=ref.gen(83)).to(dtype)
    y, lse = bw.cache_attention(q.cuda(), cache, table, i32(0, n), tl, lse=True)
    assert wide
    rows = [0, 1, 15, 16, 17, 40, 100, 320, 639, 640, 641, 655, 656, n - 1]
    check_rows(q, y, lse, k, v, scales_of(cache, table, 0, n, 16), None, 0, rows, 1)
