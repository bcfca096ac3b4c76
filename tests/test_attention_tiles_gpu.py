"""Attention of many queries a sequence in the kernel of 128-row tiles.  It is taken
where the steps of 16 rows are many, counted with the longest sequence that the
table has room for: a wide table sends small prompts there too, and they can be
checked against the definition."""

import math

import pytest
import torch

import attention_reference as ref
import bit_weight_amd as bw
import test_attention_edges_gpu as edges
import test_attention_gpu as plain
from test_attention_gpu import check, filled, scales_of, sequences

pytestmark = pytest.mark.gpu

STEPS = 32000       # of 16 rows, from which the tiles are taken


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)


@pytest.fixture
def wide(monkeypatch):
    """cache_attention with tables that have room for as long a sequence as it takes;
    -> the calls that were sent to the tiles."""
    real, sent = bw.cache_attention, []

    def call(q, cache, table, starts, lens, **kw):
        T, Hq, _ = q.shape
        page, group, S = 16 * cache.k.shape[2], Hq // cache.k.shape[1], table.shape[0]
        if T * group >= 64 * S and not kw.get("window"):
            room = 64 * (-(-STEPS // max(T * Hq // 16, 1)))
            more = torch.full((S, max(room // page + 1 - table.shape[1], 0)), -1, dtype=torch.int32, device=table.device)
            table = torch.cat([table, more], 1)
            assert T * Hq // 16 * (table.shape[1] * page // 64 + 1) >= STEPS
            sent.append(T)
        return real(q, cache, table, starts, lens, **kw)

    monkeypatch.setattr(bw, "cache_attention", call)
    return sent


@pytest.mark.parametrize("t", list(ref.TYPES))
@pytest.mark.parametrize("lens,new,page,Hq,H,D,window,sinks", [c for c in plain.PROMPTS if c[6] is None])
def test_prompts(wide, lens, new, page, Hq, H, D, window, sinks, t):
    plain.test_attention(lens, new, page, Hq, H, D, window, sinks, t)
    assert len(wide) == 2


@pytest.mark.parametrize("t", list(ref.TYPES))
@pytest.mark.parametrize("scale", [0.0, -0.2, 1e-30, 3.0])
def test_scales_of_scores(wide, scale, t):
    edges.test_scales_of_scores(scale, 130, t)
    assert wide


@pytest.mark.parametrize("t", list(ref.TYPES))
def test_blocks_of_very_different_scales(wide, t):
    edges.test_blocks_of_very_different_scales(140, t)
    assert wide


def test_rows_of_nobody_are_left_alone(wide):
    edges.test_rows_of_nobody_are_left_alone(True)
    assert wide


@pytest.mark.parametrize("S,new,group", [(70, 3, 32), (1100, 4, 32)])
def test_many_sequences(wide, S, new, group):
    edges.test_attention_of_many_sequences(S, new, group, "bf16")
    assert wide


def test_captured_runs_replay_alike(wide):
    edges.test_captured_runs_replay_alike([600, 300], [300, 70])
    assert wide


@pytest.mark.parametrize("t", ["bf16", "fp16"])
def test_a_layer_of_them_together(wide, t):
    edges.test_a_layer_of_them_together(t)
    assert wide


@pytest.mark.parametrize("t,H,D,Hq,n,new,window,sinks", [
    ("bf16", 1, 32, 64, 1300, 1200, 400, 5), ("fp32", 2, 64, 64, 1000, 1000, 500, 70), ("fp16", 1, 128, 32, 2100, 2000, 500, 0)])
def test_windows(t, H, D, Hq, n, new, window, sinks):
    """Windows bound the steps whatever the table: many heads, three of them checked,
    and of these every ninth row."""
    dtype, page = ref.TYPES[t], 16
    assert new * Hq // 16 * ((window + sinks) // 64 + 1) >= STEPS
    cache, table, tl, held = filled([n], page, H, D, 61)
    q = (2 * torch.randn(new, Hq, D, generator=ref.gen(62))).to(dtype)
    y, lse = bw.cache_attention(q.cuda(), cache, table, edges.i32(0, new), tl, window=window, sinks=sinks, lse=True)
    k, v, units = held[0][0].read(n), held[0][1].read(n), scales_of(cache, table, 0, n, page)
    for h in (0, Hq // 2 - 1, Hq - 1):
        kv = slice(h // (Hq // H), h // (Hq // H) + 1)
        for j in range(0, new, 9):
            end = n - new + j + 1       # the row as the last of its tokens
            want, want_lse = ref.attention(q[j:j + 1, h:h + 1], k[:end, kv], v[:end, kv], D ** -0.5, window, sinks, dtype,
                                           units[:end, kv])
            check("y", y[j:j + 1, h:h + 1], *want)
            check("lse", lse[j:j + 1, h:h + 1], *want_lse)


@pytest.mark.parametrize("t", list(ref.TYPES))
def test_what_is_not_finite_or_has_no_page(wide, t):
    """A token that is not finite, or a page out of range, spoils the queries that see
    a token of it and no others."""
    dtype, page, H, D, n, new = ref.TYPES[t], 16, 2, 64, 300, 250
    cache, table, starts, tl = sequences([n], [n], page, H, D, 65)
    g = ref.gen(66)
    k, v = torch.randn(n, H, D, generator=g), torch.randn(n, H, D, generator=g)
    q = torch.randn(new, 4, D, generator=g).to(dtype)
    bw.cache_write(cache, k.cuda(), v.cuda(), table, starts, tl)
    held = []
    for x in (k, v):
        held.append(ref.Blocks(H, D))
        held[-1].write(0, x.double())
    want = ref.attention(q, held[0].read(n), held[1].read(n), D ** -0.5, None, 0, dtype, scales_of(cache, table, 0, n, page))
    k[180, 0, 3], v[250, 1, 9] = math.inf, math.nan        # block 11 of head 0's keys, block 15 of head 1's values
    bw.cache_write(cache, k.cuda(), v.cuda(), table, starts, tl)
    q[7, 1, 0] = math.nan
    bad = table.clone()
    bad[0, 17] = cache.k.shape[0]                           # tokens 272 ..
    y, lse = (x.cpu() for x in bw.cache_attention(q.cuda(), cache, bad, edges.i32(0, new), tl, lse=True))
    pos = n - new + torch.arange(new)
    lost = torch.zeros(new, 4, dtype=torch.bool)
    lost[:, :2] |= (pos >= 176)[:, None]
    lost[:, 2:] |= (pos >= 240)[:, None]
    lost[pos >= 272] = True
    lost[7, 1] = True
    assert y[lost].isnan().all() and lse[lost].isnan().all()
    check("y", y[~lost], want[0][0][~lost], want[0][1][~lost])
    check("lse", lse[~lost], want[1][0][~lost], want[1][1][~lost])
    assert wide
