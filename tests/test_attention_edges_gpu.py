"""The attention operators on the GPU where they can go wrong: captured graphs,
streams, many sequences, masks and scales at their ends, long caches, refusals,
and a layer's run of them."""

import math

import pytest
import torch

import attention_reference as ref
import bit_weight_amd as bw
from test_attention_gpu import check, cuda, filled, freqs_of, rope_case, scales_of, sequences

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)


def i32(*v):
    return torch.tensor(v, dtype=torch.int32).cuda()


def running(new):
    return i32(*(sum(new[:i]) for i in range(len(new) + 1)))


def held_rows(held, lens):
    return [[b.read(n) for b in pair] for pair, n in zip(held, lens)]


def check_attention(q, y, lse, cache, table, lens, new, held, scale, window, sinks, page, only=None):
    at = 0
    for i, (n, m) in enumerate(zip(lens, new)):
        if m and (only is None or i in only):
            want, want_lse = ref.attention(q[at:at + m].cpu(), held[i][0], held[i][1], scale, window, sinks, q.dtype,
                                           scales_of(cache, table, i, n, page))
            check(f"y of sequence {i}", y[at:at + m], *want)
            check(f"lse of sequence {i}", lse[at:at + m], *want_lse)
        at += m


# ----------------------------------------------------------------- many sequences
@pytest.mark.parametrize("t", ["bf16", "fp32"])
@pytest.mark.parametrize("S,new,group", [(70, 1, 4), (130, 1, 1), (600, 1, 2), (1100, 2, 1), (70, 3, 32), (1100, 4, 16)])
def test_attention_of_many_sequences(S, new, group, t):
    """More sequences than a scan of 64 takes at once, some of them without rows or
    tokens; with one or a few queries each and (T group >= 64 S) in tiles."""
    dtype, D, page = ref.TYPES[t], 32, 16
    g = ref.gen(S)
    lens = [int(n) for n in torch.randint(0, 60, (S,), generator=g)]
    lens[0], lens[S // 2], lens[-1] = 0, 333, 47
    count = [min(n, new) if i % 5 else 0 for i, n in enumerate(lens)]
    count[S // 2], count[-1] = new, new
    cache, table, tl, held = filled(lens, page, 1, D, S)
    T = sum(count)
    q = torch.randn(T, group, D, generator=g).to(dtype).cuda()
    y, lse = bw.cache_attention(q, cache, table, running(count), tl, lse=True)
    only = {1, 2, 63, 64, 65, S // 2, S - 1, S - 2}
    check_attention(q, y, lse, cache, table, lens, count, held_rows(held, lens), D ** -0.5, None, 0, page, only)


def test_write_and_read_of_many_sequences():
    S, D, page = 1100, 16, 16
    lens = [1 + (7 * i) % 40 for i in range(S)]
    cache, table, tl, held = filled(lens, page, 1, D, 3)
    k, v = bw.cache_read(cache, table, running(lens), tl, sum(lens))
    for kind, got in enumerate((k, v)):
        assert torch.equal(got.cpu(), torch.cat([h[kind].read(n) for h, n in zip(held, lens)]).float())


# ------------------------------------------------------- rows of nobody, bad starts
@pytest.mark.parametrize("many", [False, True])
def test_rows_of_nobody_are_left_alone(many):
    """Rows behind the last sequence's, before the first's, and of starts that do
    not ascend (which give no rows)."""
    group, page, D = (64 if many else 2), 16, 32
    lens = [40, 50, 60, 30]
    cache, table, tl, held = filled(lens, page, 1, D, 5)
    T = 14
    q = torch.randn(T, group, D, generator=ref.gen(6)).cuda()
    out = torch.full((T, group, D), 7.0, device="cuda")
    starts = i32(4, 4, 8, 3, 3)       # sequences: none, rows 4 .. 7, none (8, 3), none
    y = bw.cache_attention(q, cache, table, starts, tl, out=out)
    assert y.data_ptr() == out.data_ptr() and bool((y[:4] == 7).all()) and bool((y[8:] == 7).all())
    want, _ = ref.attention(q[4:8].cpu(), held[1][0].read(50), held[1][1].read(50), D ** -0.5, None, 0, q.dtype,
                            scales_of(cache, table, 1, 50, page))
    check("y", y[4:8], *want)
    starts = i32(9, 4, 4, 8, 1 << 30)       # none, none, rows 4 .. 7, rows 8 .. 13 (to the end)
    y = bw.cache_attention(q, cache, table, starts, tl, out=out.fill_(7.0))
    assert bool((y[:4] == 7).all())
    for i, (a, b) in ((2, (4, 8)), (3, (8, 14))):
        want, _ = ref.attention(q[a:b].cpu(), held[i][0].read(lens[i]), held[i][1].read(lens[i]), D ** -0.5, None, 0, q.dtype,
                                scales_of(cache, table, i, lens[i], page))
        check("y", y[a:b], *want)
    # nobody has rows; lengths below 0
    y = bw.cache_attention(q, cache, table, i32(0, 0, 0, 0, 0), tl, out=out.fill_(7.0))
    assert bool((y == 7).all())
    y, lse = bw.cache_attention(q, cache, table, i32(0, 3, 3, 3, 3), i32(-5, 1, 1, 1), lse=True)
    assert bool((y[:3] == 0).all()) and bool((lse[:3] == -math.inf).all())


# ------------------------------------------------------------- scales and masks
@pytest.mark.parametrize("t", list(ref.TYPES))
@pytest.mark.parametrize("new", [3, 130])
@pytest.mark.parametrize("scale", [0.0, -0.2, 1e-30, 3.0])
def test_scales_of_scores(scale, new, t):
    dtype, page, H, D = ref.TYPES[t], 32, 2, 64
    cache, table, tl, held = filled([200], page, H, D, 15)
    q = torch.randn(new, 4, D, generator=ref.gen(16)).to(dtype).cuda()
    y, lse = bw.cache_attention(q, cache, table, i32(0, new), tl, scale=scale, lse=True)
    scale = torch.tensor(scale).item()      # as fp32
    check_attention(q, y, lse, cache, table, [200], [new], held_rows(held, [200]), scale, None, 0, page)


@pytest.mark.parametrize("t", list(ref.TYPES))
@pytest.mark.parametrize("new", [2, 140])
def test_blocks_of_very_different_scales(new, t):
    """Values (and keys) of neighbouring blocks from 2^-100 to 2^6, a block of zeros
    among them; queries of very different sizes, one of zeros."""
    dtype, page, H, D = ref.TYPES[t], 16, 1, 32
    n = 260
    cache, table, _, _ = sequences([n], [n], page, H, D, 25)
    g = ref.gen(26)
    size = torch.tensor([2.0 ** e for e in (-100, 0, -20, 6, -126, -8, 3, -40, 0, 5, -3, 1, -60, 2, 6, -1, 4)])
    size = size.repeat_interleave(16)[:n, None, None]
    k, v = torch.randn(n, H, D, generator=g) * size.clamp(max=1.0), torch.randn(n, H, D, generator=g) * size
    k[64:80] = v[32:48] = 0.0
    starts, tl = i32(0, n), i32(n)
    bw.cache_write(cache, k.cuda(), v.cuda(), table, starts, tl)
    held = []
    for x in (k, v):
        b = ref.Blocks(H, D)
        b.write(0, x.double())
        held.append(b)
    q = (torch.randn(new, 3, D, generator=g) * torch.tensor([1e-3, 1.0, 8.0])[None, :, None]).to(dtype)
    q[-1, 1] = 0.0
    q = q.cuda()
    y, lse = bw.cache_attention(q, cache, table, i32(0, new), tl, lse=True)
    check_attention(q, y, lse, cache, table, [n], [new], held_rows([held], [n]), D ** -0.5, None, 0, page)


@pytest.mark.parametrize("t", list(ref.TYPES))
@pytest.mark.parametrize("new", [4, 240])
def test_what_is_not_finite_stays_where_it_is(new, t):
    """A token that is not finite spoils its block for the queries that see a token
    of it and for no others; a query that is not finite spoils its own row."""
    dtype, page, H, D = ref.TYPES[t], 16, 2, 64
    n, window = 300, 64
    cache, table, starts, tl = sequences([n], [n], page, H, D, 35)
    g = ref.gen(36)
    k, v = torch.randn(n, H, D, generator=g), torch.randn(n, H, D, generator=g)
    q = torch.randn(new, 4, D, generator=g).to(dtype)
    want, held = [], []
    for spoiled in (False, True):
        if spoiled:
            k[5, 0, 3], v[250, 1, 9] = math.inf, math.nan        # block 0 of head 0's keys, block 15 of head 1's values
        bw.cache_write(cache, k.cuda(), v.cuda(), table, starts, tl)
        if not spoiled:
            for x in (k, v):
                held.append(ref.Blocks(H, D))
                held[-1].write(0, x.double())
            want = ref.attention(q, held[0].read(n), held[1].read(n), D ** -0.5, window, 0, dtype, scales_of(cache, table, 0, n, page))
    q[new - 2, 1, 0] = math.nan
    y, lse = bw.cache_attention(q.cuda(), cache, table, i32(0, new), tl, window=window, lse=True)
    pos = n - new + torch.arange(new)
    lost = torch.zeros(new, 4, dtype=torch.bool)
    lost[:, :2] |= (pos - window < 15)[:, None]                  # some of tokens 0 .. 15 in sight
    lost[:, 2:] |= ((pos >= 240) & (pos - window < 255))[:, None]
    lost[new - 2, 1] = True
    y, lse = y.cpu(), lse.cpu()
    assert y[lost].isnan().all() and lse[lost].isnan().all()
    check("y", y[~lost], want[0][0][~lost], want[0][1][~lost])
    check("lse", lse[~lost], want[1][0][~lost], want[1][1][~lost])


# ------------------------------------------------------------------ far addresses
def test_far_pages_and_rows():
    """Pages past 2^31 bytes of the cache, in both kernels, and stacked rows past
    2^31 values."""
    H, D, page = 8, 128, 64
    pages = (1 << 31) // (page * H * D) + 40
    cache = bw.kv_cache(pages, page, H, D)
    n, g = 150, ref.gen(45)
    k, v = torch.randn(n, H, D, generator=g), torch.randn(n, H, D, generator=g)
    table, tl = i32(pages - 1, 3, pages - 7)[None], i32(n)
    bw.cache_write(cache, k.cuda(), v.cuda(), table, i32(0, n), tl)
    held = []
    for x in (k, v):
        b = ref.Blocks(H, D)
        b.write(0, x.double())
        held.append(b)
    rk, rv = bw.cache_read(cache, table, i32(0, n), tl, n)
    assert torch.equal(rk.cpu(), held[0].read(n).float()) and torch.equal(rv.cpu(), held[1].read(n).float())
    for new in (1, 70):
        q = torch.randn(new, H, D, generator=g).to(torch.bfloat16).cuda()
        y, lse = bw.cache_attention(q, cache, table, i32(0, new), tl, lse=True)
        check_attention(q, y, lse, cache, table, [n], [new], held_rows([held], [n]), D ** -0.5, None, 0, page)
    del cache
    T, Hq, Hk = 430000, 32, 8
    x = torch.zeros(T, (Hq + Hk) * D, dtype=torch.bfloat16, device="cuda")
    last = torch.randn(5, (Hq + Hk) * D, generator=g).to(torch.bfloat16)
    x[-5:] = last.cuda()
    pos = torch.arange(T, dtype=torch.int32).cuda()
    fr = freqs_of(D)
    q, k = bw.qk_norm_rope(x, pos, fr.cuda(), Hq, Hk, D)
    some = bw.qk_norm_rope(last.cuda(), pos[-5:].contiguous(), fr.cuda(), Hq, Hk, D)
    assert torch.equal(q[-5:], some[0]) and torch.equal(k[-5:], some[1]) and bool((q[:1000] == 0).all())
    bw.qk_norm_rope_backward(q, k, x, pos, fr.cuda(), out=x)
    assert torch.equal(x[-5:], bw.qk_norm_rope_backward(*some, last.cuda(), pos[-5:].contiguous(), fr.cuda())[0])


# --------------------------------------------------------------- graphs, streams
def layer_step(S, lens, new, dtype=torch.bfloat16, Hq=8, H=2, D=64, page=16, seed=55):
    """A call's worth of inputs and a function that runs norm, write and attention on
    them; the cache's state before is put back first."""
    cache, table, tl, _ = filled(lens, page, H, D, seed)
    starts = running(new)
    T = sum(new)
    g = ref.gen(seed + 1)
    x = torch.randn(T, (Hq + 2 * H) * D, generator=g).to(dtype).cuda()
    lastly = torch.cat([torch.arange(n - m, n) for n, m in zip(lens, new)]).to(torch.int32).cuda()
    fr, w = freqs_of(D).cuda(), torch.rand(D, generator=g).cuda()
    saved = [c.clone() for c in cache]

    def run(x=x):
        for c, s in zip(cache, saved):
            c.copy_(s)
        q, k = bw.qk_norm_rope(x, lastly, fr, Hq, H, D, w, w)
        bw.cache_write(cache, k, x[:, (Hq + H) * D:].unflatten(1, (H, D)), table, starts, tl)
        y, lse = bw.cache_attention(q, cache, table, starts, tl, lse=True)
        dx, dwq, dwk = bw.qk_norm_rope_backward(q, k, x, lastly, fr, w, w)
        return y, lse, dx, dwq, dwk, *bw.cache_read(cache, table, starts, tl, T)

    return x, run


@pytest.mark.parametrize("lens,new", [([2000], [1]), ([400, 37, 900], [1, 1, 1]), ([600, 300], [300, 70])])
def test_captured_runs_replay_alike(lens, new):
    """Captured and replayed with other inputs and eager calls between: each replay
    is the eager run's to the last bit, also where two graphs replay side by side."""
    x, run = layer_step(len(lens), lens, new)
    other, run_other = layer_step(len(lens), lens, new, seed=75)
    inputs = [torch.randn_like(x) for _ in range(4)]
    eager = [[v.clone() for v in run(i)] for i in inputs]
    want_other = [v.clone() for v in run_other()]
    torch.cuda.synchronize()
    graph, graph_other = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = run()
    with torch.cuda.graph(graph_other):
        outs_other = run_other()
    sides = [torch.cuda.Stream(), torch.cuda.Stream()]
    for n, i in enumerate(inputs):
        x.copy_(i)
        torch.cuda.synchronize()
        if n % 2:
            run_other()       # eager work between
            torch.cuda.synchronize()
        with torch.cuda.stream(sides[0]):
            graph.replay()
        with torch.cuda.stream(sides[1]):
            graph_other.replay()
        torch.cuda.synchronize()
        for a, b in zip((*outs, *outs_other), (*eager[n], *want_other)):
            assert torch.equal(a, b), n
    assert all(not bool(b.any()) for b in bw._workspaces._bufs.values())


def test_two_streams_at_once():
    steps = [layer_step(1, [3000 + 100 * i], [1], seed=85 + 10 * i) for i in range(2)]
    alone = [[v.clone() for v in run()] for _, run in steps]
    torch.cuda.synchronize()
    sides = [torch.cuda.Stream() for _ in steps]
    for _ in range(5):
        got = []
        for side, (_, run) in zip(sides, steps):
            with torch.cuda.stream(side):
                got.append(run())
        torch.cuda.synchronize()
        for a, b in zip(alone, got):
            assert all(torch.equal(x, y) for x, y in zip(a, b))


# ------------------------------------------------------------ gradients, refusals
def test_gradients_are_not_lost_silently():
    T, Hq, Hk, D = 3, 4, 2, 32
    x, w, pos = rope_case(T, Hq, Hk, D, True, torch.float32, 95)
    x, wq, wk, pos, fr = x.cuda(), cuda(w[0]), cuda(w[1]), pos.cuda(), freqs_of(D).cuda()
    on = lambda t: t.clone().requires_grad_()
    cache, table, tl, _ = filled([20], 16, Hk, D, 96)
    q, k = bw.qk_norm_rope(x, pos, fr, Hq, Hk, D, wq, wk)
    starts = i32(0, T)
    cases = {
        "qk_norm_rope": [lambda f: bw.qk_norm_rope(f(x), pos, fr, Hq, Hk, D, wq, wk),
                         lambda f: bw.qk_norm_rope(x, pos, f(fr), Hq, Hk, D, wq, wk),
                         lambda f: bw.qk_norm_rope(x, pos, fr, Hq, Hk, D, f(wq), wk),
                         lambda f: bw.qk_norm_rope(x, pos, fr, Hq, Hk, D, wq, f(wk))],
        "qk_norm_rope_backward": [lambda f: bw.qk_norm_rope_backward(f(q), k, x, pos, fr, wq, wk),
                                  lambda f: bw.qk_norm_rope_backward(q, k, f(x), pos, fr, wq, wk)],
        "cache_attention": [lambda f: bw.cache_attention(f(q), cache, table, starts, tl, lse=True),
                            lambda f: bw.cache_attention(q, cache._replace(k_scale=f(cache.k_scale)), table, starts, tl, lse=True),
                            lambda f: bw.cache_attention(q, cache._replace(v_scale=f(cache.v_scale)), table, starts, tl, lse=True)],
        "cache_read": [lambda f: bw.cache_read(cache._replace(v_scale=f(cache.v_scale)), table, starts, tl, T)],
    }
    for name, calls in cases.items():
        for call in calls:
            plain, tracked = call(lambda t: t), call(on)
            with torch.no_grad():
                without = call(on)
            for a, b, c in zip(plain, tracked, without):
                assert torch.equal(a, b) and torch.equal(a, c) and b.requires_grad and not a.requires_grad and not c.requires_grad
                with pytest.raises(RuntimeError, match=f"bit_weight_amd.{name} .*not implemented"):
                    b.sum().backward()
    for call in (lambda: bw.cache_attention(on(q), cache, table, starts, tl, out=torch.empty_like(q)),
                 lambda: bw.qk_norm_rope_backward(q, k, on(x), pos, fr, wq, wk, out=torch.empty_like(x))):
        with pytest.raises(RuntimeError, match="out="):
            call()
        with torch.no_grad():
            call()
    for a, b in ((on(k), k), (k, on(k))):
        with pytest.raises(RuntimeError, match="gradients"):
            bw.cache_write(cache, a, b, table, starts, tl)
        with torch.no_grad():
            bw.cache_write(cache, a, b, table, starts, tl)


def test_a_hand_written_autograd_function():
    """Training through the norm and rotation: a torch.autograd.Function of the two
    operators, its gradients the backward's, captured beside a live eager graph."""
    T, Hq, Hk, D = 9, 4, 2, 64
    x, w, pos = rope_case(T, Hq, Hk, D, True, torch.float32, 105)
    pos, fr = pos.cuda(), freqs_of(D).cuda()
    x, wq, wk = (t.cuda().requires_grad_() for t in (x, *w))

    class NormRope(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, wq, wk):
            ctx.save_for_backward(x, wq, wk)
            return bw.qk_norm_rope(x, pos, fr, Hq, Hk, D, wq, wk)

        @staticmethod
        def backward(ctx, dq, dk):
            x, wq, wk = ctx.saved_tensors
            return bw.qk_norm_rope_backward(dq, dk, x, pos, fr, wq, wk)

    q, k = NormRope.apply(x, wq, wk)
    dq, dk = torch.randn_like(q), torch.randn_like(k)
    torch.autograd.backward((q, k), (dq, dk))
    with torch.no_grad():
        want = bw.qk_norm_rope_backward(dq, dk, x, pos, fr, wq, wk)
    assert all(torch.equal(a.grad, b) for a, b in zip((x, wq, wk), want))
    q = k = None
    with torch.no_grad():       # the operators themselves are what a graph holds
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            held = bw.qk_norm_rope_backward(dq, dk, x, pos, fr, wq, wk)
        for _ in range(3):
            for h in held:
                h.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(held, want))


def test_refusals():
    Hq, H, D, page, n = 4, 2, 32, 16, 20
    cache, table, tl, _ = filled([n], page, H, D, 115)
    starts, fr = i32(0, 3), freqs_of(D).cuda()
    q, k = torch.zeros(3, Hq, D, device="cuda"), torch.zeros(3, H, D, device="cuda")
    x, pos, w = torch.zeros(3, (Hq + H) * D, device="cuda"), i32(0, 1, 2), torch.ones(D, device="cuda")
    attend = lambda **kw: bw.cache_attention(**{**dict(q=q, cache=cache, table=table, starts=starts, lens=tl), **kw})
    write = lambda **kw: bw.cache_write(**{**dict(cache=cache, k=k, v=k, table=table, starts=starts, lens=tl), **kw})
    read = lambda **kw: bw.cache_read(**{**dict(cache=cache, table=table, starts=starts, lens=tl, tokens=3), **kw})
    rope = lambda **kw: bw.qk_norm_rope(**{**dict(x=x, positions=pos, freqs=fr, q_heads=Hq, k_heads=H, dim=D, q_weight=w), **kw})
    back = lambda **kw: bw.qk_norm_rope_backward(**{**dict(dq=q, dk=k, x=x, positions=pos, freqs=fr, q_weight=w), **kw})
    for call in (attend, write, read, rope, back):
        call()
    errors = (RuntimeError, ValueError, TypeError)
    shared = [dict(table=table[0]), dict(table=table.long()), dict(table=table.cpu()), dict(starts=starts[:1]), dict(lens=i32(1, 2)),
              dict(starts=starts.long()), dict(lens=tl.cpu()), dict(cache=cache._replace(k=cache.k[0])),
              dict(cache=cache._replace(v=cache.v.float())), dict(cache=cache._replace(v=cache.v[:1])),
              dict(cache=cache._replace(k_scale=cache.k_scale[:1])), dict(cache=cache._replace(v_scale=cache.v_scale.double())),
              dict(cache=cache._replace(k=cache.k.transpose(4, 5)))]
    bad = {attend: [dict(q=q[0]), dict(q=q[:, :3]), dict(q=q.double()), dict(q=q[:, :, :16]), dict(q=q.cpu()), dict(window=0),
                    dict(window=-3), dict(sinks=-1), dict(scale=math.nan), dict(out=q), dict(out=q.half()), dict(out=q[:2]),
                    dict(q=q.transpose(0, 1)), dict(q=q[:0], starts=i32(0, 0))],
           write: [dict(k=k[0]), dict(k=k[:, :1]), dict(v=k.half()), dict(v=k[:2]), dict(k=k.double()), dict(v=k.cpu()),
                   dict(k=k[:, :, ::2])],
           read: [dict(tokens=0), dict(tokens=-1), dict(tokens=(1 << 20) + 1), dict(dtype=torch.int8), dict(dtype=torch.float64)],
           rope: [dict(x=x[0]), dict(x=x[:, :-1]), dict(x=x.double()), dict(x=x.cpu()), dict(positions=pos.long()), dict(positions=pos[:2]),
                  dict(freqs=fr.float()), dict(freqs=freqs_of(2 * D).cuda()), dict(freqs=fr[:3]), dict(q_weight=w.half()),
                  dict(k_weight=w[:16]), dict(eps=0.0), dict(eps=-1.0), dict(norm=False), dict(q_heads=0), dict(k_heads=-1),
                  dict(dim=24), dict(dim=0), dict(q_heads=5), dict(x=x[:0], positions=pos[:0])],
           back: [dict(dq=q[0]), dict(dq=q.half()), dict(dk=k[:2]), dict(dk=k[:, :, :16]), dict(x=x[:, :-8]), dict(out=x[:2]),
                  dict(out=x[:, :-8]), dict(out=x.half()), dict(out=x.t()), dict(norm=False), dict(eps=math.nan)]}
    for call, cases in bad.items():
        for kw in cases + (shared if call in (attend, write, read) else []):
            with pytest.raises(errors):
                call(**kw)
    torch.cuda.synchronize()


# ---------------------------------------------------------------- a layer's run
@pytest.mark.parametrize("t", ["bf16", "fp16"])
def test_a_layer_of_them_together(t):
    """Prompts, then single tokens, then drafts of a layer: the stacked 1.25-bit q/k/v
    product, norm and rotation, the cache, attention, and the output product.  Every
    operator against its definition on what it was given."""
    dtype, Hq, H, D, page, hidden = ref.TYPES[t], 8, 2, 64, 32, 256
    g = ref.gen(125)
    width = (Hq + 2 * H) * D
    packed, alpha = bw.quantize_pack(torch.randn(width, hidden, generator=g).cuda())
    packed_o, alpha_o = bw.quantize_pack(torch.randn(hidden, Hq * D, generator=g).cuda())
    wq, wk = 1 + 0.1 * torch.randn(D, generator=g), 1 + 0.1 * torch.randn(D, generator=g)
    fr = freqs_of(D)
    S = 3
    lens, each = [0] * S, 8
    cache, _, _, _ = sequences([page * each] * S, [1] * S, page, H, D, 126)
    table = torch.randperm(cache.k.shape[0], generator=g)[:S * each].view(S, each).to(torch.int32).cuda()
    blocks = [[ref.Blocks(H, D), ref.Blocks(H, D)] for _ in range(S)]
    for new in ([100, 33, 64], [1, 1, 1], [1, 1, 1], [4, 0, 2]):
        lens = [a + b for a, b in zip(lens, new)]
        T = sum(new)
        pos = torch.cat([torch.arange(n - m, n) for n, m in zip(lens, new)]).to(torch.int32)
        hid = torch.randn(T, hidden, generator=g).cuda()
        xq, s = bw.quantize_act(hid)
        x = bw.gemm_fused(xq, s, packed, alpha, width, hidden, dtype=dtype)
        q, k = bw.qk_norm_rope(x, pos.cuda(), fr.cuda(), Hq, H, D, wq.cuda(), wk.cuda())
        v = x[:, (Hq + H) * D:].unflatten(1, (H, D))
        starts, tl = running(new), i32(*lens)
        bw.cache_write(cache, k, v, table, starts, tl)
        y, lse = bw.cache_attention(q, cache, table, starts, tl, lse=True)
        yq, ys = bw.quantize_act(y.reshape(T, Hq * D).float())
        out = bw.gemm_fused(yq, ys, packed_o, alpha_o, hidden, Hq * D, residual=hid.to(dtype), dtype=dtype)
        assert torch.isfinite(out).all()
        xc = x.cpu()
        check("q", q, *ref.norm_rope(xc[:, :Hq * D].reshape(T, Hq, D), pos, fr, wq, 1e-6, True, False, dtype))
        check("k", k, *ref.norm_rope(xc[:, Hq * D:(Hq + H) * D].reshape(T, H, D), pos, fr, wk, 1e-6, True, False, dtype))
        at = 0
        for i, (n, m) in enumerate(zip(lens, new)):
            if m:
                blocks[i][0].write(n - m, k[at:at + m].cpu().double())
                blocks[i][1].write(n - m, v[at:at + m].cpu().double())
            at += m
        check_attention(q, y, lse, cache, table, lens, new, held_rows(blocks, lens), D ** -0.5, None, 0, page)
