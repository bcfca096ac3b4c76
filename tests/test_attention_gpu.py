"""The attention operators on the GPU against their definitions in 64 bits."""

import math

import pytest
import torch

import attention_reference as ref
import bit_weight_amd as bw

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)


def check(what, got, want, bound):
    got = got.double().cpu()
    assert got.shape == want.shape, what
    off = (got - want).abs()
    worst = (off / bound).max().item()
    assert torch.isfinite(got).all() and worst <= 1, f"{what}: {worst:.3g} of the bound, off {off.max().item():.3g}"


def freqs_of(R):
    return 10000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64) / max(R, 1))


# ------------------------------------------------------------ norm and rotation
ROPE = [
    # T, Hq, Hk, D, R, interleaved, norm
    (1, 32, 8, 128, 128, False, True), (5, 4, 4, 64, 64, True, True), (7, 3, 1, 80, 32, False, True),
    (33, 12, 4, 96, 96, True, True), (2, 1, 1, 16, 16, False, True), (9, 2, 2, 32, 8, True, True),
    (130, 8, 2, 256, 128, False, True), (3, 5, 3, 112, 0, False, True), (17, 6, 2, 192, 192, False, True),
    (65, 40, 8, 128, 64, True, False), (4, 2, 1, 48, 24, False, False), (300, 7, 7, 64, 56, False, True),
    (2100, 3, 1, 32, 32, False, True),
]


def rope_case(T, Hq, Hk, D, norm, dtype, seed, extra=0):
    g = ref.gen(seed)
    x = torch.randn(T, (Hq + Hk) * D + extra, generator=g) * (0.1 + 3 * torch.rand(T, 1, generator=g))
    w = [1 + 0.3 * torch.randn(D, generator=g) if norm else None for _ in range(2)]
    pos = torch.randint(0, 1 << 20, (T,), generator=g, dtype=torch.int32)
    pos[0] = 0
    return x.to(dtype), w, pos


def cuda(t):
    return None if t is None else t.cuda()


@pytest.mark.parametrize("t", list(ref.TYPES))
@pytest.mark.parametrize("T,Hq,Hk,D,R,interleaved,norm", ROPE)
def test_norm_rope(T, Hq, Hk, D, R, interleaved, norm, t):
    dtype, eps = ref.TYPES[t], 1e-6
    x, w, pos = rope_case(T, Hq, Hk, D, norm, dtype, 1, extra=Hk * D)
    fr = freqs_of(R)
    got = bw.qk_norm_rope(x.cuda(), pos.cuda(), fr.cuda(), Hq, Hk, D, cuda(w[0]), cuda(w[1]), eps, norm, interleaved)
    for name, z, part, wt in (("q", got[0], x[:, :Hq * D].view(T, Hq, D), w[0]),
                              ("k", got[1], x[:, Hq * D:(Hq + Hk) * D].reshape(T, Hk, D), w[1])):
        check(name, z, *ref.norm_rope(part, pos, fr, wt, eps, norm, interleaved, dtype))


@pytest.mark.parametrize("t", list(ref.TYPES))
@pytest.mark.parametrize("T,Hq,Hk,D,R,interleaved,norm", ROPE)
def test_norm_rope_backward(T, Hq, Hk, D, R, interleaved, norm, t):
    dtype, eps = ref.TYPES[t], 1e-6
    x, w, pos = rope_case(T, Hq, Hk, D, norm, dtype, 2, extra=16)
    g = ref.gen(3)
    dq, dk = (torch.randn(T, h, D, generator=g).to(dtype) for h in (Hq, Hk))
    fr = freqs_of(R)
    args = [dq.cuda(), dk.cuda(), x.cuda(), pos.cuda(), fr.cuda(), cuda(w[0]), cuda(w[1]), eps, norm, interleaved]
    dx, dwq, dwk = bw.qk_norm_rope_backward(*args)
    for name, part, dz, wt, dw, to in (("q", x[:, :Hq * D].view(T, Hq, D), dq, w[0], dwq, dx[:, :Hq * D]),
                                       ("k", x[:, Hq * D:(Hq + Hk) * D].reshape(T, Hk, D), dk, w[1], dwk, dx[:, Hq * D:])):
        want, want_w = ref.norm_rope_backward(dz, part, pos, fr, wt, eps, norm, interleaved, dtype)
        check("d" + name, to.reshape(T, -1, D), *want)
        if norm:
            check("dw" + name, dw, *want_w)
        else:
            assert dw is None
    # into rows of a wider gradient, and over x itself: the same bits, the rest left as it was
    wide = torch.full((T, (Hq + Hk) * D + 24), 7.0, dtype=dtype, device="cuda")
    again = bw.qk_norm_rope_backward(*args, out=wide)
    assert torch.equal(wide[:, :(Hq + Hk) * D], dx) and bool((wide[:, (Hq + Hk) * D:] == 7).all())
    args[2] = args[2].clone()
    bw.qk_norm_rope_backward(*args, out=args[2])
    assert torch.equal(args[2][:, :(Hq + Hk) * D], dx) and torch.equal(args[2][:, (Hq + Hk) * D:].cpu(), x[:, (Hq + Hk) * D:])
    if norm:
        assert torch.equal(again[1], dwq) and torch.equal(again[2], dwk)


def test_norm_rope_gradients_against_differences():
    T, Hq, Hk, D, R, eps = 3, 2, 1, 32, 16, 1e-2
    x, w, pos = rope_case(T, Hq, Hk, D, True, torch.float32, 5)
    x = x * 0.2
    fr = freqs_of(R)
    g = ref.gen(6)
    dq, dk = torch.randn(T, Hq, D, generator=g), torch.randn(T, Hk, D, generator=g)

    def loss(x, wq, wk):       # the definition, in 64 bits
        x, total = x.double(), 0.0
        for part, wt, dz in ((x[:, :Hq * D].reshape(T, Hq, D), wq, dq), (x[:, Hq * D:].reshape(T, Hk, D), wk, dk)):
            y = part * ref.inverse_rms(part, eps) * wt.double()
            total += (ref.turn(y, pos, fr, True) * dz.double()).sum().item()
        return total

    got = [v.cpu().double() for v in bw.qk_norm_rope_backward(dq.cuda(), dk.cuda(), x.cuda(), pos.cuda(), fr.cuda(), cuda(w[0]),
                                                              cuda(w[1]), eps, True, True)]
    args, h = [x.double(), w[0].double(), w[1].double()], 1e-5
    for n, (a, d) in enumerate(zip(args, got)):
        flat = a.reshape(-1)
        for i in range(0, flat.numel(), 7):
            ends = []
            for s in (h, -h):
                moved = flat.clone()
                moved[i] += s
                ends.append(loss(*(moved.view(a.shape) if m == n else v for m, v in enumerate(args))))
            slope = (ends[0] - ends[1]) / (2 * h)
            assert abs(slope - d.reshape(-1)[i].item()) <= 1e-4 * (1 + abs(slope)), (n, i)


@pytest.mark.parametrize("t", list(ref.TYPES))
def test_norm_rope_of_extreme_rows(t):
    dtype = ref.TYPES[t]
    top = torch.finfo(dtype).max
    D, fr, eps = 64, freqs_of(64), 1e-6
    x = torch.randn(6, 2 * D, generator=ref.gen(8))
    x[0] = 0.0
    x[1] *= top / 8
    x[2] *= torch.finfo(dtype).tiny * 4
    x[3, :D] = top
    x = x.to(dtype)
    pos = torch.arange(6, dtype=torch.int32) * 1000
    q, k = bw.qk_norm_rope(x.cuda(), pos.cuda(), fr.cuda(), 1, 1, D, eps=eps)
    for z, part in ((q, x[:, :D]), (k, x[:, D:])):
        check("z", z, *ref.norm_rope(part.reshape(6, 1, D), pos, fr, None, eps, True, False, dtype))
    bad = x.clone()
    bad[4, 3], bad[5, 70] = math.nan, math.inf
    q2, k2 = bw.qk_norm_rope(bad.cuda(), pos.cuda(), fr.cuda(), 1, 1, D, eps=eps)
    assert q2[4].isnan().all() and torch.equal(k2[4], k[4]) and torch.equal(q2[:4], q[:4]) and torch.equal(q2[5], q[5])
    assert not torch.isfinite(k2[5]).all()


# --------------------------------------------------------------------- the cache
def sequences(lens, new, page, H, D, seed, spare=2):
    """A cache whose unused parts hold anything, tables of shuffled pages, starts
    and lens."""
    each = [-(-n // page) for n in lens]
    pages = sum(each) + spare
    g = ref.gen(seed)
    order = torch.randperm(pages, generator=g).tolist()
    width = max(max(each), 1)
    table = torch.full((len(lens), width), -5, dtype=torch.int32)
    for i, n in enumerate(each):
        for j in range(n):
            table[i, j] = order.pop()
    cache = bw.kv_cache(pages, page, H, D)
    for c in cache[:2]:
        c.copy_(torch.randint(-128, 128, c.shape, generator=g, dtype=torch.int8))
    for s in cache[2:]:
        s.fill_(math.nan)
    starts = torch.tensor([sum(new[:i]) for i in range(len(new) + 1)], dtype=torch.int32)
    return cache, table.cuda(), starts.cuda(), torch.tensor(lens, dtype=torch.int32).cuda()


def filled(lens, page, H, D, seed, dtype=torch.float32, spread=1.0):
    """Such a cache with whole sequences written at once, and what it should hold."""
    cache, table, starts, tl = sequences(lens, lens, page, H, D, seed)
    g = ref.gen(seed + 1)
    rows = [torch.randn(sum(lens), H, D, generator=g) * (0.3 + spread * torch.rand(sum(lens), H, 1, generator=g)) for _ in range(2)]
    rows = [r.to(dtype) for r in rows]
    bw.cache_write(cache, rows[0].cuda(), rows[1].cuda(), table, starts, tl)
    held = []
    at = 0
    for n in lens:
        pair = []
        for r in rows:
            b = ref.Blocks(H, D)
            b.write(0, r[at:at + n].double())
            pair.append(b)
        held.append(pair)
        at += n
    return cache, table, tl, held


CACHES = [
    # lens, new, page, H, D
    ([1], [1], 16, 1, 16), ([16], [16], 16, 2, 64), ([17, 40], [1, 24], 16, 3, 128), ([100, 0, 33], [7, 0, 33], 32, 2, 80),
    ([64, 65, 63], [1, 2, 3], 64, 1, 256), ([300], [290], 128, 2, 96), ([5] * 70, [1] * 70, 16, 1, 32),
    ([200, 31, 16, 15], [16, 31, 1, 15], 16, 2, 192), ([1030], [6], 1024, 1, 48),
]


@pytest.mark.parametrize("t", list(ref.TYPES))
@pytest.mark.parametrize("lens,new,page,H,D", CACHES)
def test_cache_write_and_read(lens, new, page, H, D, t):
    """In two writes, the second of growing size, through slices of wider rows:
    what is read back is the definition's to the last bit."""
    dtype = ref.TYPES[t]
    cache, table, starts, tl = sequences(lens, new, page, H, D, 11)
    g = ref.gen(12)
    held = [[ref.Blocks(H, D), ref.Blocks(H, D)] for _ in lens]
    for first, count, size in (([0] * len(lens), [a - b for a, b in zip(lens, new)], 0.2), ([a - b for a, b in zip(lens, new)], new, 2.0)):
        T = sum(count)
        if T == 0:
            continue
        rows = (size * torch.randn(T, 2 * H * D + 8, generator=g) * torch.exp(torch.randn(T, 1, generator=g))).to(dtype)
        k, v = rows[:, :H * D].unflatten(1, (H, D)), rows[:, H * D:2 * H * D].unflatten(1, (H, D))
        on = rows.cuda()
        begin = torch.tensor([sum(count[:i]) for i in range(len(count) + 1)], dtype=torch.int32).cuda()
        ends = torch.tensor([a + b for a, b in zip(first, count)], dtype=torch.int32).cuda()
        before = [c.clone() for c in cache]
        for _ in range(2):       # writing the same again changes nothing
            bw.cache_write(cache, on[:, :H * D].unflatten(1, (H, D)), on[:, H * D:2 * H * D].unflatten(1, (H, D)), table, begin, ends)
        at = 0
        for i, n in enumerate(count):
            held[i][0].write(first[i], k[at:at + n].double())
            held[i][1].write(first[i], v[at:at + n].double())
            at += n
        used = torch.zeros(cache.k.shape[0], dtype=torch.bool)
        for i, n in enumerate(lens):
            used[table[i, :-(-n // page)].long().cpu()] = True
        for c, b in zip(cache, before):      # pages of nobody are as they were
            assert torch.equal(c[~used.cuda()].nan_to_num(9.0), b[~used.cuda()].nan_to_num(9.0))
    for out in ref.TYPES.values():
        total = sum(lens)
        all_starts = torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32).cuda()
        got = bw.cache_read(cache, table, all_starts, tl, total, dtype=out)
        for kind in range(2):
            want = torch.cat([held[i][kind].read(n) for i, n in enumerate(lens)])
            assert torch.equal(got[kind].cpu(), want.to(out)), (kind, out)
        part = bw.cache_read(cache, table, starts, tl, sum(new), dtype=out)      # the last ones only
        for kind in range(2):
            want = torch.cat([held[i][kind].read(n)[n - m:] for i, (n, m) in enumerate(zip(lens, new))])
            assert torch.equal(part[kind].cpu(), want.to(out)), (kind, out)


@pytest.mark.parametrize("t", list(ref.TYPES))
def test_cache_token_by_token(t):
    """One token at a time with growing, shrinking, zero, tiny, huge and equal to
    127 steps: scales and values after every write."""
    dtype, H, D = ref.TYPES[t], 2, 32
    info = torch.finfo(dtype)
    sizes = [0.0, 1e-3, info.tiny, 127.0, 126.9, 128.0, 0.5, 1.0, info.max / 2, 1.0, info.max, 3.0, 0.0, 63.5, 1e-6, 2.0, 5.0, 0.0, 1.0, 254.0]
    cache, table, _, _ = sequences([len(sizes)], [1], 16, H, D, 21)
    starts = torch.tensor([0, 1], dtype=torch.int32).cuda()
    held = [ref.Blocks(H, D), ref.Blocks(H, D)]
    g = ref.gen(22)
    for n, size in enumerate(sizes):
        x = [(2 * torch.rand(1, H, D, generator=g) - 1) for _ in range(2)]
        for v in x:
            v[0, 0, 5] = 1.0
        x = [(v.double() * size).to(dtype) for v in x]
        lens = torch.tensor([n + 1], dtype=torch.int32).cuda()
        bw.cache_write(cache, x[0].cuda(), x[1].cuda(), table, starts, lens)
        got = bw.cache_read(cache, table, torch.tensor([0, n + 1], dtype=torch.int32).cuda(), lens, n + 1)
        for kind in range(2):
            held[kind].write(n, x[kind].double())
            assert torch.equal(got[kind].cpu(), held[kind].read(n + 1).float()), (n, kind)


def test_cache_values_that_are_not_finite():
    H, D = 2, 32
    cache, table, starts, lens = sequences([40], [40], 16, H, D, 31)
    k, v = (torch.randn(40, H, D, generator=ref.gen(32)) for _ in range(2))
    k[3, 0, 4], v[20, 1, 0], v[39, 0, 31] = math.nan, math.inf, -math.inf
    bw.cache_write(cache, k.cuda(), v.cuda(), table, starts, lens)
    rk, rv = (x.cpu() for x in bw.cache_read(cache, table, starts, lens, 40))
    bad_k, bad_v = torch.zeros(40, H, dtype=torch.bool), torch.zeros(40, H, dtype=torch.bool)
    bad_k[:16, 0], bad_v[16:32, 1], bad_v[32:, 0] = True, True, True
    for r, x, bad in ((rk, k, bad_k), (rv, v, bad_v)):
        assert r[bad].isnan().all() and torch.isfinite(r[~bad]).all() and (r[~bad] - x[~bad]).abs().max() < 0.05
    # a later token joins a block that is NaN; a new sequence in the same page starts afresh
    one = torch.tensor([0, 1], dtype=torch.int32).cuda()
    bw.cache_write(cache, k[:1].cuda(), v[:1].cuda(), table, one, torch.tensor([41], dtype=torch.int32).cuda())
    assert cache.v_scale.isnan().sum() >= 2
    bw.cache_write(cache, k[5:21].cuda(), v[:16].cuda(), table, torch.tensor([0, 16], dtype=torch.int32).cuda(),
                   torch.tensor([16], dtype=torch.int32).cuda())
    again = bw.cache_read(cache, table, torch.tensor([0, 16], dtype=torch.int32).cuda(), torch.tensor([16], dtype=torch.int32).cuda(), 16)
    assert torch.isfinite(again[0]).all()


def test_cache_positions_without_a_page():
    """Pages out of range, slots past the table and positions below 0 are not
    written, read as NaN and make attention NaN; nothing else changes."""
    H, D, page = 1, 32, 16
    cache, table, _, _ = sequences([64, 64], [64, 64], page, H, D, 41)
    starts = torch.tensor([0, 64, 128], dtype=torch.int32).cuda()
    lens = torch.tensor([64, 64], dtype=torch.int32).cuda()
    k, v = (torch.randn(128, H, D, generator=ref.gen(42)).cuda() for _ in range(2))
    bad = table.clone()
    bad[0, 1], bad[1, 3] = cache.k.shape[0], -1
    before = [c.clone() for c in cache]
    bw.cache_write(cache, k, v, bad, starts, lens)
    for c, b in zip(cache, before):
        for p in (table[0, 1], table[1, 3]):
            assert torch.equal(c[p.long()].nan_to_num(9.0), b[p.long()].nan_to_num(9.0))
    rk, rv = bw.cache_read(cache, bad, starts, lens, 128)
    lost = torch.zeros(128, dtype=torch.bool)
    lost[16:32], lost[112:] = True, True
    assert rk[lost].isnan().all() and rv[lost].isnan().all() and torch.isfinite(rk[~lost]).all() and torch.isfinite(rv[~lost]).all()
    y = bw.cache_attention(k.view(128, 1, D), cache, bad, starts, lens)
    nan = torch.zeros(128, dtype=torch.bool)
    nan[16:64], nan[112:] = True, True
    assert y[nan].isnan().all() and torch.isfinite(y[~nan]).all()
    # longer than the table, and more rows than tokens
    long = torch.tensor([65, 10], dtype=torch.int32).cuda()
    bw.cache_write(cache, k, v, table, starts, long)
    y, lse = bw.cache_attention(k.view(128, 1, D), cache, table, starts, long, lse=True)
    assert y[:64].isnan().all() and lse[:64].isnan().all()
    assert bool((y[64:118] == 0).all()) and bool((lse[64:118] == -math.inf).all()) and torch.isfinite(y[118:]).all()
    rk, _ = bw.cache_read(cache, table, starts, long, 128)
    assert torch.isfinite(rk[:63]).all() and rk[63].isnan().all() and rk[64:118].isnan().all() and torch.isfinite(rk[118:]).all()


# --------------------------------------------------------------------- attention
ATTENTION = [
    # lens, new, page, Hq, H, D, window, sinks
    ([1], [1], 16, 1, 1, 16, None, 0), ([1, 2, 3], [1, 1, 3], 16, 4, 2, 64, None, 0), ([64], [1], 16, 8, 2, 128, None, 0),
    ([65, 63, 1], [1, 1, 1], 32, 4, 1, 128, None, 0), ([300, 7, 0, 129], [1, 3, 0, 2], 16, 6, 2, 80, None, 0),
    ([1000], [1], 64, 32, 8, 128, None, 0), ([700, 40], [5, 40], 128, 7, 1, 96, None, 0), ([130], [130], 16, 3, 3, 32, None, 0),
    ([500, 33], [4, 33], 16, 16, 1, 256, None, 0), ([260], [17], 32, 12, 4, 192, None, 0),
    ([400, 100, 30], [1, 1, 1], 16, 4, 2, 64, 50, 0), ([900], [3], 16, 4, 2, 64, 100, 4), ([900, 70], [70, 70], 32, 2, 1, 48, 65, 70),
    ([600], [6], 64, 20, 1, 112, 1, 1), ([333], [200], 16, 5, 5, 64, 33, 17), ([2000], [2], 16, 3, 1, 64, 128, 300),
    ([257] * 9, [2] * 9, 256, 8, 8, 64, None, 0), ([90], [90], 16, 40, 2, 64, None, 0),
]


def scales_of(cache, table, seq, n, page):
    """The values' scale of each token, [n, H]."""
    t = torch.arange(n)
    return cache.v_scale.cpu()[table[seq].cpu().long()[t // page], :, (t % page) // 16]


@pytest.mark.parametrize("t", list(ref.TYPES))
@pytest.mark.parametrize("lens,new,page,Hq,H,D,window,sinks", ATTENTION)
def test_attention(lens, new, page, Hq, H, D, window, sinks, t):
    dtype = ref.TYPES[t]
    cache, table, tl, held = filled(lens, page, H, D, 51)
    starts = torch.tensor([sum(new[:i]) for i in range(len(new) + 1)], dtype=torch.int32).cuda()
    T = sum(new)
    rows = (2 * torch.randn(T, Hq * D + 16, generator=ref.gen(52))).to(dtype)
    q = rows[:, :Hq * D].unflatten(1, (Hq, D))
    on = rows.cuda()[:, :Hq * D].unflatten(1, (Hq, D))
    y, lse = bw.cache_attention(on, cache, table, starts, tl, window=window, sinks=sinks, lse=True)
    at = 0
    for i, (n, m) in enumerate(zip(lens, new)):
        if m == 0:
            continue
        want, want_lse = ref.attention(q[at:at + m], held[i][0].read(n), held[i][1].read(n), D ** -0.5, window, sinks, dtype,
                                       scales_of(cache, table, i, n, page))
        check("y", y[at:at + m], *want)
        check("lse", lse[at:at + m], *want_lse)
        at += m
    assert torch.equal(y, bw.cache_attention(on, cache, table, starts, tl, window=window, sinks=sinks))      # equal bits


PROMPTS = [
    # lens, new, page, Hq, H, D, window, sinks: many queries a sequence
    ([64], [64], 16, 1, 1, 64, None, 0), ([200], [200], 16, 4, 1, 128, None, 0), ([700, 65, 300], [300, 65, 100], 32, 4, 2, 128, None, 0),
    ([500], [140], 64, 3, 3, 80, None, 0), ([330, 0, 90], [130, 0, 90], 16, 7, 1, 48, None, 0), ([257], [257], 128, 2, 1, 256, None, 0),
    ([400, 128], [129, 128], 16, 6, 2, 192, None, 0), ([600], [400], 16, 2, 1, 64, 70, 5), ([1000], [100], 32, 8, 4, 96, 200, 90),
    ([300], [300], 16, 2, 2, 32, 1, 0), ([150, 1, 500], [150, 1, 200], 16, 16, 1, 112, None, 0), ([90] * 5, [80] * 5, 16, 4, 4, 16, 33, 3),
]


@pytest.mark.parametrize("t", list(ref.TYPES))
@pytest.mark.parametrize("lens,new,page,Hq,H,D,window,sinks", PROMPTS)
def test_attention_of_prompts(lens, new, page, Hq, H, D, window, sinks, t):
    test_attention(lens, new, page, Hq, H, D, window, sinks, t)
