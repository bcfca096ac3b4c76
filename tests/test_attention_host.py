"""Host-only checks of the attention operators' entry points: every bad argument
is refused before any HIP call, and the sizes they ask for hold."""

import ctypes

import pytest
import torch

import bit_weight_amd as bw

NULL, SHAPE, ALIGN, WS, ARG = -1, -2, -3, -4, -8
FAKE = 0x10000        # 64 KiB-aligned dummy device address (never dereferenced)
BIG = 1 << 40


class KV(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("k", "v", "k_scale", "v_scale")] + \
               [(n, ctypes.c_int64) for n in ("pages", "page_size", "heads", "dim")]


def _kv(kw):
    c = dict(ck=FAKE, cv=FAKE, cks=FAKE, cvs=FAKE, pages=10, page=32, heads=2, dim=64)
    c.update({k: kw.pop(k) for k in list(kw) if k in c})
    return ctypes.byref(KV(*c.values())) if kw.pop("cache", True) else None


def _rope(**kw):
    a = dict(x=FAKE, xs=384, wq=FAKE, wk=FAKE, eps=1e-6, norm=1, f=FAKE, R=64, inter=0, pos=FAKE, q=FAKE, k=FAKE, dt=0, T=3,
             Hq=4, Hk=2, D=64)
    a.update(kw)
    return bw.lib().sherry_qk_norm_rope(*a.values(), None)


def _rope_back(**kw):
    a = dict(q=FAKE, k=FAKE, x=FAKE, xs=384, wq=FAKE, wk=FAKE, eps=1e-6, norm=1, f=FAKE, R=64, inter=0, pos=FAKE, dx=FAKE,
             dxs=384, dwq=FAKE, dwk=FAKE, dt=0, T=3, Hq=4, Hk=2, D=64, sc=FAKE, scb=BIG)
    a.update(kw)
    return bw.lib().sherry_qk_norm_rope_backward(*a.values(), None)


def _write(**kw):
    kv = _kv(kw)
    a = dict(k=FAKE, ks=128, v=FAKE, vs=128, dt=0, t=FAKE, w=4, st=FAKE, ln=FAKE, S=2, T=3)
    a.update(kw)
    return bw.lib().sherry_cache_write(kv, *a.values(), None)


def _read(**kw):
    kv = _kv(kw)
    a = dict(k=FAKE, v=FAKE, dt=0, t=FAKE, w=4, st=FAKE, ln=FAKE, S=2, T=3)
    a.update(kw)
    return bw.lib().sherry_cache_read(kv, *a.values(), None)


def _attend(**kw):
    kv = _kv(kw)
    a = dict(q=FAKE, qs=256, Hq=4, kv=kv, t=FAKE, w=4, st=FAKE, ln=FAKE, S=2, T=3, scale=0.1, win=0, sinks=0, y=1 << 50, lse=FAKE,
             dt=0, ws=FAKE, wsb=BIG, sc=FAKE, scb=BIG)
    a.update(kw)
    return bw.lib().sherry_cache_attention(*a.values(), None)


BAD_HEADS = [dict(T=0), dict(T=-1), dict(T=(1 << 20) + 1), dict(T=2 ** 62), dict(Hq=0), dict(Hk=0), dict(Hq=1025), dict(Hk=1025),
             dict(Hq=2 ** 62), dict(D=0), dict(D=8), dict(D=72), dict(D=272), dict(D=2 ** 62), dict(R=-8), dict(R=4), dict(R=72),
             dict(xs=376), dict(xs=388), dict(xs=(1 << 30) + 8), dict(xs=-384)]


@pytest.mark.parametrize("call", [_rope, _rope_back])
def test_norm_rope_refusals(call):
    for k in ("x", "f", "pos", "q", "k") + (("dx",) if call is _rope_back else ()):
        assert call(**{k: None}) == NULL, k
    for kw in BAD_HEADS:
        assert call(**kw) == SHAPE, kw
    for kw in (dict(dt=3), dict(dt=-1), dict(eps=0.0), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf"))):
        assert call(**kw) == ARG, kw
    assert call(norm=0) == ARG and call(norm=0, wq=None) == ARG and call(norm=0, wk=None) == ARG      # weights without the norm
    for k in ("x", "q", "k", "wq", "wk"):
        assert call(**{k: FAKE + 8}) == ALIGN, k
    assert call(f=FAKE + 4) == ALIGN and call(pos=FAKE + 2) == ALIGN
    if call is _rope_back:
        assert call(norm=0, wq=None, wk=None) == ARG and call(norm=0, wq=None, wk=None, dwq=None) == ARG
        assert call(dxs=376) == SHAPE and call(dxs=388) == SHAPE
        assert call(dx=FAKE + 8) == ALIGN and call(dwq=FAKE + 2) == ALIGN and call(dwk=FAKE + 2) == ALIGN


def test_norm_rope_scratch():
    """A row of both weights' partial sums for every workgroup, at most two workgroups a CU."""
    L = bw.lib()
    query = L.sherry_qk_norm_rope_backward_scratch_bytes
    for T, Hq, Hk, D in ((1, 1, 1, 16), (8, 32, 8, 128), (8192, 32, 8, 128), (777, 12, 4, 80), (1 << 20, 1024, 1024, 256)):
        need = query(T, Hq, Hk, D)
        assert 2 * D * 4 <= need <= 512 * 2 * D * 4 and need % 256 == 0
        kw = dict(T=T, Hq=Hq, Hk=Hk, D=D, R=0, xs=(Hq + Hk) * D, dxs=(Hq + Hk) * D)
        assert _rope_back(sc=None, **kw) == WS and _rope_back(scb=need - 1, **kw) == WS and _rope_back(sc=FAKE + 64, **kw) == ALIGN
    for bad in ((0, 1, 1, 16), (1, 0, 1, 16), (1, 1, 1025, 16), (1, 1, 1, 24), (2 ** 62, 1, 1, 16)):
        assert query(*bad) == 0


BAD_CACHES = [dict(pages=0), dict(pages=-1), dict(pages=2 ** 62), dict(page=8), dict(page=48), dict(page=2048), dict(page=0),
              dict(heads=0), dict(heads=513), dict(heads=2 ** 62), dict(dim=8), dict(dim=72), dict(dim=272),
              dict(pages=1 << 30), dict(w=0), dict(w=-1), dict(w=(1 << 25) + 1), dict(w=2 ** 62), dict(S=0), dict(S=-1),
              dict(S=(1 << 20) + 1), dict(T=0), dict(T=-1), dict(T=(1 << 20) + 1), dict(T=2 ** 62)]


@pytest.mark.parametrize("call", [_write, _read, _attend])
def test_cache_refusals(call):
    for k in ("ck", "cv", "cks", "cvs", "t", "st", "ln") + (("q", "y") if call is _attend else ("k", "v")):
        assert call(**{k: None}) == NULL, k
    assert call(cache=False) == NULL
    for kw in BAD_CACHES:
        assert call(**kw) == SHAPE, kw
    assert call(dt=3) == ARG and call(dt=-1) == ARG
    for k in ("ck", "cv") + (("q", "y") if call is _attend else ("k", "v")):
        assert call(**{k: FAKE + 8}) == ALIGN, k
    for k in ("cks", "cvs", "t", "st", "ln"):
        assert call(**{k: FAKE + 2}) == ALIGN, k


def test_row_refusals():
    for bad in (120, 132, -128, (1 << 30) + 8):
        assert _write(ks=bad) == SHAPE and _write(vs=bad) == SHAPE, bad
        assert _attend(qs=bad) == SHAPE, bad
    for bad in (0, 3, 5, 1026, -2, 2 ** 62):
        assert _attend(Hq=bad, qs=1 << 20) == SHAPE, bad
    for kw in (dict(scale=float("nan")), dict(scale=float("inf")), dict(win=-1), dict(sinks=-1)):
        assert _attend(**kw) == ARG, kw
    assert _attend(lse=FAKE + 2) == ALIGN
    # the output over the queries, or a part of them
    for y in (FAKE, FAKE + 256, FAKE - 256):
        assert _attend(y=y) == ARG, y


def test_attention_memory():
    L = bw.lib()
    query, need_ws = L.sherry_cache_attention_scratch_bytes, L.sherry_cache_attention_workspace_bytes()
    assert 0 < need_ws <= 1 << 20
    for T, S, Hq, H, D in ((1, 1, 32, 8, 128), (64, 64, 32, 8, 128), (4096, 4, 32, 8, 128), (1 << 20, 1 << 20, 1024, 512, 256),
                           (5, 3, 7, 1, 16)):
        need = query(T, S, Hq, H, D)
        assert 0 < need <= 1 << 28 and need % 256 == 0, (T, S, Hq, H, D)
        kw = dict(T=T, S=S, Hq=Hq, heads=H, dim=D, qs=Hq * D, pages=1)
        assert _attend(sc=None, **kw) == WS and _attend(scb=need - 1, **kw) == WS and _attend(sc=FAKE + 64, **kw) == ALIGN
        assert _attend(ws=None, **kw) == WS and _attend(wsb=need_ws - 1, **kw) == WS and _attend(ws=FAKE + 64, **kw) == ALIGN
    for bad in ((0, 1, 1, 1, 16), (1, 0, 1, 1, 16), (1, 1, 3, 2, 16), (1, 1, 0, 1, 16), (1, 1, 1, 0, 16), (1, 1, 1, 1, 24),
                (1, 1, 513, 513, 16), (2 ** 62, 1, 1, 1, 16), (1, 2 ** 62, 1, 1, 16)):
        assert query(*bad) == 0


def test_python_refusals():
    for bad in ((0, 16, 1, 16), (1, 8, 1, 16), (1, 48, 1, 16), (1, 2048, 1, 16), (1, 16, 0, 16), (1, 16, 1, 24), (1, 16, 1, 272),
                (1, 16, 1, 0)):
        with pytest.raises(ValueError):
            bw.kv_cache(*bad, device="cpu")
    cache = bw.kv_cache(3, 32, 2, 64, device="cpu")
    assert cache.k.shape == (3, 2, 2, 4, 16, 16) and cache.v.shape == cache.k.shape and cache.k_scale.shape == (3, 2, 2)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32)
    table, starts, lens, rows = i32(0, 1)[None], i32(0, 5), i32(9), torch.zeros(5, 2, 64)
    freqs = torch.ones(32, dtype=torch.float64)
    x = torch.zeros(5, 256)
    for call in (lambda: bw.qk_norm_rope(x, i32(0, 1, 2, 3, 4), freqs, 2, 2, 64),
                 lambda: bw.qk_norm_rope_backward(rows, rows, x, i32(0, 1, 2, 3, 4), freqs),
                 lambda: bw.cache_write(cache, rows, rows, table, starts, lens),
                 lambda: bw.cache_read(cache, table, starts, lens, 5),
                 lambda: bw.cache_attention(rows, cache, table, starts, lens)):
        with pytest.raises(RuntimeError):      # not on a GPU
            call()
    for bad in (None, "x", 3):
        with pytest.raises(TypeError):
            bw.qk_norm_rope(bad, i32(0), freqs, 2, 2, 64)
        with pytest.raises(TypeError):
            bw.cache_write(bw.KVCache(bad, *cache[1:]), rows, rows, table, starts, lens)
