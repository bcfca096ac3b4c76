"""Host-only checks of the feed-forward operators' entry points: every bad
argument is refused before any HIP call, and the plans' workspaces hold."""

import ctypes

import pytest
import torch

import bit_weight_amd as bw

NULL, SHAPE, ALIGN, WS, ARG = -1, -2, -3, -4, -8
FAKE = 0x10000        # 64 KiB-aligned dummy device address (never dereferenced)
BIG = 1 << 40


def _fused(**kw):
    a = dict(x=FAKE, s=FAKE, p=FAKE, al=FAKE, b=None, act=0, r=None, y=FAKE, dt=0, M=1, N=64, K=128, ws=FAKE, wsb=BIG)
    a.update(kw)
    return bw.lib().sherry_gemm_fused(*a.values(), None)


def _glu(**kw):
    a = dict(x=FAKE, s=FAKE, pg=FAKE, ag=FAKE, pu=FAKE, au=FAKE, act=3, h=FAKE, dt=0, M=1, N=64, K=128, ws=FAKE, wsb=BIG)
    a.update(kw)
    return bw.lib().sherry_glu(*a.values(), None)


def _fused_back(**kw):
    a = dict(dy=FAKE, x=FAKE, s=FAKE, p=FAKE, al=FAKE, b=None, act=0, dx=FAKE, da=FAKE, db=FAKE, dt=0, M=1, N=64, K=128,
             ws=FAKE, wsb=BIG)
    a.update(kw)
    return bw.lib().sherry_gemm_fused_backward(*a.values(), None)


def _glu_back(**kw):
    a = dict(dy=FAKE, x=FAKE, s=FAKE, pg=FAKE, ag=FAKE, pu=FAKE, au=FAKE, act=3, dx=FAKE, dg=FAKE, du=FAKE, dt=0, M=1,
             N=64, K=128, ws=FAKE, wsb=BIG)
    a.update(kw)
    return bw.lib().sherry_glu_backward(*a.values(), None)


def _norm(**kw):
    a = dict(x=FAKE, w=FAKE, b=FAKE, eps=1e-5, y=FAKE, mean=FAKE, rstd=FAKE, dt=0, M=1, K=128)
    a.update(kw)
    return bw.lib().sherry_layernorm(*a.values(), None)


def _norm_q(**kw):
    a = dict(x=FAKE, w=FAKE, b=FAKE, eps=1e-5, q=FAKE, s=FAKE, mean=None, rstd=None, dt=0, M=1, K=128)
    a.update(kw)
    return bw.lib().sherry_layernorm_quantize(*a.values(), None)


def _norm_back(**kw):
    a = dict(dy=FAKE, x=FAKE, mean=FAKE, rstd=FAKE, w=FAKE, dx=FAKE, dw=FAKE, db=FAKE, dt=0, M=1, K=128, sc=FAKE, scb=BIG)
    a.update(kw)
    return bw.lib().sherry_layernorm_backward(*a.values(), None)


BAD_SHAPES = [dict(M=0), dict(N=0), dict(K=0), dict(K=100), dict(N=65), dict(M=-1), dict(M=(1 << 20) + 1),
              dict(K=(1 << 20) + 16), dict(N=2 ** 62), dict(M=2 ** 63 - 1)]


@pytest.mark.parametrize("call,pointers,aligned16", [
    (_fused, ("x", "s", "p", "al", "y"), ("x", "p", "y", "r")),
    (_glu, ("x", "s", "pg", "ag", "pu", "au", "h"), ("x", "pg", "pu", "h"))])
def test_product_refusals(call, pointers, aligned16):
    for k in pointers:
        assert call(**{k: None}) == NULL, k
    for kw in BAD_SHAPES:
        assert call(**kw) == SHAPE, kw
    for k in aligned16:
        assert call(**{k: FAKE + 8}) == ALIGN, k
    assert call(s=FAKE + 2) == ALIGN
    assert call(act=6) == ARG and call(act=-1) == ARG and call(dt=3) == ARG and call(dt=-1) == ARG
    query = bw.lib().sherry_glu_workspace_bytes if call is _glu else bw.lib().sherry_gemm_fused_workspace_bytes
    M, N, K = 2, 1024, 8192
    need = query(M, N, K)
    assert need == M * N * 8
    assert call(M=M, N=N, K=K, ws=None) == WS and call(M=M, N=N, K=K, wsb=need - 1) == WS
    assert call(M=M, N=N, K=K, ws=FAKE + 64) == ALIGN
    for kw in BAD_SHAPES:
        assert query(kw.get("M", 1), kw.get("N", 64), kw.get("K", 128)) == 0


@pytest.mark.parametrize("call,pointers,aligned16", [
    (_fused_back, ("dy", "x", "s", "p", "al", "dx"), ("dy", "x", "p", "dx")),
    (_glu_back, ("dy", "x", "s", "pg", "ag", "pu", "au", "dx"), ("dy", "x", "pg", "pu", "dx"))])
def test_backward_refusals(call, pointers, aligned16):
    for k in pointers:
        assert call(**{k: None}) == NULL, k
    for kw in BAD_SHAPES:
        assert call(**kw) == SHAPE, kw
    for k in aligned16:
        assert call(**{k: FAKE + 8}) == ALIGN, k
    assert call(act=6) == ARG and call(act=-1) == ARG and call(dt=3) == ARG
    L = bw.lib()
    query = L.sherry_glu_backward_scratch_bytes if call is _glu_back else L.sherry_gemm_fused_backward_scratch_bytes
    parts = 2 if call is _glu_back else 1
    for M, N, K, dt in ((1, 64, 128, 0), (300, 1100, 2064, 2), (2048, 14336, 4096, 1), (7, 4, 1 << 20, 0)):
        need, rows = query(M, N, K, dt), parts * -(-N // 64)
        # the fp16 terms and the weights' 2-bit form are the least it holds
        assert need >= M * rows * 64 * 2 * (1 if dt == 2 else 2) + -(-K // 128) * rows * 2048
        kw = dict(M=M, N=N, K=K, dt=dt)
        assert call(ws=None, **kw) == WS and call(wsb=need - 1, **kw) == WS and call(ws=FAKE + 64, **kw) == ALIGN
    for kw in BAD_SHAPES:
        assert query(kw.get("M", 1), kw.get("N", 64), kw.get("K", 128), 0) == 0
    assert query(1, 64, 128, 3) == 0


def test_norm_refusals():
    for call, outs in ((_norm, ("y",)), (_norm_q, ("q", "s"))):
        for k in ("x", *outs):
            assert call(**{k: None}) == NULL, k
        assert call(mean=FAKE, rstd=None) == NULL and call(mean=None, rstd=FAKE) == NULL
        for kw in (dict(M=0), dict(K=0), dict(K=6), dict(K=2), dict(M=(1 << 20) + 1), dict(K=(1 << 20) + 4), dict(M=2 ** 62)):
            assert call(**kw) == SHAPE, kw
        for kw in (dict(dt=3), dict(eps=0.0), dict(eps=-1e-5), dict(eps=float("nan")), dict(eps=float("inf"))):
            assert call(**kw) == ARG, kw
        for k in ("x", "w", "b"):
            assert call(**{k: FAKE + 8}) == ALIGN, k
    assert _norm(y=FAKE + 4) == ALIGN and _norm_q(q=FAKE + 2) == ALIGN and _norm_q(s=FAKE + 1) == ALIGN
    for k in ("dy", "x", "mean", "rstd", "dx"):
        assert _norm_back(**{k: None}) == NULL, k
    for k in ("dy", "x", "dx", "w"):
        assert _norm_back(**{k: FAKE + 8}) == ALIGN, k
    assert _norm_back(K=6) == SHAPE and _norm_back(dt=7) == ARG
    need = bw.lib().sherry_layernorm_backward_scratch_bytes(1, 128)
    assert need >= 2 * 128 * 4
    assert _norm_back(sc=None) == WS and _norm_back(scb=need - 1) == WS and _norm_back(sc=FAKE + 64) == ALIGN
    assert bw.lib().sherry_layernorm_backward_scratch_bytes(1, 6) == 0
    assert bw.lib().sherry_layernorm_backward_scratch_bytes(2 ** 62, 128) == 0


def test_workspaces_follow_the_plan():
    """One 64-bit cell per output of a launch (64 tokens at most) where K is
    split, none where it is not, whatever the shape or the override."""
    L = bw.lib()
    for M in (1, 5, 16, 17, 64, 65, 100, 128, 129, 4096, 1 << 20):
        for N, K in ((4, 16), (64, 1 << 20), (4096, 4096), (1100, 2064), (28672, 8192), (1 << 20, 16)):
            for query in (L.sherry_glu_workspace_bytes, L.sherry_gemm_fused_workspace_bytes):
                assert query(M, N, K) in (0, min(M, 64) * N * 8), (M, N, K)
    try:
        bw.plan_override("lut_gemv", rw=2, ch=2, splits=8)
        assert L.sherry_gemm_fused_workspace_bytes(1, 4096, 4096) == 4096 * 8     # as the matrix-core GEMV
    finally:
        bw.plan_override()


def test_python_refusals():
    q, s = torch.zeros((2, 128), dtype=torch.int8), torch.ones(2)
    packed, alpha = torch.zeros(bw.packed_bytes(64, 128), dtype=torch.uint8), torch.ones(64)
    with pytest.raises(RuntimeError):      # not on a GPU
        bw.gemm_fused(q, s, packed, alpha, 64, 128)
    with pytest.raises(RuntimeError):
        bw.glu(q, s, packed, alpha, packed, alpha, 64, 128)
    with pytest.raises(RuntimeError):
        bw.layernorm(torch.zeros(2, 128))
    with pytest.raises(RuntimeError):
        bw.layernorm(torch.zeros(2, 128, dtype=torch.float64))
    for bad in (None, "x", 3):
        with pytest.raises(TypeError):
            bw.gemm_fused(bad, s, packed, alpha, 64, 128)
        with pytest.raises(TypeError):
            bw.layernorm(bad)
    with pytest.raises(TypeError):
        bw.glu(q, s, packed, alpha, packed, alpha, "64", 128)
