"""Gradients of the head norms written over their inputs: refused where they would
overwrite what is still to be read.  The addresses are dummies: where there is a
GPU, which a call that were not refused would reach, nothing here runs."""

import pytest
import torch

import bit_weight_amd as bw
from test_attention_host import ARG, BIG, FAKE

SIZE = {0: 4, 1: 2, 2: 2}      # bytes of a value


pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="dummy addresses")


def back(**kw):
    """Arrays of a call of 3 tokens, 4 + 2 heads of 64, each far from the others. No
    call here is valid: all are refused before the device is looked for."""
    a = dict(q=1 << 40, k=2 << 40, x=3 << 40, xs=384, wq=4 << 40, wk=5 << 40, eps=1e-6, norm=1, f=6 << 40, R=64, inter=0,
             pos=7 << 40, dx=8 << 40, dxs=384, dwq=9 << 40, dwk=10 << 40, dt=0, T=3, Hq=4, Hk=2, D=64, sc=FAKE, scb=BIG)
    a.update(kw)
    return bw.lib().sherry_qk_norm_rope_backward(*a.values(), None)


@pytest.mark.parametrize("dt", SIZE)
def test_overlaps_are_refused(dt):
    row = 384 * SIZE[dt]
    q, k, x = 1 << 40, 2 << 40, 3 << 40
    for dx in (q, q + 16, q - 16, q + 3 * 256 * SIZE[dt] - 16, q - 3 * row + 16):      # over dq or a part of it
        assert back(dx=dx, dt=dt) == ARG, dx - q
    for dx in (k, k + 16, k + 3 * 128 * SIZE[dt] - 16, k - 3 * row + 16):
        assert back(dx=dx, dt=dt) == ARG, dx - k
    # rows of x other than the own, or a part of them
    for dx in (x + 16, x - 16, x + row, x - row, x + 2 * row, x + 2 * row + 16, x - 3 * row + 16):
        assert back(dx=dx, dt=dt) == ARG, dx - x
    assert back(dx=x, dxs=392, dt=dt) == ARG and back(dx=x, xs=392, dt=dt) == ARG      # other rows than x's
    wide = 1024
    assert back(dx=x + 368 * SIZE[dt], xs=wide, dxs=wide, dt=dt) == ARG              # columns that begin in x's
    assert back(dx=x - 368 * SIZE[dt], xs=wide, dxs=wide, dt=dt) == ARG
    assert back(dx=x + (wide - 368) * SIZE[dt], xs=wide, dxs=wide, dt=dt) == ARG     # or reach into its next row's
    for name in ("wq", "wk", "f", "pos"):
        at = dict(wq=4, wk=5, f=6, pos=7)[name] << 40
        assert back(dx=at, dt=dt) == ARG and back(dx=at - 3 * row + 16, dt=dt) == ARG, name
    # (the norm without weights, the rotation alone)
    assert back(dx=x + 16, wq=None, wk=None, dt=dt) == ARG
    assert back(dx=q + 16, wq=None, wk=None, dwq=None, dwk=None, norm=0, x=None, dt=dt) == ARG
