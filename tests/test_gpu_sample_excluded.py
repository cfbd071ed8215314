"""Tokens that are excluded, and rows that a mask leaves little or nothing of, in each
type's own values: infinities of either sign, NaN, the lowest and the largest finite
value. Tokens and logarithms as the float64 oracle's, within the bounds that
test_gpu_sample_borders.py derives."""
import math

import numpy as np
import pytest
import torch

import quantization_quality_eval_amd as qqe
import synth
from oracle import answer as oa
from tests.gpu_util import say

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
INF, NAN = math.inf, math.nan


def rows_of(dtype, vocab):
    """14 rows of that type, none of its values changed by a conversion."""
    lowest, most = torch.finfo(TYPES[dtype]).min, torch.finfo(TYPES[dtype]).max
    g = torch.Generator().manual_seed(vocab)
    z = (torch.randn(14, vocab, generator=g) * 3).to(TYPES[dtype])
    last = vocab - 1
    z[0] = -INF
    z[1] = NAN
    z[2] = INF
    z[3, ::2], z[3, 1::4] = NAN, INF              # a quarter of the tokens is left
    z[4] = -INF
    z[4, last] = -7.0                             # one is
    z[5], z[5, 3] = lowest, 1.0                   # masked by the lowest value
    z[6] = lowest
    z[7], z[7, :5] = -INF, lowest
    z[8, 0] = most
    z[9, :last] = -INF
    z[10], z[10, 1], z[10, 2] = -INF, lowest, most
    z[11] = -1e30
    z[12], z[12, last // 2] = INF, lowest         # the only finite one
    z[13, 7] = INF                                # a row of ordinary ones but for this
    assert torch.isposinf(z[2]).all() and (z[6] == lowest).all() and torch.isfinite(z[6]).all() and (z[5] == lowest).sum() == vocab - 1
    assert torch.isposinf(z[3]).sum() > 0 and torch.isnan(z[3]).sum() > 0 and torch.isposinf(z[12]).sum() == vocab - 1 and z[10, 2] == most
    return z.to(DEV)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("vocab", [9, 1000, 8192, 9000, 40001])
def test_excluded_tokens(vocab, dtype):
    z = rows_of(dtype, vocab)
    for i, s in enumerate([dict(), dict(temperature=0.0), dict(top_k=5), dict(temperature=0.8, top_k=5, top_p=0.9, min_p=0.01),
                           dict(top_p=0.5), dict(min_p=0.3), dict(temperature=1e30, top_p=0.7), dict(temperature=1e-30),
                           dict(temperature=1e38), dict(temperature=INF, top_k=vocab - 1)]):
        for u in (0.0, float(np.float32(0.37)), 1 - 2.0 ** -24):
            say(f"[sample] {vocab} {dtype} {s} {u}")
            t, lp = qqe.sample(z, torch.full((14,), u, device=DEV), **s)
            want, want_lp = oa.sample(synth.to_numpy_bits(z), np.full(14, u), **s)
            t, lp = t.cpu().numpy(), lp.double().cpu().numpy()
            assert np.array_equal(t, want), (s, u)
            none = want < 0
            assert none[:3].all() and none.sum() == 3 and (lp[none] == -INF).all()
            assert (np.abs(lp - want_lp)[~none] <= 2.0 ** -24 * np.abs(want_lp[~none]) + 2.0 ** -44).all(), (s, u)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_excluded_tokens_are_never_drawn(dtype):
    """Rows that differ in their excluded tokens alone give the same draws."""
    g = torch.Generator(device=DEV).manual_seed(2)
    z = (torch.randn(30, 20000, generator=g, device=DEV) * 3).to(TYPES[dtype])
    gone = torch.rand(30, 20000, generator=g, device=DEV) < 0.7
    u = torch.rand(30, generator=g, device=DEV)
    for s in (dict(), dict(top_p=0.9), dict(top_k=100, min_p=0.01)):
        t, lp = qqe.sample(z.masked_fill(gone, -INF), u, **s)
        assert not gone[torch.arange(30), t.long()].any()
        for other in (INF, NAN):
            a, b = qqe.sample(z.masked_fill(gone, other), u, **s)
            assert torch.equal(a, t) and torch.equal(b, lp)
