"""Draws that hang on a border, on the GPU: equal logits at the edge between two
bins in different slices of a row; shares of a row that lie next to the uniform
number or to top-p.

A weight is within 2^-45.7 of itself, a sum of weights likewise, so that a share of
a sum is within 2^-44.7 of itself, and a border that lies further than that and
2^-44, at which sums count as equal, from what it is compared with decides as
it does in exact arithmetic. A logarithm is within half a step of float32, 2^-24 of
its value, and 2^-44.7 of that of the share; the oracle's own float64, whose
exponents are rounded at up to 44.4, within 2^-46: 2^-44 for both."""
import math
import random
from decimal import Decimal, getcontext
from fractions import Fraction

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
INF = math.inf
SLICE = 8192        # tokens that one workgroup looks at


def at_edges(dtype, n):
    """(v, T): with c = 4 log2(e) / T, c v is so near to a half-integer that float64 rounds its distance from
    0 and that from about c v itself to different sides of it."""
    log2e, rng, found = 1.4426950408889634, random.Random(1), []
    while len(found) < n:
        v = torch.tensor(-rng.uniform(0.5, 2.0)).to(TYPES[dtype]).item()
        heat = 4 * log2e / ((rng.randint(150, 240) + 0.5) / -v)
        exact = Fraction(v) * Fraction(4 * log2e / heat)
        far, near = (round(float(exact - base)) + base for base in (2, math.floor(exact) + 2))
        if near > far:
            found.append((v, heat))
    return found


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_equal_logits_of_two_slices_at_the_edge_of_a_bin(dtype):
    """The largest logit and one of two equal ones are kept: that of the lowest id, which the smallest number draws.
    The equal ones lie in a slice with the largest and in one of their own."""
    for v, heat in at_edges(dtype, 12):
        say(f"[sample] {dtype} {v.hex()} at temperature {heat.hex()}")
        for first, best, second in ((5, 8000, 9000), (5, 12000, 9000), (5, 20000, 8999), (8191, 8192, 8193), (0, 16383, 16384)):
            z = torch.full((1, 3 * SLICE), -INF, device=DEV)
            z[0, [first, second]], z[0, best] = v, 0.0
            for s in (dict(top_k=2), dict(top_k=2, top_p=1 - 2.0 ** -60), dict(top_k=2, min_p=2.0 ** -63)):
                t, _ = qqe.sample(z.to(TYPES[dtype]), torch.zeros(1, device=DEV), temperature=heat, **s)
                assert int(t) == min(first, best), (v, heat, first, best, second, s)
            # the second one is kept by a third place alone
            z[0, first] = -INF
            z[0, second + 1:second + 3] = v
            t, _ = qqe.sample(z.to(TYPES[dtype]), torch.full((1,), 1 - 2.0 ** -24, device=DEV), temperature=heat, top_k=3)
            assert int(t) == best


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_two_tokens_whose_share_is_next_to_the_number_drawn(dtype):
    """Shares 2^-42.5 to 2^-37 away from a float32 number: the token hangs on the weights' last places."""
    getcontext().prec = 40
    g = np.random.default_rng(0)
    rows, seen = [], 0
    while len(rows) < 96:
        if dtype == "f32":
            x, heat = g.uniform(-0.7, 0.7, 1_000_000).astype(np.float32).astype(np.float64), 1.0
        else:   # few logits, so many temperatures: one for all rows of a call
            x, heat = np.full(1_000_000, 0.5), g.uniform(0.5, 4.0, 1_000_000)
        share = 1 / (1 + np.exp(-x / heat))
        k = np.rint(share * 2 ** 24)
        gap = np.abs(share - k / 2 ** 24) / share
        for i in np.nonzero((gap < 2.0 ** -37) & (gap > 2.0 ** -42))[0][:96]:
            t = heat if dtype == "f32" else float(heat[i])
            p = Decimal(1) / (1 + (-Decimal(float(x[i])) / Decimal(t)).exp())
            u = Decimal(int(k[i])) / Decimal(2 ** 24)
            assert abs(p - u) > p * Decimal(2.0 ** -42.5)
            rows.append((float(x[i]), t, float(u), 0 if p > u else 1))
        seen += 1
        assert seen < 50
    if dtype == "f32":
        z = torch.zeros((len(rows), 2), device=DEV)
        z[:, 0] = torch.tensor([r[0] for r in rows])
        t, _ = qqe.sample(z, torch.tensor([r[2] for r in rows], device=DEV))
        assert t.tolist() == [r[3] for r in rows]
        wide = torch.full((len(rows), 40000), -INF, device=DEV)     # in two slices
        wide[:, 77], wide[:, 33333] = z[:, 0], 0.0
        t, _ = qqe.sample(wide, torch.tensor([r[2] for r in rows], device=DEV), top_k=5)
        assert t.tolist() == [(77, 33333)[r[3]] for r in rows]
    else:
        for x, heat, u, want in rows:
            t, _ = qqe.sample(torch.tensor([[x, 0.0]], dtype=torch.bfloat16, device=DEV), torch.tensor([u], device=DEV), temperature=heat)
            assert int(t) == want


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("vocab,sigma", [(300, 1.0), (5000, 2.0), (40000, 1.0), (40000, 3.0)])
def test_nuclei_that_end_next_to_top_p(dtype, vocab, sigma):
    """top-p just below and just above the share of the first n tokens: n tokens are kept, and n + 1."""
    g = torch.Generator(device=DEV).manual_seed(vocab)
    z = (torch.randn(1, vocab, generator=g, device=DEV) * sigma).to(TYPES[dtype])
    x = np.sort(z[0].double().cpu().numpy())[::-1]
    w = np.exp(x - x[0])
    total = math.fsum(w)
    for n in (1, 2, 7, 40, 120):
        share = math.fsum(w[:n]) / total
        for away, kept in ((-2.0 ** -40, n), (2.0 ** -40, n + 1), (-2.0 ** -38, n), (2.0 ** -38, n + 1)):
            say(f"[sample] {vocab} {dtype}, sigma {sigma}: {n} tokens, {away}")
            for u in (0.0, 0.4, 1 - 2.0 ** -24):
                t, lp = qqe.sample(z, torch.full((1,), u, device=DEV), top_p=share * (1 + away))
                mass = math.fsum(w[:kept])
                want = float(z[0, int(t)].double()) - x[0] - math.log(mass)
                assert abs(float(lp.double()) - want) <= 2.0 ** -24 * abs(want) + 2.0 ** -44, (n, away, u)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,vocab", [(40, 100), (9, 1023), (6, 4096), (4, 32001), (2, 151936)])
def test_random_draws_are_those_of_float64(rows, vocab, dtype):
    """Tokens are equal and logarithms within the bound above, no border is moved: none lies next to one by chance."""
    g = torch.Generator(device=DEV).manual_seed(rows)
    for s in (dict(), dict(temperature=0.7, top_p=0.9), dict(top_k=40), dict(top_p=0.97, min_p=0.01), dict(temperature=1.3, top_k=200, top_p=0.95),
              dict(temperature=3.0, top_p=0.7)):
        say(f"[sample] {rows} x {vocab} {dtype} {s}")
        z = (torch.randn(rows, vocab, generator=g, device=DEV) * 3).to(TYPES[dtype])
        u = torch.rand(rows, generator=g, device=DEV)
        t, lp = qqe.sample(z, u, **s)
        want, want_lp = oa.sample(synth.to_numpy_bits(z), u.cpu().numpy(), **s)
        assert np.array_equal(t.cpu().numpy(), want)
        assert (np.abs(lp.double().cpu().numpy() - want_lp) <= 2.0 ** -24 * np.abs(want_lp) + 2.0 ** -44).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,vocab", [(4500, 8192), (3001, 16385), (9001, 3000), (70001, 60)])
def test_rows_of_several_passes(rows, vocab, dtype):
    """More rows than one pass over the workspace holds: what a call for each few rows draws."""
    need, one = qqe.sample_workspace_bytes(vocab, rows, dtype), qqe.sample_workspace_bytes(vocab, 1, dtype)
    say(f"[sample] {rows} x {vocab} {dtype}: {need} bytes, {one} a row")
    assert need < rows * one
    g = torch.Generator(device=DEV).manual_seed(rows)
    z = (torch.randn(rows, vocab, generator=g, device=DEV) * 3).to(TYPES[dtype])
    u = torch.rand(rows, generator=g, device=DEV)
    k = torch.randint(0, 400, (rows,), generator=g, device=DEV, dtype=torch.int32)
    ws = torch.full((need + 256,), 255, dtype=torch.uint8, device=DEV)
    t, lp = qqe.sample(z, u, top_k=k, top_p=0.9, workspace=ws[:need])
    assert (ws[need:] == 255).all()
    for r in range(0, rows, 997):
        part = slice(r, min(r + 997, rows))
        a, b = qqe.sample(z[part], u[part], top_k=k[part], top_p=0.9)
        assert torch.equal(a, t[part]) and torch.equal(b, lp[part]), r


def test_captured_draws_of_several_passes():
    """A graph whose passes share the workspace, replayed with other logits, eager work between the replays."""
    rows, vocab = 4500, 8192
    g = torch.Generator(device=DEV).manual_seed(11)
    z, u = torch.empty((rows, vocab), dtype=torch.bfloat16, device=DEV), torch.empty(rows, device=DEV)
    out = (torch.empty(rows, dtype=torch.int32, device=DEV), torch.empty(rows, device=DEV))
    ws = torch.full((qqe.sample_workspace_bytes(vocab, rows),), 255, dtype=torch.uint8, device=DEV)
    s = dict(temperature=0.8, top_k=300, top_p=0.9, min_p=0.01)

    def fill():
        z.copy_(torch.randn(rows, vocab, generator=g, device=DEV) * 3)
        u.copy_(torch.rand(rows, generator=g, device=DEV))

    fill()
    qqe.sample(z, u, out=out, workspace=ws, **s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qqe.sample(z, u, out=out, workspace=ws, **s)
    for _ in range(4):
        fill()
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in out]
        want = qqe.sample(z, u, **s)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
