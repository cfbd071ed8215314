"""The order of beam selection at the edge of what float32 normalisers can tell:
near ties that continue behind the last place, rows that rise for many tiles,
logits whose range passes float32's, and scores of long outputs.

Tolerances. A score s + z - lse is formed in float64 and rounded once to
float32: 2^-24 of itself. lse is off by at most 2^-24 (24 + log2 V), the bound
that the selection's own order rests on: an exponential's argument is rounded
once (2^-24 of itself; weighted by the probabilities the arguments average at
most log2 V + 2 binary units, of ln 2 nats each), the exponential by one step
(2), no value passes through more than 10 float32 additions (10), the logarithm
by 3 binary units (2.1), log2 e by a quarter of the entropy (0.16 log2 V):
16 + 0.86 log2 V in all. Rescalings are by powers of two and exact."""
import numpy as np
import pytest
import torch

import quantization_quality_eval_amd as qqe
import synth
from oracle import vocab as ov
from tests.gpu_util import say

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
UNIT = 2.0 ** -24


def same_choice(got, want, ctx):
    s, p, t, f = (x.cpu().numpy() for x in got)
    ws, wp, wt, wf = want
    bad = np.unique(np.argwhere((p != wp) | (t != wt))[:, 0])
    assert bad.size == 0, (f"{ctx}: {bad.size} of {len(p)} items differ, e.g. item {bad[0]}: beams {p[bad[0]].tolist()} "
                           f"tokens {t[bad[0]].tolist()}, expected {wp[bad[0]].tolist()} {wt[bad[0]].tolist()}")
    assert np.array_equal(f, wf), ctx


def choose_and_compare(z, scores, k, ctx, finished=None, eos=-1):
    say(f"[beam order] {ctx} {tuple(scores.shape)} k={k} V={z.shape[1]} {z.dtype}")
    got = qqe.beam_select(z, scores, k, finished=finished, eos_token=eos)
    torch.cuda.synchronize()
    want = ov.beam_select(synth.to_numpy_bits(z), scores.cpu().numpy(), k,
                          None if finished is None else finished.cpu().numpy(), eos)
    same_choice(got, want, ctx)
    return got, want


def with_equal_tops(items, beams, vocab, copies, dtype, seed):
    """Rows whose largest logit stands at `copies` places."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    z = torch.randn(items * beams, vocab, generator=g, device=DEV).mul_(3.0)
    at = torch.rand(items * beams, vocab, generator=g, device=DEV).argsort(1)[:, :copies]
    top = z.amax(1, keepdim=True) + 0.25
    return z.scatter_(1, at, top.expand(-1, copies)).to(TYPES[dtype])


# with 700 copies more candidates are tied than the merge ranks at once
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("copies,k", [(2, 1), (3, 2), (9, 1), (9, 7), (700, 1), (700, 5)])
def test_equal_beams_with_equal_tops(copies, k, dtype):
    """Equal beams of equal score: the first k are the lowest beam's, although the
    candidates that decide it stand behind place k + 1."""
    items, beams, vocab = 200, 3, 3001
    z = with_equal_tops(items, beams, vocab, copies, dtype, seed=copies)
    z = z.view(items, beams, vocab)[:, :1].expand(items, beams, vocab).reshape(items * beams, vocab).contiguous()
    scores = torch.full((items, beams), -0.75, device=DEV)
    choose_and_compare(z, scores, k, f"equal beams, {copies} equal tops")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("copies,k", [(2, 1), (2, 3), (3, 2), (9, 1), (9, 12), (700, 1), (700, 5)])
def test_near_equal_beams_with_equal_tops(copies, k, dtype):
    """Beams whose best candidates differ by less than a float32 normaliser can
    tell, each several times: the order is that of the float64 scores."""
    items, beams, vocab = 200, 4, 3001
    z = with_equal_tops(items, beams, vocab, copies, dtype, seed=50 + copies)
    zd = z.double().cpu().numpy()
    best = (zd.max(1) - ov.log_normalisers(zd)).reshape(items, beams)
    s = (np.float32(-0.25) + best[:, :1] - best).astype(np.float32)   # leaves gaps of up to half a step
    scores = torch.tensor(s, device=DEV)
    choose_and_compare(z, scores, k, f"near-equal beams, {copies} equal tops")


def test_finished_beams_next_to_equal_tops():
    """A finished beam's score against a live beam's candidates of nearly that score."""
    items, beams, vocab = 200, 3, 3001
    z = with_equal_tops(items, beams, vocab, 4, "bf16", seed=3)
    zd = z.double().cpu().numpy()
    best = (zd.max(1) - ov.log_normalisers(zd)).reshape(items, beams)
    s = (np.float32(-0.25) + best[:, :1] - best).astype(np.float32)
    fin = torch.zeros(items, beams, dtype=torch.uint8, device=DEV)
    fin[:, 1] = 1
    s[:, 1] = (s[:, 0] + best[:, 0]).astype(np.float32)
    for k in (1, 2, 4, 5):
        choose_and_compare(z, torch.tensor(s, device=DEV), k, "finished beams", fin, 11)


# ---- rows that rise for many tiles of one slice ----------------------------

STEPS = [1e-5, 1e-4, 1e-3, 1e-2, 1e-1]
ROWS = 8192   # from here on one wave reads a whole row


def rising(vocab, step, seed):
    """float32 logits that rise by `step` from one tile of 1024 to the next."""
    g = np.random.default_rng(seed)
    tile = np.arange(vocab) // 1024
    return (step * (tile + 0.25 * g.random(vocab)) - 3.0).astype(np.float32)


def many_rows(vocab, beams):
    """Logits of 8192 rows of which only the ones that are filled are read: the others' beams are empty."""
    z = torch.empty(ROWS, vocab, device=DEV)
    return z, torch.full((ROWS // beams, beams), float("-inf"), device=DEV)


@pytest.mark.parametrize("vocab", [65536, 262144, 1 << 20])
def test_normaliser_of_rising_rows(vocab):
    z, scores = many_rows(vocab, 1)
    rows = [rising(vocab, st, i) for i, st in enumerate(STEPS)]
    rows += [r[::-1].copy() for r in rows]
    for i, r in enumerate(rows):
        z[i] = torch.from_numpy(r).to(DEV)
        scores[i] = 0.0
    say(f"[beam order] rising rows of {vocab}")
    s, p, t, _ = (x.cpu().numpy() for x in qqe.beam_select(z, scores, 2))
    for i, r in enumerate(rows):
        x = r.astype(np.float64)
        lse = ov.log_normalisers(x[None])[0]
        order = np.lexsort((np.arange(vocab), -x))[:2]
        assert t[i].tolist() == order.tolist() and p[i].tolist() == [0, 0]
        want = x[order] - lse
        err = np.abs(s[i].astype(np.float64) - want)
        tol = UNIT * (np.abs(want) + 24 + np.log2(vocab))
        assert (err <= tol).all(), f"row {i}: off by {(err / UNIT).max():.0f} units, bound {(tol / UNIT).max():.0f}"


def test_order_of_rising_beams():
    """A rising row against the same logits falling, the scores a few steps apart
    either way: the candidates stand in the order of the scores."""
    vocab = 1 << 20
    z, scores = many_rows(vocab, 2)
    gaps = [-61, -13, 13, 61]   # odd: never a difference of two logits
    items, want = 0, []
    for i, st in enumerate(STEPS):
        r = rising(vocab, st, i)
        both = np.stack([r, r[::-1]])
        for gap in gaps:
            s = np.array([[-0.5, -0.5 + gap * UNIT]], np.float32)
            z[2 * items:2 * items + 2] = torch.from_numpy(both).to(DEV)
            scores[items] = torch.from_numpy(s[0]).to(DEV)
            want.append(ov.beam_select(both, s, 2))
            items += 1
    say(f"[beam order] rising and falling beams of {vocab}")
    got = qqe.beam_select(z, scores, 2)
    assert (got[1][items:] == -1).all()
    same_choice([x[:items] for x in got], [np.concatenate(x) for x in zip(*want)], "rising and falling beams")


# ---- ranges past float32's ---------------------------------------------------

def compare_far(z, scores, k, ctx):
    """As above; a score past float32's range is rounded to -inf and keeps its parent and token."""
    got, want = choose_and_compare(z, scores, k, ctx)
    s, ws = got[0].cpu().numpy(), want[0]
    with np.errstate(over="ignore"):
        w32 = ws.astype(np.float32)
    far = ~np.isfinite(w32)
    assert np.array_equal(s[far], w32[far]), ctx
    tol = UNIT * (np.abs(ws[~far]) + 24 + np.log2(z.shape[1]))
    assert (np.abs(s[~far].astype(np.float64) - ws[~far]) <= tol).all(), ctx


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("vocab", [3000, 3001])
def test_candidates_far_below_the_best(vocab, dtype):
    """A token of the type's lowest value beside 1e38, so that its score lies past
    float32's range: it is chosen when nothing else is left, wherever it stands."""
    low, inf = torch.finfo(TYPES[dtype]).min, float("inf")
    places = [0, 1, 40, 63, 64, 127, 1500, 2047, 2999]
    z = torch.full((2 * len(places), vocab), -inf, device=DEV)
    for i, at in enumerate(places):
        z[2 * i, [200, 1400]] = 1e38
        z[2 * i, at] = low
        z[2 * i + 1, 2500] = 3.0e38
        z[2 * i + 1, [at, (at + 700) % 2500]] = low
    scores = torch.full((len(places), 2), -1.0, device=DEV)
    scores[::2, 1] = -inf
    for k in (2, 3, 4, 6, 8):
        compare_far(z.to(TYPES[dtype]), scores, k, "far below the best")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_scores_and_normalisers_of_any_size(dtype):
    """score - lse passes float32's range either way while the sums do not."""
    vocab, sizes = 2050, [0.0, 1.0, 1e30, 3e38]
    pairs = [(a * s, b * t) for a in sizes for b in sizes for s in (-1, 1) for t in (-1, 1)]
    g = torch.Generator(device=DEV).manual_seed(8)
    z = torch.randn(2 * len(pairs), vocab, generator=g, device=DEV)
    scores = torch.zeros(len(pairs), 2, device=DEV)
    for i, (score, base) in enumerate(pairs):
        z[2 * i] += base
        scores[i, 0] = score
        scores[i, 1] = score if i % 2 else -5.0
    z = z.to(TYPES[dtype])
    for k in (1, 6, 64):
        compare_far(z, scores, k, "any size")


# ---- scores of long outputs --------------------------------------------------

@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("score", [-60.0, -600.0, -1200.0, -5000.0, -40000.0])
def test_scores_of_long_outputs(score, dtype):
    """Beams that have generated hundreds of tokens."""
    g = torch.Generator(device=DEV).manual_seed(13)
    z = torch.randn(12, 50001, generator=g, device=DEV).mul_(3.0).to(TYPES[dtype])
    scores = score - (torch.rand(3, 4, generator=g, device=DEV) * 6).sort(1).values
    for k in (1, 4, 16):
        compare_far(z, scores, k, f"scores of {score}")


def test_scores_of_long_outputs_cost_no_more():
    """The candidates that are ranked are the ones near the k-th best, however far
    the scores lie from zero: a bound of 16 bits let nearly all groups pass at -600
    and took 130 times as long."""
    g = torch.Generator(device=DEV).manual_seed(14)
    z = torch.randn(128, 151936, generator=g, device=DEV).mul_(3.0).to(torch.bfloat16)
    beams = -(torch.rand(32, 4, generator=g, device=DEV) * 6).sort(1).values

    def best_of(scores):
        times = []
        for _ in range(12):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            qqe.beam_select(z, scores, 8)
            b.record()
            b.synchronize()
            times.append(a.elapsed_time(b))
        return sorted(times)[3]

    near = best_of(beams)
    for score in (-600.0, -1200.0, -5000.0):
        far = best_of(beams + score)
        say(f"[beam order] scores of {score}: {far * 1e3:.0f} us, near zero {near * 1e3:.0f} us")
        assert far < 5 * near
