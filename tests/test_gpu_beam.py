"""Beam selection on the GPU against the float64 oracle: chosen parents, tokens
and finished flags equal, scores within their rounding.

Score tolerance. A score s + z - lse is formed in float64 and rounded once to
float32: half a step, 2^-24 |score|. The normaliser is a float32 sum: an
argument z log2 e - M is rounded once (2^-24 of itself; weighted by the
probabilities the arguments average at most log2 V, and one binary unit is ln 2
in nats), an exponential by one step (2 x 2^-24), and no value passes through
more than 60 float32 additions: lse is off by at most 2^-24 (64 + log2 V)."""
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


def norm_tol(vocab):
    return 2.0 ** -24 * (64 + np.log2(vocab))


def check(got, want, vocab, ctx=""):
    s, p, t, f = (x.cpu().numpy() for x in got)
    ws, wp, wt, wf = want
    assert np.array_equal(p, wp), f"{ctx}: parents differ at {np.argwhere(p != wp)[:4].tolist()}"
    assert np.array_equal(t, wt), f"{ctx}: tokens differ at {np.argwhere(t != wt)[:4].tolist()}"
    assert np.array_equal(f, wf), f"{ctx}: finished flags differ"
    none = np.isneginf(ws)
    assert np.isneginf(s[none]).all(), ctx
    err = np.abs(s[~none].astype(np.float64) - ws[~none])
    tol = 2.0 ** -24 * np.abs(ws[~none]) + norm_tol(vocab)
    assert (err <= tol).all(), f"{ctx}: score off by {err.max()}"


def make(items, beams, vocab, dtype, seed=0, sigma=3.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    z = torch.randn(items * beams, vocab, generator=g, device=DEV).mul_(sigma).to(TYPES[dtype])
    scores = -(torch.rand(items, beams, generator=g, device=DEV) * 6).sort(1).values
    return z, scores, g


def run_and_check(z, scores, k, finished=None, eos=-1, ctx="", **kw):
    say(f"[beam] {ctx} {tuple(scores.shape)} k={k} V={z.shape[-1]} {z.dtype}")
    got = qqe.beam_select(z, scores, k, finished=finished, eos_token=eos, **kw)
    torch.cuda.synchronize()
    want = ov.beam_select(synth.to_numpy_bits(z.reshape(-1, z.shape[-1])), scores.cpu().numpy(), k,
                          None if finished is None else finished.cpu().numpy(), eos)
    check(got, want, z.shape[-1], ctx)
    return got


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("items,beams,k,vocab", [
    (1, 1, 1, 1), (2, 1, 3, 2), (3, 2, 5, 7), (2, 3, 8, 63), (2, 4, 8, 64), (3, 2, 64, 65), (2, 64, 64, 130),
    (5, 3, 6, 1000), (1, 4, 4, 2048), (2, 4, 16, 2049), (7, 2, 64, 4099), (1, 5, 10, 32001), (1, 1, 64, 151936),
    (3, 4, 8, 151936), (40, 1, 2, 20000), (1, 64, 64, 8191)])
def test_shapes(items, beams, k, vocab, dtype):
    z, scores, _ = make(items, beams, vocab, dtype, seed=vocab + k)
    run_and_check(z, scores, k, eos=vocab // 2, ctx="shapes")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_many_rows(dtype):
    """More workgroups than the chip holds at once."""
    z, scores, _ = make(700, 3, 1500, dtype, seed=3)
    run_and_check(z, scores, 6, ctx="many rows")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("vocab", [50, 5000, 40001])
def test_excluded_tokens(vocab, dtype):
    """Masks that leave many, few, one and no tokens of a row; NaN and both
    infinities among the excluded; rows of the type's lowest value."""
    z, scores, g = make(12, 2, vocab, dtype, seed=vocab)
    inf, lowest = float("inf"), torch.finfo(TYPES[dtype]).min
    z[0:4][torch.rand(4, vocab, generator=g, device=DEV) < 0.9] = -inf
    z[4] = -inf
    z[5] = float("nan")
    z[6] = -inf
    z[6, vocab - 1] = 2.5
    z[7] = inf
    z[7, 0] = -1.0
    z[8, ::2] = float("nan")
    z[8, 1] = inf
    z[9, vocab // 2:] = inf
    z[10] = -inf   # an item with no candidate at all
    z[11] = float("nan")
    z[12] = lowest
    z[13] = lowest
    z[13, 3] = 0.0
    z[14, 5:] = lowest
    z[15] = -inf
    z[15, :3] = lowest
    z[16] = torch.finfo(TYPES[dtype]).max
    z[17, ::3] = torch.finfo(TYPES[dtype]).max
    z[18] = z[18] * 1e-30
    z[19] = 0.0
    z[19, ::2] = -0.0
    run_and_check(z, scores, 9, eos=0, ctx="excluded")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("vocab,k", [(70, 64), (9000, 33), (30011, 64), (151936, 8)])
def test_ties(vocab, k, dtype):
    """Few distinct logits, flat rows, rising and falling rows, equal beams."""
    z, scores, g = make(6, 2, vocab, dtype, seed=k)
    z[0:2] = torch.randint(-2, 3, (2, vocab), generator=g, device=DEV).to(z.dtype)
    z[2:4] = 1.25
    z[4] = torch.linspace(-4, 4, vocab, device=DEV).to(z.dtype)
    z[5] = torch.linspace(4, -4, vocab, device=DEV).to(z.dtype)
    z[7] = z[6]
    scores[3] = -1.0     # equal beams of equal score: every candidate is tied with the other beam's
    z[9] = 0.0
    z[9, vocab // 3] = 20.0
    z[8] = z[9]
    scores[4] = -2.0
    z[10, -k:] = 9.0
    run_and_check(z, scores, k, ctx="ties")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_finished_and_empty_beams(dtype):
    z, scores, _ = make(8, 4, 3001, dtype, seed=8)
    fin = torch.zeros(8, 4, dtype=torch.uint8, device=DEV)
    fin[0, 1] = 1
    fin[1] = 1
    fin[2, ::2] = 255
    scores[3, 1:] = float("-inf")
    scores[4] = float("-inf")
    scores[5, 0] = float("nan")
    scores[5, 1] = float("inf")
    scores[6, 2] = float("-inf")
    fin[6, 2] = 1                  # finished and empty: empty
    scores[7] = -1e30              # adding a log-probability changes nothing
    z[4 * 1] = float("nan")        # a finished beam's logits are not looked at
    run_and_check(z, scores, 6, fin, 17, ctx="finished")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_first_step_and_greedy(dtype):
    z, scores, _ = make(5, 4, 10007, dtype, seed=2)
    scores[:, 0] = 0
    scores[:, 1:] = float("-inf")
    run_and_check(z, scores, 4, ctx="first step")
    greedy = qqe.beam_select(z, torch.zeros(20, 1, device=DEV), 1)
    assert torch.equal(greedy[2][:, 0].long(), z.float().argmax(1))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_near_ties_across_beams(dtype):
    """Two beams whose best candidates differ by less than a float32 normaliser
    can tell, in either direction: the order is that of the float64 scores."""
    items, vocab = 300, 3000
    z, scores, _ = make(items, 2, vocab, dtype, seed=11)
    zd = z.double().cpu().numpy()
    lse = ov.log_normalisers(zd).reshape(items, 2)
    best = zd.max(1).reshape(items, 2) - lse
    s0 = np.float32(-0.25)
    s1 = (s0 + best[:, 0] - best[:, 1]).astype(np.float32)  # rounding leaves gaps of up to half a step
    scores = torch.tensor(np.stack([np.full(items, s0), s1], 1), device=DEV)
    gap = np.abs(s0 + best[:, 0] - (s1.astype(np.float64) + best[:, 1]))
    assert (gap < 5e-7).all() and (gap < 5e-8).mean() > 0.2
    run_and_check(z, scores, 3, ctx="near ties")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("scale", [1e-3, 40.0, 3e4, 1e37])
def test_logits_of_any_size(scale, dtype):
    z, scores, _ = make(4, 3, 6000, dtype, seed=5, sigma=scale)
    z[0] += scale * 50
    run_and_check(z, scores, 6, ctx=f"sigma {scale}")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_strides_and_alignments(dtype):
    items, beams, vocab = 3, 4, 9001
    z, scores, g = make(items, beams, vocab, dtype, seed=6)
    for pad, shift in ((7, 0), (0, 1), (8, 3), (64, 0), (5, 5)):
        buf = torch.full((items * beams * (vocab + pad) + shift,), 50.0, dtype=z.dtype, device=DEV)
        view = buf[shift:].view(items * beams, vocab + pad)[:, :vocab]
        view.copy_(z)
        run_and_check(view, scores, 8, ctx=f"pad {pad} shift {shift}")
    run_and_check(z.view(items, beams, vocab), scores, 8, ctx="3-d")
    wide = torch.full((items, beams, vocab + 3), 60.0, dtype=z.dtype, device=DEV)
    wide[..., :vocab] = z.view(items, beams, vocab)
    run_and_check(wide[..., :vocab], scores, 8, ctx="3-d padded")


def test_rows_past_32_bit_offsets():
    """Rows 2^27 elements apart: the last ones start past 2^32 elements."""
    rows, vocab, stride = 36, 5003, 1 << 27
    buf = torch.empty(stride * (rows - 1) + vocab, dtype=torch.bfloat16, device=DEV)
    view = buf.as_strided((rows, vocab), (stride, 1))
    g = torch.Generator(device=DEV).manual_seed(4)
    view.copy_(torch.randn(rows, vocab, generator=g, device=DEV).mul_(3))
    scores = -torch.rand(12, 3, generator=g, device=DEV)
    run_and_check(view, scores, 6, ctx="far rows")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_outputs_in_place_and_untouched_neighbours(dtype):
    items, beams, vocab = 9, 5, 4000
    z, scores, _ = make(items, beams, vocab, dtype, seed=9)
    fin = torch.zeros(items, beams, dtype=torch.uint8, device=DEV)
    fin[::2, 1] = 1
    want = qqe.beam_select(z, scores, finished=fin, eos_token=3)
    s, f = scores.clone(), fin.clone()
    parents = torch.full((items + 2, beams), 77, dtype=torch.int32, device=DEV)
    tokens = torch.full((items + 2, beams), 77, dtype=torch.int32, device=DEV)
    nbytes = qqe.beam_workspace_bytes(vocab, items, beams, beams, dtype)
    ws = torch.full((nbytes + 64,), 171, dtype=torch.uint8, device=DEV)
    got = qqe.beam_select(z, s, finished=f, eos_token=3, out=(s, parents[1:-1], tokens[1:-1], f), workspace=ws[:nbytes])
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    for x in (parents, tokens):
        assert (x[0] == 77).all() and (x[-1] == 77).all()
    assert (ws[nbytes:] == 171).all()
    with pytest.raises(ValueError, match="workspace"):
        qqe.beam_select(z, scores, workspace=ws[:nbytes - 1])


@pytest.mark.parametrize("junk", [0.0, float("inf"), float("-inf"), float("nan"), 3e38])
def test_whatever_the_workspace_holds(junk):
    """Finished and empty beams leave their part of the workspace unwritten:
    what it held before does not show."""
    z, scores, _ = make(5, 4, 6000, "bf16", seed=14)
    fin = torch.zeros(5, 4, dtype=torch.uint8, device=DEV)
    fin[0, 1], fin[1], fin[2, 0] = 1, 1, 1
    scores[2, 3], scores[3], scores[4, :3] = float("-inf"), float("-inf"), float("nan")
    nbytes = qqe.beam_workspace_bytes(6000, 5, 4, 4, "bf16")
    ws = torch.full(((nbytes + 3) // 4,), junk, device=DEV).view(torch.uint8)
    run_and_check(z, scores, 4, fin, 9, ctx=f"workspace of {junk}", workspace=ws)


def test_threads_on_streams_of_their_own():
    """Four threads at once, each on its own stream, some with equal beams (rows
    taken again in float64): each gets what it gets alone."""
    import threading
    cases = []
    for i in range(4):
        z, scores, _ = make(3 + i, 3, 5000 + 7 * i, ("f32", "bf16")[i % 2], seed=30 + i)
        if i > 1:
            z[1], scores[0, 1] = z[0], scores[0, 0]
        cases.append((z, scores, qqe.beam_select(z, scores, 6)))
    torch.cuda.synchronize()
    bad = []

    def work(z, scores, want):
        stream = torch.cuda.Stream()
        for _ in range(25):
            got = qqe.beam_select(z, scores, 6, stream=stream)
            stream.synchronize()
            if not all(torch.equal(a.cpu(), b.cpu()) for a, b in zip(got, want)):
                bad.append(tuple(z.shape))

    threads = [threading.Thread(target=work, args=c) for c in cases]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert not bad


def test_same_bits_every_time_and_on_another_stream():
    z, scores, _ = make(16, 4, 151936, "bf16", seed=10)
    first = qqe.beam_select(z, scores, 8)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(3):
        again = qqe.beam_select(z, scores, 8)
        other = qqe.beam_select(z, scores, 8, stream=side)
        torch.cuda.synchronize()
        for a, b, c in zip(first, again, other):
            assert torch.equal(a, b) and torch.equal(a, c)


def test_captured_and_replayed():
    """A graph of two steps, replayed on changing inputs with eager calls of the
    same sizes in between."""
    items, beams, vocab = 6, 4, 20001
    z, scores, g = make(items, beams, vocab, "bf16", seed=12)
    s, f = scores.clone(), torch.zeros(items, beams, dtype=torch.uint8, device=DEV)
    qqe.beam_select(z, scores, finished=f, eos_token=1)   # loads the kernels before the capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a = qqe.beam_select(z, s, finished=f, eos_token=1)
        b = qqe.beam_select(z, a[0], finished=a[3], eos_token=1)
    for step in range(4):
        z.copy_(torch.randn(items * beams, vocab, generator=g, device=DEV).mul_(3))
        s.copy_(-torch.rand(items, beams, generator=g, device=DEV))
        say(f"[beam] replay {step}")
        graph.replay()
        torch.cuda.synchronize()
        ea = qqe.beam_select(z, s, finished=f, eos_token=1)
        eb = qqe.beam_select(z, ea[0], finished=ea[3], eos_token=1)
        torch.cuda.synchronize()
        for x, y in zip((*a, *b), (*ea, *eb)):
            assert torch.equal(x, y)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_as_many_items_as_a_call_takes(dtype):
    """2^22 items of one beam: more workgroups than one launch may have."""
    items, vocab = 1 << 22, 8
    g = torch.Generator(device=DEV).manual_seed(1)
    z = torch.randn(items, vocab, generator=g, device=DEV).to(TYPES[dtype])
    s, p, t, f = qqe.beam_select(z, torch.zeros(items, 1, device=DEV), 2)
    logp = torch.log_softmax(z.double(), 1)
    top = z.float().max(1)
    assert torch.equal(t[:, 0].long(), top.indices) and not p.any() and not f.any()
    assert ((s[:, 0].double() - logp.gather(1, top.indices[:, None])[:, 0]).abs() <= 2.0 ** -24 * 8 + norm_tol(vocab)).all()
    with pytest.raises(qqe.KldEvalError, match="4194304"):
        qqe.beam_select(torch.zeros(items + 1, 1, device=DEV), torch.zeros(items + 1, 1, device=DEV))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("items,beams,k,vocab", [(2, 12, 24, 151936), (1, 64, 8, 32000), (1, 16, 64, 262144),
                                                 (2, 1, 64, 5000), (3, 2, 2, 600000)])
def test_many_groups(items, beams, k, vocab, dtype):
    """More group maxima than a workgroup keeps in registers, and few of them
    for a large k."""
    z, scores, g = make(items, beams, vocab, dtype, seed=21)
    run_and_check(z, scores, k, eos=3, ctx="many groups")
    z[:, vocab // 3:] = float("-inf")
    run_and_check(z, scores, k, eos=3, ctx="many groups, masked")


def test_refusals_with_device_tensors():
    z, scores, _ = make(2, 3, 100, "f32")
    ok = dict(dtype=torch.float32, device=DEV)
    for bad in (dict(logits=z.half()), dict(logits=z[:5]), dict(logits=z.t().contiguous().t()), dict(scores=scores.cpu()),
                dict(scores=scores.double()), dict(scores=scores[:, :2]), dict(k=0), dict(k=65), dict(eos_token=100),
                dict(finished=torch.zeros(2, 3, dtype=torch.bool, device=DEV), eos_token=1),
                dict(finished=torch.zeros(2, 2, dtype=torch.uint8, device=DEV), eos_token=1),
                dict(finished=torch.zeros(2, 3, dtype=torch.uint8, device=DEV)),
                dict(out=(torch.empty(2, 3, **ok),)), dict(workspace=torch.empty(1 << 20, **ok))):
        args = dict(logits=z, scores=scores)
        args.update(bad)
        with pytest.raises((ValueError, TypeError, qqe.KldEvalError)):
            qqe.beam_select(**args)
    assert qqe.beam_select(z[:0], scores[:0])[0].shape == (0, 3)


@pytest.mark.parametrize("seed", range(40))
def test_random(seed):
    g = np.random.default_rng(1000 + seed)
    items, beams = int(g.integers(1, 9)), int(g.integers(1, 9))
    vocab = int(np.exp(g.uniform(np.log(2), np.log(60000))))
    k, dtype = int(g.integers(1, 65)), ("f32", "bf16")[seed % 2]
    z, scores, tg = make(items, beams, vocab, dtype, seed=seed, sigma=float(g.uniform(0.1, 8)))
    if seed % 3 == 0:
        z.masked_fill_(torch.rand(z.shape, generator=tg, device=DEV) < g.uniform(0, 1), float("-inf"))
    fin = (torch.rand(items, beams, generator=tg, device=DEV) < 0.2).to(torch.uint8)
    run_and_check(z, scores, k, fin, int(g.integers(0, vocab)), ctx=f"random {seed}")
