"""The order of beam selection at the edge of what float32 normalisers can tell:
near ties that continue behind the last place."""
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
