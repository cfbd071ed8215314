"""The vocabulary operators together, as a user's program calls them: a decoding
loop (lookup, model, selection, reordering) and a tuning step (lookup, model, KL
rows and their gradient, model backward, embedding gradient), against the same
programs in float64."""
import math

import numpy as np
import pytest
import torch

import quantization_quality_eval_amd as qqe
import synth
from oracle import grad as ograd
from oracle import vocab as ov
from tests.gpu_util import say

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


class Tiny:
    """A recurrent stand-in for a model: state' = tanh(state A + x), logits = state' E^T."""

    def __init__(self, vocab, dim, seed):
        g = torch.Generator(device=DEV).manual_seed(seed)
        self.table = torch.randn(vocab, dim, generator=g, device=DEV)
        self.mix = torch.randn(dim, dim, generator=g, device=DEV) / math.sqrt(dim)

    def step(self, state, x):
        state = torch.tanh(state @ self.mix + x)
        return state, state @ self.table.t()


@pytest.mark.parametrize("vocab,dim,items,beams", [(997, 24, 3, 4), (4104, 64, 5, 1), (300, 40, 2, 7)])
def test_decoding_loop(vocab, dim, items, beams):
    """Twelve steps: tokens, parents and finished flags equal those of the oracle
    run on the logits of the loop itself; histories and states follow."""
    model, steps, eos = Tiny(vocab, dim, vocab), 12, 5
    scores = torch.full((items, beams), float("-inf"), device=DEV)
    scores[:, 0] = 0
    fin = torch.zeros(items, beams, dtype=torch.uint8, device=DEV)
    tokens = torch.full((items, beams), 1, dtype=torch.int32, device=DEV)
    state = torch.zeros(items * beams, dim, device=DEV)
    history = torch.full((items * beams, steps), -7, dtype=torch.int32, device=DEV)
    host = np.full((items * beams, steps), -7, np.int32)
    for t in range(steps):
        x = qqe.embed(model.table, tokens, 1.0 / math.sqrt(dim)).view(items * beams, dim)
        state, logits = model.step(state, x)
        want = ov.beam_select(logits.cpu().numpy(), scores.cpu().numpy(), beams, fin.cpu().numpy(), eos)
        want_state = ov.beam_reorder(state.cpu().numpy(), want[1])
        host = ov.beam_reorder(host, want[1], np.full(items, t), 1)
        scores, parents, tokens, fin = qqe.beam_select(logits, scores, finished=fin, eos_token=eos)
        qqe.beam_reorder(state, parents)
        qqe.beam_reorder(history, parents, lengths=torch.full((items,), t, dtype=torch.int32, device=DEV), length_dim=1)
        history[:, t] = tokens.view(-1)
        host[:, t] = want[2].reshape(-1)
        assert np.array_equal(parents.cpu().numpy(), want[1]) and np.array_equal(tokens.cpu().numpy(), want[2]), t
        assert np.array_equal(fin.cpu().numpy(), want[3])
        assert np.array_equal(state.cpu().numpy(), want_state) and np.array_equal(history.cpu().numpy(), host)
    say(f"[loop] {vocab} x {dim}, {items} x {beams}: best {scores[:, 0].tolist()}")


def test_decoding_loop_as_one_graph():
    """A step captured once (every call of it allocates nothing outside the
    graph) and replayed gives the eager loop's tokens and states."""
    vocab, dim, items, beams, eos = 1500, 32, 4, 3, 7
    model = Tiny(vocab, dim, 1)

    def fresh():
        s = torch.full((items, beams), float("-inf"), device=DEV)
        s[:, 0] = 0
        return [s, torch.zeros(items, beams, dtype=torch.uint8, device=DEV),
                torch.ones(items, beams, dtype=torch.int32, device=DEV), torch.zeros(items * beams, dim, device=DEV)]

    def step(v):
        x = qqe.embed(model.table, v[2], 0.2).view(items * beams, dim)
        state, logits = model.step(v[3], x)
        scores, parents, tokens, fin = qqe.beam_select(logits, v[0], finished=v[1], eos_token=eos)
        qqe.beam_reorder(state, parents)
        for old, new in zip(v, (scores, fin, tokens, state)):
            old.copy_(new)

    eager, held = fresh(), fresh()
    step(fresh())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(held)
    for old, new in zip(held, fresh()):
        old.copy_(new)
    for t in range(6):
        graph.replay()
        step(eager)
        torch.cuda.synchronize()
        for a, b in zip(held, eager):
            assert torch.equal(a, b), t


@pytest.mark.parametrize("vocab,dim,n", [(1001, 48, 200), (4104, 64, 513)])
def test_tuning_step(vocab, dim, n):
    """Loss: mean KL of logits embed(E) W against fixed base rows. The gradient of
    E by the operators against the formula in float64, and against differences."""
    g = torch.Generator(device=DEV).manual_seed(vocab)
    table = torch.randn(vocab, dim, generator=g, device=DEV) * 0.3
    weight = torch.randn(dim, vocab, generator=g, device=DEV) * 0.3
    base = torch.randn(n, vocab, generator=g, device=DEV)
    tokens = torch.randint(0, 37, (n,), generator=g, device=DEV, dtype=torch.int32)
    tokens[::19] = -1
    scale = math.sqrt(dim)
    x = qqe.embed(table, tokens, scale)
    logits = x @ weight
    with qqe.Evaluator(vocab, n, "f32", "f32", device=DEV) as ev:
        ev.rows(base, logits)
        dlogits = ev.grad(base, logits, scale=1.0 / n)
        torch.cuda.synchronize()
    dx = dlogits @ weight.t()
    dtable = qqe.embed_grad(dx, tokens, vocab, scale)

    # the formula in float64 from the operators' own inputs
    nb, nq = base.cpu().numpy(), logits.cpu().numpy()
    lb, lq = (ov.log_normalisers(a.astype(np.float64)) for a in (nb, nq))
    dl, _, _ = ograd.grad_rows(nb, nq, lb, lq, 1.0 / n)
    want_dx = dl @ weight.double().cpu().numpy().T
    t = tokens.cpu().numpy()
    want = np.zeros((vocab, dim))
    np.add.at(want, t[t >= 0], want_dx[t >= 0])
    want *= scale
    err = np.abs(dtable.cpu().numpy() - want).max() / np.abs(want).max()
    # dlogits 1e-5 of q + p as the gradient kernel states; the product sums `vocab` such terms with
    # signs, and its own float32 rounding is of the same order
    assert err < 1e-4, err
    assert not dtable[37:].any()

    def loss(e):
        z = torch.where((tokens < 0)[:, None], 0.0, e.double()[tokens.clamp(min=0).long()]) * scale @ weight.double()
        p = torch.log_softmax(base.double(), 1)
        return (p.exp() * (p - torch.log_softmax(z, 1))).sum(1).mean()

    h = 1e-5
    for v, c in ((0, 0), (3, 7), (36, dim - 1)):
        up, down = table.double().clone(), table.double().clone()
        up[v, c] += h
        down[v, c] -= h
        diff = ((loss(up) - loss(down)) / (2 * h)).item()
        # truncation h^2 and the float32 gradient's own error above
        assert abs(diff - dtable[v, c].item()) <= 1e-4 * np.abs(want).max() + 1e-7
    again = qqe.embed_grad(dx, tokens, vocab, scale, out=dtable.clone(), accumulate=True)
    assert torch.allclose(again, 2 * dtable, rtol=2 ** -23, atol=0)
    say(f"[tuning] {vocab} x {dim}, {n} tokens: gradient within {err:.2e}")
