"""The float64 oracle of the vocabulary operators, pinned by values worked out
by hand and by enumeration in plain Python."""
import math

import numpy as np
import pytest

from oracle import vocab as ov


def test_one_beam_is_the_log_softmax_in_order():
    z = np.log(np.array([[1.0, 4.0, 2.0, 1.0]], np.float64)).astype(np.float32)   # probabilities 1/8, 1/2, 1/4, 1/8
    s, p, t, f = ov.beam_select(z, np.array([[-1.0]], np.float32), 4)
    assert t.tolist() == [[1, 2, 0, 3]] and p.tolist() == [[0, 0, 0, 0]] and not f.any()
    want = [-1 + math.log(q) for q in (0.5, 0.25, 0.125, 0.125)]
    assert np.allclose(s[0], want, atol=1e-7)


def test_finished_empty_and_excluded():
    inf = np.float32(np.inf)
    z = np.array([[0, 0, -inf, inf], [5, 5, 5, 5], [1, 2, 3, 4]], np.float32)
    scores = np.array([[-1.0, -0.5, -inf]], np.float32)
    s, p, t, f = ov.beam_select(z, scores, 5, np.array([[0, 1, 0]], np.uint8), eos=2)
    # beam 1 stays with its end token, beam 0 offers its two finite logits, beam 2 is empty
    assert t.tolist() == [[2, 0, 1, -1, -1]] and p.tolist() == [[1, 0, 0, -1, -1]] and f.tolist() == [[1, 0, 0, 0, 0]]
    assert s[0, :3].tolist() == [-0.5, -1 - math.log(2), -1 - math.log(2)] and np.isneginf(s[0, 3:]).all()


@pytest.mark.parametrize("seed", range(20))
def test_select_equals_enumeration(seed):
    g = np.random.default_rng(seed)
    items, beams, vocab, k = 3, int(g.integers(1, 5)), int(g.integers(1, 9)), int(g.integers(1, 12))
    # equal logits within a row, none across rows
    z = (g.integers(-3, 4, size=(items * beams, vocab)) * g.uniform(0.5, 2, size=(items * beams, 1))).astype(np.float32)
    scores = -g.uniform(0, 3, size=(items, beams)).astype(np.float32)
    s, p, t, f = ov.beam_select(z, scores, k, eos=0)
    for i in range(items):
        row = [[float(x) for x in z[i * beams + w]] for w in range(beams)]
        rows = [(float(scores[i, w]) + row[w][v] - math.log(sum(math.exp(x) for x in row[w])), -w, -v)
                for w in range(beams) for v in range(vocab)]
        best = sorted(rows, key=lambda c: (-round(c[0], 12), -c[1], -c[2]))[:k]
        assert np.allclose([c[0] for c in best], s[i, :len(best)], atol=1e-12)
        assert [(-c[1], -c[2]) for c in best] == list(zip(p[i, :len(best)].tolist(), t[i, :len(best)].tolist()))
        assert (t[i, len(best):] == -1).all() and (f[i] == (t[i] == 0)).all()


def test_reorder_moves_only_the_stated_positions():
    x = np.arange(2 * 3 * 4).reshape(6, 4)
    y = ov.beam_reorder(x, np.array([[2, 0, -1], [1, 1, 1]]), np.array([3, 9]), 1)
    assert y.tolist() == [[8, 9, 10, 3], [0, 1, 2, 7], [8, 9, 10, 11], [16, 17, 18, 19], [16, 17, 18, 19],
                          [16, 17, 18, 19]]


def test_embed_and_its_gradient():
    table = np.array([[1, 2], [3, 4], [5, 6]], np.float32)
    e = ov.embed(table, [2, -1, 0, 3, 2], 0.5)
    assert e[0].tolist() == [2.5, 3] and e[1].tolist() == [0, 0] and np.isnan(e[3]).all()
    grad = np.array([[1, 1], [9, 9], [2, 3], [9, 9], [4, 5]], np.float32)
    d, mag, count = ov.embed_grad(grad, [2, -1, 0, 3, 2], 3, 0.5)
    assert d.tolist() == [[1, 1.5], [0, 0], [2.5, 3]] and count.tolist() == [1, 0, 2]


def test_embed_gradient_is_the_derivative():
    """Central differences of L = sum(grad * embed(table)); L is linear, so a
    step of 1 gives the derivative up to float64 rounding."""
    g = np.random.default_rng(0)
    table, tokens = g.normal(size=(5, 3)), [4, 1, 1, -1, 0, 4, 4, 7]
    grad = g.normal(size=(8, 3))
    seen = [n for n, t in enumerate(tokens) if t < 5]

    def loss(e):
        return (grad[seen] * ov.embed(e, tokens, 1.7)[seen]).sum()

    d, _, _ = ov.embed_grad(grad, tokens, 5, 1.7)
    for v in range(5):
        for c in range(3):
            up, down = table.copy(), table.copy()
            up[v, c] += 1
            down[v, c] -= 1
            assert abs((loss(up) - loss(down)) / 2 - d[v, c]) <= 1e-12
