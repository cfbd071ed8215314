"""Float64 oracle of the operators around the vocabulary: one step of beam
search, reordering of beam states, embedding lookup with scaling and its
gradient, each from its definition (NumPy loops and sums)."""
from __future__ import annotations

import math

import numpy as np

from . import to_f64


def log_normalisers(z: np.ndarray) -> np.ndarray:
    """log sum exp of each row over its finite entries (0 where there is none)."""
    out = np.zeros(z.shape[0])
    for r in range(z.shape[0]):
        x = z[r][np.isfinite(z[r])]
        if x.size:
            m = x.max()
            out[r] = m + math.log(np.exp(x - m).sum())
    return out


def beam_select(logits, scores, k, finished=None, eos=-1):
    """(scores float64, parents, tokens, finished) [items, k] of one step;
    ``logits`` [items * beams, vocab] float32 or bf16 bits."""
    z = to_f64(logits)
    items, beams = scores.shape
    vocab = z.shape[1]
    lse = log_normalisers(z).reshape(items, beams)
    z = z.reshape(items, beams, vocab)
    s_out = np.full((items, k), -np.inf)
    p_out = np.full((items, k), -1, np.int64)
    t_out = np.full((items, k), -1, np.int64)
    f_out = np.zeros((items, k), np.uint8)
    for i in range(items):
        c = np.full((beams, vocab), -np.inf)
        for w in range(beams):
            s = float(scores[i, w])
            if not math.isfinite(s):
                continue
            if finished is not None and finished[i, w]:
                c[w, eos] = s
            else:
                ok = np.isfinite(z[i, w])
                c[w, ok] = s + (z[i, w, ok] - lse[i, w])
        flat = c.reshape(-1)
        top = np.argpartition(-flat, min(k, flat.size) - 1)[:k] if flat.size > 4 * k else np.arange(flat.size)
        least = np.sort(flat[top])[::-1][:k][-1]  # everything at or above the k-th value, lowest places first
        at = np.nonzero(flat >= least)[0]
        # by score, then by beam, and within a beam by the logit: logits too close for their scores to differ keep
        # their order
        at = at[np.lexsort((at, -z[i].reshape(-1)[at], at // vocab, -flat[at]))][:k]
        at = at[flat[at] > -np.inf]
        n = at.size
        s_out[i, :n], p_out[i, :n], t_out[i, :n] = flat[at], at // vocab, at % vocab
        for j in range(n):
            ended = finished is not None and finished[i, p_out[i, j]]
            f_out[i, j] = bool(ended) or t_out[i, j] == eos
    return s_out, p_out, t_out, f_out


def beam_reorder(state, parents, lengths=None, length_dim=None):
    """A copy of ``state`` [items * beams, ...] after the reordering."""
    items, beams = parents.shape
    new = state.copy()
    for i in range(items):
        for w in range(beams):
            p = parents[i, w]
            if not 0 <= p < beams:
                continue
            at = [slice(None)] * (state.ndim - 1)
            if length_dim is not None:
                at[length_dim - 1] = slice(0, max(0, min(int(lengths[i]), state.shape[length_dim])))
            new[(i * beams + w, *at)] = state[(i * beams + p, *at)]
    return new


def embed(table, tokens, scale=1.0):
    """float64 [n, dim]."""
    e = to_f64(table)
    out = np.zeros((len(tokens), e.shape[1]))
    for n, t in enumerate(tokens):
        if t >= e.shape[0]:
            out[n] = np.nan
        elif t >= 0:
            out[n] = e[t] * scale
    return out


def embed_grad(grad, tokens, vocab, scale=1.0):
    """(float64 [vocab, dim] gradient, float64 [vocab, dim] sums of magnitudes, counts [vocab])."""
    g = to_f64(grad)
    out, mag = np.zeros((vocab, g.shape[1])), np.zeros((vocab, g.shape[1]))
    count = np.zeros(vocab, np.int64)
    for n, t in enumerate(tokens):
        if 0 <= t < vocab:
            out[t] += g[n]
            mag[t] += np.abs(g[n])
            count[t] += 1
    return out * scale, mag * abs(scale), count
