"""Embedding lookup and its gradient on the GPU against the float64 oracle.

Tolerances. A lookup is one product rounded once: half a step of the output
type (2^-24 or 2^-8 of the value; the product may be rounded to float32 before
it is rounded to bfloat16, 2^-24 more). A gradient row sums c rows in float32:
at most (c - 1) 2^-24 of the sum of magnitudes, then the scaled (and, when
accumulating, added) value is rounded like a lookup."""
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
PAIRS = [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32"), ("f32", "bf16")]


def half_step(name):
    return 2.0 ** -24 if name == "f32" else 2.0 ** -8 + 2.0 ** -24


def f64(t):
    return t.double().cpu().numpy()


def close(got, want, tol, ctx):
    assert got.shape == want.shape, ctx
    nan = np.isnan(want)
    assert np.array_equal(np.isnan(got), nan), f"{ctx}: NaN where none belongs, or the reverse"
    err = np.abs(got - want)
    bad = ~nan & ~(err <= tol)
    assert not bad.any(), f"{ctx}: off by {err[bad].max()} at {np.argwhere(bad)[:3].tolist()}"


def rand(shape, dtype, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn(*shape, generator=g, device=DEV).to(TYPES[dtype])


def ids(n, vocab, seed, kind="uniform"):
    g = np.random.default_rng(seed)
    if kind == "one":
        t = np.full(n, vocab // 2)
    elif kind == "words":
        p = 1.0 / (np.arange(vocab) + 2.7)
        t = g.permutation(vocab)[g.choice(vocab, n, p=p / p.sum())]
    elif kind == "few":
        t = g.integers(0, min(3, vocab), n)
    elif kind == "none":
        t = np.full(n, -1)
    else:
        t = g.integers(0, vocab, n)
    if kind in ("uniform", "words") and n > 3:
        t[g.integers(0, n, max(1, n // 20))] = -1
        t[g.integers(0, n)] = vocab
        t[g.integers(0, n)] = 2**31 - 1
        t[g.integers(0, n)] = -2**31
    return torch.tensor(t.astype(np.int32), device=DEV)


SIZES = [(1, 1, 1), (7, 3, 5), (1000, 8, 64), (37, 64, 300), (32000, 100, 33), (501, 257, 100), (64, 1000, 2048),
         (5000, 1024, 777), (200, 4096, 129), (17, 5001, 64)]


@pytest.mark.parametrize("ti,to", PAIRS)
@pytest.mark.parametrize("vocab,dim,n", SIZES)
def test_lookup(vocab, dim, n, ti, to):
    table, tok = rand((vocab, dim), ti, n), ids(n, vocab, dim)
    scale = float(np.sqrt(dim))
    say(f"[embed] {vocab} x {dim}, {n} ids, {ti} -> {to}")
    got = f64(qqe.embed(table, tok, scale, dtype=to))
    want = ov.embed(synth.to_numpy_bits(table), tok.cpu().numpy(), scale)
    close(got, want, half_step(to) * np.abs(want), "lookup")


def test_lookup_shapes_strides_and_edges():
    table = rand((300, 40), "bf16", 1)
    tok = ids(24, 300, 2, "few").view(2, 3, 4)
    assert qqe.embed(table, tok).shape == (2, 3, 4, 40) and qqe.embed(table, tok).dtype == torch.bfloat16
    assert torch.equal(qqe.embed(table, tok).view(24, 40), table[tok.view(-1).long()])
    for cols in (37, 32, 33):      # rows of a wider table into rows of a wider output, at an odd offset
        wide = torch.full((24, 51), 9.0, dtype=torch.float32, device=DEV)
        qqe.embed(table[:, 3:3 + cols], tok, 2.0, out=_view(wide, tok, 5, cols))
        assert torch.equal(wide[:, 5:5 + cols], table[tok.view(-1).long(), 3:3 + cols].float() * 2)
        assert (wide[:, :5] == 9).all() and (wide[:, 5 + cols:] == 9).all()
    inf = torch.tensor([[float("inf"), float("nan"), -0.0]], device=DEV)
    one = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = qqe.embed(inf, one, -1.0)
    assert got[0, 0] == float("-inf") and got[0, 1].isnan() and got[0, 2] == 0
    assert qqe.embed(inf, one, -1.0, dtype="bf16")[0, 1].isnan()
    assert qqe.embed(table, one[:0]).shape == (0, 40)


def _view(wide, tok, at, cols):
    return wide[:, at:at + cols].unflatten(0, tuple(tok.shape))


def test_lookup_past_32_bits():
    dim, vocab = 1 << 20, 2600      # 2.7e9 elements
    table = torch.empty((vocab, dim), dtype=torch.bfloat16, device=DEV)
    rows = torch.tensor([0, 2599, 2100, 5], dtype=torch.int32, device=DEV)
    for r in rows.tolist():
        table[r].fill_(float(r % 100))
        table[r, -1] = 3.0
    got = qqe.embed(table, rows, 1.0)
    for i, r in enumerate(rows.tolist()):
        assert torch.equal(got[i], table[r])


@pytest.mark.parametrize("ti,to", PAIRS)
@pytest.mark.parametrize("kind", ["uniform", "words", "one", "few", "none"])
@pytest.mark.parametrize("vocab,dim,n", SIZES)
def test_gradient(vocab, dim, n, kind, ti, to):
    grad, tok = rand((n, dim), ti, vocab), ids(n, vocab, n, kind)
    say(f"[embed_grad] {vocab} x {dim}, {n} ids ({kind}), {ti} -> {to}")
    out = torch.full((vocab, dim), float("nan"), dtype=TYPES[to], device=DEV)
    got = f64(qqe.embed_grad(grad, tok, vocab, 0.75, out=out))
    want, mag, count = ov.embed_grad(synth.to_numpy_bits(grad), tok.cpu().numpy(), vocab, 0.75)
    tol = half_step(to) * np.abs(want) + 2.0 ** -24 * np.maximum(count - 1, 0)[:, None] * mag * (1 + half_step(to))
    close(got, want, tol, "gradient")
    assert not got[count == 0].any()
    old = rand((vocab, dim), to, 5)
    base = f64(old)
    got = f64(qqe.embed_grad(grad, tok, vocab, 0.75, out=old, accumulate=True))
    tol = half_step(to) * np.abs(base + want) + 2.0 ** -24 * np.maximum(count - 1, 0)[:, None] * mag * (1 + half_step(to))
    close(got, base + want, tol, "accumulated")
    assert np.array_equal(got[count == 0], base[count == 0])


@pytest.mark.parametrize("ti,to", [("bf16", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("n,vocab,dim,kind", [(70000, 1000, 24, "one"), (70000, 40000, 24, "words"),
                                              (200000, 3, 9, "uniform"), (131072, 151936, 8, "words"),
                                              (40000, 300, 520, "words"), (1537, 1 << 20, 4, "words"),
                                              (20000, (1 << 20) + 1, 4, "words"), (1536, 5, 100, "few"),
                                              (3000, 1 << 24, 1, "uniform")])
def test_gradient_of_long_runs(n, vocab, dim, kind, ti, to):
    """Runs of thousands of positions, against sums in float64."""
    grad, tok = rand((n, dim), ti, 3), ids(n, vocab, 4, kind)
    say(f"[embed_grad] long {n} ids ({kind}) of {vocab} x {dim}")
    got = f64(qqe.embed_grad(grad, tok, vocab, 1.0, dtype=to))
    t = tok.cpu().numpy().astype(np.int64)
    ok = (t >= 0) & (t < vocab)
    g = f64(grad)
    want, mag = np.zeros((vocab, dim)), np.zeros((vocab, dim))
    np.add.at(want, t[ok], g[ok])
    np.add.at(mag, t[ok], np.abs(g[ok]))
    count = np.bincount(t[ok], minlength=vocab)
    tol = half_step(to) * np.abs(want) + 2.0 ** -24 * np.maximum(count - 1, 0)[:, None] * mag * (1 + half_step(to))
    close(got, want, tol, "long runs")


def test_gradient_strides_and_untouched_bytes():
    n, vocab, dim = 333, 97, 60
    tok = ids(n, vocab, 1, "words")
    wide = rand((n, 80), "f32", 2)
    want, _, count = ov.embed_grad(f64(wide)[:, 7:67].astype(np.float32), tok.cpu().numpy(), vocab, 1.0)
    out = torch.full((vocab, 90), 5.0, device=DEV)
    nbytes = qqe.embed_grad_workspace_bytes(vocab, dim, n)
    ws = torch.full((nbytes + 64,), 171, dtype=torch.uint8, device=DEV)
    qqe.embed_grad(wide[:, 7:67], tok, vocab, out=out[:, 11:71], workspace=ws[:nbytes])
    assert (out[:, :11] == 5).all() and (out[:, 71:] == 5).all() and (ws[nbytes:] == 171).all()
    assert np.abs(f64(out[:, 11:71]) - want).max() < 1e-4
    three = qqe.embed_grad(wide[:, :60].contiguous().view(9, 37, 60), tok.view(9, 37), vocab)
    assert torch.equal(three, qqe.embed_grad(wide[:, :60], tok, vocab))


@pytest.mark.parametrize("fill", [0, 255, 127])
@pytest.mark.parametrize("n", [70, 5000])
def test_gradient_whatever_the_workspace_holds(n, fill):
    vocab, dim = 400, 36
    grad, tok = rand((n, dim), "f32", n), ids(n, vocab, n, "words")
    ws = torch.full((qqe.embed_grad_workspace_bytes(vocab, dim, n),), fill, dtype=torch.uint8, device=DEV)
    got = f64(qqe.embed_grad(grad, tok, vocab, workspace=ws))
    want, mag, count = ov.embed_grad(synth.to_numpy_bits(grad), tok.cpu().numpy(), vocab)
    close(got, want, half_step("f32") * np.abs(want) + 2.0 ** -24 * np.maximum(count - 1, 0)[:, None] * mag * 1.001,
          f"workspace of {fill}")


def test_gradient_of_no_tokens_and_bad_rows():
    out = rand((50, 33), "f32", 1)
    keep = out.clone()
    empty = torch.empty((0, 33), device=DEV)
    no = torch.empty(0, dtype=torch.int32, device=DEV)
    qqe.embed_grad(empty, no, 50, out=out, accumulate=True)
    assert torch.equal(out, keep)
    assert not qqe.embed_grad(empty, no, 50, out=out).any()
    grad = torch.full((3, 33), float("nan"), device=DEV)    # rows without a valid id add nothing, NaN or not
    grad[1] = 2.0
    got = qqe.embed_grad(grad, torch.tensor([-1, 4, 50], dtype=torch.int32, device=DEV), 50)
    assert (got[4] == 2).all() and got.sum() == 66
    got = qqe.embed_grad(grad, torch.tensor([3, 4, 5], dtype=torch.int32, device=DEV), 50, dtype="bf16")
    assert got[3].isnan().all() and (got[4] == 2).all() and not got[6].any()


def test_gradient_past_32_bits():
    """A table of more than 2^32 elements, the last rows among the named."""
    vocab, dim = 4200, 1 << 20
    grad = rand((3, dim), "bf16", 1)
    out = torch.empty((vocab, dim), dtype=torch.bfloat16, device=DEV)
    out[-3:].fill_(7.0)
    out[2000].fill_(7.0)
    qqe.embed_grad(grad, torch.tensor([4199, 0, 4100], dtype=torch.int32, device=DEV), vocab, out=out)
    assert torch.equal(out[4199], grad[0]) and torch.equal(out[0], grad[1]) and torch.equal(out[4100], grad[2])
    assert not out[4198].any() and not out[4197].any() and not out[2000].any()


def test_difference_quotients():
    """The gradient against differences of the lookup it belongs to: the loss is
    linear in the table, so a step of 1/2 is exact up to rounding."""
    vocab, dim, n = 11, 5, 40
    table, grad, tok = rand((vocab, dim), "f32", 1), rand((n, dim), "f32", 2), ids(n, vocab, 3, "few")
    d = f64(qqe.embed_grad(grad, tok, vocab, 1.5))
    for v, c in ((0, 0), (1, 3), (2, 4), (7, 2)):
        up, down = table.clone(), table.clone()
        up[v, c] += 0.5
        down[v, c] -= 0.5
        gap = (qqe.embed(up, tok, 1.5).double() - qqe.embed(down, tok, 1.5).double()) * grad.double()
        # 40 products of magnitude <= 8 x |grad|, each lookup rounded by 2^-24 of it, and the step itself
        assert abs(gap.sum().item() - d[v, c]) <= 40 * 4 * 8 * 4 * 2.0 ** -24


def test_same_bits_streams_and_graphs():
    n, vocab, dim = 5000, 2000, 256
    grad, tok = rand((n, dim), "bf16", 1), ids(n, vocab, 2, "words")
    first = qqe.embed_grad(grad, tok, vocab)
    look = qqe.embed(grad, tok)          # any table will do
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        assert torch.equal(first, qqe.embed_grad(grad, tok, vocab))
        a, b = qqe.embed_grad(grad, tok, vocab, stream=side), qqe.embed(grad, tok, stream=side)
        torch.cuda.synchronize()
        assert torch.equal(a, first) and torch.equal(b.view(torch.int16), look.view(torch.int16))   # NaN rows among them
    graph = torch.cuda.CUDAGraph()
    out = torch.zeros((vocab, dim), device=DEV)
    with torch.cuda.graph(graph):
        qqe.embed_grad(grad, tok, vocab, out=out)
        qqe.embed_grad(grad, tok, vocab, out=out, accumulate=True)
        row = qqe.embed(out, tok, dtype="bf16")
    for step in range(4):
        tok.copy_(ids(n, vocab, 10 + step, "words"))
        graph.replay()
        eager = qqe.embed_grad(grad, tok, vocab)
        qqe.embed_grad(grad, tok, vocab, out=eager, accumulate=True)
        torch.cuda.synchronize()
        assert torch.equal(out, eager), step
        assert torch.equal(row.view(torch.int16), qqe.embed(eager, tok, dtype="bf16").view(torch.int16)), step


def test_refusals_with_device_tensors():
    table, tok = rand((10, 4), "f32", 1), ids(5, 10, 2, "few")
    for bad in (dict(table=table.half()), dict(table=table.t()), dict(table=table[0]), dict(tokens=tok.long()),
                dict(tokens=tok.cpu()), dict(scale=float("inf")), dict(out=torch.empty(5, 3, device=DEV)),
                dict(out=torch.empty(5, 4, device=DEV), dtype="bf16"), dict(out=torch.empty(5, 4))):
        args = dict(table=table, tokens=tok)
        args.update(bad)
        with pytest.raises((ValueError, TypeError, qqe.KldEvalError)):
            qqe.embed(**args)
    grad = rand((5, 4), "f32", 1)
    for bad in (dict(grad=grad.half()), dict(grad=grad[:4]), dict(tokens=tok.long()), dict(vocab=0), dict(accumulate=True),
                dict(out=torch.empty(9, 4, device=DEV)), dict(out=torch.empty(10, 4)), dict(scale=float("nan")),
                dict(workspace=torch.empty(1, dtype=torch.uint8, device=DEV)), dict(grad=grad.cpu())):
        args = dict(grad=grad, tokens=tok, vocab=10)
        args.update(bad)
        with pytest.raises((ValueError, TypeError, qqe.KldEvalError)):
            qqe.embed_grad(**args)
