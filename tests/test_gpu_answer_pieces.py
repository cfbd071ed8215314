"""8-bit rows and products whose grids exceed what one launch may hold (the dispatch
packet counts work-items in 32 bits) and are cut into pieces: sizes just past the
first piece, outputs filled before with what no result is, samples around the
boundary, at the ends and elsewhere against the oracle."""
import numpy as np
import pytest
import torch

import quantization_quality_eval_amd as qqe
import synth
from oracle import answer as oa
from tests.gpu_util import say

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
PIECE = (2 ** 31 - 1) // 256   # workgroups of 256 threads in one piece


def around(n, *boundaries):
    g = np.random.default_rng(n)
    some = [np.arange(5), np.arange(n - 5, n), g.integers(0, n, 200)] + [np.arange(b - 40, min(b + 40, n)) for b in boundaries]
    return torch.as_tensor(np.unique(np.concatenate(some)), device=DEV)


def random_bytes(n, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randint(-128, 128, (n,), generator=g, device=DEV, dtype=torch.int8)


def test_rounding_past_one_launch():
    n = PIECE * 16 + 1000      # sixteen rows to a workgroup
    g = torch.Generator(device=DEV).manual_seed(1)
    x = torch.randn(n, 2, generator=g, device=DEV).bfloat16()
    q, s = torch.full((n, 2), -128, dtype=torch.int8, device=DEV), torch.full((n,), float("nan"), device=DEV)
    say(f"[pieces] rounding of {n} rows")
    qqe.quantize_int8(x, out=(q, s))
    assert not bool((q == -128).any()) and not bool(s.isnan().any())
    at = around(n, PIECE * 16)
    wq, ws = oa.quantize(synth.to_numpy_bits(x[at]))
    assert np.array_equal(q[at].cpu().numpy(), wq) and np.array_equal(s[at].cpu().numpy(), ws)


@pytest.mark.parametrize("m,cols,what", [(3, 32, "few rows"), (17, 128, "tiles of 64 x 128")])
def test_products_past_one_launch(m, cols, what):
    n = PIECE * cols + 1000
    x, w = random_bytes(m, 2).view(m, 1), random_bytes(n, 3).view(n, 1)
    g = torch.Generator(device=DEV).manual_seed(4)
    xs, ws = torch.rand(m, generator=g, device=DEV), torch.rand(n, generator=g, device=DEV)
    out = torch.full((m, n), float("nan"), dtype=torch.bfloat16, device=DEV)
    say(f"[pieces] product of {m} x 1 by {n}: {what}, {out.numel() * 2 / 2 ** 30:.1f} GiB")
    qqe.matmul_int8(x, xs, w, ws, out=out)
    at = around(n, PIECE * cols)
    got = out[:, at].double().cpu().numpy()
    assert not any(bool(row.isnan().any()) for row in out)
    want = oa.matmul(x.cpu().numpy(), xs.cpu().numpy(), w[at].cpu().numpy(), ws[at].cpu().numpy())
    tol = 3.0001 * 2.0 ** -24 * np.abs(want) + 2.0 ** -150
    assert (np.abs(got - want) <= tol + 2.0 ** -8 * (np.abs(want) + tol) + 2.0 ** -134).all()
    del out, w, ws
    torch.cuda.empty_cache()
