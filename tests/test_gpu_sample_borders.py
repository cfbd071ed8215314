"""Draws that hang on a border, on the GPU: equal logits at the edge between two
bins in different slices of a row."""
import math
import random
from fractions import Fraction

import numpy as np
import pytest
import torch

import quantization_quality_eval_amd as qqe
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
