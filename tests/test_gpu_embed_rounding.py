"""The embedding calls round once: a product, or a scaled sum, formed in float64
goes straight to the output's type. Expected values are rounded from float64 by
comparing the neighbouring bfloat16 values, and every bit is compared."""
import numpy as np
import pytest
import torch

import quantization_quality_eval_amd as qqe
from tests.gpu_util import say

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def nearest_bf16(x):
    """float64 -> bfloat16 bits, to nearest, ties to even (finite values)."""
    x = np.asarray(x, np.float64)
    with np.errstate(over="ignore"):
        near = np.abs(x).astype(np.float32).view(np.uint32).astype(np.int64) >> 16
    low = np.maximum(near - 1, 0)
    places = low[..., None] + np.arange(4)   # the float32 may have been rounded past a bfloat16, no further
    places = np.minimum(places, 0x7f80)
    value = (places.astype(np.uint32) << 16).view(np.float32).astype(np.float64)
    value[places == 0x7f80] = 2.0 ** 128     # where the next value would be
    gap = np.abs(np.abs(x)[..., None] - value)
    pick = np.lexsort((places & 1, gap), axis=-1)[..., :1]
    bits = np.take_along_axis(places, pick, -1)[..., 0]
    return (bits | np.where(np.signbit(x), 0x8000, 0)).astype(np.uint16)


def bits(t):
    return t.cpu().view(torch.int16).numpy().view(np.uint16)


# a scale beside a midpoint of two bfloat16 values, by less than float32 can tell
BESIDE = [1 + 2.0 ** -8 + 2.0 ** -40, 1 + 3 * 2.0 ** -8 - 2.0 ** -40, -(1 + 2.0 ** -8 + 2.0 ** -52),
          (2 - 2.0 ** -8) * 2.0 ** 127 * (1 - 2.0 ** -40),   # below the border to infinity
          2.0 ** -134 * (1 + 2.0 ** -40),                     # above half of the smallest subnormal value
          5 * 2.0 ** -134 * (1 - 2.0 ** -40), 2.0 ** -160]


def test_the_reference_rounding():
    assert nearest_bf16([1.0, -2.5, 0.0, 3.0]).tolist() == [0x3f80, 0xc020, 0, 0x4040]
    assert nearest_bf16([1 + 2.0 ** -8, 1 + 3 * 2.0 ** -8]).tolist() == [0x3f80, 0x3f82]
    assert nearest_bf16(BESIDE).tolist() == [0x3f81, 0x3f81, 0xbf81, 0x7f7f, 1, 2, 0]
    assert nearest_bf16([2.0 ** 127 * 1.9999, -3.4e38]).tolist() == [0x7f80, 0xff80]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("dim", [5, 64])
def test_lookup_beside_midpoints(dim, dtype):
    table = torch.ones(3, dim, dtype=torch.float32 if dtype == "f32" else torch.bfloat16, device=DEV)
    tok = torch.tensor([0, 2, -1], dtype=torch.int32, device=DEV)
    for scale in BESIDE:
        got = bits(qqe.embed(table, tok, scale, dtype="bf16"))
        want = int(nearest_bf16(scale))
        assert (got[:2] == want).all() and (got[2] == 0).all(), f"scale {scale!r}: {got[0, 0]:#x}, expected {want:#x}"


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_lookup_of_random_rows(dtype):
    g = torch.Generator(device=DEV).manual_seed(5)
    table = torch.randn(2000, 2048, generator=g, device=DEV).to(torch.float32 if dtype == "f32" else torch.bfloat16)
    tok = torch.arange(2000, dtype=torch.int32, device=DEV)
    for scale in (1.0, 45.254833995939045, -1e-3):
        say(f"[embed rounding] {dtype} scale {scale}")
        got = bits(qqe.embed(table, tok, scale, dtype="bf16"))
        want = nearest_bf16(table.double().cpu().numpy() * scale)
        assert np.array_equal(got, want), f"scale {scale}: {(got != want).sum()} of {got.size} differ"


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n", [1, 64, 4096])   # one position, a run of several pieces, the sort of many positions
def test_gradient_beside_midpoints(n, dtype):
    """n equal rows of a power of two: their sum is exact."""
    grad = torch.full((n, 24), 1.0 / n, dtype=torch.float32 if dtype == "f32" else torch.bfloat16, device=DEV)
    tok = torch.full((n,), 7, dtype=torch.int32, device=DEV)
    for scale in BESIDE:
        say(f"[embed rounding] gradient of {n} x {dtype}, scale {scale!r}")
        got = bits(qqe.embed_grad(grad, tok, 10, scale, dtype="bf16"))
        want = int(nearest_bf16(scale))
        assert (got[7] == want).all(), f"scale {scale!r}: {got[7, 0]:#x}, expected {want:#x}"
        out = torch.full((10, 24), 1.0, dtype=torch.bfloat16, device=DEV)
        got = bits(qqe.embed_grad(grad, tok, 10, 2.0 ** -8 + 2.0 ** -40, out=out, accumulate=True))
        assert (got[7] == 0x3f81).all() and (got[:7] == 0x3f80).all() and (got[8:] == 0x3f80).all()
