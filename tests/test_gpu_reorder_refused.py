"""States of several geometries, one of them refused: none has been moved."""
import pytest
import torch

import quantization_quality_eval_amd as qqe

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
KINDS = ["beams at one place", "heads at one place", "beams overlap", "given twice"]


def refused(kind):
    """States [6, ...] that the reordering cannot take."""
    if kind == "beams at one place":
        return [torch.ones(1, 2, 10, 8, device=DEV).expand(6, 2, 10, 8)]
    if kind == "heads at one place":
        return [torch.ones(6, 1, 10, 8, device=DEV).expand(6, 2, 10, 8)]
    if kind == "beams overlap":
        return [torch.ones(1000, device=DEV).as_strided((6, 2, 10, 8), (100, 80, 8, 1))]
    x = torch.ones(6, 2, 10, 8, device=DEV)
    return [x, x]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("ragged", [True, False])
@pytest.mark.parametrize("first", [True, False])
def test_nothing_moves(kind, ragged, first):
    parents = torch.tensor([[1, 2, 0], [2, 2, 0]], dtype=torch.int32, device=DEV)
    good = [torch.randn(6, 4, 10, 16, device=DEV), torch.randn(6, 1, 10, 3, device=DEV)]
    kept = [x.clone() for x in good]
    kw = dict(lengths=torch.tensor([10, 7], dtype=torch.int32, device=DEV), length_dim=2) if ragged else {}
    bad = refused(kind)
    with pytest.raises((ValueError, qqe.KldEvalError)):
        qqe.beam_reorder(good + bad if not first else bad + good, parents, **kw)
    torch.cuda.synchronize()
    for x, was in zip(good, kept):
        assert torch.equal(x, was)
    qqe.beam_reorder(good, parents, **kw)
    for x, was in zip(good, kept):
        assert not torch.equal(x, was)
