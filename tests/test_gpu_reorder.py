"""Reordering of beam states on the GPU, in place, against the oracle's copy:
equal bytes, and every byte outside the moved positions as it was."""
import numpy as np
import pytest
import torch

import quantization_quality_eval_amd as qqe
from oracle import vocab as ov
from tests.gpu_util import say

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def bytes_of(t):
    return t.contiguous().cpu().view(torch.uint8).numpy().reshape(*t.shape, t.element_size())


def expect(x, parents, lengths, dim):
    return ov.beam_reorder(bytes_of(x), parents.cpu().numpy(), None if lengths is None else lengths.cpu().numpy(), dim)


def random_state(shape, dtype, g):
    n = int(np.prod(shape)) * torch.empty(0, dtype=dtype).element_size()
    return torch.randint(0, 256, (n,), generator=g, device=DEV, dtype=torch.uint8).view(dtype).view(shape)


def check(states, parents, lengths=None, dim=None, ctx="", **kw):
    say(f"[reorder] {ctx} {[tuple(x.shape) for x in states]} beams {tuple(parents.shape)}")
    want = [expect(x, parents, lengths, dim) for x in states]
    qqe.beam_reorder(states, parents, lengths=lengths, length_dim=dim, **kw)
    torch.cuda.synchronize()
    for i, (x, w) in enumerate(zip(states, want)):
        assert np.array_equal(bytes_of(x), w), f"{ctx}: state {i} differs"


def beams_of(items, beams, g, low=-1):
    return torch.randint(low, beams, (items, beams), generator=g, device=DEV, dtype=torch.int32)


@pytest.mark.parametrize("beams", [1, 2, 3, 4, 5, 8, 9, 16, 17, 32, 33, 64])
@pytest.mark.parametrize("shape,dim,dtype", [((2, 40, 64), 2, torch.bfloat16), ((33, 3), 1, torch.float32),
                                             ((5, 7, 3), 2, torch.bfloat16), ((19,), 1, torch.uint8),
                                             ((1, 1), 1, torch.int64), ((3, 2, 9, 10), 3, torch.float32)])
def test_geometries(beams, shape, dim, dtype):
    g = torch.Generator(device=DEV).manual_seed(beams)
    items = 3
    parents = beams_of(items, beams, g)
    lengths = torch.tensor([0, shape[dim - 1], max(1, shape[dim - 1] // 2)], dtype=torch.int32, device=DEV)
    states = [random_state((items * beams, *shape), dtype, g) for _ in range(2)]
    check(states, parents, lengths, dim, ctx=f"{dtype}")
    check(states, parents, ctx=f"{dtype} whole")


def test_cycles_swaps_and_broadcasts():
    g = torch.Generator(device=DEV).manual_seed(1)
    parents = torch.tensor([[1, 2, 3, 0], [1, 0, 3, 2], [0, 1, 2, 3], [3, 3, 3, 3], [0, 0, 1, 2], [-1, 4, 2**30, -2**31]],
                           dtype=torch.int32, device=DEV)
    check([random_state((24, 2, 70, 32), torch.bfloat16, g)], parents, torch.full((6,), 70, dtype=torch.int32, device=DEV),
          2, ctx="cycles")


def test_lengths_outside_the_state_are_taken_into_it():
    g = torch.Generator(device=DEV).manual_seed(2)
    lengths = torch.tensor([-5, 1000, 2**31 - 1, -2**31], dtype=torch.int32, device=DEV)
    check([random_state((8, 3, 21, 8), torch.float32, g)], beams_of(4, 2, g), lengths, 2, ctx="lengths")


def test_views_leave_the_rest_alone():
    """Part of a cache: some heads, the first positions, a slice of a wider
    buffer, beams behind the heads; odd byte offsets."""
    g = torch.Generator(device=DEV).manual_seed(3)
    parents, lengths = beams_of(3, 4, g), torch.tensor([9, 30, 17], dtype=torch.int32, device=DEV)
    full = random_state((12, 6, 40, 16), torch.bfloat16, g)
    for name, view in (("heads", full[:, 1:4]), ("positions", full[:, :, 3:33]), ("both", full[:, 2:3, 5:])):
        before = full.clone()
        check([view], parents, lengths.clamp(max=view.shape[2]), 2, ctx=name)
        changed = torch.zeros_like(full, dtype=torch.bool)
        (changed[:, 1:4] if name == "heads" else changed[:, :, 3:33] if name == "positions" else changed[:, 2:3, 5:]).fill_(True)
        assert torch.equal(full.view(torch.int16)[~changed], before.view(torch.int16)[~changed])
    behind = random_state((5, 12, 33, 8), torch.float32, g).transpose(0, 1)   # [beams, heads, ...] over [heads, beams, ...]
    check([behind], parents, lengths, 2, ctx="beams inside heads")
    odd = random_state((12 * 37 + 1,), torch.uint8, g)
    check([odd[1:].view(12, 37)], parents, lengths, 1, ctx="odd offset")
    kv = random_state((12, 2, 4, 40, 16), torch.bfloat16, g)                  # keys and values of one buffer
    check([kv[:, 0], kv[:, 1]], parents, lengths, 2, ctx="interleaved")


def test_many_states_items_and_outer():
    g = torch.Generator(device=DEV).manual_seed(4)
    check([random_state((6, 2, 16, 8), torch.bfloat16, g) for _ in range(130)], beams_of(2, 3, g),
          torch.tensor([16, 5], dtype=torch.int32, device=DEV), 2, ctx="130 states")
    check([random_state((70000 * 2, 3), torch.int32, g)], beams_of(70000, 2, g), ctx="70000 items")
    check([random_state((4, 70001, 2, 2), torch.bfloat16, g)], beams_of(1, 4, g),
          torch.tensor([2], dtype=torch.int32, device=DEV), 2, ctx="70001 outer")


def test_states_past_32_bits():
    """Beams 3 GiB apart."""
    beam = 3 << 30
    buf = torch.empty(beam * 3 + 4096, dtype=torch.uint8, device=DEV)
    x = buf.as_strided((4, 4096), (beam, 1))
    g = torch.Generator(device=DEV).manual_seed(5)
    x.copy_(torch.randint(0, 256, (4, 4096), generator=g, device=DEV, dtype=torch.uint8))
    check([x], torch.tensor([[3, 0, 1, 2]], dtype=torch.int32, device=DEV), ctx="far beams")
    big = torch.empty((2, (5 << 30) // 2), dtype=torch.bfloat16, device=DEV)   # one beam alone passes 4 GiB
    big[0].fill_(1.0)
    big[1].fill_(2.0)
    big[1, -1], big[0, -3] = 7.0, 5.0
    qqe.beam_reorder(big, torch.tensor([[1, 0]], dtype=torch.int32, device=DEV))
    assert big[0, -1] == 7 and big[1, -3] == 5
    big[0, -1], big[1, -3] = 2.0, 1.0
    assert bool((big[0] == 2).all()) and bool((big[1] == 1).all())


def test_streams_graphs_and_refusals():
    g = torch.Generator(device=DEV).manual_seed(6)
    parents = beams_of(4, 4, g)
    x = random_state((16, 4, 50, 64), torch.bfloat16, g)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    check([x], parents, torch.full((4,), 50, dtype=torch.int32, device=DEV), 2, ctx="stream", stream=side)
    graph = torch.cuda.CUDAGraph()
    y = x.clone()
    with torch.cuda.graph(graph):
        qqe.beam_reorder([y], parents)
    for step in range(4):
        parents.copy_(beams_of(4, 4, g))
        y.copy_(x)
        z = x.clone()
        graph.replay()
        qqe.beam_reorder(z, parents)
        torch.cuda.synchronize()
        assert torch.equal(y.view(torch.int16), z.view(torch.int16)), step
    with pytest.raises(qqe.KldEvalError, match="overlap"):
        qqe.beam_reorder([x, x], parents)
    for bad in (dict(states=x[:15]), dict(states=x.cpu()), dict(parents=parents.long()), dict(parents=parents[0]),
                dict(lengths=parents[0].contiguous()), dict(length_dim=2), dict(states=x.transpose(1, 2)),
                dict(states=x, lengths=parents[0].contiguous(), length_dim=4),
                dict(states=x, lengths=parents[0].contiguous(), length_dim=0),
                dict(states=x[:1].expand(16, 4, 50, 64)), dict(states=x[:, :, ::2], lengths=parents[0].contiguous(), length_dim=2)):
        args = dict(states=x, parents=parents)
        args.update(bad)
        with pytest.raises((ValueError, qqe.KldEvalError)):
            qqe.beam_reorder(**args)
    qqe.beam_reorder([], parents)
