"""Argument checks of the vocabulary operators, on the CPU: every bad call is
refused before a device is touched, empty calls return, and a good call on a
machine without a GPU reports that there is none."""
import ctypes

import pytest
import torch

import quantization_quality_eval_amd as qqe

OK, BAD, RANGE, NODEV = qqe.KLD_OK, qqe.KLD_ERR_INVALID_ARG, qqe.KLD_ERR_RANGE, qqe.KLD_ERR_NO_DEVICE
no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-device path")
P = 4096   # an address that is never followed: the calls below end in the host's checks


def lib():
    return qqe.load_library()


def select(**kw):
    a = dict(logits=P, dtype=0, vocab=100, row_stride=100, n_items=2, n_beams=3, n_select=4, scores=P, finished=P,
             eos=5, so=P, po=P, to=P, fo=P, ws=P, ws_bytes=1 << 40, stream=None)
    assert not set(kw) - set(a)
    a.update(kw)
    return lib().kld_eval_beam_select(*a.values())


def reorder(states=(P,), **kw):
    a = dict(n_items=2, n_beams=3, parents=P, beam=64, outer=1, outer_stride=0, positions=4, nbytes=16, lengths=P,
             stream=None)
    assert not set(kw) - set(a)
    a.update(kw)
    arr = (ctypes.c_void_p * max(len(states), 1))(*states)
    return lib().kld_eval_beam_reorder(arr, len(states), *a.values())


def embed(**kw):
    a = dict(table=P, tt=1, vocab=100, dim=8, stride=8, tokens=P, n=5, scale=1.0, out=P, ot=1, out_stride=8, stream=None)
    assert not set(kw) - set(a)
    a.update(kw)
    return lib().kld_eval_embed(*a.values())


def embed_grad(**kw):
    a = dict(grad=P, gt=1, gstride=8, tokens=P, n=5, vocab=100, dim=8, scale=1.0, out=P, ot=0, ostride=8, acc=0, ws=P,
             ws_bytes=1 << 40, stream=None)
    assert not set(kw) - set(a)
    a.update(kw)
    return lib().kld_eval_embed_grad(*a.values())


@pytest.mark.parametrize("kw", [
    dict(dtype=2), dict(dtype=-1), dict(vocab=0), dict(vocab=2**31), dict(row_stride=99), dict(n_items=-1),
    dict(n_beams=0), dict(n_beams=65), dict(n_select=0), dict(n_select=65), dict(logits=None), dict(logits=P + 2),
    dict(scores=None), dict(scores=P + 2), dict(so=None), dict(po=None), dict(to=None), dict(fo=None), dict(eos=-2),
    dict(eos=100), dict(eos=-1), dict(ws=None), dict(ws=P + 8), dict(ws_bytes=0), dict(row_stride=2**60),
    dict(so=P + 1), dict(po=P + 2), dict(to=P + 3)])
def test_select_refuses(kw):
    assert select(**kw) == BAD
    assert "kld_eval_beam_select" in qqe.kld_eval_last_error()


def test_select_limits_and_empty():
    assert select(n_items=(1 << 22) // 3 + 1) == RANGE
    assert select(n_items=2**62) == RANGE
    assert select(n_items=0, logits=None, scores=None, ws=None, ws_bytes=0) == OK
    need = qqe.kld_eval_beam_select_workspace(100, 0, 2, 3, 4)
    assert need > 0 and select(ws_bytes=need - 1) == BAD
    with pytest.raises(qqe.KldEvalError):
        qqe.kld_eval_beam_select_workspace(100, 0, 2, 3, 0)
    assert lib().kld_eval_beam_select_workspace(100, 0, 2, 3, 4, None) == BAD


@pytest.mark.parametrize("kw", [
    dict(n_items=-1), dict(n_beams=0), dict(n_beams=65), dict(parents=None), dict(parents=P + 2), dict(lengths=P + 1),
    dict(outer=-1), dict(positions=-1), dict(nbytes=-1), dict(states=(P, None)), dict(beam=63), dict(beam=-64),
    dict(outer=2, outer_stride=63, beam=128), dict(outer=2, outer_stride=64, beam=127),
    dict(outer=2, outer_stride=0, beam=128), dict(outer=2, outer_stride=6 * 64 - 1, beam=64),
    dict(positions=2**40, nbytes=2**40), dict(beam=2**60), dict(states=(P, P)), dict(states=(P, P + 63)),
    dict(states=(P, P + 6 * 64 - 1)), dict(states=(P + 64, P)), dict(states=(P, P + 96), outer=2, outer_stride=64, beam=256),
    dict(states=(P, P + 256 * 5 + 64 + 63), outer=2, outer_stride=64, beam=256)])
def test_reorder_refuses(kw):
    assert reorder(**kw) == BAD
    assert "kld_eval_beam_reorder" in qqe.kld_eval_last_error()


def test_reorder_limits_and_empty():
    assert reorder(n_items=(1 << 22) // 3 + 1) == RANGE
    for kw in (dict(states=()), dict(n_items=0), dict(outer=0), dict(positions=0), dict(nbytes=0)):
        assert reorder(parents=None, **kw) == OK


@no_gpu
@pytest.mark.parametrize("kw", [
    dict(), dict(lengths=None), dict(states=(P, P + 6 * 64)), dict(states=(P, P + 128), outer=2, outer_stride=64, beam=256),
    dict(states=(P, P + 64), beam=128), dict(outer=2, outer_stride=6 * 64, beam=64),
    dict(states=(P, P + 64), outer=2, outer_stride=6 * 128, beam=128),
    dict(n_items=1, n_beams=1, beam=0), dict(outer_stride=-5)])
def test_reorder_takes_these_layouts(kw):
    assert reorder(**kw) == NODEV


@pytest.mark.parametrize("kw", [
    dict(tt=2), dict(ot=-1), dict(vocab=0), dict(vocab=2**31), dict(dim=0), dict(dim=2**24 + 1), dict(n=-1),
    dict(stride=7), dict(out_stride=7), dict(table=None), dict(table=P + 1), dict(tokens=None), dict(tokens=P + 2),
    dict(out=None), dict(out=P + 1), dict(scale=float("nan")), dict(scale=float("inf")), dict(stride=2**58)])
def test_embed_refuses(kw):
    assert embed(**kw) == BAD
    assert "kld_eval_embed" in qqe.kld_eval_last_error()


@pytest.mark.parametrize("kw", [
    dict(gt=2), dict(ot=-1), dict(vocab=0), dict(vocab=2**31), dict(dim=0), dict(dim=2**24 + 1), dict(n=-1),
    dict(gstride=7), dict(ostride=7), dict(grad=None), dict(grad=P + 1), dict(tokens=None), dict(tokens=P + 2),
    dict(out=None), dict(out=P + 2), dict(scale=float("nan")), dict(ws=None), dict(ws=P + 4), dict(ws_bytes=0),
    dict(n=0, out=None)])
def test_embed_grad_refuses(kw):
    assert embed_grad(**kw) == BAD
    assert "kld_eval_embed_grad" in qqe.kld_eval_last_error()


def test_embed_limits_and_empty():
    assert embed(n=0, table=None, tokens=None, out=None) == OK
    assert embed_grad(n=0, acc=1, grad=None, tokens=None, out=None, ws=None) == OK
    assert embed_grad(n=2**22 + 1) == RANGE and embed_grad(vocab=2**24 + 1) == RANGE
    with pytest.raises(qqe.KldEvalError) as e:
        qqe.kld_eval_embed_grad_workspace(100, 8, 2**22 + 1)
    assert e.value.status == RANGE
    need = qqe.kld_eval_embed_grad_workspace(100, 8, 5)
    assert need > 0 and embed_grad(ws_bytes=need - 1) == BAD


@no_gpu
def test_good_calls_without_a_device():
    assert select() == NODEV and embed() == NODEV and embed_grad() == NODEV and embed_grad(n=0) == NODEV
    assert select(finished=None, eos=-1, row_stride=1000) == NODEV
    assert embed(stride=100, out_stride=9, ot=0) == NODEV


@pytest.mark.parametrize("n_select", [1, 64])
@pytest.mark.parametrize("vocab", [1, 2**31 - 1])
@pytest.mark.parametrize("items,beams", [(1, 1), (1 << 22, 1), (1 << 16, 64)])
def test_workspace_sizes_at_the_limits(items, beams, vocab, n_select):
    for code in (qqe.KLD_DTYPE_F32, qqe.KLD_DTYPE_BF16):
        n = qqe.kld_eval_beam_select_workspace(vocab, code, items, beams, n_select)
        rows = items * beams   # a sixteenth of the largest logits, a tile and a slice per row, a full chip's slices
        assert 0 < n <= rows * (vocab // 4 + 256) + 16 * 8192 and n < 2**62
    assert 0 < qqe.kld_eval_embed_grad_workspace(min(vocab, 2**24), 2**24, items) < 2**52


# ---- the torch-facing functions: host tensors and wrong shapes are refused ----

def test_binding_refuses_host_tensors():
    z, s = torch.zeros(4, 10), torch.zeros(2, 2)
    with pytest.raises(ValueError, match="device tensor"):
        qqe.beam_select(z, s)
    with pytest.raises(ValueError, match="device tensor"):
        qqe.beam_reorder(torch.zeros(4, 3), torch.zeros(2, 2, dtype=torch.int32))
    with pytest.raises(ValueError, match="device tensor"):
        qqe.embed(z, torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError, match="device tensor"):
        qqe.embed_grad(z, torch.zeros(4, dtype=torch.int32), 10)


def test_state_geometry():
    g = qqe._state_geometry
    x = torch.zeros(6, 4, 10, 8)
    assert g(x, 2, "x") == (4, 320, 10, 32, 1280)
    assert g(x, 1, "x") == (1, 0, 4, 320, 1280)
    assert g(x[:, :, :7], 2, "x") == (4, 320, 7, 32, 1280)
    assert g(x[:, 1:3], 2, "x") == (2, 320, 10, 32, 1280)
    assert g(x.transpose(0, 1).contiguous().transpose(0, 1), 2, "x") == (4, 6 * 320, 10, 32, 320)
    assert g(torch.zeros(6, 2, 3, 10, 8, dtype=torch.bfloat16), 3, "x") == (6, 160, 10, 16, 960)
    assert g(torch.zeros(6, 11, dtype=torch.int32), 1, "x") == (1, 0, 11, 4, 44)
    assert g(torch.zeros(6, 1, 10, 1, 8), 2, "x") == (1, 0, 10, 32, 320)
    for bad in (x.transpose(2, 3), x[:, :, ::2], x[..., :5], torch.zeros(6, 2, 3, 10, 8).transpose(1, 2)):
        with pytest.raises(ValueError):
            g(bad, bad.dim() - 2, "x")


def test_rows_of():
    d = torch.device("cpu")
    x = torch.zeros(4, 10)
    assert qqe._rows_of(x, "x", d) == 10 and qqe._rows_of(x[:, :7], "x", d) == 10 and qqe._rows_of(x[::2], "x", d) == 20
    assert qqe._rows_of(x[:1].expand(1, 10), "x", d) == 10
    for bad in (x[:1].expand(4, 10), x.t(), x[:, ::2]):
        with pytest.raises(ValueError):
            qqe._rows_of(bad, "x", d)
    with pytest.raises(TypeError):
        qqe._rows_of(x, "x", d, torch.bfloat16)
    with pytest.raises(ValueError, match="one stride"):
        qqe._as_rows(torch.zeros(4, 3, 10).transpose(0, 1), 12, 10, "x")
