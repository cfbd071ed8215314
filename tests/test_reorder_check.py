"""The check of a reordering's states and geometry, which a caller with states of
several geometries makes before the first of its calls: on the host, without a
device, refusing what the call refuses and nothing else."""
import ctypes

import pytest

import quantization_quality_eval_amd as qqe

OK, BAD, RANGE = qqe.KLD_OK, qqe.KLD_ERR_INVALID_ARG, qqe.KLD_ERR_RANGE
P = 4096   # an address that is never followed


def check(states=(P,), **kw):
    a = dict(n_items=2, n_beams=3, beam=64, outer=1, outer_stride=0, positions=4, nbytes=16)
    assert not set(kw) - set(a)
    a.update(kw)
    arr = (ctypes.c_void_p * max(len(states), 1))(*states)
    return qqe.load_library().kld_eval_beam_reorder_check(arr, len(states), *a.values())


@pytest.mark.parametrize("kw", [
    dict(n_items=-1), dict(n_beams=0), dict(n_beams=65), dict(outer=-1), dict(positions=-1), dict(nbytes=-1),
    dict(states=(P, None)), dict(beam=0), dict(beam=63), dict(beam=-64), dict(outer=2, outer_stride=63, beam=128),
    dict(outer=2, outer_stride=64, beam=127), dict(outer=2, outer_stride=0, beam=128),
    dict(positions=2**40, nbytes=2**40), dict(beam=2**60), dict(states=(P, P)), dict(states=(P, P + 63)),
    dict(states=(P, P + 6 * 64 - 1)), dict(states=(P + 64, P))])
def test_refuses(kw):
    assert check(**kw) == BAD
    assert "kld_eval_beam_reorder_check" in qqe.kld_eval_last_error()


def test_refuses_no_states_and_too_many_rows():
    assert qqe.load_library().kld_eval_beam_reorder_check(None, 1, 2, 3, 64, 1, 0, 4, 16) == BAD
    assert check(n_items=(1 << 22) // 3 + 1) == RANGE
    with pytest.raises(qqe.KldEvalError, match="overlap"):
        qqe.kld_eval_beam_reorder_check([P, P], 2, 3, 64, 1, 0, 4, 16)


@pytest.mark.parametrize("kw", [
    dict(), dict(states=(P, P + 6 * 64)), dict(states=(P, P + 128), outer=2, outer_stride=64, beam=256),
    dict(states=(P, P + 64), beam=128), dict(outer=2, outer_stride=6 * 64, beam=64),
    dict(n_items=1, n_beams=1, beam=0), dict(outer_stride=-5), dict(states=()), dict(n_items=0), dict(outer=0),
    dict(positions=0), dict(nbytes=0), dict(positions=0, beam=0)])
def test_takes(kw):
    assert check(**kw) == OK
