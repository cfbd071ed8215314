"""What drawing tokens asks of its workspace (no GPU): in proportion to the logits
whatever their shape, and enough for at least one row."""
import pytest

import quantization_quality_eval_amd as qqe

SIZES = {0: 4, 1: 2}
PASS = 1 << 28      # what a pass may take where the logits themselves take less


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("rows,vocab", [(1, 1), (1, 60), (1, 32000), (64, 151936), (32768, 60), (32768, 1024), (32768, 8192), (8192, 32000),
                                        (1 << 22, 1), (1 << 22, 8), (1 << 22, 60), (100000, 4000), (3, 1 << 22), (1 << 22, 1 << 22)])
def test_workspace_is_in_proportion(rows, vocab, dtype):
    need = qqe.kld_eval_sample_workspace(vocab, dtype, rows)
    one = qqe.kld_eval_sample_workspace(vocab, dtype, 1)
    assert 0 < one <= need <= max(PASS, rows * vocab * SIZES[dtype], one)
    assert need == qqe.kld_eval_sample_workspace(vocab, 1 - dtype, rows)      # one workspace serves either type
    # a row: its slices' bins, its own, and a list of no more tokens than it has
    assert one <= -(-vocab // 8192) * 3000 + 4000 + 8 * min(vocab, 16384)
    assert need == qqe.sample_workspace_bytes(vocab, rows, ("f32", "bf16")[dtype])


def test_workspace_of_ordinary_batches_holds_all_rows():
    for rows, vocab in ((1, 151936), (64, 151936), (1024, 151936), (512, 32000), (16384, 2000)):
        assert qqe.kld_eval_sample_workspace(vocab, 1, rows) == rows * qqe.kld_eval_sample_workspace(vocab, 1, 1) or (
            rows * qqe.kld_eval_sample_workspace(vocab, 1, 1) > PASS)


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("vocab", [1, 60, 3000, 8192, 16385, 32000, 151936, 1 << 22])
def test_workspace_of_a_batch_serves_smaller_ones(vocab, dtype):
    counts = sorted({int(1.07 ** i) for i in range(225)} | {1 << 22})
    needs = [qqe.kld_eval_sample_workspace(vocab, dtype, n) for n in counts]
    assert all(a <= b for a, b in zip(needs, needs[1:]))
