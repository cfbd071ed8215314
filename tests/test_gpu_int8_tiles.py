"""Every form of the 8-bit product's kernels on the GPU against the oracle: each
size of tile with each way of filling it, both output types, sizes that leave
remainders everywhere. The tolerances are those of test_gpu_int8.py.

Which form a call takes follows from its sizes by the launcher's rule, whose
figures are read from the source here: a rule that sends these sizes elsewhere
fails the first test, without a GPU."""
import os
import re

import pytest

import quantization_quality_eval_amd as qqe

SOURCE = os.path.join(os.path.dirname(os.path.abspath(qqe.__file__)), "csrc", "kld_int8.hip")
UNITS = 256      # compute units


def rule():
    text = open(SOURCE).read()
    tiles = [tuple(int(x) for x in m) for m in re.findall(r"\bc[0-9x]+ = cost\((\d+), (\d+), (\d+)\)", text)]
    assert len(tiles) == 4 and "kUnits = 256" in text and "return (tiles + kUnits - 1) / kUnits * step_ns;" in text
    assert "if (a.n_rows <= 16)\n        return a.n_rows > 8 && a.n_cols >= 16384 ? launch_few<O, 1, 4>(a, stream) : launch_few<O, 1, 2>(a, stream);" in text
    assert "if (a.n_rows <= 64 && a.n_cols <= 8192) return launch_few<O, 2, 2>(a, stream);" in text
    assert "lines && a.dim % (4 * kDepth) == 0 && tiles > kUnits" in text and "kDepth = 64" in text
    return tiles


def form(m, k, n, aligned):
    """(rows, columns of a tile, feed) of a product m x k by n; few rows: groups of 16 rows and of 16 columns."""
    if m <= 16:
        return ("few", 1, 4 if m > 8 and n >= 16384 else 2)
    if m <= 64 and n <= 8192:
        return ("few", 2, 2)
    count = lambda bm, bn: -(-m // bm) * -(-n // bn)  # noqa: E731
    costs = [(-(-count(bm, bn) // UNITS) * ns, -bm * bn, bm, bn) for bm, bn, ns in rule()]
    _, _, bm, bn = min(costs)                       # of equal ones the larger tile
    stream = (bm, bn) == (256, 256) and aligned and k % 256 == 0 and count(bm, bn) > UNITS
    return (bm, bn, "stream" if stream else "lines" if aligned else "registers")


# (k, bytes between rows, bytes past a boundary): three whole stages; seven and a part of one; a part of one alone;
# rows that start anywhere, with and without a whole stage
FEEDS = [(192, 192, 0), (465, 480, 0), (40, 48, 0), (133, 141, 3), (31, 31, 1)]
SIZES = {("few", 1, 2): [(7, 1001)], ("few", 1, 4): [(13, 16401)], ("few", 2, 2): [(45, 1001)],
         (64, 64): [(70, 333)], (64, 128): [(45, 60001), (450, 4001)], (128, 128): [(900, 3001), (101, 30001)],
         (256, 256): [(333, 32001)]}
CASES = [(m, k, n, stride, shift, (*tile, "lines" if (stride | shift) % 16 == 0 else "registers") if tile[0] != "few" else tile)
         for tile, sizes in SIZES.items() for m, n in sizes for k, stride, shift in FEEDS]
CASES += [(m, k, n, k, 0, (256, 256, "stream")) for m, n in ((513, 40001), (1000, 33000)) for k in (256, 768)]
CASES += [(333, 512, 32001, 512, 0, (256, 256, "lines"))]       # whole groups of stages, but a tile for each workgroup


def test_the_cases_take_every_form():
    taken = {form(m, k, n, (stride | shift) % 16 == 0) for m, k, n, stride, shift, _ in CASES}
    assert [form(m, k, n, (stride | shift) % 16 == 0) for m, k, n, stride, shift, _ in CASES] == [c[5] for c in CASES]
    tiles = [(64, 64), (64, 128), (128, 128), (256, 256)]
    assert taken == {("few", 1, 2), ("few", 1, 4), ("few", 2, 2), (256, 256, "stream"),
                     *((*t, feed) for t in tiles for feed in ("lines", "registers"))}


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("m,k,n,stride,shift,what", CASES)
def test_product_of_every_form(m, k, n, stride, shift, what, dtype):
    from tests.gpu_util import say
    from tests.test_gpu_int8 import DEV, TYPES, bytes_, check_product, scales
    import torch
    say(f"[product] {m} x {k} by {n} {dtype}, rows {stride} apart, {shift} past a boundary: {what}")
    x, w = bytes_(m, k, 3, stride - k, shift), bytes_(n, k, 4, stride - k, shift)
    assert all((t.data_ptr() | t.stride(0)) % 16 == 0 for t in (x, w)) == ((stride | shift) % 16 == 0)
    wide = torch.full((m, n + 9), 5.0, dtype=TYPES[dtype], device=DEV)
    check_product(x, scales(m, 1), w, scales(n, 2), dtype, f"{m} x {k} by {n}: {what}", out=wide[:, 5:5 + n])
    assert (wide[:, :5] == 5).all() and (wide[:, 5 + n:] == 5).all()
