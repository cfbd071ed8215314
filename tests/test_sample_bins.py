"""The arithmetic that drawing tokens places logits with (csrc/kld_bins.h), on
the host: compiled with the undefined-behaviour sanitizer, which ends the
program at a conversion out of range, and compared with exact fractions."""
import math
import os
import subprocess
from decimal import Decimal, getcontext
from fractions import Fraction

import numpy as np
import pytest

import quantization_quality_eval_amd as qqe
from quantization_quality_eval_amd import build

CSRC = os.path.join(os.path.dirname(os.path.abspath(qqe.__file__)), "csrc")
BINS = 272
INF = math.inf
MOST = 3.4028234663852886e38
NO_GPU_CODE = ["-std=c++17", "-O1", "-ffp-contract=off", "--cuda-host-only", "-Wno-unused-command-line-argument",
               "-Xarch_host", "-fsanitize=float-cast-overflow", "-Xarch_host", "-fno-sanitize-recover=all",
               "-Xarch_host", "-fsanitize-minimal-runtime"]


def program(tmp_path_factory, name, body):
    """A program that reads words from stdin and answers each line by the body's code."""
    folder = tmp_path_factory.mktemp(name)
    source, out = folder / f"{name}.hip", folder / name
    source.write_text('#include "kld_bins.h"\n#include <stdio.h>\nusing namespace kldk;\n' + body)
    subprocess.run([build.hipcc(), *NO_GPU_CODE, "-I", CSRC, str(source), "-o", str(out)], check=True, capture_output=True)

    def ask(lines):
        text = "\n".join(" ".join(float(x).hex() if math.isfinite(x) else str(x) for x in line) for line in lines)
        done = subprocess.run([str(out)], input=text, capture_output=True, text=True, timeout=60)
        assert done.returncode == 0, done.stderr
        return [[float.fromhex(w) if "x" in w else float(w) for w in line.split()] for line in done.stdout.splitlines()]
    return ask


@pytest.fixture(scope="module")
def scanned(tmp_path_factory):
    """(z, largest logit of the slice, temperature) -> the bin that the scan adds z to."""
    return program(tmp_path_factory, "scanned", r"""
int main() {
    double z, m, heat;
    while (scanf("%la %la %la", &z, &m, &heat) == 3) {
        const int bin = spot_of(static_cast<float>(z), frame_of(static_cast<float>(m), heat_of(heat))).bin;
        printf("%d\n", bin < kBins ? bin : kBins);
    }
}
""")


@pytest.fixture(scope="module")
def placed(tmp_path_factory):
    """(z, m, temperature) -> bin and r of z below the largest logit m, and c."""
    return program(tmp_path_factory, "placed", r"""
int main() {
    double z, m, heat;
    while (scanf("%la %la %la", &z, &m, &heat) == 3) {
        const Frame f = frame_of(static_cast<float>(m), heat_of(heat));
        const int bin = bin_of(static_cast<float>(z), f);
        printf("%d %a %a\n", bin, bin >= 0 && bin < kBins ? spot_of(static_cast<float>(z), f).r : 0.0, f.per);
    }
}
""")


def test_every_logit_of_a_scan_has_a_bin_or_none(scanned):
    """Excluded tokens, logits that a small temperature puts far below and an infinite temperature's NaN are
    placed behind the bins without a conversion out of range."""
    log2e = 1.4426950408889634
    cases = []
    for heat in (5e-324, 1e-300, 1e-45, 1e-30, 1e-6, 0.01, 0.7, 1.0, 50.0, 1e12, 1e30, 1e300, 1.7e308, INF):
        for m in (0.0, 1e-30, 1.0, -1.0, 37.5, -2000.0, 1e5, 2.0 ** -149, -2.0 ** -149, MOST, -MOST):
            m = float(np.float32(m))
            for z in (-INF, math.nan, -MOST, max(m - 1e6 * (1 + abs(m)), -MOST), max(m - 1.0, -MOST), m):
                cases.append((float(np.float32(z)), m, heat))
    answers = scanned(cases)
    assert len(answers) == len(cases) > 500
    for (z, m, heat), (got,) in zip(cases, answers):
        if not math.isfinite(z):
            assert got == BINS, (z, m, heat)
        else:
            below = 0.0 if m == z else (m - z) * (4 * log2e / heat if heat > 1e-300 else INF)
            assert got == BINS if below > BINS + 2 else 0 <= got <= BINS and abs(got - below) <= 1, (z, m, heat, got)


def test_a_logit_has_one_bin_whatever_it_lies_below(placed):
    """Logits next to the edge between two bins, below largest logits of any distance: the bins differ by those
    of the largest logits. The first two were told apart by the precision of their distance."""
    log2e = 1.4426950408889634
    cases = [(float.fromhex("-0x1.c3e49cp-1"), float.fromhex("0x1.86dc6529b7038p-6")),
             (float.fromhex("-0x1.48158cp-1"), float.fromhex("0x1.8ab1de3bf08f3p-6"))]
    g = np.random.default_rng(3)
    for _ in range(300):
        z = float(np.float32(-g.uniform(0.5, 2)))
        cases.append((z, 4 * log2e / ((int(g.integers(100, 240)) + 0.5) / -z)))
    lines = []
    for z, heat in cases:
        half = float(np.float32(z / 2))
        lines += [(z, 0.0, heat), (z, z, heat), (z, half, heat), (half, 0.0, heat)]
    answers = placed(lines)
    for i, (z, heat) in enumerate(cases):
        whole, alone, half, shift = (a[0] for a in answers[4 * i:4 * i + 4])
        assert alone == 0 and whole == shift + half, (z, heat, whole, half, shift)


def test_places_are_those_of_exact_fractions(placed):
    """c z is the whole number at the top, less the bin, plus r: r within half a step of float64, at most one half."""
    g = np.random.default_rng(4)
    lines = []
    for _ in range(2000):
        heat = float(10.0 ** g.uniform(-9, 12))
        m = float(np.float32(g.standard_normal() * 10.0 ** g.uniform(-3, 3)))
        if abs(m) / heat < 2.0 ** 42:
            lines.append((float(np.float32(m - g.uniform(0, 50) * heat)), m, heat))
    answers, tops = placed(lines), placed([(m, m, heat) for _, m, heat in lines])
    seen = 0
    for (z, m, heat), (bin_, r, per), (zero, top_r, _) in zip(lines, answers, tops):
        assert zero == 0 and abs(per * heat / (4 * 1.4426950408889634) - 1) < 2.0 ** -51
        below = (Fraction(m) - Fraction(z)) * Fraction(per)
        if bin_ == BINS:
            assert below > BINS - 1
            continue
        seen += 1
        assert 0 <= bin_ < BINS and abs(r) <= 0.5
        err = below - (Fraction(int(bin_)) + Fraction(top_r) - Fraction(r))
        assert abs(err) <= Fraction(1, 2 ** 53), (z, m, heat)
    assert seen > 1000


def test_steep_rows_keep_their_largest_logit_alone(placed):
    for m, heat in ((1.0, 2.0 ** -43), (-3.0, 1e-200), (MOST, 1.0), (-MOST, 1.0), (2.0 ** -149, 5e-324), (0.0, 1e-100)):
        with np.errstate(over="ignore"):
            below = float(np.nextafter(np.float32(m), np.float32(-INF)))
            above = float(np.nextafter(np.float32(m), np.float32(INF)))
        answers = placed([(m, m, heat), (below, m, heat), (above, m, heat), (-INF, m, heat), (math.nan, m, heat)])
        assert [a[0] for a in answers] == [0, BINS, -1, BINS, BINS], (m, heat)


@pytest.fixture(scope="module")
def summed(tmp_path_factory):
    """(r, n) -> the mantissa of r, and what a word to which n such tokens were added says of their count and sum."""
    return program(tmp_path_factory, "summed", r"""
int main() {
    const Raise raise;
    double r, n;
    while (scanf("%la %la", &r, &n) == 2) {
        uint64_t word = 0;
        for (int i = 0; i < static_cast<int>(n); ++i) word += __builtin_bit_cast(uint64_t, raise(r));
        printf("%a %d %a %a\n", mantissa_of(raise(r)), count_in(word), static_cast<double>(units_in(word)),
               static_cast<double>(units_of(raise(r))));
    }
}
""")


def test_mantissas_and_their_sums(summed):
    """A mantissa is within 2^-45.7 of 2^(r / 4), as a whole number of 2^-45; sums and counts of up to 1024 are exact."""
    getcontext().prec = 40
    g = np.random.default_rng(5)
    cases = [(float(r), float(n)) for r in np.concatenate([[-0.5, 0.5, 0.0, -2.0 ** -60], g.uniform(-0.5, 0.5, 400)])
             for n in (0, 1, 2, int(g.integers(3, 1024)), 1023, 1024)]
    for (r, n), (mantissa, count, total, units) in zip(cases, summed(cases)):
        want = (Decimal(2).ln() * Decimal(r) / 4).exp()
        assert abs(Decimal(mantissa) / want - 1) <= Decimal(2.0 ** -45.7), r
        assert units == mantissa * 2.0 ** 45 and units == int(units)
        assert (count, total) == (n, n * units), (r, n)       # below 2^56: even where float64 rounds it alike
