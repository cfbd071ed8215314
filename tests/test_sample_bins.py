"""The arithmetic that drawing tokens places logits with (csrc/kld_bins.h), on
the host: compiled with the undefined-behaviour sanitizer, which ends the
program at a conversion out of range, and compared with exact fractions."""
import math
import os
import subprocess

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
    """(z, largest logit of the slice, c) -> the bin that the scan adds z to."""
    return program(tmp_path_factory, "scanned", r"""
int main() {
    double z, m, per;
    while (scanf("%la %la %la", &z, &m, &per) == 3) {
        const double base = base_of(static_cast<float>(m), per);
        printf("%d\n", bin_or_none(rint(fma(z, per, -base))));
    }
}
""")


def test_every_logit_of_a_scan_has_a_bin_or_none(scanned):
    """Excluded tokens, logits that a small temperature puts far below and an infinite temperature's NaN are
    placed behind the bins without a conversion out of range."""
    log2e = 1.4426950408889634
    cases = []
    for heat in (1e-300, 1e-45, 1e-30, 1e-6, 0.01, 0.7, 1.0, 50.0, 1e12, 1e30, 1e300, INF):
        per = min(4 * log2e / heat, 1e200)
        for m in (0.0, 1e-30, 1.0, -1.0, 37.5, -2000.0, 1e5, MOST, -MOST):
            if abs(m * per) >= 2.0 ** 45:
                continue
            m = float(np.float32(m))
            for z in (-INF, -MOST, max(m - 1e6 * (1 + abs(m)), -MOST), max(m - 1.0, -MOST), m):
                cases.append((float(np.float32(z)), m, per))
    answers = scanned(cases)
    assert len(answers) == len(cases) > 200
    for (z, m, per), (got,) in zip(cases, answers):
        if z == -INF:
            assert got == BINS, (z, m, per)
        else:
            below = (m - z) * per
            assert got == BINS if below > BINS + 2 else 0 <= got <= BINS, (z, m, per, got)
            assert z != m or got <= 2
