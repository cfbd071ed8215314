"""What the kernel sources have to keep to, read from their text: properties
that no run shows, since today's compiler happens to give the code they ask for."""
import glob
import os
import re

import quantization_quality_eval_amd as qqe

CSRC = os.path.join(os.path.dirname(os.path.abspath(qqe.__file__)), "csrc")


def code_lines(path):
    """The file's lines with their comments and blank lines left out."""
    text = re.sub(r"/\*.*?\*/", "", open(path).read(), flags=re.S)
    lines = (re.sub(r"//.*", "", line).strip() for line in text.splitlines())
    return [line for line in lines if line]


def test_lanes_of_a_wave_exchange_lds_across_fences():
    """A wave barrier orders the lanes' execution, not what the compiler does
    with their memory accesses: the writes before it need a release and the
    reads behind it an acquire, at the scope of the wave."""
    seen = 0
    for path in sorted(glob.glob(os.path.join(CSRC, "*.hip")) + glob.glob(os.path.join(CSRC, "*.h"))):
        lines = code_lines(path)
        for i, line in enumerate(lines):
            if "__builtin_amdgcn_wave_barrier" not in line:
                continue
            seen += 1
            where = f"{os.path.basename(path)}: {line}"
            assert lines[i - 1] == '__builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");', where
            assert lines[i + 1] == '__builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");', where
    assert seen > 0
