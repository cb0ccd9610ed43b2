"""Order of waits and releases in the sources of the matrices' kernels
(CPU): what no run on one GPU would show."""
import pathlib

import pytest

CSRC = pathlib.Path(__file__).resolve().parent.parent / "deformable_convolution_gb300" / "csrc"
KERNELS = ("fp8.cu", "fp8_matmul.cu", "fp8_pointwise.cu", "muon.cu", "muon_products.cu", "muon_small.cu")


def lines(name):
    """(indentation, code) of the lines that are not comments alone."""
    out = []
    for line in (CSRC / name).read_text().splitlines():
        code = line.split("//")[0].rstrip()
        if code:
            out.append((len(code) - len(code.lstrip()), code.strip()))
    return out


@pytest.mark.parametrize("name", KERNELS)
def test_dependents_are_released_after_the_own_wait(name):
    """A kernel that lets its dependent start has itself waited: what runs in a
    dependent's prologue may read what was produced two launches earlier."""
    code = lines(name)
    for i, (indent, text) in enumerate(code):
        if "pdl_release()" in text:
            # the statement before it, under the same conditions
            assert code[i - 1] == (indent, "pdl_wait();"), f"{name}: a release that does not follow a wait"
