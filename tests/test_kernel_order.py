"""Order of waits, releases and fences in the sources of the matrices' kernels
(CPU): what no run on one GPU would show."""
import pathlib
import re

import pytest

CSRC = pathlib.Path(__file__).resolve().parent.parent / "deformable_convolution_gb300" / "csrc"
KERNELS = ("fp8.cu", "fp8_matmul.cu", "fp8_pointwise.cu", "muon.cu", "muon_products.cu", "muon_small.cu")


def source(name):
    """A file without comments and empty lines."""
    code = (line.split("//")[0].rstrip() for line in (CSRC / name).read_text().splitlines())
    return "".join(line + "\n" for line in code if line)


def lines(name):
    """(indentation, code) of its lines."""
    return [(len(line) - len(line.lstrip()), line.strip()) for line in source(name).splitlines()]


@pytest.mark.parametrize("name", KERNELS)
def test_dependents_are_released_after_the_own_wait(name):
    """A kernel that lets its dependent start has itself waited: what runs in a
    dependent's prologue may read what was produced two launches earlier."""
    code = lines(name)
    for i, (indent, text) in enumerate(code):
        if "pdl_release()" in text:
            # the statement before it, under the same conditions
            assert code[i - 1] == (indent, "pdl_wait();"), f"{name}: a release that does not follow a wait"


def test_what_one_lane_has_waited_for_is_ordered_for_the_warp():
    """A vote does not order memory among a warp's lanes: where one lane polled, a
    warp barrier stands between the vote and what the others read."""
    text = source("muon_products.cu")
    votes = [m.end() for m in re.finditer(r"if \(lane == 0\) here = inputs_done\(q\);", text)]
    assert len(votes) == 2
    for at in votes:
        assert re.match(r"\s*here = __all_sync\(0xffffffffu, here\);\s*__syncwarp\(\);", text[at:])
    wait = re.search(r"bool warp_wait\(.*?\n}\n", source("tc_pair.cuh"), re.S).group(0)
    assert re.search(r"done = __all_sync\(0xffffffffu, done\);\s*__syncwarp\(\);\s*return done;", wait)
