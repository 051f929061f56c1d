"""Rules that the kernel sources keep so that a wait which runs out ends the kernel and
does not hang it.  They are read from the sources: breaking one shows only where a GPU
stops answering."""

import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bit_nf4_quantized_27_b200", "csrc")
KERNELS = sorted(os.path.basename(p) for p in glob.glob(os.path.join(CSRC, "*.cuh")))

# Warp-wide instructions with the full mask: every lane has to arrive.
WARP_WIDE = r"(?:ptx::)?elect_one\s*\(|__(?:shfl|ballot|all|any|match_any)\w*_sync\s*\(|__(?:shfl|ballot|all|any)_sync\s*\("


def _code(name):
    text = open(os.path.join(CSRC, name)).read()
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", text, flags=re.S)


@pytest.mark.parametrize("name", KERNELS)
def test_no_lane_skips_a_warp_wide_instruction(name):
    """`ok` is a lane's own record of a wait that ran out: behind `ok && ...` the other
    lanes would wait for this one."""
    found = re.findall(r"\bok\s*&&[^;{]*?(?:%s)[^;{]*" % WARP_WIDE, _code(name))
    assert not found, found


def test_one_lanes_failure_reaches_its_warp():
    """A branch that only the elected lane takes may set `ok`; the warp shares it before its
    next tile."""
    text = _code("pool_kernels.cuh")
    branches = [m.end() for m in re.finditer(r"if \((?:ok && [^{]*)?(?:one|ptx::elect_one\(\))\) \{", text)]
    assert len(branches) >= 6
    for at in branches:
        depth, i = 1, at
        while depth:
            depth += {"{": 1, "}": -1}.get(text[i], 0)
            i += 1
        if re.search(r"\bok = (?!__all_sync)", text[at:i]):
            assert re.match(r"\s*ok = __all_sync\(0xffffffffu, ok\);", text[i:]), text[at:i + 80]
