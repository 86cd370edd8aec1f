"""Tensor-memory loads are asynchronous: what they load may be read only after tcgen05.wait::ld.
Held in the sources, since a build that reads too early can still give right results."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(__file__), "..", "rmsnorm_fwd_02_gb300", "csrc")


def sources(*names):
    """The kernels' sources (by name) without comments."""
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu*"))):
        if not names or os.path.basename(path) in names:
            text = re.sub(r"//[^\n]*|/\*.*?\*/", "", open(path).read(), flags=re.S)
            yield os.path.basename(path), text


def behind(text, at):
    """What follows position `at` up to the end of the block that it stands in."""
    depth, i = 0, at
    while depth >= 0:
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        i += 1
    return text[at:i - 1]


def test_a_load_returns_registers_that_nothing_has_read():
    seen = 0
    for name, text in sources():
        for m in re.finditer(r'"tcgen05\.ld\.', text):
            rest = behind(text, text.index(";", text.index('"memory")', m.end())) + 1)
            assert not rest.strip(), (name, rest)
            seen += 1
    assert seen >= 3


@pytest.mark.parametrize("source", ["blk_bwd.cuh", "ln_bwd.cu", "rmsn_bwd_rows.cuh"])
def test_a_wait_stands_before_the_first_use(source):
    calls = 0
    (_, text), = sources(source)
    for m in re.finditer(r"(?:tmem_ld(?:8|16)|load_cells)\([^;{]*?(\w+)(?:\[\w+\])?\);", text):
        between = text[m.end():text.index("tmem_wait_ld", m.end())]
        between = re.sub(r"(tmem_ld(8|16)|load_cells)\([^;]*;", "", between)
        assert not re.search(rf"\b{m[1]}\b", between), (source, m[0])
        calls += 1
    assert calls >= 2


def test_every_wait_holds_registers():
    """Packing a register into a pair is no memory access, so nothing but the operands of the wait
    keeps a compiler from moving it ahead."""
    calls = 0
    for name, text in sources():
        assert not re.search(r"tmem_wait_ld\(\s*\)", text), name
        calls += len(re.findall(r"tmem_wait_ld\(\w+(?:\[0\])?\);", text))
    assert calls >= 8
