"""Launch plans of every kernel of a block's boundary and of the norm that keeps 8 bits, over every
width, and which builds the GPU tests' shapes take.  Without a GPU."""
import pytest

from block_builds import NO_GATE, NO_POST, NO_PRE, NORM8, ONE, build, builds, most_threads, plans
from test_abi_host import lib  # noqa: F401  (the module fixture)
from test_block_builds_gpu import MANY, SHAPES
from test_block_long_gpu import LONG, PART

from rmsnorm_fwd_02_gb300 import _native as N

ROWS = (1, 7, 152, 153, 2000, 100000, (1 << 31) - (1 << 16))


@pytest.mark.parametrize("rows", ROWS)
def test_every_forms_plan_fits_the_device(lib, rows):
    size = N.rmsnorm_block_train_bwd_workspace_bytes
    for h in range(8, 8193, 8):
        floats = 0
        for backward, form, packed, p in plans(rows, h):
            where = (rows, h, backward, form, packed, p)
            assert p["stages"] >= 2 and p["smem"] <= 227 * 1024 and 1 <= p["ctas"] <= 152, where
            assert p["threads"] <= most_threads(h, backward, form, packed, p), where
            assert 8 * p["vectors"] * p["row_threads"] >= h, where
            side = 32 // p["row_threads"] if p["row_threads"] < 32 else 1
            assert p["threads"] == p["teams"] * side * p["row_threads"], where
            assert p["rows"] % side == 0, where
            if backward:
                floats = max(floats, p["ctas"] * h * ((form != "post") + (form != "norm")))
        assert size(rows, h, 1) >= 4 * floats


@pytest.mark.parametrize("backward,flags,packed,n", [
    (0, NO_POST | NO_PRE, 0, 1), (1, NO_POST | NO_PRE, 0, 1), (0, ONE, 0, 1), (1, ONE | NO_PRE, 0, 1),
    (1, NORM8, 0, 1), (0, NORM8 | NO_POST, 0, 1), (1, NORM8 | NO_GATE, 1, 1), (0, NORM8, 0, 2),
    (1, NO_GATE, 0, 2), (0, 64, 0, 1), (0, -2, 0, 1), (0, 0, 2, 1),
])
def test_plans_that_no_call_has_are_refused(lib, backward, flags, packed, n):
    with pytest.raises(N.RmsnError):
        N.rmsnorm_block_train_launch_plan(64, 256, n, backward, packed, flags)


def test_the_long_tests_shapes_have_two_levels_in_every_form(lib):
    for rows, h in LONG:
        assert rows % (3 * PART) == 0
        for backward, form, packed, p in plans(rows, h):
            assert not backward or p["lane_rows"] > 64, (rows, h, form, packed, p)


def test_the_gpu_tests_take_every_build(lib):
    there = set().union(*(builds(rows, h) for h in range(8, 8193, 8) for rows in ROWS))
    taken = set().union(*(builds(rows, h) for rows, h in SHAPES + MANY + LONG))
    assert taken == there, sorted(there - taken, key=str)


@pytest.mark.parametrize("packed", [0, 1])
def test_which_widths_take_a_third_more_rows(lib, packed):
    """As the rule's comment says (blk_launch.h): rows of one or two warps of three vectors a thread."""
    norm = NO_POST | NO_GATE
    threads = {h: N.rmsnorm_block_train_launch_plan(100000, h, 1, 1, packed, norm)["threads"]
               for h in range(8, 6145, 8)}
    assert [h for h in threads if threads[h] > 384] == [768, 1536] * packed
