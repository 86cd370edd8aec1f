"""Which build of the block boundary's kernels a shape takes, from the library's launch plans."""
from rmsnorm_fwd_02_gb300 import _native as N

NO_POST, NO_PRE, NO_GATE = N.BLOCK_PLAN_NO_NORM_BEHIND, N.BLOCK_PLAN_NO_NORM_BEFORE, \
    N.BLOCK_PLAN_NO_GATE
ONE, NORM8 = N.BLOCK_PLAN_ONE_INPUT, N.BLOCK_PLAN_ACT8_NORM

# (name, flags): the kernels' forms, each with every combination of what it stages
FORWARD = [("both", 0), ("pre", NO_POST), ("post", NO_PRE), ("norm8", NORM8), ("norm8", NORM8 | ONE)]
BACKWARD = [("both", 0), ("both", ONE), ("both", NO_GATE), ("pre", NO_POST), ("pre", NO_POST | ONE),
            ("norm", NO_POST | NO_GATE), ("norm", NO_POST | NO_GATE | ONE), ("post", NO_PRE),
            ("post", NO_PRE | NO_GATE)]
NORM8_BACKWARD = [("norm", NORM8), ("norm", NORM8 | ONE)]


def plans(rows, h):
    """(backward, form, packed, plan) of every kernel that rows of h values are given to."""
    for form, flags in FORWARD:
        yield 0, form, 0, N.rmsnorm_block_train_launch_plan(rows, h, 1, 0, 0, flags)
    for packed in (0, 1):
        for form, flags in BACKWARD + (NORM8_BACKWARD if packed else []):
            p = N.rmsnorm_block_train_launch_plan(rows, h, 1, 1, packed, flags)
            p["dh"], p["lane_rows"] = not flags & ONE, lane_rows(p, rows)
            yield 1, form, packed, p


def lane_rows(p, rows):
    """Rows that a thread sums up."""
    side = 32 // p["row_threads"] if p["row_threads"] < 32 else 1
    return -(-rows // (p["ctas"] * p["teams"] * side))


def additions(p, rows):
    """Most additions one after another in a column sum, of one level or of two (runs of about the
    root of the rows, in whole ring slots)."""
    side = 32 // p["row_threads"] if p["row_threads"] < 32 else 1
    slots = -(-(-(-rows // p["ctas"])) // p["rows"])      # of a CTA, which its teams take in turns
    n = -(-slots // p["teams"]) * (p["rows"] // side)
    n = max(n, lane_rows(p, rows) + 1)                    # or each a run of its own
    if lane_rows(p, rows) <= 64:
        return n + 9
    f = 16
    while f * f < lane_rows(p, rows):
        f *= 2
    f = -(-f * side // p["rows"]) * (p["rows"] // side)
    return f + -(-n // f) + 9


def most_threads(h, backward, form, packed, p):
    """Of a CTA of the build that a plan p names."""
    if not backward:
        return 512 if form == "norm8" else 384
    if form == "norm":
        three = p["vectors"] == 3 and p["row_threads"] in (32, 64)
        return 512 if packed and (three or h > 6144) else 384
    return 384 if form == "both" and packed and h <= 6144 else 256


def build(h, backward, form, packed, p):
    """What tells a plan's build from the others of its activation type."""
    even = p["vectors"] >= 3 and p["row_threads"] >= 32 and \
        h == 8 * p["vectors"] * p["row_threads"]
    threads = most_threads(h, backward, form, packed, p) if p["vectors"] >= 3 else 0
    levels = 0
    if backward and p["lane_rows"] > 64:
        levels = "dh" if p["dh"] else "no dh"
    return backward, form, packed, p["vectors"], even, threads, levels


def builds(rows, h):
    return {build(h, *k) for k in plans(rows, h)}
