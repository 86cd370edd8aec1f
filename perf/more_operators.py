"""Performance cases of the operators at a block's boundary in a training step:

  act8            activations kept in 8 bits: packed, and unpacked again
  rmsnorm_act8    RMSNorm (with the residual add) that keeps its input in 8 bits, and the
                  backward that reads it
  rmsnorm_block   the norm behind a block, its gate and the residual scales, and the norm before
                  the next block in one pass, and its backward from 16- or 8-bit activations

8 bits: 32 consecutive values of a row (the last block of a row may be shorter) share a power of
two 2^e, the smallest with e >= -120 (and at most 127) whose greatest magnitude times 2^(6 - e)
is below 127.5; a value x is held as the whole number nearest to x 2^(6 - e) (ties to even, at
most 127 in magnitude).  A block that holds an infinity or a NaN is NaN.  A packed row is H
bytes of these numbers, padded to 16, then a byte e + 127 for each block (255: NaN), padded to
16; the padding is zero.

The block's boundary, on rows of H values, with a gate of one row or of one row for each of n
equally long runs of rows (samples):

  h = residual_scale * residual + scale * gate * rmsnorm(x) * w_post
  y = rmsnorm(h) * w_pre    (of h before it is rounded to the 16 bits that are written)

`own` chooses between plain torch operations in 32 bits and the package's own calls.
"""
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
MOST = 65536 * 4096    # elements of the largest activation
EPS = 1e-6


# ---- the cases ---------------------------------------------------------------------------

def listed():
    return [
        # the smallest activation of the package's tests: latency alone
        dict(name="act8_small", op="act8", dtype="bf16", rows=64, cols=256),
        # a width that no vector divides, in 32 bits
        dict(name="act8_odd_fp32", op="act8", dtype="fp32", rows=4099, cols=2051),
        # a large activation of a training step: bandwidth
        dict(name="act8_large", op="act8", dtype="bf16", rows=65536, cols=4096),
        # a whole step (forward, then backward) of a sublayer's norm: a short batch, and the
        # package's residual workload
        dict(name="rmsnorm_act8_step_few", op="rmsnorm_act8", way="step", dtype="bf16", w="fp32",
             rows=96, cols=6144, residual=True, dh=True),
        dict(name="rmsnorm_act8_step_residual", op="rmsnorm_act8", way="step", dtype="bf16",
             w="bf16", rows=30720, cols=6144, residual=True, dh=True),
        # the backward alone, on the package's largest plain rows
        dict(name="rmsnorm_act8_bwd_large", op="rmsnorm_act8", way="bwd", dtype="bf16", w="bf16",
             rows=65536, cols=4096, residual=False, dh=False),
        # a block's boundary with both norms: the smallest, and the largest rows
        dict(name="block_fwd_small", op="rmsnorm_block", way="fwd", dtype="bf16", w="fp32", n=1,
             length=64, cols=256, pre=True, post=True, gate="row", act8=False),
        dict(name="block_fwd_large", op="rmsnorm_block", way="fwd", dtype="bf16", w="bf16", n=1,
             length=65536, cols=4096, pre=True, post=True, gate="none", act8=False),
        # a gate for each sample of a batch, in FP16, an odd number of rows a sample
        dict(name="block_fwd_samples_fp16", op="rmsnorm_block", way="fwd", dtype="fp16", w="fp32",
             n=8, length=4095, cols=1536, pre=True, post=False, gate="sample", act8=False),
        # the backward: a few rows; the largest rows with all that they can have; from 8 bits
        # with a gate for each sample
        dict(name="block_bwd_few", op="rmsnorm_block", way="bwd", dtype="bf16", w="bf16", n=1,
             length=96, cols=6144, pre=True, post=True, gate="none", act8=False, dh=True),
        dict(name="block_bwd_large", op="rmsnorm_block", way="bwd", dtype="bf16", w="bf16", n=1,
             length=65536, cols=4096, pre=True, post=True, gate="row", act8=False, dh=True),
        dict(name="block_bwd_samples_act8", op="rmsnorm_block", way="bwd", dtype="fp16", w="fp32",
             n=5, length=4099, cols=1536, pre=True, post=True, gate="sample", act8=True, dh=True),
    ]


def _spread(rng, low, high):
    """A whole number of [low, high], its logarithm evenly spread."""
    return min(high, max(low, int(round(low * (high / low) ** rng.random()))))


def draw(rng: random.Random):
    op = rng.choice(["act8", "rmsnorm_act8", "rmsnorm_block", "rmsnorm_block"])
    if op == "act8":
        dtype = rng.choice(["bf16", "fp16", "fp32"])
        cols = _spread(rng, 1, 16384)
        return dict(op=op, dtype=dtype, rows=_spread(rng, 1, MOST // 2 // cols), cols=cols)
    cols = 8 * _spread(rng, 1, 1024)
    dtype, w = rng.choice(["bf16", "bf16", "fp16"]), rng.choice(["same", "fp32"])
    case = dict(op=op, way=rng.choice(["bwd", "step" if op == "rmsnorm_act8" else "fwd"]),
                dtype=dtype, w=dtype if w == "same" else w, cols=cols)
    if op == "rmsnorm_act8":
        residual = rng.random() < 0.5
        case.update(rows=_spread(rng, 1, min(131072, MOST // 2 // cols)), residual=residual,
                    dh=residual or rng.random() < 0.3)
        return case
    pre, post = rng.choice([(True, True), (True, True), (True, False), (False, True)])
    gate = rng.choice(["none", "row", "sample"])
    n = _spread(rng, 1, 256) if gate == "sample" else 1
    case.update(n=n, length=_spread(rng, 1, max(1, min(131072, MOST // 2 // cols) // n)), pre=pre,
                post=post, gate=gate, act8=case["way"] == "bwd" and rng.random() < 0.5)
    if case["way"] == "bwd":
        case["dh"] = not pre or rng.random() < 0.7
    return case


def _packed_bytes(cols):
    return -(-cols // 16) * 16 + -(-(-(-cols // 32)) // 16) * 16


def work(case):
    h, e = case["cols"], BYTES[case["dtype"]]
    if case["op"] == "act8":  # x, the packed rows written and read, the values
        t = case["rows"]
        return {"bytes": 2 * t * (h * e + _packed_bytes(h)), "flops": 3 * t * h}
    w = h * BYTES[case["w"]]
    if case["op"] == "rmsnorm_act8":
        t, dh = case["rows"], case["dh"]
        n = t * h
        bwd = t * _packed_bytes(h) + (6 if dh else 4) * n + 4 * t + w + 4 * h
        if case["way"] == "bwd":  # packed x, dy [, dh], dx
            return {"bytes": bwd, "flops": 12 * n}
        fwd = t * _packed_bytes(h) + (8 if case["residual"] else 4) * n + 4 * t + w
        return {"bytes": fwd + bwd, "flops": 18 * n}
    t = case["n"] * case["length"]
    n, norms = t * h, case["pre"] + case["post"]
    rows = 0 if case["gate"] == "none" else case["n"]
    small = norms * (4 * t + w) + rows * h * BYTES[case["w"]]
    if case["way"] == "fwd":  # x, residual, h [, y]
        return {"bytes": (8 if case["pre"] else 6) * n + small, "flops": (4 + 4 * norms) * n}
    saved = t * _packed_bytes(h) if case["act8"] else 2 * n
    kept = case["pre"] + (case["post"] or rows > 0)    # h, x
    grads = case["pre"] + case["dh"] + 2               # dy, dh, dresidual, dx
    return {"bytes": kept * saved + 2 * grads * n + small + 4 * (norms + rows) * h,
            "flops": (4 + 10 * norms) * n}


# ---- inputs ------------------------------------------------------------------------------

def _rstd(x):
    return torch.cat([(part.double().square().mean(1) + EPS).rsqrt().float()
                      for part in x.split(8192)])


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, dtype=torch.float32):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)

    s, h, dtype = dict(case=case), case["cols"], DTYPES[case["dtype"]]
    if case["op"] == "act8":
        s["x"] = normal(case["rows"], h, dtype=dtype)
        return s
    wt = DTYPES[case["w"]]
    if case["op"] == "rmsnorm_act8":
        t = case["rows"]
        s["w"] = (1 + 0.1 * normal(h)).to(wt)
        s["x"] = normal(t, h, dtype=dtype)
        s["residual"] = None
        if case["way"] == "step":
            s["residual"] = normal(t, h, dtype=dtype) if case["residual"] else None
        else:
            s["rstd"] = _rstd(s["x"])
            s["x8"] = torch.cat([_pack(part) for part in s.pop("x").split(8192)])
        s["dy"] = normal(t, h, dtype=dtype)
        s["dh"] = normal(t, h, dtype=dtype) if case["dh"] else None
        return s
    n, t = case["n"], case["n"] * case["length"]
    r = random.Random(seed)
    # depth-scaled branches, and a residual that some networks shrink
    s["scale"], s["residual_scale"] = r.uniform(0.3, 1.0), r.choice([1.0, r.uniform(0.7, 1.0)])
    s["w_pre"] = (1 + 0.1 * normal(h)).to(wt) if case["pre"] else None
    s["w_post"] = (1 + 0.1 * normal(h)).to(wt) if case["post"] else None
    s["gate"] = None
    if case["gate"] != "none":
        s["gate"] = (0.5 + 0.3 * normal(*((n, h) if case["gate"] == "sample" else (h,)))).to(wt)
    s["x"] = (2 * normal(t, h)).to(dtype)
    if case["way"] == "fwd":
        s["residual"] = normal(t, h, dtype=dtype)
        return s
    s["h"] = normal(t, h, dtype=dtype)
    s["dy"] = normal(t, h, dtype=dtype) if case["pre"] else None
    s["dh"] = normal(t, h, dtype=dtype) if case["dh"] else None
    s["rstd_pre"] = _rstd(s["h"]) if case["pre"] else None
    s["rstd_post"] = _rstd(s["x"]) if case["post"] else None
    if not case["pre"]:
        s["h"] = None
    if not case["post"] and case["gate"] == "none":
        s["x"] = None
    if case["act8"]:
        for k in ("x", "h"):
            if s[k] is not None:
                s[k] = torch.cat([_pack(part) for part in s[k].split(8192)])
    return s


# ---- the plain forms ---------------------------------------------------------------------

def _blocks(x):
    """x [rows, H] in 32 bits as blocks [rows, blocks, 32], the last one filled with zeros."""
    rows, h = x.shape
    n = -(-h // 32)
    v = torch.zeros(rows, n * 32, device=x.device, dtype=torch.float32)
    v[:, :h] = x
    return v.view(rows, n, 32)


def _pack(x):
    """Packed rows, uint8."""
    rows, h = x.shape
    v = _blocks(x)
    bits = v.abs().amax(2).view(torch.int32)
    # the exponent; the addition carries into it where the number would round to 128
    e = ((bits + 0x10000) >> 23).clamp(7, 254)
    q = torch.round(v * ((260 - e) << 23).view(torch.float32)[:, :, None]).clamp(-127, 127)
    bad = bits >= 0x7F800000
    q = torch.where(bad[:, :, None], 0.0, q)
    out = torch.zeros(rows, _packed_bytes(h), device=x.device, dtype=torch.uint8)
    out[:, :h] = q.view(rows, -1)[:, :h].to(torch.int8).view(torch.uint8)
    first = -(-h // 16) * 16
    out[:, first:first + e.shape[1]] = torch.where(bad, 255, e).to(torch.uint8)
    return out


def _unpack(p, h):
    """The values of packed rows, in 32 bits."""
    first, n = -(-h // 16) * 16, -(-h // 32)
    e = p[:, first:first + n].to(torch.int32)
    unit = torch.where(e == 255, float("nan"), ((e - 6).clamp(min=0) << 23).view(torch.float32))
    q = p[:, :h].contiguous().view(torch.int8).float()
    return q * unit.repeat_interleave(32, 1)[:, :h]


def _saved(t, case):
    """A kept activation in 32 bits."""
    return _unpack(t, case["cols"]) if t.dtype == torch.uint8 else t.float()


def _norm_bwd(xhat, g, rstd):
    return rstd * (g - xhat * (g * xhat).mean(1, keepdim=True))


def _plain_rmsnorm_act8(s):
    case = s["case"]
    w, dy = s["w"].float(), s["dy"].float()
    first = ()
    if case["way"] == "step":
        h = s["x"]
        if s["residual"] is not None:
            h = (h.float() + s["residual"].float()).to(h.dtype)
            first = (h,)
        rstd = 1 / torch.sqrt(h.float().square().mean(1) + EPS)
        first = ((h.float() * rstd[:, None] * w).to(h.dtype), rstd) + first
        held = _unpack(_pack(h), case["cols"])
    else:
        rstd, held = s["rstd"], _unpack(s["x8"], case["cols"])
    xhat = held * rstd[:, None]
    dx = _norm_bwd(xhat, dy * w, rstd[:, None])
    if s["dh"] is not None:
        dx = dx + s["dh"].float()
    return first + (dx.to(s["dy"].dtype), (dy * xhat).sum(0))


def _gate_rows(s):
    """The gate's factor of every row: [rows, H], [H] or a number."""
    gate = s["gate"]
    if gate is None:
        return 1.0
    gate = gate.float()
    return gate if gate.dim() == 1 else gate.repeat_interleave(s["case"]["length"], 0)


def _plain_block_fwd(s):
    x = s["x"].float()
    rstd_post = rstd_pre = y = None
    if s["w_post"] is not None:
        rstd_post = 1 / torch.sqrt(x.square().mean(1) + EPS)
        x = x * rstd_post[:, None] * s["w_post"].float()
    h = s["residual_scale"] * s["residual"].float() + s["scale"] * _gate_rows(s) * x
    if s["w_pre"] is not None:
        rstd_pre = 1 / torch.sqrt(h.square().mean(1) + EPS)
        y = (h * rstd_pre[:, None] * s["w_pre"].float()).to(s["x"].dtype)
    return tuple(t for t in (y, h.to(s["x"].dtype), rstd_pre, rstd_post) if t is not None)


def _plain_block_bwd(s):
    case, out = s["case"], {}
    dtype = DTYPES[case["dtype"]]
    if s["w_pre"] is not None:
        dy, rstd = s["dy"].float(), s["rstd_pre"][:, None]
        hhat = _saved(s["h"], case) * rstd
        total = _norm_bwd(hhat, dy * s["w_pre"].float(), rstd)
        out["dw_pre"] = (dy * hhat).sum(0)
        if s["dh"] is not None:
            total = total + s["dh"].float()
    else:
        total = s["dh"].float()
    out["dresidual"] = (s["residual_scale"] * total).to(dtype)
    branch = s["scale"] * _gate_rows(s) * total
    if s["w_post"] is not None:
        rstd, w = s["rstd_post"][:, None], s["w_post"].float()
        xhat = _saved(s["x"], case) * rstd
        out["dw_post"] = (branch * xhat).sum(0)
        grown = xhat * w
        branch = _norm_bwd(xhat, branch * w, rstd)
    elif s["gate"] is not None:
        grown = _saved(s["x"], case)
    out["dx"] = branch.to(dtype)
    if s["gate"] is not None:
        dgate = s["scale"] * total * grown
        out["dgate"] = (dgate.sum(0) if s["gate"].dim() == 1
                        else dgate.view(case["n"], -1, case["cols"]).sum(1))
    return tuple(out[k] for k in ("dx", "dresidual", "dw_pre", "dw_post", "dgate") if k in out)


def _own(s):
    import rmsnorm_fwd_02_gb300 as R
    case = s["case"]
    if case["op"] == "act8":
        return R.act8_unpack(R.act8_pack(s["x"]), case["cols"], s["x"].dtype)
    if case["op"] == "rmsnorm_act8":
        if case["way"] == "bwd":
            return R.rmsnorm_act8_bwd(s["dy"], s["x8"], s["rstd"], s["w"], dh=s["dh"])
        y, rstd, x8, *h = R.rmsnorm_act8_fwd(s["x"], s["w"], EPS, residual=s["residual"])
        return (y, rstd, *h) + R.rmsnorm_act8_bwd(s["dy"], x8, rstd, s["w"], dh=s["dh"])
    same = dict(w_pre=s["w_pre"], w_post=s["w_post"], gate=s["gate"], scale=s["scale"],
                residual_scale=s["residual_scale"])
    if case["way"] == "fwd":
        out = R.rmsnorm_block_fwd(s["x"], s["residual"], eps=EPS, **same)
    else:
        out = R.rmsnorm_block_bwd(s["dy"], s["x"], s["h"], s["rstd_pre"], s["rstd_post"],
                                  dh=s["dh"], **same)
    return tuple(t for t in out if t is not None)


def run(state):
    if own:
        return _own(state)
    case = state["case"]
    if case["op"] == "act8":
        x = state["x"]
        return _unpack(_pack(x), case["cols"]).to(x.dtype)
    if case["op"] == "rmsnorm_act8":
        return _plain_rmsnorm_act8(state)
    return (_plain_block_fwd if case["way"] == "fwd" else _plain_block_bwd)(state)


# ---- the definitions in 64 bits ----------------------------------------------------------

def _held(x):
    """What x [rows, H] in 64 bits is worth after being held in 8 bits."""
    rows, h = x.shape
    out = torch.empty_like(x)
    for c in range(0, h, 4096):  # whole blocks at a time
        part = x[:, c:c + 4096]
        n = part.shape[1]
        full = torch.nn.functional.pad(part, (0, -n % 32)).view(rows, -1, 32)
        most = full.abs().max(2).values
        e = torch.frexp(most).exponent.double() - 1
        e = torch.where(most * torch.exp2(6 - e) >= 127.5, e + 1, e)
        e = torch.where(most > 0, e, -120.0).clamp(-120, 127)
        unit = torch.exp2(e - 6)[:, :, None]
        q = torch.round(full / unit).clamp(-127, 127)
        v = torch.where(torch.isfinite(most)[:, :, None], q * unit, float("nan"))
        out[:, c:c + n] = v.view(rows, -1)[:, :n]
    return out


def _opened(p, h):
    """The values of packed rows in 64 bits."""
    at = (h + 15) // 16 * 16
    q = p[:, :h].double()
    q = torch.where(q > 127, q - 256, q)
    e = p[:, at:at + (h + 31) // 32].double()
    unit = torch.where(e < 255, torch.exp2(e - 133), float("nan"))
    return q * unit[:, torch.arange(h, device=p.device) // 32]


def _value(t, h):
    return _opened(t, h) if t.dtype == torch.uint8 else t.double()


def exact(case, seed):
    s, h = prepare(case, seed), case["cols"]
    if case["op"] == "act8":
        return torch.cat([_held(part.double()) for part in s["x"].split(8192)])
    root = lambda v: (v.pow(2).sum(1) / h + EPS).pow(-0.5)  # noqa: E731
    if case["op"] == "rmsnorm_act8":
        w, lead = s["w"].double(), []
        if case["way"] == "step":
            v = s["x"].double()
            if s["residual"] is not None:
                hid = v + s["residual"]
                v = hid.to(s["x"].dtype).double()  # the norm is taken of h as it is written
            rstd = root(v)
            lead = [v * rstd[:, None] * w, rstd] + ([hid] if s["residual"] is not None else [])
            xhat = _held(v)
        else:
            rstd, xhat = s["rstd"].double(), _opened(s["x8"], h)
        xhat *= rstd[:, None]
        dw = torch.einsum("th,th->h", s["dy"].double(), xhat)
        grad = s["dy"].double() * w
        dot = torch.einsum("th,th->t", grad, xhat) / h
        grad.sub_(xhat.mul_(dot[:, None])).mul_(rstd[:, None])
        if s["dh"] is not None:
            grad += s["dh"]
        return (*lead, grad, dw)
    a, b, n, length = s["residual_scale"], s["scale"], case["n"], case["length"]
    gate = torch.ones(1, h, device="cuda", dtype=torch.float64)
    if s["gate"] is not None:
        gate = s["gate"].double().view(-1, h)
    gate = gate.expand(n, h)
    by_sample = (n, length, h)
    if case["way"] == "fwd":
        branch, rstd_post, last = s["x"].double(), None, []
        if s["w_post"] is not None:
            rstd_post = root(branch)
            branch = branch * rstd_post[:, None] * s["w_post"].double()
        hid = a * s["residual"].double() + b * (branch.view(by_sample) * gate[:, None]).view(-1, h)
        if s["w_pre"] is not None:
            rstd_pre = root(hid)
            last = [hid * rstd_pre[:, None] * s["w_pre"].double(), hid, rstd_pre]
        else:
            last = [hid]
        return (*last, rstd_post) if rstd_post is not None else tuple(last)
    dw = []
    if s["w_pre"] is not None:
        rstd = s["rstd_pre"].double()[:, None]
        hhat = _value(s["h"], h) * rstd
        total = s["dy"].double()
        dw.append(torch.einsum("th,th->h", total, hhat))
        total = total * s["w_pre"].double()
        dot = torch.einsum("th,th->t", total, hhat) / h
        total = total.sub_(hhat.mul_(dot[:, None])).mul_(rstd)
        if s["dh"] is not None:
            total += s["dh"]
    else:
        total = s["dh"].double()
    dres = a * total
    if s["w_post"] is None and s["gate"] is None:
        return (b * total, dres, *dw)
    w = torch.ones(h, device="cuda", dtype=torch.float64)
    xhat = _value(s["x"], h)
    if s["w_post"] is not None:
        w = s["w_post"].double()
        rstd = s["rstd_post"].double()[:, None]
        xhat *= rstd
    sums = torch.einsum("nlh,nlh->nh", total.view(by_sample), xhat.view(by_sample)) * b
    dx = (total.view(by_sample) * (gate * w * b)[:, None]).view(-1, h)
    if s["w_post"] is not None:
        dw.append((sums * gate).sum(0))
        dot = torch.einsum("th,th->t", dx, xhat) / h
        dx.sub_(xhat.mul_(dot[:, None])).mul_(rstd)
    if s["gate"] is not None:
        dw.append((sums * w).view(s["gate"].shape))
    return (dx, dres, *dw)
