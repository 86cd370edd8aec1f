"""Performance cases of the operators that stand beside the norms in a training step:

  dropout           y = [residual +] keep * x / (1 - p'), the keep mask drawn from a
                    counter-based generator and never stored; the backward draws it again
  rmsnorm_dropout   h = residual + dropout(x), y = rmsnorm(h) * w, and its backward
                    (gradients of x, of the residual and of w)
  groupnorm         group norm with an activation, channels last, and its backward

The generator is Philox4x32 with ten rounds (Salmon, Moraes, Dror and Shaw, "Parallel random
numbers: as easy as 1, 2, 3", SC 2011).  Eight consecutive elements of the flattened tensor
share one block: element i takes the 16-bit half (i & 1) of word (i >> 1) & 3 of the block
with counter (i >> 3, offset) and key seed, both 64 bits, low word first.  It is kept when
that number is at least t = floor(65536 p + 1/2), so p' = t / 65536.

`own` chooses between plain torch operations in 32 bits and the package's own calls.
"""
import random

import torch

own = False

LOW = 0xFFFFFFFF
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
MOST = 65536 * 4096    # elements of the largest activation
MOST_GN = 2 * 262144 * 128
EPS = 1e-6
EPS_GN = 1e-5


# ---- the cases ---------------------------------------------------------------------------

def listed():
    return [
        # the smallest activation of the package's tests: latency alone
        dict(name="dropout_fwd_small", op="dropout", way="fwd", dtype="bf16", rows=64, cols=256,
             p=0.1, residual=False),
        # sizes that no vector width divides, with the residual added, in 32 bits
        dict(name="dropout_add_odd_fp32", op="dropout", way="fwd", dtype="fp32", rows=4099,
             cols=2051, p=0.25, residual=True),
        # the gradient of a large 16-bit activation: bandwidth
        dict(name="dropout_bwd_large_fp16", op="dropout", way="bwd", dtype="fp16", rows=65536,
             cols=4096, p=0.1, residual=False),
        # a sublayer's end in a short batch, and the package's residual workload
        dict(name="rmsnorm_dropout_fwd_small", op="rmsnorm_dropout", way="fwd", w="fp32", rows=64,
             cols=256, p=0.1, dh=False),
        dict(name="rmsnorm_dropout_fwd_residual", op="rmsnorm_dropout", way="fwd", w="bf16",
             rows=30720, cols=6144, p=0.1, dh=False),
        # its backward: a few rows, and the package's largest plain rows with the gradient
        # that comes down the residual branch
        dict(name="rmsnorm_dropout_bwd_few", op="rmsnorm_dropout", way="bwd", w="bf16", rows=96,
             cols=6144, p=0.1, dh=True),
        dict(name="rmsnorm_dropout_bwd_large", op="rmsnorm_dropout", way="bwd", w="bf16",
             rows=65536, cols=4096, p=0.2, dh=True),
        # group norm: the deepest, smallest images of an image model; the widest stage of a
        # batch, with ten channels a group; one large decoded image in 32 bits
        dict(name="groupnorm_fwd_small", op="groupnorm", way="fwd", dtype="bf16", n=2, s=64,
             c=1280, groups=32, act="silu"),
        dict(name="groupnorm_fwd_batch", op="groupnorm", way="fwd", dtype="bf16", n=8, s=4096,
             c=320, groups=32, act="silu"),
        dict(name="groupnorm_fwd_image_fp32", op="groupnorm", way="fwd", dtype="fp32", n=1,
             s=262144, c=128, groups=32, act="silu"),
        # the backward in 16 bits with an odd number of places, and over two large images
        dict(name="groupnorm_bwd_odd_fp16", op="groupnorm", way="bwd", dtype="fp16", n=5, s=1023,
             c=640, groups=32, act="silu"),
        dict(name="groupnorm_bwd_large", op="groupnorm", way="bwd", dtype="bf16", n=2, s=262144,
             c=128, groups=32, act="silu"),
    ]


def _spread(rng, low, high):
    """A whole number of [low, high], its logarithm evenly spread."""
    return min(high, max(low, int(round(low * (high / low) ** rng.random()))))


def draw(rng: random.Random):
    op = rng.choice(["dropout", "rmsnorm_dropout", "groupnorm"])
    way = rng.choice(["fwd", "bwd"])
    p = rng.choice([0.0, rng.uniform(0.01, 0.6), rng.uniform(0.01, 0.6), rng.uniform(0.01, 0.6)])
    if op == "dropout":
        dtype = rng.choice(["bf16", "fp16", "fp32"])
        cols = _spread(rng, 1, 16384)
        rows = _spread(rng, 1, MOST // 2 // cols)
        return dict(op=op, way=way, dtype=dtype, rows=rows, cols=cols, p=p,
                    residual=way == "fwd" and rng.random() < 0.5)
    if op == "rmsnorm_dropout":
        cols = 8 * _spread(rng, 1, 1024)
        rows = _spread(rng, 1, min(131072, MOST // cols))
        return dict(op=op, way=way, w=rng.choice(["bf16", "fp32"]), rows=rows, cols=cols, p=p,
                    dh=way == "bwd" and rng.random() < 0.5)
    dtype = rng.choice(["bf16", "fp16", "fp32"])
    groups = rng.choice([1, 4, 8, 16, 32, 32, 32, 64])
    width = _spread(rng, 1, 2048 // groups)
    while groups * width % 8:
        width += 1
    c = groups * width
    # groups of 32 values at least: the gradient through two or three cancels to nothing
    s = _spread(rng, -(-32 // width), min(262144, MOST_GN // 2 // c))
    n = _spread(rng, 1, max(1, min(64, MOST_GN // 2 // (c * s))))
    return dict(op=op, way=way, dtype=dtype, n=n, s=s, c=c, groups=groups,
                act=rng.choice(["none", "gelu", "silu", "silu"]))


def work(case):
    if case["op"] == "dropout":
        n = case["rows"] * case["cols"]
        return {"bytes": n * BYTES[case["dtype"]] * (3 if case["residual"] else 2), "flops": 2 * n}
    if case["op"] == "rmsnorm_dropout":
        n, t, h = case["rows"] * case["cols"], case["rows"], case["cols"]
        w = h * (4 if case["w"] == "fp32" else 2)
        if case["way"] == "fwd":  # x, residual, h, y; rstd
            return {"bytes": 8 * n + 4 * t + w, "flops": 6 * n}
        # h, dy [, dh], dx, dresidual; rstd; dw
        return {"bytes": (10 if case["dh"] else 8) * n + 4 * t + w + 4 * h, "flops": 13 * n}
    n = case["n"] * case["s"] * case["c"]
    stats = 8 * case["n"] * case["groups"]
    if case["way"] == "fwd":  # x, y
        return {"bytes": 2 * n * BYTES[case["dtype"]] + stats + 8 * case["c"], "flops": 9 * n}
    # x, dy, dx; dw, db
    return {"bytes": 3 * n * BYTES[case["dtype"]] + stats + 16 * case["c"], "flops": 20 * n}


# ---- inputs ------------------------------------------------------------------------------

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, dtype=torch.float32):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)

    r = random.Random(seed)
    s = dict(case=case, seed=r.getrandbits(63), offset=r.getrandbits(40))
    if case["op"] == "dropout":
        t, h, dtype = case["rows"], case["cols"], DTYPES[case["dtype"]]
        s["x"] = normal(t, h, dtype=dtype)  # the activation, or the gradient of the output
        s["residual"] = normal(t, h, dtype=dtype) if case["residual"] else None
    elif case["op"] == "rmsnorm_dropout":
        t, h, bf = case["rows"], case["cols"], torch.bfloat16
        s["w"] = (1 + 0.1 * normal(h)).to(DTYPES[case["w"]])
        if case["way"] == "fwd":
            s["x"] = normal(t, h, dtype=bf)
            s["residual"] = normal(t, h, dtype=bf)
        else:
            s["h"] = normal(t, h, dtype=bf)
            s["dy"] = normal(t, h, dtype=bf)
            s["dh"] = normal(t, h, dtype=bf) if case["dh"] else None
            s["rstd"] = torch.cat([(part.double().square().mean(1) + EPS).rsqrt().float()
                                   for part in s["h"].split(8192)])
    else:
        n, sp, c, dtype = case["n"], case["s"], case["c"], DTYPES[case["dtype"]]
        s["x"] = (normal(n, sp, c) + 0.5 * normal(c)).to(dtype)  # channels with means of their own
        s["w"] = 1 + 0.1 * normal(c)
        s["b"] = 0.1 * normal(c)
        if case["way"] == "bwd":
            s["dy"] = normal(n, sp, c, dtype=dtype)
            x = s["x"].view(n, sp, case["groups"], -1)
            mean = torch.stack([part.double().mean((0, 2)) for part in x])
            var = torch.stack([(part.double() - m[:, None]).square().mean((0, 2))
                               for part, m in zip(x, mean)])
            s["mean"], s["rstd"] = mean.float(), (var + EPS_GN).rsqrt().float()
    return s


# ---- the plain forms ---------------------------------------------------------------------

def _keep(n, p, seed, offset):
    """The keep mask of n elements, and the factor of those kept."""
    q = torch.arange((n + 7) // 8, device="cuda", dtype=torch.int64)
    a, b = q & LOW, q >> 32
    c, d = torch.full_like(q, offset & LOW), torch.full_like(q, offset >> 32)
    k0, k1 = seed & LOW, seed >> 32
    for _ in range(10):
        u, v = a * 0xD2511F53, c * 0xCD9E8D57  # modulo 2^64: both halves of the product
        a, b, c, d = ((v >> 32) & LOW) ^ b ^ k0, v & LOW, ((u >> 32) & LOW) ^ d ^ k1, u & LOW
        k0, k1 = (k0 + 0x9E3779B9) & LOW, (k1 + 0xBB67AE85) & LOW
    words = torch.stack([a, b, c, d], 1)
    bits = torch.stack([words & 0xFFFF, words >> 16], 2).view(-1)[:n]
    t = int(65536 * p + 0.5)
    return bits >= t, 65536.0 / (65536 - t)


def _dropped(x, keep, scale):
    return torch.where(keep.view(x.shape), x * scale, 0.0)


def _act(z, act):
    if act == "silu":
        return z / (1 + torch.exp(-z))
    return 0.5 * z * (1 + torch.erf(z * 0.5 ** 0.5)) if act == "gelu" else z


def _act_slope(z, act):
    if act == "silu":
        s = 1 / (1 + torch.exp(-z))
        return s * (1 + z * (1 - s))
    if act == "gelu":
        density = torch.exp(-0.5 * z * z) / (2 * torch.pi) ** 0.5
        return 0.5 * (1 + torch.erf(z * 0.5 ** 0.5)) + z * density
    return torch.ones_like(z)


def _plain_dropout(s):
    x = s["x"]
    keep, scale = _keep(x.numel(), s["case"]["p"], s["seed"], s["offset"])
    y = _dropped(x.float(), keep, scale)
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return y.to(x.dtype)


def _plain_rmsnorm_dropout_fwd(s):
    x, w = s["x"], s["w"].float()
    keep, scale = _keep(x.numel(), s["case"]["p"], s["seed"], s["offset"])
    h = (s["residual"].float() + _dropped(x.float(), keep, scale)).to(x.dtype)
    rstd = 1 / torch.sqrt(h.float().square().mean(1) + EPS)
    return (h.float() * rstd[:, None] * w).to(x.dtype), rstd, h


def _plain_rmsnorm_dropout_bwd(s):
    h, dy, w, rstd = s["h"].float(), s["dy"].float(), s["w"].float(), s["rstd"][:, None]
    keep, scale = _keep(h.numel(), s["case"]["p"], s["seed"], s["offset"])
    xhat, g = h * rstd, dy * w
    total = rstd * (g - xhat * (g * xhat).mean(1, keepdim=True))
    if s["dh"] is not None:
        total = total + s["dh"].float()
    dw = (dy * xhat).sum(0)
    return _dropped(total, keep, scale).bfloat16(), total.bfloat16(), dw


def _plain_groupnorm_fwd(s):
    case, x = s["case"], s["x"]
    xg = x.float().view(case["n"], case["s"], case["groups"], -1)
    mean = xg.mean((1, 3))
    d = xg - mean[:, None, :, None]
    rstd = 1 / torch.sqrt(d.square().mean((1, 3)) + EPS_GN)
    z = (d * rstd[:, None, :, None]).view(x.shape) * s["w"] + s["b"]
    return _act(z, case["act"]).to(x.dtype), mean, rstd


def _plain_groupnorm_bwd(s):
    case, x, w = s["case"], s["x"], s["w"]
    xg = x.float().view(case["n"], case["s"], case["groups"], -1)
    rstd = s["rstd"][:, None, :, None]
    xhat = (xg - s["mean"][:, None, :, None]) * rstd
    z = xhat.view(x.shape) * w + s["b"]
    dz = s["dy"].float() * _act_slope(z, case["act"])
    dw, db = (dz * xhat.view(x.shape)).sum((0, 1)), dz.sum((0, 1))
    g = (dz * w).view(xg.shape)
    dx = rstd * (g - g.mean((1, 3), keepdim=True) - xhat * (g * xhat).mean((1, 3), keepdim=True))
    return dx.view(x.shape).to(x.dtype), dw, db


def _own(s):
    import rmsnorm_fwd_02_gb300 as R
    case = s["case"]
    op, way = case["op"], case["way"]
    if op == "dropout":
        if way == "bwd":
            return R.dropout_bwd(s["x"], case["p"], s["seed"], s["offset"])
        return R.dropout_fwd(s["x"], case["p"], s["seed"], s["offset"], residual=s["residual"])
    if op == "rmsnorm_dropout":
        if way == "fwd":
            return R.rmsnorm_dropout_fwd(s["x"], s["residual"], s["w"], case["p"], s["seed"],
                                         s["offset"], eps=EPS)
        return R.rmsnorm_dropout_bwd(s["dy"], s["h"], s["rstd"], s["w"], case["p"], s["seed"],
                                     s["offset"], dh=s["dh"])
    if way == "fwd":
        return R.groupnorm_fwd(s["x"], s["w"], s["b"], case["groups"], eps=EPS_GN, act=case["act"])
    return R.groupnorm_bwd(s["dy"], s["x"], s["mean"], s["rstd"], s["w"], s["b"], case["groups"],
                           act=case["act"])


def run(state):
    if own:
        return _own(state)
    op, way = state["case"]["op"], state["case"]["way"]
    if op == "dropout":
        return _plain_dropout(state)
    if op == "rmsnorm_dropout":
        return (_plain_rmsnorm_dropout_fwd if way == "fwd" else _plain_rmsnorm_dropout_bwd)(state)
    return (_plain_groupnorm_fwd if way == "fwd" else _plain_groupnorm_bwd)(state)


# ---- the definitions in 64 bits ----------------------------------------------------------

def _mul_parts(k, v):
    """High and low 32 bits of k * v (both below 2^32), from 16-bit parts of k."""
    low, high = (k & 0xFFFF) * v, (k >> 16) * v       # each below 2^48
    low = low + ((high & 0xFFFF) << 16)               # below 2^49
    return (high >> 16) + (low >> 32), low & LOW


def _kept_factor(n, p, seed, offset):
    """0 for a dropped element and 1 / (1 - p') for a kept one, in 64 bits."""
    dev = "cuda"
    block = torch.arange(-(-n // 8), device=dev, dtype=torch.int64)
    ctr = [block % 2 ** 32, block // 2 ** 32, torch.full_like(block, offset % 2 ** 32),
           torch.full_like(block, offset // 2 ** 32)]
    for i in range(10):
        key = [(seed + i * 0x9E3779B9) % 2 ** 32, (seed // 2 ** 32 + i * 0xBB67AE85) % 2 ** 32]
        h0, l0 = _mul_parts(0xD2511F53, ctr[0])
        h1, l1 = _mul_parts(0xCD9E8D57, ctr[2])
        ctr = [h1 ^ ctr[1] ^ key[0], l1, h0 ^ ctr[3] ^ key[1], l0]
    out = torch.empty(block.numel(), 8, device=dev, dtype=torch.float64)
    threshold = int(65536 * p + 0.5)
    for j in range(8):
        u = (ctr[j // 2] // 65536 ** (j % 2)) % 65536
        out[:, j] = (u >= threshold).double() / (1 - threshold / 65536)
    return out.view(-1)[:n]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "dropout":
        y = _kept_factor(s["x"].numel(), case["p"], s["seed"], s["offset"]).view(s["x"].shape)
        y *= s["x"]
        return y if s["residual"] is None else y + s["residual"]
    if case["op"] == "rmsnorm_dropout":
        t, h = case["rows"], case["cols"]
        f = _kept_factor(t * h, case["p"], s["seed"], s["offset"]).view(t, h)
        w = s["w"].double()
        if case["way"] == "fwd":
            # the norm is taken of h as it is written, in bf16
            hid = (f.mul_(s["x"]) + s["residual"])
            held = hid.bfloat16().double()
            rstd = (held.pow(2).sum(1) / h + EPS).pow(-0.5)
            return held * rstd[:, None] * w, rstd, hid
        xhat = s["h"].double() * s["rstd"].double()[:, None]
        dw = torch.einsum("th,th->h", s["dy"].double(), xhat)
        g = s["dy"].double() * w
        dot = torch.einsum("th,th->t", g, xhat) / h
        total = (g - xhat * dot[:, None]) * s["rstd"].double()[:, None]
        if s["dh"] is not None:
            total += s["dh"]
        return f * total, total, dw
    n, c, k = case["n"], case["c"], case["groups"]
    x = s["x"].double().view(n, -1, k, c // k)
    per = x.shape[1] * x.shape[3]
    wide = (1, 1, k, c // k)
    w, b = s["w"].double().view(wide), s["b"].double().view(wide)
    if case["way"] == "fwd":
        mean = x.sum((1, 3), keepdim=True) / per
        rstd = ((x - mean).pow(2).sum((1, 3), keepdim=True) / per + EPS_GN).pow(-0.5)
        z = (x - mean) * rstd * w + b
        y = z
        if case["act"] == "silu":
            y = z * torch.sigmoid(z)
        elif case["act"] == "gelu":
            y = z * torch.special.ndtr(z)
        return y.view(s["x"].shape), mean.view(n, k), rstd.view(n, k)
    rstd = s["rstd"].double().view(n, 1, k, 1)
    xhat = (x - s["mean"].double().view(n, 1, k, 1)) * rstd
    z = xhat * w + b
    slope = torch.ones_like(z)
    if case["act"] == "silu":
        sig = torch.sigmoid(z)
        slope = sig + z * sig * (1 - sig)
    elif case["act"] == "gelu":
        slope = torch.special.ndtr(z) + z * torch.exp(-z.pow(2) / 2) / (2 * torch.pi) ** 0.5
    dz = s["dy"].double().view(x.shape) * slope
    dw, db = (dz * xhat).sum((0, 1)).view(c), dz.sum((0, 1)).view(c)
    first = (dz * w).sum((1, 3), keepdim=True) / per
    second = (dz * w * xhat).sum((1, 3), keepdim=True) / per
    return ((dz * w - first - xhat * second) * rstd).view(s["x"].shape), dw, db
