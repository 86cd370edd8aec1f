"""8-bit activations and a block's boundary where they are used in ways the other tests do not: views
and gradients at any address, infinities, captured and replayed graphs, side streams, two calls at
once, workspaces with anything in them, offsets past 32 bits, and a network of both."""
import pytest
import torch

import rmsnorm_fwd_02_gb300 as R
from block_cases import DEV, check, check_bwd, check_fwd, f64, normal
from oracle import act8 as OA
from rmsnorm_fwd_02_gb300 import _native as N
from rmsnorm_fwd_02_gb300 import act8 as A8
from test_block_gpu import case

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def equal(a, b):
    return all((p is None and q is None) or torch.equal(p, q) for p, q in zip(a, b, strict=True))


def at_odd_address(t):
    return torch.cat([t.new_zeros(3), t.flatten()])[3:].view_as(t)


def test_views_and_gradients_at_any_address():
    c, f, dy, dh = case(60, 264, 3, True, True, "sample", BF, torch.float32)
    wide = normal(1, 60, 640)
    wide[:, 64:328] = c["x"]
    x, res = wide[:, 64:328], c["residual"].view(3, 20, 264)
    out = R.rmsnorm_block_fwd(**c, **f)
    assert equal(R.rmsnorm_block_fwd(x, c["residual"], **f), out)
    cube = R.rmsnorm_block_fwd(c["x"].view(3, 20, 264), res, **f)
    assert cube[0].shape == (3, 20, 264) and cube[2].shape == (3, 20)
    assert equal([t.reshape(s.shape) for t, s in zip(cube, out)], out)
    odd = {k: at_odd_address(v) if isinstance(v, torch.Tensor) else v for k, v in f.items()}
    assert equal(R.rmsnorm_block_fwd(x, c["residual"], **odd), out)
    grads = R.rmsnorm_block_bwd(dy, c["x"], *out[1:], **f, dh=dh)
    assert equal(R.rmsnorm_block_bwd(at_odd_address(dy), x, *out[1:], **odd, dh=dh.t().contiguous().t()),
                 grads)
    for bad in (wide[:, 4:268], wide[:, 64:592:2], wide.t()[:60, :40]):
        with pytest.raises(ValueError):
            R.rmsnorm_block_fwd(bad, torch.zeros(bad.shape, dtype=BF, device=DEV), w_pre=f["w_pre"])
    with pytest.raises(ValueError, match="residual"):
        R.rmsnorm_block_fwd(c["x"], c["residual"].half(), **f)
    with pytest.raises(ValueError, match="both"):
        R.rmsnorm_block_bwd(dy, R.act8_pack(c["x"]), *out[1:], **f, dh=dh)
    with pytest.raises(ValueError, match="packed"):
        R.rmsnorm_block_bwd(dy, R.act8_pack(c["x"])[1:], *out[1:], **f, dh=dh)
    with pytest.raises(ValueError, match="rstd_pre"):
        R.rmsnorm_block_bwd(dy, c["x"], out[1], out[2].double(), out[3], **f, dh=dh)
    with pytest.raises(ValueError, match="one device"):
        R.rmsnorm_block_fwd(c["x"], c["residual"], w_pre=f["w_pre"].cpu())


def test_no_rows():
    x, w = torch.empty(0, 64, dtype=BF, device=DEV), torch.ones(64, device=DEV)
    gate = torch.ones(3, 64, device=DEV)
    y, h, r2, r1 = R.rmsnorm_block_fwd(x, x, w, w, gate)
    assert y.shape == h.shape == (0, 64) and r1.shape == (0,)
    dx, dres, dw_pre, dw_post, dgate = R.rmsnorm_block_bwd(y, x, h, r2, r1, w, w, gate)
    assert dx.shape == (0, 64) and not (dw_pre.any() or dw_post.any() or dgate.any())


@pytest.mark.parametrize("h", [64, 264, 1536])
@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_one_bad_row_stays_alone(h, bad):
    c, f, dy, dh = case(90, h, 1, True, True, "row", BF, torch.float32)
    rows = torch.arange(90, device=DEV) != 41
    good = R.rmsnorm_block_fwd(**c, **f, act8=True)
    for name in ("x", "residual"):
        c2 = dict(c, **{name: c[name].clone()})
        c2[name][41, h - 3] = bad
        out = R.rmsnorm_block_fwd(**c2, **f, act8=True)
        assert all(torch.equal(p[rows], q[rows]) for p, q in zip(out, good))
        assert not out[0][41].isfinite().all()
    first = R.rmsnorm_block_bwd(dy, c["x"], *good[1:4], **f, dh=dh)
    dy2 = dy.clone()
    dy2[41, 5] = bad
    got = R.rmsnorm_block_bwd(dy2, c["x"], *good[1:4], **f, dh=dh)
    assert torch.equal(got[0][rows], first[0][rows]) and torch.equal(got[1][rows], first[1][rows])
    # the sum over dy meets it in its column alone, and an infinity stays one
    cols = torch.arange(h, device=DEV) != 5
    assert torch.equal(got[2][cols], first[2][cols])
    assert got[2][5].isinf() if bad == float("inf") else got[2][5].isnan()


def test_infinite_gradients_without_a_norm_before():
    c, f, dy, dh = case(700, 264, 1, False, True, "none", BF, torch.float32)
    out = R.rmsnorm_block_fwd(**c, **f)
    dh[300, 9] = float("inf")
    dx, dres, _, dw_post, _ = R.rmsnorm_block_bwd(None, c["x"], None, None, out[3], **f, dh=dh)
    cols = torch.arange(264, device=DEV) != 9
    assert dres[300, 9].isinf() and dw_post[9].isinf() and dw_post[cols].isfinite().all()


def test_zero_rows_and_zero_gates():
    c, f, dy, dh = case(40, 264, 4, True, True, "sample", BF, torch.float32)
    c["x"][7] = 0
    f["gate"][2] = 0
    out = R.rmsnorm_block_fwd(**c, **f)
    check_fwd(out, c["x"], c["residual"], f["w_pre"], f["w_post"], f["gate"], 0.7, 0.9)
    got = R.rmsnorm_block_bwd(dy, c["x"], *out[1:], **f, dh=dh)
    check_bwd(got, dy, dh, c["x"], *out[1:], f["w_pre"], f["w_post"], f["gate"], 0.7, 0.9)
    assert not got[0][20:30].any() and got[4][2].any()


def test_negative_and_zero_scales():
    c, f, dy, dh = case(40, 512, 1, True, False, "row", torch.float16, torch.float32)
    for f["scale"], f["residual_scale"] in ((-1.5, 0.0), (0.0, -1.0)):
        out = R.rmsnorm_block_fwd(**c, **f)
        check_fwd(out, c["x"], c["residual"], f["w_pre"], None, f["gate"], f["scale"], f["residual_scale"])
        got = R.rmsnorm_block_bwd(dy, c["x"], *out[1:], **f, dh=dh)
        check_bwd(got, dy, dh, c["x"], out[1], out[2], None, f["w_pre"], None, f["gate"], f["scale"],
                  f["residual_scale"])


def test_a_broadcast_gate_and_an_x_that_is_the_residual():
    c, f, dy, dh = case(48, 264, 1, True, True, "none", BF, torch.float32)
    x = c["x"].requires_grad_()
    g = torch.tensor(0.3, device=DEV, requires_grad=True)
    y, h = R.rmsnorm_block_train(x, x, f["w_pre"], f["w_post"], g.expand(264), 0.7, 0.9)
    torch.autograd.backward([y, h], [dy, dh])
    plain = R.rmsnorm_block_fwd(x.detach(), x.detach(), f["w_pre"], f["w_post"],
                                torch.full((264,), 0.3, device=DEV), 0.7, 0.9)
    got = R.rmsnorm_block_bwd(dy, x.detach(), *plain[1:], f["w_pre"], f["w_post"],
                              torch.full((264,), 0.3, device=DEV), 0.7, 0.9, dh=dh)
    assert torch.equal(x.grad, got[0] + got[1])
    assert abs(g.grad - got[4].sum()) <= 264 * 2.0 ** -24 * got[4].abs().sum()


def test_workspaces_hold_anything():
    c, f, dy, dh = case(1500, 264, 5, True, True, "sample", BF, torch.float32)
    out = R.rmsnorm_block_fwd(**c, **f)
    want = R.rmsnorm_block_bwd(dy, c["x"], *out[1:], **f, dh=dh)
    nbytes = N.rmsnorm_block_train_bwd_workspace_bytes(1500, 264, 5)
    for fill in (0x00, 0xFF, 0x7F):
        ws = torch.full((nbytes,), fill, dtype=torch.uint8, device=DEV)
        got = [torch.full_like(t, 3.0) for t in want]
        N.rmsnorm_block_train_bwd(dy, dh, c["x"], out[1], 0, N.ACT8_BF16, out[2], out[3], f["w_pre"],
                                  f["w_post"], 1, f["gate"], 1, 5, *got, ws, nbytes, 1500, 264, 264,
                                  0.7, 0.9)
        assert equal(got, want)
    with pytest.raises(N.RmsnError, match="workspace"):
        N.rmsnorm_block_train_bwd(dy, dh, c["x"], out[1], 0, N.ACT8_BF16, out[2], out[3], f["w_pre"],
                                  f["w_post"], 1, f["gate"], 1, 5, *got, ws, nbytes // 4, 1500, 264,
                                  264, 0.7, 0.9)


@pytest.mark.parametrize("act8", [False, True])
def test_captured_steps_replay_on_new_inputs(act8):
    shape = (777, 520)
    w = [(1 + 0.1 * normal(i, 520, dtype=torch.float32)).requires_grad_() for i in (1, 2, 3)]

    def step(x, res, dy):
        y, h = R.rmsnorm_block_train(x, res, w[0], w[1], w[2], 0.5, act8=act8)
        z, h2 = R.rmsnorm_act8_train(y, w[0], residual=h)
        return torch.autograd.grad([z, h2], [x, res, *w], [dy, dy])

    x, res = (normal(i, *shape).requires_grad_() for i in (4, 5))
    dy = normal(6, *shape)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(x, res, dy)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            out = step(x, res, dy)
    torch.cuda.synchronize()
    for seed in (10, 20):
        with torch.no_grad():
            x.copy_(normal(seed, *shape))
            res.copy_(normal(seed + 1, *shape))
            dy.copy_(normal(seed + 2, *shape))
        graph.replay()
        torch.cuda.synchronize()
        want = step(x.detach().clone().requires_grad_(), res.detach().clone().requires_grad_(), dy.clone())
        assert equal(out, want)


def test_two_graphs_and_two_streams_at_once():
    cases = [case(400 + 100 * i, 1536, 1, True, True, "row", BF, torch.float32, seed=i) for i in range(2)]
    streams, graphs, outs, wants = [torch.cuda.Stream() for _ in range(2)], [], [], []
    alive = []      # what the graphs read
    for (c, f, dy, dh), s in zip(cases, streams):
        kept = R.rmsnorm_block_fwd(**c, **f, act8=True)
        alive.append(kept)
        run = lambda c=c, f=f, dy=dy, dh=dh, k=kept: (  # noqa: E731
            *R.rmsnorm_block_fwd(**c, **f, act8=True),
            *R.rmsnorm_block_bwd(dy, k[4], k[5], k[2], k[3], **f, dh=dh))
        wants.append(run())
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            run()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                outs.append(run())
        graphs.append(g)
    torch.cuda.synchronize()
    for _ in range(5):
        for t in (t for o in outs for t in o):
            t.zero_()
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
                g.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, wants):
            assert equal(o, w)


def test_a_producer_on_the_same_side_stream():
    s = torch.cuda.Stream()
    base = normal(3, 3000, 1536)
    w = torch.ones(1536, device=DEV)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        for k in range(1, 4):
            x = base * k
            y, rstd, x8 = R.rmsnorm_act8_fwd(x, w)
            back = R.act8_unpack(x8, 1536)
            z = y + 0
    s.synchronize()
    want = R.rmsnorm_act8_fwd(base * 3, w)
    assert torch.equal(z, want[0]) and torch.equal(back, R.act8_unpack(want[2], 1536))


def test_offsets_past_32_bits():
    rows, h = 540000, 8192          # 4.4e9 elements, 8.8e9 bytes a tensor
    w = (1 + 0.1 * normal(1, h, dtype=torch.float32))
    some = torch.tensor([0, 300000, rows - 2, rows - 1], device=DEV)
    c, f, dy, dh = case(4, h, 1, True, True, "none", BF, torch.float32)
    f["w_pre"] = w

    def spread(t):
        out = torch.zeros(rows, h, dtype=BF, device=DEV)
        out[some] = t
        return out

    x, res = spread(c["x"]), spread(c["residual"])
    y, hid, r2, r1, x8, h8 = R.rmsnorm_block_fwd(x, res, **f, act8=True)
    check_fwd((y[some], hid[some], r2[some], r1[some]), c["x"], c["residual"], w, f["w_post"], None, 0.7,
              0.9)
    assert not y[1:1000].any() and torch.equal(x8[some], R.act8_pack(c["x"]))
    del res, y
    big_dy, big_dh = spread(dy), spread(dh)
    for kx, kh in ((x, hid), (x8, h8)):
        got = R.rmsnorm_block_bwd(big_dy, kx, kh, r2, r1, **f, dh=big_dh)
        small = [got[0][some], got[1][some], *got[2:]]
        check_bwd(small, dy, dh, kx[some], kh[some], r2[some], r1[some], w, f["w_post"], None, 0.7, 0.9)
        assert not got[1][2000:3000].any()
        del got


def test_a_network_of_both_is_its_calls_by_hand():
    # two blocks on a residual stream: gated sublayers with norms on both sides, kept in 8 bits
    T, H = 300, 1536
    w = [(1 + 0.1 * normal(i, H, dtype=torch.float32)).requires_grad_() for i in range(4)]
    gate = normal(9, 3, H, dtype=torch.float32).requires_grad_()
    x = normal(10, T, H).requires_grad_()
    dy, dh = normal(11, T, H), normal(12, T, H)
    y0 = R.rmsnorm_act8_train(x, w[0])
    y1, h1 = R.rmsnorm_block_train(y0, x, w[1], w[2], gate, 0.5, act8=True)
    y2, h2 = R.rmsnorm_block_train(y1, h1, w[3], None, None, 1.0, 0.9, act8=True)
    torch.autograd.backward([y2, h2], [dy, dh])

    d = [t.detach() for t in w]
    a, ra, a8 = R.rmsnorm_act8_fwd(x.detach(), d[0])
    b, hb, rb, pb, xb8, hb8 = R.rmsnorm_block_fwd(a, x.detach(), d[1], d[2], gate.detach(), 0.5, act8=True)
    e, he, re, _, _, he8 = R.rmsnorm_block_fwd(b, hb, d[3], None, None, 1.0, 0.9, act8=True)
    assert torch.equal(y2, e) and torch.equal(h2, he)
    gb, ghb, gw3, _, _ = R.rmsnorm_block_bwd(dy, None, he8, re, None, d[3], None, None, 1.0, 0.9, dh=dh)
    ga, gx, gw1, gw2, gg = R.rmsnorm_block_bwd(gb, xb8, hb8, rb, pb, d[1], d[2], gate.detach(), 0.5, dh=ghb)
    gx0, gw0 = R.rmsnorm_act8_bwd(ga, a8, ra, d[0])
    assert torch.equal(x.grad, gx + gx0)
    assert equal([t.grad for t in w] + [gate.grad], [gw0, gw1, gw2, gw3, gg])


def test_gradients_of_one_output_alone():
    c, f, dy, dh = case(40, 264, 1, True, True, "row", BF, torch.float32)
    for first in (True, False):
        leaves = [t.detach().clone().requires_grad_() for t in
                  (c["x"], c["residual"], f["w_pre"], f["w_post"], f["gate"])]
        out = R.rmsnorm_block_train(*leaves, 0.7, 0.9)
        out[0 if first else 1].backward(dy if first else dh)
        kept = R.rmsnorm_block_fwd(**c, **f)
        want = R.rmsnorm_block_bwd(dy if first else torch.zeros_like(dy), c["x"], *kept[1:], **f,
                                   dh=None if first else dh)
        assert equal([t.grad for t in leaves], want)
    x = c["x"].clone().requires_grad_()       # without a norm before there is no y
    y, h = R.rmsnorm_block_train(x, c["residual"], None, f["w_post"])
    assert y is None
    h.backward(dh)
    assert x.grad.isfinite().all()


@pytest.mark.parametrize("name", ["_current_device", "_empty_strided"])
def test_without_the_private_calls(monkeypatch, name):
    from rmsnorm_fwd_02_gb300 import block as B8
    from rmsnorm_fwd_02_gb300 import dropout as D
    c, f, dy, dh = case(40, 264, 1, True, True, "row", BF, torch.float32)
    want = R.rmsnorm_block_fwd(**c, **f, act8=True)
    if name == "_current_device":
        monkeypatch.setattr(A8, name, torch.cuda.current_device)
    else:
        monkeypatch.setattr(A8, name, D._empty_strided_dispatched)
        monkeypatch.setattr(B8, name, D._empty_strided_dispatched)
    assert equal(R.rmsnorm_block_fwd(**c, **f, act8=True), want)
    assert torch.equal(R.act8_pack(c["x"]), want[4])


def test_held_values_of_the_forward_are_those_of_its_outputs():
    for h in (8, 40, 136, 520, 1544, 8192):
        c, f, _, _ = case(37, h, 1, True, True, "none", BF, torch.float32)
        _, hid, _, _, x8, h8 = R.rmsnorm_block_fwd(**c, **f, act8=True)
        assert (x8.cpu().numpy() == OA.pack(f64(c["x"]))).all()
        assert (h8.cpu().numpy() == OA.pack(f64(hid))).all()
        check(R.act8_unpack(h8, h), OA.held(f64(hid)), 0 * f64(hid))


def test_no_wait_gave_up():
    assert N.rmsnorm_block_train_device_error() == 0
