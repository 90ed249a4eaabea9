"""The training-step operators where their formulas reach the ends of the number
range, where calls are very large, and where layouts are unusual."""
import numpy as np
import pytest
import torch

import adaptive_residual_gradient_amd as A
import operator_refs as R
from test_gpu_adamw import P
from test_gpu_gated_scan import Case

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


# ---- AdamW ----

@pytest.mark.parametrize("size", [1e14, 1e16, 1e17, 1e18, 1e20, 1e25, 1e30, 1e38])
def test_packed_step_of_large_gradients(size):
    """Gradients up to float32's end, beside ones of any smaller size: every weight takes its step."""
    n = 8192
    gen = torch.Generator(device=DEV).manual_seed(1)
    g = torch.randn(n, generator=gen, device=DEV).clamp_(-3, 3) * size
    g[::3] *= 10.0 ** (-30 * torch.rand(n, generator=gen, device=DEV)[::3])
    w = torch.randn(n, generator=gen, device=DEV)
    w0, p = R.f64(w), dict(P, step=1)
    opt = A.Optimizer([(0, n, 0.1, 1.0)])
    mc, vc = (torch.zeros(n, dtype=torch.uint8, device=DEV) for _ in range(2))
    A.adamw_packed(opt, w, g, mc, vc, opt.moment_scales(DEV), seed=1, **p)
    m, v = R.moments(R.f64(g) * p["scale"], np.zeros(n), np.zeros(n), p)
    new, step, denom = R.adamw_weights(w0, m, v, p, 0.1, 1.0)
    R.assert_within(w, new, R.weight_bound(w0, new, m, R.U * np.abs(m), step, denom), "w")


@pytest.mark.parametrize("packed", [False, True])
def test_decay_and_step_size_are_rounded_once(packed):
    """Without a gradient a weight of 1 becomes the decay factor; with a denominator of 1 a weight of 0
    becomes the step size times m.  Both factors are formed in float64."""
    rng = np.random.default_rng(2)
    table = [(4 * i, 4, R.f32(rng.uniform(0.01, 30.0)), R.f32(rng.uniform(0.1, 3.0))) for i in range(500)]
    opt = A.Optimizer(table)
    n = 4 * len(table)
    dt = torch.uint8 if packed else torch.float32
    p = dict(lr=R.f32(0.0123), beta1=0.9, beta2=0.999, eps=1.0, step=3)
    step = A.adamw_packed if packed else A.adamw
    extra = lambda: (opt.moment_scales(DEV),) if packed else ()
    w, zero = torch.ones(n, device=DEV), torch.zeros(n, device=DEV)
    m, v = (torch.zeros(n, dtype=dt, device=DEV) for _ in range(2))
    step(opt, w, zero, m, v, *extra(), **p)
    lr = np.array([p["lr"] * t[3] for t in table])
    keep = (1.0 - lr * np.array([t[2] for t in table])).astype(np.float32)
    assert np.array_equal(w.cpu().numpy(), np.repeat(keep, 4))
    if not packed:
        w, m, v = torch.zeros(n, device=DEV), torch.randn(n, device=DEV), torch.zeros(n, device=DEV)
        step(opt, w, zero, m, v, **p)
        size = (lr / (1.0 - R.f32(0.9) ** 3)).astype(np.float32)
        assert np.array_equal(w.cpu().numpy(), -np.repeat(size, 4) * m.cpu().numpy())


# ---- gated scan ----

def check_any(got, want, bound, what):
    """Finite values within their bound; infinities and NaN in the same places."""
    got = R.f64(got)
    assert np.array_equal(np.isnan(got), np.isnan(want)), what
    far = np.isinf(want)
    assert np.array_equal(got[far], want[far]) and not np.isinf(got[~far]).any(), what
    fine = np.isfinite(want)
    R.assert_within(got[fine], want[fine], bound[fine], what)


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,T,D", [(2, 15, 40),      # one thread a channel
                                   (2, 120, 40),     # one tile
                                   (3, 3000, 40),    # few chains of tiles
                                   (70, 900, 20)])   # many
@np.errstate(invalid="ignore", over="ignore")
def test_infinite_states_stay(B, T, D, dtype, sigmoid):
    """A carried infinity stays one under gates whose products are far below the smallest number, and
    turns to NaN at a gate of 0; neighbouring channels stay finite."""
    c = Case(B, T, D, dtype, sigmoid, seed=8)
    if sigmoid:
        c.z.fill_(-0.4)
    else:
        c.z.fill_(0.4)
        c.z[:, :, 1::5] *= -1
        c.z[:, T // 2, 2::5] = 0
    c.h0[:, :D // 2], c.h0[:, D // 4:D // 2] = float("inf"), float("-inf")
    (h, e), (last, el) = R.scan_forward(R.f64(c.z), R.f64(c.x), R.f64(c.h0), c.n, sigmoid, dtype)
    c.forward()
    check_any(c.h, h, R.rounded(h, e, dtype), "h")
    check_any(c.last, last, R.rounded(last, el, torch.float32), "h_last")
    c.h0 = torch.randn(B, D, device=DEV)
    c.forward()
    c.dl[:, :D // 2], c.dl[:, D // 4:D // 2] = float("inf"), float("-inf")
    want = R.scan_backward(R.f64(c.z), R.f64(c.x), R.f64(c.h), R.f64(c.dh), R.f64(c.h0), R.f64(c.dl), c.n, sigmoid,
                           dtype)
    c.backward()
    for got, (v, err), what, dt in ((c.dz, want[0], "dgate", dtype), (c.dx, want[1], "dx", dtype),
                                    (c.dh0, want[2], "dh0", torch.float32)):
        check_any(got, v, R.rounded(v, err, dt), what)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T", [1, 40])
def test_gate_factors_of_16_bit_types(T, dtype):
    """The states of 16-bit calls are float32: gates of any size give them as many right bits as float32
    gates do."""
    B, D = 3, 1500
    c = Case(B, T, D, dtype, True, seed=9)
    c.z.copy_(torch.linspace(-30, 60, D, device=DEV).expand(B, T, D))
    for h0 in (torch.zeros_like(c.h0), c.h0):
        c.h0 = h0
        c.forward()
        _, (last, el) = R.scan_forward(R.f64(c.z), R.f64(c.x), R.f64(h0), c.n, True, torch.float32)
        R.assert_within(c.last, last, R.rounded(last, el, torch.float32), "h_last")
        c.backward()
        want = R.scan_backward(R.f64(c.z), R.f64(c.x), R.f64(c.h), R.f64(c.dh), R.f64(h0), R.f64(c.dl), c.n, True,
                               torch.float32)
        R.assert_within(c.dh0, want[2][0], R.rounded(want[2][0], want[2][1], torch.float32), "dh0")


def test_factors_of_far_float32_gates():
    """Either factor keeps its bits down to float32's smallest normal numbers."""
    D = 4000
    z = torch.linspace(-86.9, 86.9, D, device=DEV).view(1, 1, D)
    one, zero, last = torch.ones(1, D, device=DEV), torch.zeros(1, D, device=DEV), torch.empty(1, D, device=DEV)
    h = torch.empty_like(z)
    for x, h0, want in ((zero, one, 1 / (1 + np.exp(-R.f64(z)))), (one, zero, 1 / (1 + np.exp(R.f64(z))))):
        A.gated_scan(z, x.view(1, 1, D), h, h0=h0, h_last=last)
        R.assert_within(last, want[0], R.rounded(want[0], 10 * R.U * want[0], torch.float32), "factor")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_long_chains_give_the_same_bits(dtype):
    """Few long chains of tiles, many times: with other work beside them, and a sequence by itself."""
    B, T, D = 2, 20000, 130
    c = Case(B, T, D, dtype, True, seed=10)
    c.z.add_(8.0)      # gates so close to 1 that a state reaches across many tiles
    keys = ("h", "last", "dz", "dx", "dh0")
    c.forward()
    c.backward()
    first = {k: getattr(c, k).clone() for k in keys}
    side, room = torch.cuda.Stream(), torch.empty(1 << 28, device=DEV)
    for i in range(30):
        if i % 2:
            torch.cuda.synchronize()
            with torch.cuda.stream(side):
                room.add_(1.0)
        c.forward()
        c.backward()
        torch.cuda.synchronize()
        for k in keys:
            assert torch.equal(getattr(c, k), first[k]), (i, k)
    for b in range(B):
        one = Case(1, T, D, dtype, True)
        for k in ("z", "x", "dh", "h0", "dl"):
            setattr(one, k, getattr(c, k)[b:b + 1].contiguous())
        one.forward()
        one.backward()
        for k in keys:
            assert torch.equal(getattr(one, k), first[k][b:b + 1]), (b, k)


def test_one_sequence_of_millions_of_steps():
    """The two parts of one very long sequence, the state handed over, give what the whole does."""
    B, T, D, cut = 1, 16_600_000, 64, 8_000_000
    gen = torch.Generator(device=DEV).manual_seed(11)
    z, x = (torch.randn(B, T, D, generator=gen, device=DEV) for _ in range(2))
    h, part = torch.empty_like(z), torch.empty_like(z)
    last, state = torch.empty(B, D, device=DEV), torch.empty(B, D, device=DEV)
    ws = A.gated_scan_workspace(B, T, D, DEV)
    A.gated_scan(z, x, h, h_last=last, ws=ws)
    A.gated_scan(z[:, :cut], x[:, :cut], part[:, :cut], h_last=state, ws=ws)
    tail = torch.empty_like(state)
    A.gated_scan(z[:, cut:], x[:, cut:], part[:, cut:], h0=state, h_last=tail, ws=ws)
    # a state is a mean of inputs of about 1 over the few steps that its gates reach back, with 10 roundings a step
    bound = 10 * 64 * R.U * float(x.abs().max())
    assert float((h - part).abs().max()) <= bound and float((last - tail).abs().max()) <= bound


@pytest.mark.parametrize("B,T", [(4, 1), (3, 2), (1, 1), (1, 300), (5, 40)])
@pytest.mark.parametrize("time_first", [False, True])
def test_halves_of_one_projection(B, T, time_first):
    """gate and input, and their gradients, as halves of one buffer, for one step and with time first in memory."""
    D = 64
    c = Case(B, T, D, torch.bfloat16, True)
    c.forward()
    c.backward()
    size = (T, B, 2 * D) if time_first else (B, T, 2 * D)
    both, grads = (torch.full(size, 7.0, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    if time_first:
        both, grads = both.transpose(0, 1), grads.transpose(0, 1)
    both[:, :, :D], both[:, :, D:] = c.z, c.x
    h, dh0 = torch.empty_like(c.h), torch.empty_like(c.dh0)
    A.gated_scan(both[:, :, :D], both[:, :, D:], h, h0=c.h0, ws=c.ws)
    A.gated_scan_backward(both[:, :, :D], both[:, :, D:], h, c.dh, grads[:, :, :D], grads[:, :, D:], h0=c.h0,
                          dh_last=c.dl, dh0=dh0, ws=c.ws)
    assert torch.equal(h, c.h) and torch.equal(dh0, c.dh0)
    assert torch.equal(grads[:, :, :D], c.dz) and torch.equal(grads[:, :, D:], c.dx)
    # the input's half of the buffer receives the states
    out = both.clone(memory_format=torch.preserve_format)
    x = c.x.clone()
    A.gated_scan(out[:, :, :D], x, out[:, :, D:], h0=c.h0, ws=c.ws)
    assert torch.equal(out[:, :, D:], c.h) and torch.equal(out[:, :, :D], c.z)
    # halves that share a channel
    with pytest.raises(A.AdaCompError):
        A.gated_scan(out[:, :, :D], x, out[:, :, D - 1:2 * D - 1], h0=c.h0, ws=c.ws)


def test_example_with_one_step():
    """The example's layers on one token of several sequences."""
    import pathlib
    import sys
    sys.path.insert(0, str(pathlib.Path(__file__).resolve().parent.parent / "examples"))
    import train_gated_layers as E
    losses = E.train(layers=1, width=64, batch=4, length=1, learners=2, steps=3, log=lambda s: None)
    assert all(x == x for x in losses)


# ---- layer norm ----

def test_layer_norm_of_parts_of_wider_rows():
    """Any leading axes whose rows lie at one distance, and axes of one place wherever they lie."""
    B, T, D = 3, 50, 96
    gen = torch.Generator(device=DEV).manual_seed(3)
    both, grads = (torch.randn(B, T, 2 * D, generator=gen, device=DEV) for _ in range(2))
    x, dy = both[:, :, :D], both[:, :, D:]
    y, dx = grads[:, :, :D], grads[:, :, D:]
    kept = [torch.empty(B * T, device=DEV) for _ in range(4)]
    sums = [torch.empty(D, device=DEV) for _ in range(4)]
    ws = A.layer_norm_workspace(B * T, D, DEV)
    A.layer_norm(x, None, None, y, *kept[:2])
    A.layer_norm_backward(dy, x, None, *kept[:2], dx, *sums[:2], ws)
    x2, dy2 = x.contiguous(), dy.contiguous()
    y2, dx2 = torch.empty_like(x2), torch.empty_like(x2)
    A.layer_norm(x2, None, None, y2, *kept[2:])
    A.layer_norm_backward(dy2, x2, None, *kept[2:], dx2, *sums[2:], ws)
    assert torch.equal(y, y2) and torch.equal(dx, dx2) and torch.equal(sums[0], sums[2])
    assert torch.equal(kept[0], kept[2]) and torch.equal(sums[1], sums[3])
    last = both[:, -1:, :D]          # [B, 1, D]: one distance between its rows
    A.layer_norm(last, None, None, y2[:, :1].contiguous())
    out = torch.empty(B, 1, D, device=DEV)
    A.layer_norm(last, None, None, out)
    assert torch.equal(out[:, 0], y2[:, -1])
    spread = torch.zeros(B, 1, D, device=DEV).expand(B, T, D)
    for bad in (both[:, ::2, :D].transpose(0, 1), both[:2, :7, :D], both[:, :, ::2], spread, spread.transpose(0, 1)):
        with pytest.raises(TypeError):
            A.layer_norm(bad, None, None, torch.empty(bad.shape, device=DEV))
    with pytest.raises(A.AdaCompError):      # one row for all of them
        A.layer_norm(torch.zeros(D, device=DEV).expand(B, T, D), None, None, torch.empty(B, T, D, device=DEV))


def test_layer_norm_of_more_rows_than_one_workgroup_each():
    """67 million rows: as the two halves of them give, and the weight's sums within their bound."""
    rows, cols, half = (1 << 26) + 77, 4, 1 << 25
    gen = torch.Generator(device=DEV).manual_seed(4)
    new = lambda: torch.randn(rows, cols, generator=gen, device=DEV, dtype=torch.float16)
    x, dy = new(), new()
    w = 1 + 0.2 * torch.randn(cols, generator=gen, device=DEV)
    y, y2 = torch.empty_like(x), torch.empty_like(x)
    kept = [torch.empty(rows, device=DEV) for _ in range(4)]
    parts = (slice(0, half), slice(half, rows))
    A.layer_norm(x, w, None, y, *kept[:2])
    for s in parts:
        A.layer_norm(x[s], w, None, y2[s], *(k[s] for k in kept[2:]))
    assert torch.equal(y, y2) and torch.equal(kept[0], kept[2]) and torch.equal(kept[1], kept[3])
    dw, db = torch.empty(cols, device=DEV), torch.empty(cols, device=DEV)
    A.layer_norm_backward(dy, x, w, *kept[:2], y, dw, db, A.layer_norm_workspace(rows, cols, DEV))
    for s in parts:
        A.layer_norm_backward(dy[s], x[s], w, *(k[s] for k in kept[:2]), y2[s])
    assert torch.equal(y, y2)
    want = [torch.zeros(cols, dtype=torch.float64, device=DEV) for _ in range(4)]
    for i in range(0, rows, 1 << 23):
        s = slice(i, min(rows, i + (1 << 23)))
        hat = (x[s].double() - kept[0][s, None].double()) * kept[1][s, None].double()
        d = dy[s].double()
        for t, v in zip(want, (d * hat, d, (d * hat).abs(), d.abs())):
            t += v.sum(0)
    # 256 workgroups of 64 teams: a team's rows one after the other, the teams, the partial rows
    chain = rows / (256 * 64) + 64 + R.SUM
    for got, value, size in ((dw, want[0], want[2]), (db, want[1], want[3])):
        R.assert_within(got, R.f64(value), chain * R.U * R.f64(size), "weight's sums")
