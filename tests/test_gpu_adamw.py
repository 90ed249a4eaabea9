"""Gradient norm and AdamW on the GPU against the 64-bit forms: tables of odd
tensors with gaps, every gradient type, float32 and 8-bit moments (codes and
scales equal), clipping, the bf16 copy, many steps, graphs and streams."""
import math

import numpy as np
import pytest
import torch

import adaptive_residual_gradient_amd as A
import operator_refs as R

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
P = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, step=7, scale=0.125)
TABLES = {
    # one element; a block's edge on either side; a tile's edge on either side; gaps of 4 and more
    "edges": [(0, 1, 0.1, 1.0), (4, 31, 0.0, 0.5), (36, 32, 0.1, 1.0), (76, 33, 0.0, 2.0), (120, 4095, 0.1, 1.0),
              (4216, 4096, 0.01, 1.0), (8312, 4097, 0.0, 1.0), (12412, 3, 0.1, 0.0)],
    # table order is not memory order
    "backwards": [(20000, 9001, 0.1, 1.0), (100, 64, 0.0, 0.5), (9000, 10007, 0.0, 1.0)],
    "one": [(0, 100000, 0.125, 1.0)],
    # more tiles than the norm's first pass has workgroups
    "large": [(0, 2048 * 4096 + 5, 0.1, 1.0)],
}
GRADS = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def make(table, grad, seed, outlier=True):
    span = max(o + n for o, n, _, _ in table)
    span = (span + 3) // 4 * 4 + 4
    gen = torch.Generator(device=DEV).manual_seed(seed)
    rand = lambda s: torch.randn(span, generator=gen, device=DEV) * s
    inside = torch.zeros(span, dtype=torch.bool, device=DEV)
    for o, n, _, _ in table:
        inside[o:o + n] = True
    g = rand(1e-2)
    if outlier:
        g[::97] *= 50
    s = {"w": rand(0.05), "g": g.to(grad), "m": rand(1e-3), "v": rand(1e-3) ** 2, "inside": inside, "span": span}
    # whatever lies between the tensors is not used
    s["g"][~inside] = float("nan")
    return s


def places(o, n):
    return np.arange(o, o + n, dtype=np.uint64)


@pytest.mark.parametrize("name", TABLES)
@pytest.mark.parametrize("grad", GRADS)
def test_grad_norm(name, grad):
    table = TABLES[name]
    s = make(table, GRADS[grad], 1)
    opt = A.Optimizer(table)
    clip = torch.full((2,), -1.0, device=DEV)
    total = math.sqrt(sum(float((s["g"][o:o + n].double() ** 2).sum()) for o, n, _, _ in table))
    for max_norm in (0.0, 0.125 * total * 0.3, 0.125 * total * 3):
        A.grad_norm(opt, s["g"], clip, opt.norm_workspace(DEV), max_norm, scale=0.125)
        norm, coef = clip.tolist()
        assert abs(norm - 0.125 * total) <= 2 * R.U * 0.125 * total
        want = min(1.0, R.f32(max_norm) / (0.125 * total))
        assert abs(coef - want) <= 2 * R.U * want


@pytest.mark.parametrize("bad,coef", [(float("inf"), 0.0), (float("nan"), 1.0)])
def test_grad_norm_not_finite(bad, coef):
    opt = A.Optimizer([(0, 5000, 0.0, 1.0)])
    g = torch.ones(5000, device=DEV)
    g[4997] = bad
    clip = torch.zeros(2, device=DEV)
    A.grad_norm(opt, g, clip, opt.norm_workspace(DEV), 1.0)
    assert not math.isfinite(float(clip[0])) and float(clip[1]) == coef


@pytest.mark.parametrize("name", TABLES)
@pytest.mark.parametrize("grad", GRADS)
@pytest.mark.parametrize("clip,copy", [(False, True), (True, False)])
def test_adamw_float_moments(name, grad, clip, copy):
    table = TABLES[name]
    s = make(table, GRADS[grad], 2)
    opt = A.Optimizer(table)
    c = torch.tensor([3.0, 0.7], device=DEV) if clip else None
    w16 = torch.full((s["span"],), 9.0, dtype=torch.bfloat16, device=DEV) if copy else None
    old = {k: s[k].clone() for k in "wmv"}
    A.adamw(opt, s["w"], s["g"], s["m"], s["v"], clip=c, weights_bf16=w16, **P)
    out = ~s["inside"]
    for k in "wmv":
        assert torch.equal(s[k][out], old[k][out])      # between the tensors nothing is written
    factor = P["scale"] * (float(c[1]) if clip else 1.0)
    for o, n, decay, lr_scale in table:
        part = slice(o, o + n)
        g, w0, m0, v0 = (R.f64(t[part]) for t in (s["g"], old["w"], old["m"], old["v"]))
        g = g * factor
        m, v = R.moments(g, m0, v0, P)
        # factor, product, 1 - beta and their product: 4 roundings; v's square: twice and one more
        em = R.U * (5 * 0.1 * np.abs(g) + np.abs(m)) + 2.0 ** -149
        R.assert_within(s["m"][part], m, em, "m")
        R.assert_within(s["v"][part], v, R.U * (9 * 0.001 * g * g + v) + 2.0 ** -148, "v")
        new, size, denom = R.adamw_weights(w0, m, v, P, decay, lr_scale)
        R.assert_within(s["w"][part], new, R.weight_bound(w0, new, m, em, size, denom), "w")
        if copy:
            assert torch.equal(w16[part], s["w"][part].bfloat16())
    if copy:
        assert bool((w16[out] == 9.0).all())


def pack(table, m, v, span, seed):
    """8-bit moments of float values (rounded down)."""
    mc, vc = (torch.full((span,), 0x55, dtype=torch.uint8, device=DEV) for _ in range(2))
    scales = []
    for o, n, _, _ in table:
        both = []
        for codes, x, positive in ((mc, m, False), (vc, v, True)):
            q, scale = R.quantise(R.f64(x[o:o + n]), np.zeros(n), positive)
            codes[o:o + n] = torch.tensor(q, device=DEV).float().to(torch.float8_e4m3fn).view(torch.uint8)
            both.append(scale)
        scales.append(np.stack(both, 1).reshape(-1))
    return mc, vc, torch.tensor(np.concatenate(scales), dtype=torch.uint8, device=DEV)


def unpack(codes, scale, o, n):
    x = R.f64(codes[o:o + n].view(torch.float8_e4m3fn).float())
    return np.ldexp(x, np.repeat(scale.astype(np.int64) - 127, R.BLOCK)[:n])


def check_packed(table, s, old, w, mc, vc, scales, p, seed, factor):
    at = 0
    for o, n, decay, lr_scale in table:
        nb = (n + R.BLOCK - 1) // R.BLOCK
        before = old["scales"][2 * at:2 * (at + nb)].cpu().numpy()
        after = scales[2 * at:2 * (at + nb)].cpu().numpy()
        m0, v0 = unpack(old["m"], before[0::2], o, n), unpack(old["v"], before[1::2], o, n)
        m, v = R.moments(R.f64(s["g"][o:o + n]) * factor, m0, v0, p)
        bits = R.random_bits(places(o, n), seed, p["step"])
        for codes, x, k, r in ((mc, m, 0, bits & np.uint64(0xFFFF)), (vc, v, 1, bits >> np.uint64(16))):
            q, scale = R.quantise(x, r.astype(np.float64), bool(k))
            np.testing.assert_array_equal(after[k::2], scale)
            np.testing.assert_array_equal(R.f64(codes[o:o + n].view(torch.float8_e4m3fn).float()), q)
        w0 = R.f64(old["w"][o:o + n])
        new, size, denom = R.adamw_weights(w0, m, v, p, decay, lr_scale)
        R.assert_within(w[o:o + n], new, R.weight_bound(w0, new, m, R.U * np.abs(m), size, denom), "w")
        at += nb


@pytest.mark.parametrize("name", TABLES)
@pytest.mark.parametrize("grad", ["f32", "bf16", "f16"])
def test_adamw_packed_moments(name, grad):
    table = TABLES[name]
    s = make(table, GRADS[grad], 3)
    opt = A.Optimizer(table)
    mc, vc, scales = pack(table, s["m"], s["v"], s["span"], 5)
    clip = torch.tensor([3.0, 0.7], device=DEV)
    w16 = torch.full((s["span"],), 9.0, dtype=torch.bfloat16, device=DEV)
    old = {"w": s["w"].clone(), "m": mc.clone(), "v": vc.clone(), "scales": scales.clone()}
    A.adamw_packed(opt, s["w"], s["g"], mc, vc, scales, seed=11, clip=clip, weights_bf16=w16, **P)
    check_packed(table, s, old, s["w"], mc, vc, scales, P, 11, P["scale"] * float(clip[1]))
    out = ~s["inside"]
    assert torch.equal(mc[out], old["m"][out]) and torch.equal(vc[out], old["v"][out])
    assert torch.equal(s["w"][out], old["w"][out]) and bool((w16[out] == 9.0).all())
    assert torch.equal(w16[s["inside"]], s["w"][s["inside"]].bfloat16())


def test_adamw_packed_from_zero_many_steps():
    """From zeroed codes and scales, gradients of very different sizes (zero blocks, tiny and huge
    ones): each step from the codes the step before left."""
    table = TABLES["edges"]
    s = make(table, torch.float32, 4)
    opt = A.Optimizer(table)
    mc, vc = (torch.zeros(s["span"], dtype=torch.float8_e4m3fn, device=DEV) for _ in range(2))
    scales = opt.moment_scales(DEV)
    size = torch.ones(s["span"], device=DEV)
    for i, x in enumerate((0.0, 1e-18, 1e-6, 1e6, 1e15)):
        size[300 + 64 * i:300 + 64 * (i + 1)] = x
    for step in range(1, 6):
        gen = torch.Generator(device=DEV).manual_seed(100 + step)
        s["g"] = torch.randn(s["span"], generator=gen, device=DEV) * size
        p = dict(P, step=step)
        old = {"w": s["w"].clone(), "m": mc.clone(), "v": vc.clone(), "scales": scales.clone()}
        A.adamw_packed(opt, s["w"], s["g"], mc, vc, scales, seed=3, **p)
        check_packed(table, s, old, s["w"], mc, vc, scales, p, 3, p["scale"])
    first = vc[4312:4320].view(torch.uint8)
    assert bool((first > 0).all())      # a second moment above zero stays above


@pytest.mark.parametrize("value", [3.0, 3.1, 0.07, 1e-4])
def test_adamw_packed_rounding_is_unbiased(value):
    """The mean of many codes of one value is the value: a value that a code holds stays, any other of
    2^17 elements goes up with probability p, so the share that does is within 6 standard deviations of p."""
    n = 1 << 17
    opt = A.Optimizer([(0, n, 0.0, 1.0)])
    g = torch.full((n,), value, device=DEV)
    g[::32] = 4.48          # every block's scale comes from its first element
    w = torch.zeros(n, device=DEV)
    mc, vc = (torch.zeros(n, dtype=torch.uint8, device=DEV) for _ in range(2))
    scales = opt.moment_scales(DEV)
    A.adamw_packed(opt, w, g, mc, vc, scales, lr=0.0, beta1=0.0, beta2=0.5, step=1, seed=9)
    scale = 2.0 ** (int(scales[0]) - 127)
    q = mc.view(torch.float8_e4m3fn).float().double() * scale
    rest = torch.ones(n, dtype=torch.bool, device=DEV)
    rest[::32] = False
    vals = q[rest].unique().tolist()
    if value == 3.0:
        assert vals == [3.0]
        return
    value = R.f32(value)
    assert len(vals) == 2 and vals[0] < value < vals[1]
    p = (value - vals[0]) / (vals[1] - vals[0])
    share = float((q[rest] == vals[1]).double().mean())
    assert abs(share - p) < 6 * math.sqrt(p * (1 - p) / int(rest.sum())) + 2.0 ** -16


def test_nan_stays_in_its_element_and_block():
    n = 4096
    opt = A.Optimizer([(0, n, 0.0, 1.0)])
    g = torch.ones(n, device=DEV)
    g[40] = float("nan")
    w, m, v = (torch.zeros(n, device=DEV) for _ in range(3))
    A.adamw(opt, w, g, m, v, lr=1e-3)
    assert torch.isnan(w).nonzero().flatten().tolist() == [40]
    w = torch.zeros(n, device=DEV)
    mc, vc = (torch.zeros(n, dtype=torch.uint8, device=DEV) for _ in range(2))
    A.adamw_packed(opt, w, g, mc, vc, opt.moment_scales(DEV), lr=1e-3)
    assert torch.isnan(w).nonzero().flatten().tolist() == [40]
    codes = mc.view(torch.float8_e4m3fn).float()
    assert torch.isnan(codes).nonzero().flatten().tolist() == [40]


def test_packed_random_bits_go_by_the_element_index():
    """The same tensor at two places of the buffer takes different random bits; the same call twice the
    same ones."""
    n = 1 << 14
    table = [(0, n, 0.0, 1.0), (n, n, 0.0, 1.0)]
    opt = A.Optimizer(table)
    g = torch.randn(n, device=DEV).repeat(2)
    outs = []
    for _ in range(2):
        w = torch.zeros(2 * n, device=DEV)
        mc, vc = (torch.zeros(2 * n, dtype=torch.uint8, device=DEV) for _ in range(2))
        sc = opt.moment_scales(DEV)
        A.adamw_packed(opt, w, g, mc, vc, sc, lr=1e-3, seed=1)
        outs.append((mc, vc, sc, w))
    for a, b in zip(*outs):
        assert torch.equal(a, b)
    assert not torch.equal(outs[0][0][:n], outs[0][0][n:])


@pytest.mark.parametrize("packed", [False, True])
def test_step_in_a_graph_and_on_another_stream(packed):
    """grad_norm and the step captured once and replayed on new gradients with eager work between the
    replays: every replay equals the eager calls; so do calls on a side stream."""
    table = TABLES["backwards"]
    opt = A.Optimizer(table)
    span = int(opt.info.span)

    def state():
        gen = torch.Generator(device=DEV).manual_seed(5)
        s = {"w": torch.randn(span, generator=gen, device=DEV), "clip": torch.zeros(2, device=DEV),
             "ws": opt.norm_workspace(DEV), "g": torch.zeros(span, device=DEV)}
        dt = torch.uint8 if packed else torch.float32
        s["m"], s["v"] = torch.zeros(span, dtype=dt, device=DEV), torch.zeros(span, dtype=dt, device=DEV)
        s["sc"] = opt.moment_scales(DEV)
        return s

    def step(s, stream=None):
        A.grad_norm(opt, s["g"], s["clip"], s["ws"], 0.5, stream=stream)
        if packed:
            A.adamw_packed(opt, s["w"], s["g"], s["m"], s["v"], s["sc"], lr=1e-2, step=3, seed=2, clip=s["clip"],
                           stream=stream)
        else:
            A.adamw(opt, s["w"], s["g"], s["m"], s["v"], lr=1e-2, step=3, clip=s["clip"], stream=stream)

    eager, graph, side = state(), state(), state()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        step(graph)
    other = torch.cuda.Stream()
    for i in range(5):
        new = torch.randn(span, device=DEV) * (i + 1)
        for s in (eager, graph, side):
            s["g"].copy_(new)
        g.replay()
        step(eager)
        torch.cuda.synchronize()
        step(side, other)
        other.synchronize()
        for k in ("w", "m", "v", "sc", "clip"):
            assert torch.equal(eager[k], graph[k]), (i, k)
            assert torch.equal(eager[k], side[k]), (i, k)


def test_refusals():
    opt = A.Optimizer([(0, 1000, 0.0, 1.0)])
    f = lambda n=1000: torch.zeros(n, device=DEV)
    w, g, m, v, clip, ws = f(), f(), f(), f(), f(2), opt.norm_workspace(DEV)
    with pytest.raises(A.AdaCompError) as e:
        A.adamw(opt, w, g, m, v, lr=1e-3, step=0)
    assert e.value.status == -1
    for a in ((w, w, m, v), (w, g, w, v), (w, g, m, m)):
        with pytest.raises(A.AdaCompError) as e:
            A.adamw(opt, *a, lr=1e-3)
        assert e.value.status == -1
    with pytest.raises(A.AdaCompError) as e:
        A.adamw(opt, f(996), g, m, v, lr=1e-3)
    assert e.value.status == -5
    big = f(1004)
    with pytest.raises(A.AdaCompError) as e:
        A.adamw(opt, big[1:1001], g, m, v, lr=1e-3)
    assert e.value.status == -3
    with pytest.raises(TypeError):
        A.adamw(opt, w.bfloat16(), g, m, v, lr=1e-3)
    with pytest.raises(TypeError):
        A.adamw(opt, w, g.double(), m, v, lr=1e-3)
    with pytest.raises(TypeError):
        A.adamw(opt, w, big[::1][:2000:2], m, v, lr=1e-3)
    with pytest.raises(ValueError):
        A.adamw(opt, w, g, m, v, lr=1e-3, weights_bf16=torch.zeros(4, dtype=torch.bfloat16, device=DEV))
    with pytest.raises(ValueError):
        A.adamw_packed(opt, w, g, m.to(torch.uint8), v.to(torch.uint8), opt.moment_scales(DEV)[:-2], lr=1e-3)
    with pytest.raises(ValueError):
        A.grad_norm(opt, g, f(3), ws, 1.0)
    with pytest.raises(A.AdaCompError) as e:
        A.grad_norm(opt, g, clip, ws, -1.0)
    assert e.value.status == -1
    with pytest.raises(A.AdaCompError) as e:
        A.grad_norm(opt, g, clip, ws[:0], 1.0)
    assert e.value.status in (-1, -5)
