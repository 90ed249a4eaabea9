"""The training-step operators at the ends of their ranges: places past 32 bits,
every number of rows a workgroup of the layer norm gradients can hold, long
chains of scan tiles, and what the entry points refuse."""
import numpy as np
import pytest
import torch

import adaptive_residual_gradient_amd as A
import operator_refs as R
from test_gpu_adamw import P
from test_gpu_gated_scan import Case
from test_gpu_layer_norm import EPS, backward

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.mark.parametrize("packed", [False, True])
def test_adamw_places_past_32_bits(packed):
    """A tensor that begins before element 2^32 and ends behind it: the same steps as one call on its part alone,
    and (8 bits) random bits that go by the whole index."""
    n, at = 5003, (1 << 32) - 2504
    span = at + (n + 3) // 4 * 4
    gen = torch.Generator(device=DEV).manual_seed(1)
    old = {"w": torch.randn(n, generator=gen, device=DEV), "g": torch.randn(n, generator=gen, device=DEV).bfloat16(),
           "m": torch.zeros(n, device=DEV), "v": torch.zeros(n, device=DEV)}
    opt = A.Optimizer([(at, n, 0.1, 1.0)])
    part = slice(at, at + n)
    state = torch.uint8 if packed else torch.float32
    big = {"w": torch.empty(span, device=DEV), "g": torch.empty(span, dtype=torch.bfloat16, device=DEV),
           "m": torch.empty(span, dtype=state, device=DEV), "v": torch.empty(span, dtype=state, device=DEV)}
    for k, t in big.items():
        t[part] = old[k].to(t.dtype)
    clip = torch.empty(2, device=DEV)
    A.grad_norm(opt, big["g"], clip, opt.norm_workspace(DEV), 1e9)
    norm = float(old["g"].double().norm())
    assert abs(float(clip[0]) - norm) <= 2 * R.U * norm
    g = R.f64(old["g"]) * P["scale"]
    m, v = R.moments(g, np.zeros(n), np.zeros(n), P)
    if packed:
        scales = opt.moment_scales(DEV)
        A.adamw_packed(opt, big["w"], big["g"], big["m"], big["v"], scales, seed=4, **P)
        bits = R.random_bits(np.arange(at, at + n, dtype=np.uint64), 4, P["step"])
        for k, x, positive, r in (("m", m, False, bits & np.uint64(0xFFFF)), ("v", v, True, bits >> np.uint64(16))):
            q, scale = R.quantise(x, r.astype(np.float64), positive)
            np.testing.assert_array_equal(scales[int(positive)::2].cpu().numpy(), scale)
            np.testing.assert_array_equal(R.f64(big[k][part].view(torch.float8_e4m3fn).float()), q)
    else:
        A.adamw(opt, big["w"], big["g"], big["m"], big["v"], **P)
    new, size, denom = R.adamw_weights(R.f64(old["w"]), m, v, P, 0.1, 1.0)
    # the gradient's product with 1 - beta: 5 roundings, as in the tests of small tables
    em = R.U * (5 * 0.1 * np.abs(g) + np.abs(m)) + 2.0 ** -149
    R.assert_within(big["w"][part], new, R.weight_bound(R.f64(old["w"]), new, m, em, size, denom), "w")


def test_layer_norm_rows_past_32_bits():
    """Rows 2^21 + 64 elements apart whose last ones lie past element 2^32."""
    rows, cols, stride = 2051, 1000, (1 << 21) + 64
    gen = torch.Generator(device=DEV).manual_seed(2)
    room = lambda: torch.empty((rows - 1) * stride + cols, dtype=torch.bfloat16, device=DEV).as_strided(
        (rows, cols), (stride, 1))
    new = lambda: torch.randn(rows, cols, generator=gen, device=DEV).bfloat16()
    x, dy = new(), new()
    far_x, far_dy, far_y = room(), room(), room()
    far_x.copy_(x)
    far_dy.copy_(dy)
    stats = [torch.empty(rows, device=DEV) for _ in range(4)]
    sums = [torch.empty(cols, device=DEV) for _ in range(4)]
    y, ws = torch.empty_like(x), A.layer_norm_workspace(rows, cols, DEV)
    A.layer_norm(x, None, None, y, *stats[:2], eps=EPS)
    A.layer_norm(far_x, None, None, far_y, *stats[2:], eps=EPS)
    assert torch.equal(far_y, y) and torch.equal(stats[0], stats[2]) and torch.equal(stats[1], stats[3])
    A.layer_norm_backward(dy, x, None, *stats[:2], y, *sums[:2], ws)
    A.layer_norm_backward(far_dy, far_x, None, *stats[:2], far_y, *sums[2:], ws)
    assert torch.equal(far_y, y) and torch.equal(sums[0], sums[2]) and torch.equal(sums[1], sums[3])


def test_scan_steps_past_32_bits():
    """Steps 2^22 + 8 elements apart, the last ones past element 2^32."""
    B, T, D, stride = 1, 1030, 40, (1 << 22) + 8
    c = Case(B, T, D, torch.bfloat16, True)
    c.forward()
    c.backward()
    room = torch.empty((T - 1) * stride + 6 * D, dtype=torch.bfloat16, device=DEV)
    view = lambda k: room.as_strided((B, T, D), (T * stride, stride, 1), k * D)   # side by side in the same rows
    z, x, h, dh, dz, dx = (view(k) for k in range(6))
    for t, v in ((z, c.z), (x, c.x), (dh, c.dh)):
        t.copy_(v)
    last, dh0 = torch.empty_like(c.last), torch.empty_like(c.dh0)
    A.gated_scan(z, x, h, h0=c.h0, h_last=last, ws=c.ws)
    A.gated_scan_backward(z, x, h, dh, dz, dx, h0=c.h0, dh_last=c.dl, dh0=dh0, ws=c.ws)
    for got, want in ((h, c.h), (last, c.last), (dz, c.dz), (dx, c.dx), (dh0, c.dh0)):
        assert torch.equal(got, want)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,cols", [
    # up to 1024 columns: half of a workgroup's teams, then all of them with some without a row
    (1024, 1000), (1025, 1000), (2049, 300), (4097, 100), (33000, 30),
    # a team of 2 wavefronts (4 a workgroup), 3 (2), 4 (2), 6 (1) and 8 (1)
    (512, 1999), (513, 1999), (1031, 2048), (257, 3000), (700, 3001), (601, 4096), (300, 6000), (259, 8192)])
def test_layer_norm_gradients_by_workgroup(rows, cols, dtype):
    backward(rows, cols, dtype, seed=rows)


@pytest.mark.parametrize("sigmoid", [True, False])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_scan_long_chains(dtype, sigmoid):
    """Chains of more tiles than a look back takes at once, whole and with ends inside."""
    Case(1, 12011, 130, dtype, sigmoid, seed=6).check()
    Case(3, 9000, 66, dtype, sigmoid, lengths=[9000, 4097, 12], seed=7).check()


def test_a_closed_optimizer_is_refused():
    opt = A.Optimizer([(0, 1000, 0.0, 1.0)])
    w, g, m, v = (torch.zeros(1000, device=DEV) for _ in range(4))
    ws, clip = opt.norm_workspace(DEV), torch.zeros(2, device=DEV)
    opt.close()
    for call in (lambda: A.adamw(opt, w, g, m, v, lr=1e-3), lambda: A.grad_norm(opt, g, clip, ws, 1.0)):
        with pytest.raises(A.AdaCompError) as e:
            call()
        assert e.value.status == -1


def test_arguments_of_the_wrong_kind():
    opt = A.Optimizer([(0, 1000, 0.0, 1.0)])
    w, g, m, v = (torch.zeros(1000, device=DEV) for _ in range(4))
    with pytest.raises(TypeError):
        A.adamw(opt, w, g, m, v, lr="a")
    with pytest.raises(TypeError):
        A.adamw(opt, w, g, [0.0] * 1000, v, lr=1e-3)
    with pytest.raises(OverflowError):
        A.adamw(opt, w, g, m, v, lr=1e-3, step=-1)
    with pytest.raises(ValueError):
        A.adamw(opt, w, g, m, v, lr=1e-3, step=1 << 32)
    with pytest.raises(TypeError):
        A.adamw_packed(opt, w, g, m.to(torch.uint8), v.to(torch.uint8), None, lr=1e-3)
    with pytest.raises(AttributeError):
        A.adamw(opt, w, g, m, v, lr=1e-3, stream=7)
    with pytest.raises(TypeError):
        A.layer_norm(None, None, None, w)
    with pytest.raises(ValueError):
        A.layer_norm(torch.zeros((), device=DEV), None, None, torch.zeros((), device=DEV))
    assert not w.any() and not m.any() and not v.any()
