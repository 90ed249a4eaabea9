"""Layer norm and its gradients on the GPU against the 64-bit forms, within
bounds that count the roundings."""
import numpy as np
import pytest
import torch

import adaptive_residual_gradient_amd as A
import operator_refs as R

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
EPS = R.f32(1e-5)
# team sizes and their edges, one vector short and over, one workgroup's limits, the looping kernels
COLS = [1, 2, 3, 7, 8, 9, 16, 17, 31, 32, 33, 63, 64, 65, 100, 127, 128, 129, 255, 256, 257, 511, 512, 513, 1000,
        1023, 1024, 1025, 2048, 2500, 4096, 4101, 8192, 16384, 16385, 20000]


def strided(rows, cols, dtype, pad, seed, scale=1.0, shift=0.0):
    """A [rows, cols] tensor; pad > 0 puts its rows cols + pad apart, from an odd place on, with NaN between."""
    gen = torch.Generator(device=DEV).manual_seed(seed)
    x = (torch.randn(rows, cols, generator=gen, device=DEV) * scale + shift).to(dtype)
    if not pad:
        return x
    room = torch.full((rows * (cols + pad) + 1,), float("nan"), dtype=dtype, device=DEV)
    v = room[1:].view(rows, cols + pad)[:, :cols]
    v.copy_(x)
    return v


def affine(cols, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    return 1 + 0.2 * torch.randn(cols, generator=gen, device=DEV), 0.1 * torch.randn(cols, generator=gen, device=DEV)


def forward(rows, cols, dtype, pad=0, seed=0, scale=1.0, shift=0.3):
    x = strided(rows, cols, dtype, pad, seed, scale, shift)
    y = strided(rows, cols, dtype, pad, seed + 1)
    w, b = affine(cols, seed)
    mean, rstd = torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
    A.layer_norm(x, w, b, y, mean, rstd, eps=EPS)
    want = R.norm_forward_bounds(R.f64(x), R.f64(w), R.f64(b), EPS)
    for got, (value, err), what, dt in ((y, want[0], "y", dtype), (mean, want[1], "mean", torch.float32),
                                        (rstd, want[2], "rstd", torch.float32)):
        R.assert_within(got, value, R.rounded(value, err, dt), f"{what} {rows}x{cols}")
    return x, w, mean, rstd


def backward(rows, cols, dtype, pad=0, seed=0):
    x, w, mean, rstd = forward(rows, cols, dtype, pad, seed)
    dy, dx = strided(rows, cols, dtype, pad, seed + 2), strided(rows, cols, dtype, pad, seed + 3)
    dw, db = (torch.full((cols,), float("nan"), device=DEV) for _ in range(2))
    A.layer_norm_backward(dy, x, w, mean, rstd, dx, dw, db, A.layer_norm_workspace(rows, cols, DEV))
    want = R.norm_backward_bounds(*(R.f64(t) for t in (dy, x, w, mean, rstd)))
    for got, (value, err), what, dt in ((dx, want[0], "dx", dtype), (dw, want[1], "dweight", torch.float32),
                                        (db, want[2], "dbias", torch.float32)):
        R.assert_within(got, value, R.rounded(value, err, dt), f"{what} {rows}x{cols}")
    return dy, x, w, mean, rstd, dx


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("cols", COLS)
def test_widths(cols, dtype):
    print(f"  layer norm {dtype} cols {cols}", flush=True)
    backward(5, cols, TYPES[dtype])
    backward(3, cols, TYPES[dtype], pad=3)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols", [(1, 1000), (2, 64), (67, 16), (1025, 40), (4099, 1000), (5000, 24),
                                       (2100, 1024), (1030, 4096), (3001, 1)])
def test_rows(rows, cols, dtype):
    """Fewer rows than a workgroup's teams, more than all workgroups' teams, odd counts."""
    backward(rows, cols, TYPES[dtype], seed=3)


@pytest.mark.parametrize("scale,shift", [(1e-3, 100.0), (1e4, -3e4), (1e-20, 0.0), (0.0, 5.0)])
def test_large_offsets_small_spreads_and_constant_rows(scale, shift):
    forward(9, 1000, torch.float32, scale=scale, shift=shift)
    forward(9, 5000, torch.float32, scale=scale, shift=shift)


def test_without_weight_bias_and_statistics():
    x = strided(7, 200, torch.bfloat16, 0, 1)
    y, y2 = torch.empty_like(x), torch.empty_like(x)
    A.layer_norm(x, None, None, y, eps=EPS)
    A.layer_norm(x, torch.ones(200, device=DEV), torch.zeros(200, device=DEV), y2, eps=EPS)
    assert torch.equal(y, y2)
    dy, mean, rstd = strided(7, 200, torch.bfloat16, 0, 2), torch.zeros(7, device=DEV), torch.ones(7, device=DEV)
    dx, dx2 = torch.empty_like(x), torch.empty_like(x)
    dw, db = torch.empty(200, device=DEV), torch.empty(200, device=DEV)
    A.layer_norm_backward(dy, x, None, mean, rstd, dx)
    A.layer_norm_backward(dy, x, torch.ones(200, device=DEV), mean, rstd, dx2, dw, db,
                          A.layer_norm_workspace(7, 200, DEV))
    assert torch.equal(dx, dx2)


def test_no_rows():
    x = torch.empty(0, 64, device=DEV)
    A.layer_norm(x, None, None, torch.empty_like(x))
    dw, db = torch.full((64,), 3.0, device=DEV), torch.full((64,), 3.0, device=DEV)
    none = torch.empty(0, device=DEV)
    A.layer_norm_backward(x, x, None, none, none, torch.empty_like(x), dw, db, A.layer_norm_workspace(0, 64, DEV))
    assert not dw.any() and not db.any()


def test_a_row_of_nan_or_infinity_stays_alone():
    for cols in (24, 1000, 2048):
        x = strided(70, cols, torch.float32, 0, 4)
        x[3, 5], x[66, 7] = float("nan"), float("inf")
        y = torch.empty_like(x)
        mean, rstd = torch.empty(70, device=DEV), torch.empty(70, device=DEV)
        A.layer_norm(x, None, None, y, mean, rstd)
        bad = torch.zeros(70, dtype=torch.bool, device=DEV)
        bad[3] = bad[66] = True
        assert torch.isnan(y[bad]).all() and torch.isfinite(y[~bad]).all()


def test_leading_axes():
    x = strided(24, 100, torch.float32, 0, 5).view(2, 3, 4, 100)
    y, y2 = torch.empty_like(x), torch.empty(24, 100, device=DEV)
    A.layer_norm(x, None, None, y)
    A.layer_norm(x.view(24, 100), None, None, y2)
    assert torch.equal(y.view(24, 100), y2)


def test_gradient_against_differences():
    """The kernel's gradients along random directions against central differences of the 64-bit forward."""
    rng = np.random.default_rng(6)
    dy, x, w, mean, rstd, dx = backward(33, 257, torch.float32, seed=7)
    u = rng.standard_normal((33, 257))
    x64, w64, dy64 = R.f64(x), R.f64(w), R.f64(dy)
    loss = lambda t: (R.norm_forward(t, w64, 0.0, EPS)[0] * dy64).sum()
    diff = (loss(x64 + 1e-5 * u) - loss(x64 - 1e-5 * u)) / 2e-5
    assert abs(diff - (R.f64(dx) * u).sum()) < 1e-4 * np.abs(R.f64(dx) * u).sum()


@pytest.mark.parametrize("cols", [1000, 2048])
def test_in_a_graph(cols):
    rows = 300
    x, dy = strided(rows, cols, torch.bfloat16, 0, 8), strided(rows, cols, torch.bfloat16, 0, 9)
    w, b = affine(cols, 8)
    mean, rstd, ws = torch.empty(rows, device=DEV), torch.empty(rows, device=DEV), A.layer_norm_workspace(rows, cols, DEV)
    y, dx, dw, db = torch.empty_like(x), torch.empty_like(x), torch.empty(cols, device=DEV), torch.empty(cols, device=DEV)

    def both():
        A.layer_norm(x, w, b, y, mean, rstd)
        A.layer_norm_backward(dy, x, w, mean, rstd, dx, dw, db, ws)

    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        both()
    for i in range(4):
        x.copy_(strided(rows, cols, torch.bfloat16, 0, 20 + i))
        g.replay()
        torch.cuda.synchronize()
        replayed = [t.clone() for t in (y, mean, rstd, dx, dw, db)]
        both()
        for a, c in zip(replayed, (y, mean, rstd, dx, dw, db)):
            assert torch.equal(a, c)


def test_refusals():
    x = torch.zeros(4, 64, device=DEV)
    y, m = torch.empty_like(x), torch.zeros(4, device=DEV)
    for bad in (lambda: A.layer_norm(x, None, None, x),
                lambda: A.layer_norm(x, None, None, y, eps=-1.0),
                lambda: A.layer_norm_backward(y, x, None, m, m.clone(), torch.empty_like(x), torch.zeros(64, device=DEV),
                                              torch.zeros(64, device=DEV)),
                lambda: A.layer_norm_backward(y, x, None, m, m.clone(), y)):
        with pytest.raises(A.AdaCompError):
            bad()
    with pytest.raises(ValueError):
        A.layer_norm(x, torch.ones(63, device=DEV), None, y)
    with pytest.raises(ValueError):
        A.layer_norm(x, None, None, y[:, :32])
    with pytest.raises(ValueError):
        A.layer_norm(x, None, None, y.bfloat16())
    with pytest.raises(TypeError):
        A.layer_norm(x.double(), None, None, y.double())
    with pytest.raises(TypeError):
        A.layer_norm(x.t().contiguous().t(), None, None, y)
    with pytest.raises(TypeError):
        A.layer_norm(x, torch.ones(64, device=DEV, dtype=torch.bfloat16), None, y)
