"""The kernels that only large calls take: inputs that go past the cache, rows of the looping
layer norm kernels beyond a few, and the widest rows.  A large call has to give what calls
on parts of it give, bit for bit, and sums over rows what 64 bits give."""
import pytest
import torch

import adaptive_residual_gradient_amd as A
import operator_refs as R
from test_gpu_layer_norm import EPS, backward

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def normal(gen, *shape, dtype=torch.float32, scale=1.0):
    return torch.randn(shape, generator=gen, device=DEV).mul_(scale).to(dtype)


@pytest.mark.parametrize("sigmoid", [True, False])
@pytest.mark.parametrize("dtype,B,T,D,part", [
    # every case reads more than 96 MB, its parts less, in the same kind of call
    ("bf16", 256, 100, 1024, 64),      # one tile a sequence
    ("f32", 220, 120, 520, 55),        # the same, rows that share cache lines
    ("bf16", 16, 1600, 1024, 8),       # 64 chains of tiles and more
    ("f16", 16, 1600, 1024, 8),
    ("f32", 16, 800, 1024, 4),
    ("bf16", 4, 6300, 1024, 1),        # few chains
    ("f32", 4, 6300, 512, 1),
    ("f32", 2, 30000, 224, 1)])
def test_scan_of_large_inputs(dtype, B, T, D, part, sigmoid):
    gen = torch.Generator(device=DEV).manual_seed(T)
    dt = TYPES[dtype]
    z = normal(gen, B, T, D) + 3.0
    z = (z if sigmoid else torch.sigmoid(z)).to(dt)
    x, dh = normal(gen, B, T, D, dtype=dt), normal(gen, B, T, D, dtype=dt, scale=0.1)
    assert 2 * z.numel() * z.element_size() > 96 << 20
    h0, dl = normal(gen, B, D), normal(gen, B, D, scale=0.1)
    new = lambda: [torch.empty_like(z) for _ in range(3)] + [torch.empty(B, D, device=DEV) for _ in range(2)]
    big, small = new(), new()

    def call(at, out, ws):
        h, dz, dx, last, dh0 = (t[at] for t in out)
        A.gated_scan(z[at], x[at], h, h0=h0[at], h_last=last, sigmoid=sigmoid, ws=ws)
        A.gated_scan_backward(z[at], x[at] if sigmoid else None, h, dh[at], dz, dx, h0=h0[at], dh_last=dl[at], dh0=dh0,
                              sigmoid=sigmoid, ws=ws)

    call(slice(0, B), big, A.gated_scan_workspace(B, T, D, DEV))
    ws = A.gated_scan_workspace(part, T, D, DEV)
    for b in range(0, B, part):
        call(slice(b, b + part), small, ws)
    for a, c, what in zip(big, small, ("h", "dgate", "dx", "h_last", "dh0")):
        assert torch.equal(a, c), what


@pytest.mark.parametrize("dtype,rows,cols", [
    # past 96 MB forward and backward, by every kind of team
    ("bf16", 50001, 1024), ("f32", 25003, 1000), ("f16", 510007, 100), ("f32", 900001, 30), ("bf16", 12502, 4096),
    ("f32", 6007, 4500), ("bf16", 20000000, 3),
    # the gradients' inputs past it, their output not
    ("bf16", 32768, 1024), ("f32", 17001, 1000), ("bf16", 8001, 4096), ("f16", 300007, 100)])
def test_layer_norm_of_large_inputs(dtype, rows, cols):
    gen = torch.Generator(device=DEV).manual_seed(rows)
    dt = TYPES[dtype]
    x, dy = (normal(gen, rows, cols, dtype=dt) for _ in range(2))
    assert 2 * x.numel() * x.element_size() > 96 << 20
    w, b = 1 + normal(gen, cols, scale=0.2), normal(gen, cols, scale=0.1)
    out = lambda: (torch.empty_like(x), torch.empty(rows, device=DEV), torch.empty(rows, device=DEV))
    y, mean, rstd = out()
    y2, mean2, rstd2 = out()
    A.layer_norm(x, w, b, y, mean, rstd, eps=EPS)
    dx, dx2 = torch.empty_like(x), torch.empty_like(x)
    dw, db = torch.empty(cols, device=DEV), torch.empty(cols, device=DEV)
    A.layer_norm_backward(dy, x, w, mean, rstd, dx, dw, db, A.layer_norm_workspace(rows, cols, DEV))
    step = (rows + 3) // 4
    want = [torch.zeros(cols, dtype=torch.float64, device=DEV) for _ in range(4)]
    for r in range(0, rows, step):
        s = slice(r, min(rows, r + step))
        A.layer_norm(x[s], w, b, y2[s], mean2[s], rstd2[s], eps=EPS)
        A.layer_norm_backward(dy[s], x[s], w, mean[s], rstd[s], dx2[s])
        d, hat = dy[s].double(), (x[s].double() - mean[s, None].double()) * rstd[s, None].double()
        for t, v in zip(want, (d * hat, d, (d * hat).abs(), d.abs())):
            t += v.sum(0)
    for a, c, what in ((y, y2, "y"), (mean, mean2, "mean"), (rstd, rstd2, "rstd"), (dx, dx2, "dx")):
        assert torch.equal(a, c), what
    # as in norm_backward_bounds: a workgroup's share of the rows in one chain at most, then the joins
    chain = rows / 256 + R.SUM
    for got, value, size in ((dw, want[0], want[2]), (db, want[1], want[3])):
        R.assert_within(got, R.f64(value), chain * R.U * R.f64(size), "sums over rows")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,cols", [(200, 8193), (131, 16385), (200, 20000), (3, 65535), (2, 65536), (70, 65533)])
def test_layer_norm_of_many_wide_rows(rows, cols, dtype):
    """More rows than the 64 workgroups that sum the weight's gradient take one each, and rows up to the limit."""
    backward(rows, cols, TYPES[dtype], seed=cols)
    backward(rows, cols, TYPES[dtype], pad=5, seed=cols)
