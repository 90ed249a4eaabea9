"""Gates p * sigmoid(p) far below 0, where they are 0: nothing of what they multiply passes, and nothing goes back."""
import pytest
import torch

import model_refs as M
import test_gpu_causal_conv as conv
import test_gpu_selective_scan as scan

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
# A sigmoid below 2^-126 or so may be taken for 0; at -87, where it is there, p sigmoid(p) is 87 exp(-87).
NOTHING = 1.5e-36


def plant(t, seed):
    """Some of t far below 0, down to the type's lowest value; returns which are where the gate is 0 in float32."""
    low = torch.finfo(t.dtype).min
    far = torch.tensor([max(v, low) for v in (-90.0, -104.0, -700.0, -1e4, -1e34, -1e36, low)], device=DEV)
    gen = torch.Generator(device=DEV).manual_seed(seed)
    pick = torch.randint(0, 2 * len(far), t.shape, generator=gen, device=DEV)
    on = pick < len(far)
    t.copy_(torch.where(on, far[pick % len(far)].to(t.dtype), t))
    return t <= -200.0


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("K", [1, 2, 4, 6])
@pytest.mark.parametrize("T", [3, 90])
def test_convolution(T, K, dtype):
    c = conv.Case(2, T, 40, K, TYPES[dtype], state=False, bias=False, seed=K)
    c.w.zero_()
    c.w[:, -1] = 1.0        # p is x
    none = plant(c.x, T)
    c.forward()
    c.backward()
    assert not c.y[none].any() and not c.dx[none].any()
    x, dy = M.f64(c.x), M.f64(c.dy)
    q = torch.sigmoid(x)
    slope, flat = q + x * q * (1 - q), q + (x * q * (1 - q)).abs()
    M.assert_within(c.y, (x * q, M.GATE * M.U * (x * q).abs() + NOTHING), "y")
    eg = (M.GATE + 6) * M.U * dy.abs() * flat + NOTHING * dy.abs()
    M.assert_within(c.dx, (dy * slope, eg), "dx")
    if K == 1:              # of longer filters the other taps' sums hold the far values themselves
        g = dy * slope
        # where the slope may be taken for 0, it is below 90 exp(-87) = 1.5e-36 and x above -104
        eg = torch.where(x < -200.0, torch.zeros(()).double(), eg)
        err = (eg * x.abs()).sum((0, 1)) + (T + 260) * M.U * (g * x).abs().sum((0, 1))
        M.assert_within(c.dw, ((g * x).sum((0, 1))[:, None], err[:, None]), "dweight")


class Scan(scan.Case):
    def check(self):
        """As its own check, with what a sigmoid that is 0 leaves out of dz: the gate's slope at z below -87 is
        s (1 + z (1 - s)) with s < exp(-87) = 1.65e-38 and |z| s < 1.43e-36, so less than NOTHING times dy and what the
        gate multiplies."""
        form, ins = M.scan, {k: M.f64(v) for k, v in self.i.items()}

        def wider(dy, **kw):
            out = form(dy=dy, **kw)
            sums = form(**dict(ins, z=None), h0=kw["h0"])["y"]
            value, err = out["dz"]
            out["dz"] = (value, err + NOTHING * dy.abs() * (sums[0].abs() + sums[1]))
            return out
        M.scan = wider
        try:
            return super().check()
        finally:
            M.scan = form


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,N", [(3, 16), (8, 5), (30, 8), (100, 16), (40, 40)])
def test_selective_scan(T, N, dtype):
    """Short sequences and chunks; check() compares with the 64-bit form in both directions."""
    c = Scan(3, T, 70, N, TYPES[dtype], seed=N)
    none = plant(c.i["z"], T)
    c.check()
    assert not c.y[none].any() and not c.g["dz"][none].any()


@pytest.mark.parametrize("dtype", TYPES)
def test_selective_scan_behind_shut_gates(dtype):
    """Every gate at the type's lowest value: no output, and of the inputs' gradients what h_last has alone."""
    c = Scan(2, 50, 70, 16, TYPES[dtype])
    c.i["z"].fill_(torch.finfo(c.dtype).min)
    c.check()
    assert not any(t.any() for t in (c.y, c.g["dz"], c.g["dc"], c.g["dd"]))
    c.dl = None
    c.backward()
    assert not any(c.g[k].any() for k in scan.GRADS)
