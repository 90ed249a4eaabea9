"""Gates p * sigmoid(p) far below 0, where they are 0: nothing of what they multiply passes, and nothing goes back."""
import pytest
import torch

import model_refs as M
import test_gpu_causal_conv as conv

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
