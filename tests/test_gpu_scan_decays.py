"""Decays of whole chunks of the selective scan that float32 does not hold, while the states before and behind
them are ordinary numbers."""
import pytest
import torch

import adaptive_residual_gradient_amd as A
import model_refs as M
from test_gpu_selective_scan import Case

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
# What the inputs of these cases add lies near float32's smallest number, 2^-149, and each rounding there is off by up
# to 2^-150.  A result has at most 64 terms (channels; 32 steps, 16 states) of 4 roundings each, and is multiplied by
# a step of at most 16 behind them.  (States of 1e-33 and more do not feel them: 2^-24 of one is 6e-41.)
SMALL = 64 * 4 * 16 * 2.0 ** -150


class Swinging(Case):
    def check(self):
        form = M.scan
        M.scan = lambda **kw: {k: (v, e + SMALL) for k, (v, e) in form(**kw).items()}
        try:
            return super().check()
        finally:
            M.scan = form


def swinging(T, N, step, first, last):
    """Chunks of 8 steps: h is multiplied by exp(step) at each step of one and by exp(-step) of the next, from `first`
    on, what is carried back from `last` on.  What the steps write and read is far smaller."""
    c = Swinging(1, T, 64, N, torch.float32, softplus=False, gated=False)
    sign = torch.where(torch.arange(T, device=DEV) // 8 % 2 == 0, 1.0, -1.0)
    c.i["dt"].copy_((sign * step)[None, :, None].expand(1, T, 64))
    c.i["a"].fill_(1.0)
    c.i["dt_bias"] = None
    for t, scale in ((c.h0, first), (c.dl, last), (c.i["x"], 1e-36), (c.dy, 1e-36)):
        t.mul_(scale)
    return c


@pytest.mark.parametrize("N", [4, 16])
@pytest.mark.parametrize("step,first,last", [(12.0, 1e-30, 1e10), (15.0, 1e-32, 1e22), (-12.0, 1e10, 1e-30),
                                             (-16.0, 1e25, 1e-32)])
def test_chunks_past_float32(step, first, last, N):
    """exp(96) to exp(128) over a chunk, and one over them; every state on the way lies between 1e-33 and 1e26."""
    c = swinging(32, N, step, first, last)
    # 4 chunks of 8: b and c in rows, the chunks' ends, the sums and s
    up = lambda floats: (4 * floats + 255) // 256 * 256
    padded = 8 if N <= 8 else 16
    assert A.selective_scan_workspace(1, 32, 64, N, device="cpu").numel() == (
        up(32 * 2 * padded) + up(4 * padded * 64) + up(4 * 64) + up(32 * 64))
    c.check()
