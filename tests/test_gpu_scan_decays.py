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


@pytest.mark.parametrize("T", [7, 100])
def test_rates_of_minus_infinity(T):
    """States that keep nothing: h is what the last step wrote, behind a sequence's end too."""
    lengths = [T, 3, T // 2, 0]
    c = Case(4, T, 64, 16, torch.float32, gated=False, lengths=lengths)
    c.i["a"][::2] = float("-inf")
    c.forward(kept=False)
    d = {k: M.f64(v) for k, v in c.i.items()}
    for b, n in enumerate(lengths):
        if n == 0:
            assert torch.equal(c.last[b], c.h0[b])
            continue
        raw = d["dt"][b, n - 1] + d["dt_bias"]
        u = torch.logaddexp(raw, torch.zeros(()).double()) * d["x"][b, n - 1]
        want = (u[:, None] * d["b"][b, n - 1])[::2]
        # softplus: 12 roundings and that of its argument, and three products
        M.assert_within(c.last[b, ::2], (want, (16 + raw.abs()[::2, None]) * M.U * want.abs()), f"h_last of sequence {b}")
    assert not torch.isnan(c.y[:, :3]).any() and not torch.isnan(c.last).any()
    c.forward()
    c.backward()
    assert not any(torch.isnan(g).any() for g in c.g.values() if g is not None)
    # what h0 holds goes nowhere, and of the rates' gradients nothing is left
    assert not c.g["dh0"][:3, ::2].any() and not c.g["da"][::2].any() and torch.equal(c.g["dh0"][3], c.dl[3])
