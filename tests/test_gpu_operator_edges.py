"""The training-step operators where their formulas reach the ends of the number
range, where calls are very large, and where layouts are unusual."""
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
