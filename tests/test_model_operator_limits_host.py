"""Sizes and types of the convolution's, the selective scan's and the losses' buffers (no GPU needed)."""
import pytest
import torch

import adaptive_residual_gradient_amd as A


@pytest.fixture(scope="module", autouse=True)
def _lib_built():
    if not A.LIB_PATH.exists():
        from adaptive_residual_gradient_amd import _build
        _build.build()


@pytest.mark.parametrize("default", [torch.float32, torch.float64, torch.bfloat16])
def test_kept_states_are_float32_whatever_torch_makes_by_default(default):
    was = torch.get_default_dtype()
    torch.set_default_dtype(default)
    try:
        states = A.selective_scan_states(2, 30, 64, 16, device="cpu")
        workspaces = [A.selective_scan_workspace(2, 30, 64, 16, device="cpu"), A.causal_conv_workspace(2, 30, 64, 4, "cpu"),
                      A.linear_loss_workspace(10, 64, 300, torch.float32, device="cpu")]
    finally:
        torch.set_default_dtype(was)
    assert states.dtype == torch.float32 and states.numel() == 2 * 4 * 16 * 64
    assert all(ws.dtype == torch.uint8 for ws in workspaces)
