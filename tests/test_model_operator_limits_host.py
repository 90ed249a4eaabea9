"""Sizes and types of the convolution's, the selective scan's and the losses' buffers (no GPU needed)."""
import ctypes

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


OK, CAPACITY, TOO_LARGE = 0, -5, -7


def head_query(R, H, V, type_=1, picks=1, back=0):
    n = ctypes.c_uint64()
    head = A._Head(R, H, V, type_, H, H, None, None)
    return A.lib().adacomp_head_workspace_bytes(ctypes.byref(head), picks, back, ctypes.byref(n))


def head_call(R, H, V, picks=1, back=False):
    """Refused for its 0 bytes of workspace at the latest."""
    head, L = ctypes.byref(A._Head(R, H, V, 1, H, H, 1 << 20, 1 << 50)), A.lib()
    at = [(1 << 50) + (k << 46) for k in range(1, 9)]
    if picks > 1 and back:
        return L.adacomp_linear_distillation_backward(head, at[0], at[1], picks, 1.0, at[2], at[3], at[4], at[5], H, at[6], H,
                                                      at[7], 0, None)
    if picks > 1:
        return L.adacomp_linear_distillation(head, at[0], at[1], picks, 1.0, at[2], at[3], at[4], at[5], 0, None)
    if back:
        return L.adacomp_linear_cross_entropy_backward(head, at[0], at[1], at[2], at[3], at[4], H, at[5], H, at[6], 0, None)
    return L.adacomp_linear_cross_entropy(head, at[0], at[1], at[2], at[3], 0, None)


@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("R,H,V,picks,fits", [
    (131072, 8, 262144, 1, True), (1 << 20, 64, 1 << 18, 1, True), ((1 << 24) - 1, 8, 127 << 8, 1, True),
    ((1 << 24) - 1, 8, (127 << 8) + 1, 1, False), ((1 << 24) - 1, 8, (1 << 24) - 1, 1, False),
    (1 << 16, 64, 1000, 1023, True), (1 << 16, 64, 1000, 1024, False), ((1 << 24) - 1, 8, 1000, 3, True),
    ((1 << 24) - 1, 8, 1000, 5, False),
    ((1 << 24) - 1, 1024, 1000, 1, True), ((1 << 24) - 1, 1025, 1000, 1, False), (1 << 18, 65536, 1000, 1, False),
    ((1 << 18) - 1, 65536, 1000, 1, True)])
def test_losses_query_and_calls_take_the_same_sizes(R, H, V, picks, fits, back):
    """2^26 picks, 2^34 elements of hidden rows in whole 8, 2^23 tiles of 256 words and rows."""
    assert head_query(R, H, V, picks=picks, back=int(back)) == (OK if fits else TOO_LARGE)
    assert head_call(R, H, V, picks, back) == (CAPACITY if fits else TOO_LARGE)
