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


@pytest.mark.parametrize("B,T,C,N,fits", [
    (1, (1 << 27) - 8, 8, 16, True), (1, 1 << 27, 8, 16, False), (3, 1 << 26, 8, 16, False), (2, (1 << 25) - 8, 8, 24, True),
    (2, 1 << 25, 8, 33, False), (1 << 20, 100, 64, 64, False), ((1 << 20) - 1, 4, 64, 64, True), (1 << 20, 0, 64, 64, False)])
def test_scan_queries_and_calls_take_the_same_sizes(B, T, C, N, fits):
    """2^32 steps and states of b and c, each in whole blocks, and of channels, states and sequences."""
    L, n = A.lib(), ctypes.c_uint64()
    s = A._SsmShape(T, B, C, N, 1, 1)
    for back in (0, 1):
        assert L.adacomp_selective_scan_workspace_bytes(ctypes.byref(s), back, ctypes.byref(n)) == (OK if fits else TOO_LARGE)
    assert L.adacomp_selective_scan_kept_bytes(ctypes.byref(s), ctypes.byref(n)) == (OK if fits else TOO_LARGE)
    at = [(k << 50) for k in range(1, 16)]
    view = lambda p, width: A._View(p, T * width, width)
    i = A._SsmInputs(view(at[0], C), view(at[1], C), view(at[2], N), view(at[3], N), view(None, C), at[4], None, None, None)
    y = view(at[5], C)
    call = L.adacomp_selective_scan(ctypes.byref(s), ctypes.byref(i), ctypes.byref(y), None, None, None, 1 << 20, 0, None)
    g = A._SsmGradients(view(at[6], C), view(at[7], C), view(at[8], N), view(at[9], N), view(None, C), at[10], None, None, None)
    back = L.adacomp_selective_scan_backward(ctypes.byref(s), ctypes.byref(i), ctypes.byref(y), at[11], None, ctypes.byref(g),
                                             1 << 20, 0, None)
    assert call == back == (CAPACITY if fits else TOO_LARGE)
