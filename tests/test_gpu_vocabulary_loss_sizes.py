"""Losses over more logits than 2^35, and weights of more elements than 2^32 that nothing adds to."""
import pytest
import torch

import adaptive_residual_gradient_amd as A
import model_refs as M

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def test_many_rows_and_words():
    R, H, V = 131072 + 5, 8, 262144
    gen = torch.Generator(device=DEV).manual_seed(1)
    hidden = torch.randn(R, H, generator=gen, device=DEV).bfloat16()
    weight = torch.randn(V, H, generator=gen, device=DEV).bfloat16()
    ids = torch.randint(0, V, (R,), generator=gen, device=DEV)
    ids[::5] = -1
    loss, lse, dloss = (torch.full((R,), 0.5, device=DEV) for _ in range(3))
    dhidden = torch.empty_like(hidden)
    ws = A.linear_loss_workspace(R, H, V, torch.bfloat16, backward=True, device=DEV)
    ws[:1 << 28].fill_(0xFF)
    A.linear_cross_entropy(hidden, weight, ids, loss, lse, ws)
    A.linear_cross_entropy_backward(hidden, weight, ids, loss, lse, dloss, dhidden, None, ws)
    at = torch.cat([torch.arange(8), torch.arange(65530, 65540), torch.arange(R - 8, R)]).to(DEV)
    want = M.loss(M.f64(hidden[at]), M.f64(weight), ids[at, None].cpu(), dloss=M.f64(dloss[at]), dtype=torch.bfloat16)
    for got, what in ((loss, "loss"), (lse, "lse"), (dhidden, "dhidden")):
        M.assert_within(got[at], want[what], what)
    assert not loss[::5].any() and not dhidden[::5].any() and torch.isfinite(lse).all()


def test_no_rows_and_a_weight_past_32_bits():
    H, V = 520, (1 << 23) + 3
    dweight = torch.full((V, H), 7.0, dtype=torch.bfloat16, device=DEV)
    weight = torch.zeros(V, H, dtype=torch.bfloat16, device=DEV)
    none = torch.empty(0, device=DEV)
    hidden = torch.empty(0, H, dtype=torch.bfloat16, device=DEV)
    A.linear_cross_entropy_backward(hidden, weight, torch.empty(0, dtype=torch.int64, device=DEV), none, none, none, None,
                                    dweight, None)
    assert not dweight.any()
