"""The training-step operators together, as examples/train_gated_layers.py uses
them: the model's gradients against 64-bit autograd, and a short training run."""
import pathlib
import sys

import pytest
import torch

sys.path.insert(0, str(pathlib.Path(__file__).resolve().parent.parent / "examples"))
import train_gated_layers as E  # noqa: E402

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def plain(layout, flat, x, lengths):
    """The layers in elementary 64-bit operations."""
    D = layout.width
    for i in range(layout.layers):
        of = lambda name: layout.of(flat, i, name)
        d = x - x.mean(2, keepdim=True)
        u = d / torch.sqrt((d * d).mean(2, keepdim=True) + E.EPS) * of("weight") + of("bias")
        proj = u @ of("in").t()
        a = torch.sigmoid(proj[:, :, :D])
        state, hs = torch.zeros_like(x[:, 0]), []
        for t in range(x.shape[1]):
            state = a[:, t] * state + (1 - a[:, t]) * proj[:, t, D:]
            hs.append(state)
        h = torch.stack(hs, 1)
        if lengths is not None:
            h = h * (torch.arange(x.shape[1]) < lengths[:, None])[:, :, None]
        x = x + h @ of("out").t()
    return x


@pytest.mark.parametrize("ragged", [False, True])
def test_gradients_of_the_model(ragged):
    """float32 layers.  Every gradient is a chain of about a dozen sums of at most B T = 200 terms with
    relative errors of at most 2^-24 a term (terms add up like their roots in norm, 2^-24 * 200 at worst):
    12 * 200 * 2^-24 = 1.4e-4 of its norm."""
    B, T, D = 4, 50, 36
    layout = E.Layout(2, D)
    flat = layout.init(DEV, 1)
    gen = torch.Generator(device=DEV).manual_seed(2)
    for i in range(2):
        layout.of(flat, i, "bias").copy_(torch.randn(D, generator=gen, device=DEV) * 0.1)
    x, dy = (torch.randn(B, T, D, generator=gen, device=DEV) for _ in range(2))
    lengths = torch.tensor([50, 0, 17, 33], dtype=torch.int32, device=DEV) if ragged else None
    model = E.Model(layout, B, T, torch.float32, DEV)
    y = model.forward(flat, flat, x, lengths)
    grad = torch.zeros_like(flat)
    dx = model.backward(flat, flat, dy, grad, lengths)

    flat64, x64 = flat.double().cpu().requires_grad_(), x.double().cpu().requires_grad_()
    want = plain(layout, flat64, x64, lengths.cpu() if ragged else None)
    want.backward(dy.double().cpu())
    for i in range(2):
        for name in ("in", "out", "weight", "bias"):
            a, b = layout.of(grad, i, name).double().cpu(), layout.of(flat64.grad, i, name)
            assert float((a - b).norm()) <= 1.4e-4 * float(b.norm()), (i, name)
    assert float((y.double().cpu() - want.detach()).norm()) <= 1.4e-4 * float(want.detach().norm())
    assert float((dx.double().cpu() - x64.grad).norm()) <= 1.4e-4 * float(x64.grad.norm())


def test_training_lowers_the_loss():
    losses = E.train(layers=1, width=64, batch=4, length=40, learners=2, steps=40, log=lambda s: print(s, flush=True))
    assert all(x == x for x in losses)
    assert sum(losses[-5:]) < 0.5 * sum(losses[:5])
    assert E.train(layers=1, width=64, batch=4, length=40, learners=2, steps=3, log=lambda s: None) == losses[:3]
