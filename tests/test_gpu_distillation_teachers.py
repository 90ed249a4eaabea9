"""Teachers' logits that are no numbers, or leave a row without any probability."""
import pytest
import torch

from test_gpu_vocabulary_loss import Case

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
INF = float("inf")


def case(dtype, R, picks):
    c = Case(R, 40, 300, dtype, picks=picks, ignored=0.0, temperature=1.5, seed=picks)
    c.ids.clamp_(min=0)
    c.hidden.copy_(torch.randn(c.hidden.shape, generator=torch.Generator(device=DEV).manual_seed(1), device=DEV))
    c.off[:] = False
    return c


def results(c):
    c.forward()
    c.backward()
    return [t.clone() for t in (c.loss, c.dh, c.dw)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("R", [40, 600])
@pytest.mark.parametrize("picks", [1, 6, 70])
def test_rows_without_probability(picks, R, dtype):
    """Logits of -infinity at every pick that is a word: the row does not count, as if it had no pick, whatever its
    hidden state holds."""
    c = case(TYPES[dtype], R, picks)
    c.check()
    c.teacher[1::3] = -INF
    c.hidden[1::6] = float("nan")
    if picks > 1:
        c.ids[1::3, 0] = -1
        c.teacher[1::3, 0] = 1.0       # of no word
    got = results(c)
    assert all(torch.isfinite(t).all() for t in got)
    assert not got[0][1::3].any() and not got[1][1::3].any() and got[0][::3].all()
    c.ids[1::3] = -1
    c.teacher[1::3] = 0.0
    assert all(torch.equal(a, b) for a, b in zip(got, results(c)))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("picks", [1, 6, 70])
@pytest.mark.parametrize("value", [float("nan"), INF])
def test_rows_that_are_no_numbers(value, picks, dtype):
    """NaN or infinity among a row's logits: its loss and gradients are NaN, other rows' are what they were."""
    c = case(TYPES[dtype], 40, picks)
    loss, dh, _ = results(c)
    c.teacher[7, picks // 2] = value
    got, dgot, _ = results(c)
    rest = torch.arange(40, device=DEV) != 7
    assert torch.isnan(got[7]) and torch.isnan(dgot[7]).all()
    assert torch.equal(got[rest], loss[rest]) and torch.equal(dgot[rest], dh[rest])
    c.ids[7, picks // 2] = 300         # no word: left out
    got, dgot, dw = results(c)
    assert all(torch.isfinite(t).all() for t in (got, dgot, dw))
