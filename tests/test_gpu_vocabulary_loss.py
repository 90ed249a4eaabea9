"""The losses over a vocabulary and their gradients on the GPU against the 64-bit
form, within bounds that count the roundings."""
import pytest
import torch

import adaptive_residual_gradient_amd as A
import model_refs as M

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


class Case:
    """picks = 0: cross entropy."""

    def __init__(self, R, H, V, dtype, picks=0, temperature=1.0, ignored=0.2, scale=2.0, pad=0, even=False, seed=0):
        gen = torch.Generator(device=DEV).manual_seed(seed)
        normal = lambda *s: torch.randn(*s, generator=gen, device=DEV)
        # pad: elements between the rows, NaN
        def new(v):
            room = torch.full((v.shape[0], v.shape[1] + pad), float("nan"), dtype=dtype, device=DEV)
            out = room[:, pad // 2:pad // 2 + v.shape[1]]
            out.copy_(v)
            return out
        self.dtype, self.picks, self.t = dtype, picks, temperature
        self.hidden, self.weight = new(normal(R, H)), new(normal(V, H) * scale * H ** -0.5)
        self.ids = torch.randint(0, V, (R, max(picks, 1)), generator=gen, device=DEV)
        off = torch.rand(R, generator=gen, device=DEV) < ignored
        self.ids[off] = torch.tensor([-100, V, -1, 2 ** 40], device=DEV)[torch.arange(R, device=DEV) % 4][off][:, None]
        self.hidden[off] = float("nan")
        if picks:
            self.ids[torch.rand(R, picks, generator=gen, device=DEV) < 0.1] = -1
            off = ((self.ids < 0) | (self.ids >= V)).all(1)
            self.hidden[off] = float("inf")
            self.teacher = normal(R, picks) * 3
        self.off = off
        self.dloss = torch.full((R,), 1.0 / R, device=DEV) if even else normal(R) / R
        full = lambda *s: torch.full(s, 7.0, device=DEV)
        self.loss, self.lse, self.picked = full(R), full(R), full(R, max(picks, 1))
        self.dh, self.dw = new(full(R, H)), new(full(V, H))
        self.ws = A.linear_loss_workspace(R, H, V, dtype, backward=True, device=DEV)
        self.ws.fill_(0xFF)

    def forward(self):
        if self.picks:
            A.linear_distillation(self.hidden, self.weight, self.ids, self.teacher, self.loss, self.lse, self.picked,
                                  self.ws, temperature=self.t)
        else:
            A.linear_cross_entropy(self.hidden, self.weight, self.ids[:, 0], self.loss, self.lse, self.ws)

    def backward(self, dh=True, dw=True):
        dh, dw = self.dh if dh else None, self.dw if dw else None
        if self.picks:
            A.linear_distillation_backward(self.hidden, self.weight, self.ids, self.teacher, self.lse, self.picked,
                                           self.dloss, dh, dw, self.ws, temperature=self.t)
        else:
            A.linear_cross_entropy_backward(self.hidden, self.weight, self.ids[:, 0], self.loss, self.lse, self.dloss,
                                            dh, dw, self.ws)

    def check(self):
        on = ~self.off.cpu()
        want = M.loss(M.f64(self.hidden), M.f64(self.weight), self.ids.cpu(), M.f64(self.teacher) if self.picks else None,
                      self.t, M.f64(self.dloss), self.dtype)
        some = lambda got, what, rows: M.assert_within(got[rows.to(got.device)], tuple(v[rows] for v in want[what]), what)
        self.forward()
        some(self.lse, "lse", on)
        assert not self.loss[self.off].any()
        some(self.loss, "loss", on)
        if self.picks:
            some(self.picked, "picked", on)
        self.ws.fill_(0x3F)
        self.backward()
        M.assert_within(self.dh, want["dhidden"], "dhidden")
        M.assert_within(self.dw, want["dweight"], "dweight")
        return self


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("R", [1, 2, 31, 32, 33, 63, 64, 65, 127, 129, 255, 257, 500])
def test_rows(R, dtype):
    Case(R, 72, 700, TYPES[dtype], seed=R).check()
    Case(R, 40, 300, TYPES[dtype], picks=5, temperature=2.0, seed=R).check()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("H", [1, 2, 7, 8, 9, 63, 64, 65, 127, 128, 136, 200, 257, 520])
def test_widths(H, dtype):
    """Widths that end inside a step of the inner axis, inside 16 bytes, or with a tile."""
    Case(100, H, 500, TYPES[dtype], seed=H).check()
    Case(20, H, 300, TYPES[dtype], picks=3, seed=H).check()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("V", [1, 2, 3, 8, 100, 127, 128, 129, 255, 256, 257, 511, 1000, 5003])
def test_vocabularies(V, dtype):
    Case(70, 64, V, TYPES[dtype], seed=V).check()
    Case(30, 33, V, TYPES[dtype], picks=4, temperature=0.5, seed=V).check()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("R,H,V", [(600, 256, 9000),      # large tiles, several shares of the inner axis
                                   (900, 600, 3001),
                                   (40, 16, 70001),       # several pieces of the vocabulary
                                   (300, 24, 33000),
                                   (2000, 48, 2000)])
def test_shapes(R, H, V, dtype):
    Case(R, H, V, TYPES[dtype], seed=1).check()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("picks", [1, 2, 63, 64, 65, 200, 1024])
def test_picks(picks, dtype):
    """More picks than words make words picked twice and more."""
    Case(33, 48, 400, TYPES[dtype], picks=picks, temperature=3.0, seed=picks).check()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("pad", [1, 3, 8, 24])
def test_strides(pad, dtype):
    """Rows at any distance from each other and from 16 bytes; what lies between is not used and not written."""
    c = Case(130, 64, 700, TYPES[dtype], pad=pad, seed=pad).check()
    for t in (c.dh, c.dw):
        assert torch.isnan(t._base[:, :pad // 2]).all() and torch.isnan(t._base[:, pad // 2 + 64:]).all()
    Case(10, 64, 20000, TYPES[dtype], pad=pad, seed=pad).check()     # copied in pieces


@pytest.mark.parametrize("dtype", TYPES)
def test_even_gradients(dtype):
    """The mean's gradient over many rows: probabilities over the number of rows."""
    Case(3000, 32, 4000, TYPES[dtype], even=True, scale=0.1).check()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("picks", [0, 4])
def test_no_row_counts(dtype, picks):
    c = Case(50, 40, 300, TYPES[dtype], picks=picks, ignored=2.0)
    c.forward()
    c.backward()
    assert not c.loss.any() and not c.dh.any() and not c.dw.any()


@pytest.mark.parametrize("dtype", TYPES)
def test_sharp_rows(dtype):
    """Logits far apart: rows whose target has nearly all, or nothing, of the probability."""
    c = Case(200, 64, 500, TYPES[dtype], ignored=0.0, scale=20.0)
    best = (M.f64(c.hidden) @ M.f64(c.weight).t()).argmax(1)
    c.ids[::2, 0] = best[::2].to(DEV)
    c.check()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("picks", [0, 3])
def test_rows_of_weight_zero(picks, dtype):
    """Rows that count in the loss and whose gradient is 0, among logits whose exponentials overflow: a loss mask."""
    c = Case(90, 64, 600, TYPES[dtype], picks=picks, scale=100.0)
    c.dloss[::2] = 0
    c.check()
    assert not c.dh[::2].any()


def test_teacher_without_probability():
    """Teacher logits of -infinity have no part."""
    c = Case(40, 40, 300, torch.float32, picks=6)
    c.teacher[:, 1] = float("-inf")
    c.teacher[::2, 3] = float("-inf")
    c.ids[:, 0] = torch.arange(40, device=DEV)          # every row keeps one
    c.teacher[:, 0] = 1.0
    c.hidden.copy_(torch.randn(40, 40, device=DEV))
    c.off[:] = False
    c.check()


@pytest.mark.parametrize("dtype", TYPES)
def test_one_gradient_alone(dtype):
    c = Case(100, 40, 3000, TYPES[dtype]).check()
    dh, dw = c.dh.clone(), c.dw.clone()
    for which in (0, 1):
        c.dh.fill_(7.0)
        c.dw.fill_(7.0)
        c.backward(dh=which == 0, dw=which == 1)
        assert torch.equal(c.dh, dh) if which == 0 else (c.dh == 7).all()
        assert torch.equal(c.dw, dw) if which == 1 else (c.dw == 7).all()


@pytest.mark.parametrize("dtype", TYPES)
def test_scales_of_the_gradient(dtype):
    """Powers of two on dloss are powers of two on the gradients, bit for bit where the results do not leave the
    type's normal numbers."""
    c = Case(64, 32, 200, torch.float32 if dtype == "f32" else torch.bfloat16)
    c.forward()
    c.backward()
    dh, dw = c.dh.clone(), c.dw.clone()
    for power in (2.0 ** -60, 2.0 ** 40):
        c.dloss *= power
        c.backward()
        normal = lambda t: (t.float() * power).abs() >= 2.0 ** -120
        for got, was in ((c.dh, dh), (c.dw, dw)):
            m = normal(was)
            assert torch.equal(got[m], (was.float() * power).to(was.dtype)[m])
        c.dloss /= power


def test_repeated_calls_give_the_same_bits():
    c = Case(700, 128, 9000, torch.bfloat16, picks=9)
    c.forward()
    c.backward()
    first = [t.clone() for t in (c.loss, c.lse, c.dh, c.dw)]
    for _ in range(3):
        c.ws.fill_(0x3F)
        c.forward()
        c.backward()
        on = ~c.off
        assert all(torch.equal(a[on] if a.shape[0] == 700 else a, b[on] if b.shape[0] == 700 else b)
                   for a, b in zip(first, (c.loss, c.lse, c.dh, c.dw)))


def test_leading_axes_and_no_rows():
    c = Case(60, 40, 300, torch.bfloat16, ignored=0.0).check()
    loss, dh = torch.empty(4, 15, device=DEV), torch.empty(4, 15, 40, dtype=torch.bfloat16, device=DEV)
    h = c.hidden.view(4, 15, 40)
    A.linear_cross_entropy(h, c.weight, c.ids.view(4, 15), loss, c.lse, c.ws)
    assert torch.equal(loss.view(-1), c.loss)
    A.linear_cross_entropy_backward(h, c.weight, c.ids.view(4, 15), loss, c.lse, c.dloss, dh, None, c.ws)
    assert torch.equal(dh.view(60, 40), c.dh)
    c = Case(0, 40, 300, torch.bfloat16)
    c.forward()
    c.backward()
    assert not c.dw.any()
