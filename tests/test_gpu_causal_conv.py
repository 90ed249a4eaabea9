"""The causal convolution and its gradients on the GPU against the 64-bit form,
within bounds that count the roundings."""
import pytest
import torch

import adaptive_residual_gradient_amd as A
import model_refs as M
from test_gpu_gated_scan import as_view

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


class Case:
    def __init__(self, B, T, C, K, dtype, silu=True, lengths=None, state=True, bias=True, layout="plain", seed=0):
        gen = torch.Generator(device=DEV).manual_seed(seed)
        normal = lambda *s: torch.randn(*s, generator=gen, device=DEV)
        new = lambda v: as_view(v.to(dtype), layout, gen)
        self.silu, self.K, self.dtype = silu, K, dtype
        self.x, self.dy = new(normal(B, T, C) * 1.5), new(normal(B, T, C))
        self.y, self.dx = (new(torch.full((B, T, C), 7.0, device=DEV)) for _ in range(2))
        self.w, self.bias = normal(C, K), normal(C) if bias else None
        self.state = normal(B, K - 1, C).to(dtype) if state else None
        full = lambda *s, t=torch.float32: torch.full(s, 7.0, dtype=t, device=DEV)
        self.state_out, self.dstate = full(B, K - 1, C, t=dtype), full(B, K - 1, C, t=dtype) if state else None
        self.dw, self.db = full(C, K), full(C) if bias else None
        self.lengths = None
        if lengths is not None:
            self.lengths = torch.tensor(lengths, dtype=torch.int32, device=DEV)
            for b, n in enumerate(lengths):
                for t in (self.x, self.dy):
                    t[b, max(n, 0):] = float("nan") if b % 2 else float("inf")
        self.ws = A.causal_conv_workspace(B, T, C, K, DEV)
        self.ws.fill_(0xFF)

    def forward(self):
        A.causal_conv(self.x, self.w, self.bias, self.y, self.state, self.state_out, self.lengths, silu=self.silu)

    def backward(self):
        A.causal_conv_backward(self.dy, self.x, self.w, self.bias, self.dx, self.dw, self.db, self.state, self.dstate,
                               self.lengths, silu=self.silu, ws=self.ws)

    def check(self):
        self.forward()
        self.backward()
        n = None if self.lengths is None else self.lengths.cpu()
        want = M.conv(M.f64(self.x), M.f64(self.w), M.f64(self.bias), M.f64(self.state), n, self.silu, M.f64(self.dy))
        for got, what in ((self.y, "y"), (self.state_out, "state_out"), (self.dx, "dx"), (self.dw, "dweight"),
                          (self.db, "dbias"), (self.dstate, "dstate")):
            if got is not None:
                M.assert_within(got, want[what], what)
        return self


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("K", range(1, 9))
def test_taps(K, dtype):
    Case(3, 37, 20, K, TYPES[dtype], seed=K).check()
    Case(2, 40, 3, K, TYPES[dtype], silu=False, state=False, bias=False, seed=K).check()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T", [1, 2, 3, 4, 5, 15, 16, 17, 31, 32, 33, 64, 65, 250])
def test_lengths(T, dtype):
    Case(3, T, 70, 4, TYPES[dtype], seed=T).check()
    Case(2, T, 24, 8, TYPES[dtype], seed=T).check()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("C", [1, 2, 3, 4, 7, 8, 9, 15, 16, 33, 63, 65, 255, 257, 1000, 2100])
def test_channels(C, dtype):
    Case(2, 45, C, 4, TYPES[dtype], seed=C).check()
    Case(3, 1, C, 2, TYPES[dtype], seed=C).check()


@pytest.mark.parametrize("B,T,C", [(1, 9000, 40), (64, 130, 33), (300, 1, 7), (2, 2000, 1000), (5, 600, 2056)])
def test_shapes(B, T, C):
    """Long sequences, many of them, and sizes with many steps a thread."""
    Case(B, T, C, 4, torch.float32, seed=1).check()
    Case(B, T, C, 3, torch.bfloat16, seed=2).check()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("K", [2, 4, 7])
def test_ragged(K, dtype):
    """Empty, negative, whole and too long lengths, shorter than the filter, and NaN and infinities at the
    masked steps."""
    T = 133
    lengths = [0, -5, T, T + 100, 1, 2, 3, 4, 15, 16, 17, 31, 32, 33, 132, 64]
    Case(len(lengths), T, 41, K, TYPES[dtype], lengths=lengths).check()
    Case(3, 1, 41, K, TYPES[dtype], lengths=[0, 1, 2]).check()
    Case(2, 50, 8, K, TYPES[dtype], lengths=[0, 0], state=False).check()


@pytest.mark.parametrize("layout", ["part", "time_first"])
@pytest.mark.parametrize("dtype", TYPES)
def test_strides(layout, dtype):
    c = Case(4, 90, 37, 4, TYPES[dtype], lengths=[90, 3, 0, 89], layout=layout).check()
    if layout == "part":
        for t in (c.y, c.dx):
            assert torch.isnan(t._base[:, :, 0]).all() and torch.isnan(t._base[:, :, 1 + 37:]).all()


def test_large_values():
    """The logistic function's ends: far negative sums give 0, far positive ones themselves."""
    c = Case(1, 64, 16, 2, torch.float32, state=False, bias=False)
    c.w.fill_(1.0)
    c.x.copy_(torch.linspace(-600, 600, 64, device=DEV)[None, :, None].expand(1, 64, 16))
    c.check()


@pytest.mark.parametrize("dtype", TYPES)
def test_tokens_one_by_one(dtype):
    """A prompt and then single tokens, from state to state: the same bits as one call."""
    B, T, C, K, P = 3, 23, 40, 4, 14
    c = Case(B, T, C, K, TYPES[dtype])
    c.forward()
    y, states = torch.empty_like(c.y), [torch.empty_like(c.state_out) for _ in range(2)]
    A.causal_conv(c.x[:, :P], c.w, c.bias, y[:, :P], c.state, states[0])
    for i, t in enumerate(range(P, T)):
        A.causal_conv(c.x[:, t:t + 1], c.w, c.bias, y[:, t:t + 1], states[i % 2], states[(i + 1) % 2])
    assert torch.equal(y, c.y) and torch.equal(states[(T - P) % 2], c.state_out)


def test_repeated_calls_give_the_same_bits():
    c = Case(7, 300, 100, 4, torch.bfloat16)
    c.backward()
    first = [t.clone() for t in (c.dx, c.dw, c.db, c.dstate)]
    for _ in range(3):
        c.ws.fill_(0x3F)
        c.backward()
        assert all(torch.equal(a, b) for a, b in zip(first, (c.dx, c.dw, c.db, c.dstate)))


def test_no_steps_and_no_sequences():
    c = Case(3, 0, 10, 4, torch.float32)
    c.forward()
    assert torch.equal(c.state_out, c.state)
    c.backward()
    assert not c.dw.any() and not c.db.any() and not c.dstate.any()
    c = Case(0, 5, 10, 4, torch.float32)
    c.forward()
    c.backward()
    assert not c.dw.any() and not c.db.any()


def test_places_past_32_bits():
    """Sequences that lie 2^31 elements and more into a buffer."""
    B, T, C, K = 3, 5, 8, 4
    room = torch.empty(2 * (2 ** 30 + 8) + T * C, dtype=torch.bfloat16, device=DEV)
    view = lambda: torch.as_strided(room, (B, T, C), (2 ** 30 + 8, C, 1))
    gen = torch.Generator(device=DEV).manual_seed(3)
    c = Case(B, T, C, K, torch.bfloat16)
    c.check()
    view().copy_(c.x)
    y = torch.empty_like(c.y)
    A.causal_conv(view(), c.w, c.bias, y, c.state, None)
    assert torch.equal(y, c.y)
    A.causal_conv(c.x, c.w, c.bias, view(), c.state, None)
    assert torch.equal(view(), c.y)
    del gen
