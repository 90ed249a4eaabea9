"""The gated linear recurrence and its gradients on the GPU against the 64-bit
forms, within bounds that count the roundings."""
import numpy as np
import pytest
import torch

import adaptive_residual_gradient_amd as A
import operator_refs as R

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device=DEV)


def as_view(x, layout, gen):
    """The same values contiguous, as a part of wider rows, or with time first in memory; what lies between
    is NaN."""
    B, T, D = x.shape
    if layout == "plain":
        return x
    if layout == "part":       # from an odd element on
        room = torch.full((B, T, 2 * D + 3), float("nan"), dtype=x.dtype, device=DEV)
        v = room[:, :, 1:1 + D]
    else:
        v = torch.full((T, B, D), float("nan"), dtype=x.dtype, device=DEV).transpose(0, 1)
    v.copy_(x)
    return v


class Case:
    def __init__(self, B, T, D, dtype, sigmoid, lengths=None, layout="plain", states=True, seed=0):
        gen = torch.Generator(device=DEV).manual_seed(seed)
        self.sigmoid, self.dtype, self.shape = sigmoid, dtype, (B, T, D)
        z = normal(gen, B, T, D) * 2 + 1
        z = z if sigmoid else torch.sigmoid(z) * torch.where(normal(gen, B, T, D) < -1.5, -1.0, 1.0)
        new = lambda x: as_view(x.to(dtype), layout, gen)
        self.z, self.x, self.dh = new(z), new(normal(gen, B, T, D)), new(normal(gen, B, T, D) * 0.1)
        self.h, self.dz, self.dx = (new(torch.full((B, T, D), 7.0, device=DEV)) for _ in range(3))
        self.h0 = normal(gen, B, D) if states else None
        self.dl = normal(gen, B, D) * 0.1 if states else None
        self.last, self.dh0 = torch.full((B, D), 7.0, device=DEV), torch.full((B, D), 7.0, device=DEV)
        self.lengths = None
        self.n = np.full(B, T)
        if lengths is not None:
            self.lengths = torch.tensor(lengths, dtype=torch.int32, device=DEV)
            self.n = np.clip(np.array(lengths), 0, T)
            for b, k in enumerate(self.n):      # whatever is masked does not count
                for t in (self.z, self.x, self.dh):
                    t[b, k:] = float("nan") if b % 2 else float("inf")
        self.ws = A.gated_scan_workspace(B, T, D, DEV)
        if self.ws.numel():
            self.ws.fill_(0xFF)

    def forward(self):
        A.gated_scan(self.z, self.x, self.h, h0=self.h0, h_last=self.last, lengths=self.lengths,
                     sigmoid=self.sigmoid, ws=self.ws)

    def backward(self):
        A.gated_scan_backward(self.z, self.x if self.sigmoid else None, self.h, self.dh, self.dz, self.dx, h0=self.h0,
                              dh_last=self.dl, dh0=self.dh0, lengths=self.lengths, sigmoid=self.sigmoid, ws=self.ws)

    def check(self):
        B, T, D = self.shape
        zero = np.zeros((B, D))
        z, x, h0 = R.f64(self.z), R.f64(self.x), R.f64(self.h0) if self.h0 is not None else zero
        self.forward()
        (h, e), (last, el) = R.scan_forward(z, x, h0, self.n, self.sigmoid, self.dtype)
        R.assert_within(self.h, h, R.rounded(h, e, self.dtype), "h")
        R.assert_within(self.last, last, R.rounded(last, el, torch.float32), "h_last")
        self.backward()
        dl = R.f64(self.dl) if self.dl is not None else zero
        want = R.scan_backward(z, x, R.f64(self.h), R.f64(self.dh), h0, dl, self.n, self.sigmoid, self.dtype)
        for got, (v, err), what, dt in ((self.dz, want[0], "dgate", self.dtype), (self.dx, want[1], "dx", self.dtype),
                                        (self.dh0, want[2], "dh0", torch.float32)):
            R.assert_within(got, v, R.rounded(v, err, dt), what)
        return self


@pytest.mark.parametrize("sigmoid", [True, False])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T", [1, 2, 7, 8, 9, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 300, 1025])
def test_lengths(T, dtype, sigmoid):
    Case(3, T, 70, TYPES[dtype], sigmoid, seed=T).check()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D", [1, 2, 3, 4, 5, 7, 8, 9, 15, 16, 31, 63, 64, 65, 127, 130, 257, 513, 1000])
def test_channels(D, dtype):
    Case(2, 150, D, TYPES[dtype], True, seed=D).check()
    Case(2, 1, D, TYPES[dtype], True, seed=D).check()


@pytest.mark.parametrize("B,T,D", [(1, 5000, 24), (64, 40, 33), (5, 700, 260), (300, 1, 7), (1, 20000, 3),
                                   (16, 513, 128),
                                   # at least 64 chains of tiles: the state travels from tile to tile
                                   (64, 600, 20), (70, 300, 33), (5, 1500, 1000), (1, 3000, 4101), (130, 270, 1)])
@pytest.mark.parametrize("sigmoid", [True, False])
def test_shapes(B, T, D, sigmoid):
    Case(B, T, D, torch.float32, sigmoid, seed=1).check()
    Case(B, T, D, torch.bfloat16, sigmoid, seed=2).check()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("sigmoid", [True, False])
def test_ragged(dtype, sigmoid):
    """Empty, negative, whole and too long lengths, ends inside a chunk and on its edges, with NaN and
    infinities at the masked steps."""
    T = 333
    lengths = [0, -5, T, T + 100, 1, 16, 17, 15, 128, 127, 129, 332, 64, 200]
    Case(len(lengths), T, 65, TYPES[dtype], sigmoid, lengths=lengths).check()
    Case(3, 1, 65, TYPES[dtype], sigmoid, lengths=[0, 1, 2]).check()
    Case(2, 1000, 65, TYPES[dtype], sigmoid, lengths=[0, 0]).check()
    rng = np.random.default_rng(3)
    T = 1100
    lengths = [0, T, 1, 255, 256, 257, 511, 512, 513, 767, 768, 769] + rng.integers(0, T + 1, 60).tolist()
    Case(len(lengths), T, 40, TYPES[dtype], sigmoid, lengths=lengths).check()
    T = 3000
    Case(6, T, 40, TYPES[dtype], sigmoid, lengths=[0, T, 1, 1024, 2047, 2050]).check()


@pytest.mark.parametrize("layout", ["part", "time_first"])
@pytest.mark.parametrize("dtype", TYPES)
def test_strides(layout, dtype):
    """Parts of wider rows from an odd element on, and time-major buffers; the places between the rows are not
    written."""
    c = Case(4, 210, 37, TYPES[dtype], True, lengths=[210, 3, 0, 209], layout=layout).check()
    if layout == "part":
        for t in (c.h, c.dz, c.dx):
            assert torch.isnan(t._base[:, :, 0]).all() and torch.isnan(t._base[:, :, 1 + 37:]).all()


def test_gate_and_input_of_one_projection():
    """gate and x as halves of one [batch, length, 2 channels] tensor, their gradients as halves of another."""
    B, T, D = 2, 300, 64
    c = Case(B, T, D, torch.bfloat16, True)
    both = torch.cat([c.z, c.x], 2)
    grads = torch.full_like(both, 7.0)
    h, dh0 = torch.empty_like(c.h), torch.empty_like(c.dh0)
    c.forward()
    c.backward()
    A.gated_scan(both[:, :, :D], both[:, :, D:], h, h0=c.h0, ws=c.ws)
    A.gated_scan_backward(both[:, :, :D], both[:, :, D:], h, c.dh, grads[:, :, :D], grads[:, :, D:], h0=c.h0,
                          dh_last=c.dl, dh0=dh0, ws=c.ws)
    assert torch.equal(h, c.h) and torch.equal(dh0, c.dh0)
    assert torch.equal(grads, torch.cat([c.dz, c.dx], 2))


def test_one_gate_for_all_sequences():
    """A gate with batch stride 0."""
    c = Case(3, 120, 40, torch.float32, True)
    z = c.z[:1].expand(3, -1, -1)
    h = torch.empty_like(c.h)
    A.gated_scan(z, c.x, h, h0=c.h0, ws=c.ws)
    c.z = z.contiguous()
    c.forward()
    assert torch.equal(h, c.h)


def test_without_states():
    Case(3, 200, 40, torch.float32, True, states=False).check()
    c = Case(3, 200, 40, torch.float32, True, states=False)
    h, dz, dx = (torch.empty_like(c.h) for _ in range(3))
    A.gated_scan(c.z, c.x, h, ws=c.ws)
    A.gated_scan_backward(c.z, c.x, h, c.dh, dz, dx, ws=c.ws)
    c.forward()
    c.backward()
    assert torch.equal(h, c.h) and torch.equal(dz, c.dz) and torch.equal(dx, c.dx)


def test_no_steps_and_no_sequences():
    h0 = torch.randn(3, 8, device=DEV)
    e = torch.empty(3, 0, 8, device=DEV)
    last, dh0 = torch.zeros(3, 8, device=DEV), torch.zeros(3, 8, device=DEV)
    A.gated_scan(e, e.clone(), e.clone(), h0=h0, h_last=last, ws=A.gated_scan_workspace(3, 0, 8, DEV))
    A.gated_scan_backward(e, e.clone(), e.clone(), e.clone(), e.clone(), e.clone(), dh_last=h0, dh0=dh0,
                          ws=A.gated_scan_workspace(3, 0, 8, DEV))
    assert torch.equal(last, h0) and torch.equal(dh0, h0)
    e = torch.empty(0, 5, 8, device=DEV)
    A.gated_scan(e, e.clone(), e.clone(), ws=A.gated_scan_workspace(0, 5, 8, DEV))


def test_far_gates():
    """Gates where one of the two factors is tiny, and gates that are infinite."""
    B, T, D = 2, 100, 8
    z = torch.linspace(-120, 120, B * T * D, device=DEV).view(B, T, D).contiguous()
    c = Case(B, T, D, torch.float32, True)
    c.z.copy_(z[:, torch.randperm(T, device=DEV)])
    c.forward()
    assert torch.isfinite(c.h).all()
    zz = R.f64(c.z)
    # factors of float32's exponential below its smallest number are 0
    (h, e), _ = R.scan_forward(zz, R.f64(c.x), R.f64(c.h0), c.n, True)
    R.assert_within(c.h, h, R.rounded(h, e + 1e-36, torch.float32), "h")
    c.z[:, 10] = float("inf")      # keeps the state
    c.z[:, 20] = float("-inf")     # takes the input
    c.forward()
    assert torch.equal(c.h[:, 10], c.h[:, 9]) and torch.equal(c.h[:, 20], c.x[:, 20])


def test_one_token_steps_follow_the_whole_sequence():
    """Steps of one token from the carried state give what one call over the sequence gives."""
    B, T, D = 4, 40, 96
    c = Case(B, T, D, torch.float32, True)
    c.forward()
    s, n = c.h0.clone(), torch.empty_like(c.h0)
    for t in range(T):
        h = torch.empty(B, 1, D, device=DEV)
        A.gated_scan(c.z[:, t:t + 1], c.x[:, t:t + 1], h, h0=s, h_last=n)
        s, n = n, s
        assert torch.allclose(h[:, 0], c.h[:, t], rtol=1e-5, atol=1e-6)


def test_gradient_against_differences():
    c = Case(3, 90, 20, torch.float32, True, lengths=[90, 0, 33], seed=5)
    c.z, c.x, c.dh = (torch.nan_to_num(t, nan=0.5, posinf=0.5) for t in (c.z, c.x, c.dh))
    c.forward()
    c.backward()
    rng = np.random.default_rng(0)
    z, x, h0, dh, dl = (R.f64(t) for t in (c.z, c.x, c.h0, c.dh, c.dl))
    def loss(z_, x_, h0_):
        (h, _), (last, _) = R.scan_forward(z_, x_, h0_, c.n, True)
        return (h * dh).sum() + (last * dl).sum()
    for i, got in enumerate((c.dz, c.dx, c.dh0)):
        at = [z, x, h0]
        u = rng.standard_normal(at[i].shape)
        hi, lo = list(at), list(at)
        hi[i], lo[i] = at[i] + 1e-5 * u, at[i] - 1e-5 * u
        diff = (loss(*hi) - loss(*lo)) / 2e-5
        assert abs(diff - (R.f64(got) * u).sum()) < 1e-4 * np.abs(R.f64(got) * u).sum()


def test_in_a_graph_and_on_another_stream():
    args = (3, 700, 130, torch.bfloat16, True)
    lengths = [700, 33, 500]
    c, d, e = (Case(*args, lengths=lengths) for _ in range(3))
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        c.forward()
        c.backward()
    other = torch.cuda.Stream()
    for i in range(5):
        new = torch.randn(3, 700, 130, device=DEV).bfloat16()
        for k in (c, d, e):
            k.x.copy_(new)
        g.replay()
        torch.cuda.synchronize()
        d.forward()
        d.backward()
        torch.cuda.synchronize()
        with torch.cuda.stream(other):
            e.forward()
            e.backward()
        other.synchronize()
        for k in ("h", "last", "dz", "dx", "dh0"):
            assert torch.equal(getattr(c, k), getattr(d, k)), (i, k)
            assert torch.equal(getattr(c, k), getattr(e, k)), (i, k)


def test_refusals():
    z = torch.zeros(2, 3000, 8, device=DEV)
    x, h, ws = z.clone(), z.clone(), A.gated_scan_workspace(2, 3000, 8, DEV)
    assert ws.numel() > 64      # several tiles: a workspace is needed
    for bad in (lambda: A.gated_scan(z, x, z, ws=ws), lambda: A.gated_scan(z, x, x, ws=ws),
                lambda: A.gated_scan(z, x, h), lambda: A.gated_scan(z, x, h, ws=ws[:64]),
                lambda: A.gated_scan_backward(z, None, h, x, z.clone(), z.clone(), ws=ws),
                lambda: A.gated_scan(z, x, h[:1].expand(2, 3000, 8), ws=ws)):
        with pytest.raises(A.AdaCompError):
            bad()
    with pytest.raises(ValueError):
        A.gated_scan(z, x[:, :200], h, ws=ws)
    with pytest.raises(ValueError):
        A.gated_scan(z, x.bfloat16(), h, ws=ws)
    with pytest.raises(ValueError):
        A.gated_scan(z, x, h, h0=torch.zeros(2, 7, device=DEV), ws=ws)
    with pytest.raises(TypeError):
        A.gated_scan(z.transpose(1, 2).contiguous().transpose(1, 2), x, h, ws=ws)
    with pytest.raises(TypeError):
        A.gated_scan(z, x, h, lengths=torch.tensor([1, 2], device=DEV), ws=ws)
    with pytest.raises(ValueError):
        A.gated_scan(z, x, h, lengths=torch.tensor([1], dtype=torch.int32, device=DEV), ws=ws)
