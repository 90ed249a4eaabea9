"""The selective scan and its gradients on the GPU against the 64-bit form,
within bounds that count the roundings."""
import pytest
import torch

import adaptive_residual_gradient_amd as A
import model_refs as M
from test_gpu_gated_scan import as_view

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
GRADS = ("dx", "ddt", "da", "db", "dc", "dz", "dd", "ddt_bias", "dh0")


class Case:
    def __init__(self, B, T, C, N, dtype, gated=True, softplus=True, lengths=None, extras=True, layout="plain", seed=0,
                 dt_scale=1.0):
        gen = torch.Generator(device=DEV).manual_seed(seed)
        normal = lambda *s: torch.randn(*s, generator=gen, device=DEV)
        new = lambda v: as_view(v.to(dtype), layout, gen)
        full = lambda *s: torch.full(s, 7.0, device=DEV)
        self.softplus, self.dtype, self.shape = softplus, dtype, (B, T, C, N)
        dt = normal(B, T, C) * dt_scale - (2.0 if softplus else 0.0)
        self.i = dict(x=new(normal(B, T, C)), dt=new(dt if softplus else dt.abs() * 0.2),
                      a=-(0.2 + 3 * torch.rand(C, N, generator=gen, device=DEV)), b=new(normal(B, T, N)),
                      c=new(normal(B, T, N)), d=normal(C) if extras else None,
                      z=new(normal(B, T, C) * 2) if gated else None, dt_bias=normal(C) * 0.3 if extras else None)
        self.h0, self.dl = (normal(B, C, N), normal(B, C, N)) if extras else (None, None)
        self.dy, self.y = new(normal(B, T, C)), new(full(B, T, C))
        self.g = dict(dx=new(full(B, T, C)), ddt=new(full(B, T, C)), da=full(C, N), db=new(full(B, T, N)),
                      dc=new(full(B, T, N)), dz=new(full(B, T, C)) if gated else None, dd=full(C) if extras else None,
                      ddt_bias=full(C) if extras else None, dh0=full(B, C, N))
        self.last = full(B, C, N)
        self.lengths = None
        if lengths is not None:
            self.lengths = torch.tensor(lengths, dtype=torch.int32, device=DEV)
            for k, n in enumerate(lengths):
                for t in [self.i[s] for s in ("x", "dt", "b", "c", "z") if self.i[s] is not None] + [self.dy]:
                    t[k, max(n, 0):] = float("nan") if k % 2 else float("inf")
        self.kept = A.selective_scan_states(B, T, C, N, DEV)
        self.kept.fill_(float("nan"))
        self.ws = A.selective_scan_workspace(B, T, C, N, True, DEV)
        self.ws.fill_(0xFF)

    def forward(self, kept=True):
        i = self.i
        A.selective_scan(i["x"], i["dt"], i["a"], i["b"], i["c"], self.y, d=i["d"], z=i["z"], dt_bias=i["dt_bias"],
                         h0=self.h0, h_last=self.last, states=self.kept if kept else None, lengths=self.lengths,
                         softplus=self.softplus, ws=self.ws)

    def backward(self):
        i, g = self.i, self.g
        A.selective_scan_backward(self.dy, i["x"], i["dt"], i["a"], i["b"], i["c"], self.kept, g["dx"], g["ddt"], g["da"],
                                  g["db"], g["dc"], d=i["d"], z=i["z"], dt_bias=i["dt_bias"], dz=g["dz"], dd=g["dd"],
                                  ddt_bias=g["ddt_bias"], dh_last=self.dl, dh0=g["dh0"], lengths=self.lengths,
                                  softplus=self.softplus, ws=self.ws)

    def check(self):
        n = None if self.lengths is None else self.lengths.cpu()
        want = M.scan(**{k: M.f64(v) for k, v in self.i.items()}, h0=M.f64(self.h0), lengths=n, softplus=self.softplus,
                      dy=M.f64(self.dy), dh_last=M.f64(self.dl))
        self.forward(kept=False)     # short sequences take another kernel
        M.assert_within(self.y, want["y"], "y")
        M.assert_within(self.last, want["h_last"], "h_last")
        self.ws.fill_(0xFF)
        self.forward()
        M.assert_within(self.y, want["y"], "y with states kept")
        M.assert_within(self.last, want["h_last"], "h_last with states kept")
        self.ws.fill_(0x3F)
        self.backward()
        for k in GRADS:
            if self.g[k] is not None:
                M.assert_within(self.g[k], want[k], k)
        return self


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T", [1, 2, 3, 7, 8, 9, 15, 16, 17, 63, 64, 65, 129, 200])
def test_lengths(T, dtype):
    Case(2, T, 70, 16, TYPES[dtype], gated=T % 2 == 0, seed=T).check()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("N", [1, 2, 4, 7, 8, 9, 12, 16, 17, 24, 32, 33, 48, 63, 64])
def test_states(N, dtype):
    Case(2, 21, 33, N, TYPES[dtype], gated=N % 2 == 0, seed=N).check()
    Case(3, 1, 33, N, TYPES[dtype], seed=N).check()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("C", [1, 2, 3, 31, 63, 64, 65, 127, 128, 129, 256, 257, 300])
def test_channels(C, dtype):
    Case(2, 19, C, 16, TYPES[dtype], seed=C).check()
    Case(2, 11, C, 5, TYPES[dtype], gated=False, seed=C).check()
    Case(3, 2, C, 3, TYPES[dtype], seed=C).check()


@pytest.mark.parametrize("B,T,C,N", [(1, 1100, 20, 16),     # cut into chunks of 64 steps
                                     (1, 700, 130, 40),
                                     (9, 150, 64, 8),
                                     (2, 333, 100, 20),
                                     (40, 10, 64, 16)])
@pytest.mark.parametrize("gated", [False, True])
def test_shapes(B, T, C, N, gated):
    Case(B, T, C, N, torch.float32, gated=gated, seed=1).check()
    Case(B, T, C, N, torch.bfloat16, gated=gated, seed=2).check()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("N", [3, 16, 24])
def test_ragged(N, dtype):
    """Empty, negative, whole and too long lengths, ends inside a block and on its edges and on the edges of
    chunks, with NaN and infinities at the masked steps."""
    T = 210
    lengths = [0, -5, T, T + 100, 1, 7, 8, 9, 63, 64, 65, 128, 209, 192]
    Case(len(lengths), T, 65, N, TYPES[dtype], lengths=lengths).check()
    Case(4, 3, 65, N, TYPES[dtype], lengths=[0, 1, 2, 3]).check()
    Case(2, 100, 10, N, TYPES[dtype], lengths=[0, 0], gated=False).check()


@pytest.mark.parametrize("layout", ["part", "time_first"])
@pytest.mark.parametrize("dtype", TYPES)
def test_strides(layout, dtype):
    c = Case(4, 90, 37, 9, TYPES[dtype], lengths=[90, 3, 0, 89], layout=layout).check()
    if layout == "part":
        for k, w in (("dx", 37), ("ddt", 37), ("dz", 37), ("db", 9), ("dc", 9)):
            t = c.g[k]._base
            assert torch.isnan(t[:, :, 0]).all() and torch.isnan(t[:, :, 1 + w:]).all()


@pytest.mark.parametrize("T", [5, 100])
def test_without_the_optional_arguments(T):
    Case(2, T, 40, 16, torch.float32, gated=False, extras=False).check()
    Case(2, T, 40, 16, torch.float32, gated=True, extras=False, softplus=False).check()
    Case(2, T, 40, 16, torch.bfloat16, softplus=False).check()


@pytest.mark.parametrize("T", [4, 150])
def test_steps_of_any_size(T):
    """Steps from exp(-20) to 20: decays of nearly 1 and of nothing."""
    Case(2, T, 64, 16, torch.float32, dt_scale=8.0).check()


@pytest.mark.parametrize("dtype", TYPES)
def test_tokens_one_by_one(dtype):
    """A prompt and then single tokens, from state to state, against one call: the same steps by other kernels, each
    within its bound."""
    B, T, C, N, P = 2, 40, 50, 16, 32
    c = Case(B, T, C, N, TYPES[dtype])
    i = c.i
    want = M.scan(**{k: M.f64(v) for k, v in i.items()}, h0=M.f64(c.h0))
    h, out = c.h0, torch.empty_like(c.y)
    for t, u in [(0, P)] + [(t, t + 1) for t in range(P, T)]:
        new = torch.empty_like(c.last)
        A.selective_scan(i["x"][:, t:u], i["dt"][:, t:u], i["a"], i["b"][:, t:u], i["c"][:, t:u], out[:, t:u], d=i["d"],
                         z=i["z"][:, t:u], dt_bias=i["dt_bias"], h0=h, h_last=new, ws=c.ws)
        h = new
    M.assert_within(out, want["y"], "y")
    M.assert_within(h, want["h_last"], "h_last")


def test_parts_of_one_projection():
    """x and z halves of one tensor, dt, b and c parts of another, and their gradients of others like them."""
    B, T, C, N = 2, 70, 64, 16
    c = Case(B, T, C, N, torch.bfloat16).check()
    want = {k: v.clone() for k, v in c.g.items()}
    xz, rest = torch.empty(B, T, 2 * C, dtype=c.dtype, device=DEV), torch.empty(B, T, C + 2 * N, dtype=c.dtype, device=DEV)
    gxz, grest = torch.empty_like(xz), torch.empty_like(rest)
    parts = lambda a, r: dict(x=a[:, :, :C], z=a[:, :, C:], dt=r[:, :, :C], b=r[:, :, C:C + N], c=r[:, :, C + N:])
    for k, v in parts(xz, rest).items():
        v.copy_(c.i[k])
        c.i[k] = v
    for k, v in parts(gxz, grest).items():
        c.g["d" + k] = v
    c.forward()
    c.backward()
    assert all(torch.equal(want[k], c.g[k]) for k in GRADS)


def test_repeated_calls_give_the_same_bits():
    c = Case(2, 500, 200, 16, torch.bfloat16)
    c.forward()
    c.backward()
    first = [t.clone() for t in (c.y, c.last, *c.g.values())]
    for _ in range(3):
        c.ws.fill_(0x3F)
        c.forward()
        c.backward()
        assert all(torch.equal(a, b) for a, b in zip(first, (c.y, c.last, *c.g.values())))


def test_no_steps_and_no_sequences():
    c = Case(3, 0, 10, 16, torch.float32)
    c.forward()
    assert torch.equal(c.last, c.h0)
    c.backward()
    assert torch.equal(c.g["dh0"], c.dl)
    assert not any(c.g[k].any() for k in ("da", "dd", "ddt_bias"))
    c = Case(0, 5, 10, 16, torch.float32)
    c.forward()
    c.backward()
    assert not any(c.g[k].any() for k in ("da", "dd", "ddt_bias"))


def test_a_neighbour_s_infinity_stays_there():
    """A channel with an infinite input has no part in the others' results."""
    c = Case(1, 40, 70, 16, torch.float32)
    c.forward()
    y = c.y.clone()
    c.i["x"][0, 5, 69] = float("inf")
    c.forward()
    assert torch.equal(c.y[..., :69], y[..., :69]) and not torch.isfinite(c.y[0, 5:, 69]).any()


def test_places_past_32_bits():
    """Sequences that lie 2^31 elements and more into a buffer."""
    c = Case(3, 5, 8, 4, torch.bfloat16)
    c.check()
    y, g = c.y.clone(), {k: v.clone() for k, v in c.g.items()}
    room = torch.empty(2 * (2 ** 30 + 8) + 40, dtype=torch.bfloat16, device=DEV)
    for k in ("x", "b"):
        v = torch.as_strided(room, c.i[k].shape, (2 ** 30 + 8, c.i[k].shape[2], 1))
        old = c.i[k]
        v.copy_(old)
        c.i[k] = v
        c.forward()
        c.backward()
        assert torch.equal(y, c.y) and all(torch.equal(g[s], c.g[s]) for s in g)
        c.i[k] = old
