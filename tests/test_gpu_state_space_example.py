"""The convolution, the selective scan and the losses together, as
examples/train_state_space.py uses them: the model's gradients against 64-bit
autograd, decoding word by word against one call, a short run, graphs and
streams."""
import pathlib
import sys

import pytest
import torch

sys.path.insert(0, str(pathlib.Path(__file__).resolve().parent.parent / "examples"))
import adaptive_residual_gradient_amd as A  # noqa: E402
import train_state_space as E  # noqa: E402

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def plain(layout, flat, words, lengths):
    """The last layer's normed states in elementary 64-bit operations."""
    of, D, En, N, R = layout.of, layout.width, layout.inner, layout.states, layout.rank
    live = torch.ones(words.shape, dtype=torch.bool)
    if lengths is not None:
        live = torch.arange(words.shape[1]) < lengths[:, None]

    def norm(i, x):
        d = x - x.mean(2, keepdim=True)
        return d / torch.sqrt((d * d).mean(2, keepdim=True) + E.EPS) * of(flat, i, "weight") + of(flat, i, "bias")
    h = of(flat, None, "embed")[words]
    for i in range(layout.layers):
        proj = norm(i, h) @ of(flat, i, "in").t()
        x, z = proj[:, :, :En], proj[:, :, En:]
        rows = torch.nn.functional.pad(x, (0, 0, layout.taps - 1, 0))
        p = of(flat, i, "conv_bias") + sum(of(flat, i, "conv")[:, k] * rows[:, k:k + x.shape[1]] for k in range(layout.taps))
        xc = p * torch.sigmoid(p) * live[:, :, None]
        low = xc @ of(flat, i, "low").t()
        s = torch.nn.functional.softplus(low[:, :, :R] @ of(flat, i, "dt").t() + of(flat, i, "dt_bias"))
        state, a, ys = torch.zeros(words.shape[0], En, N).double(), -torch.exp(of(flat, i, "rate")), []
        for t in range(words.shape[1]):
            b, c = low[:, t, None, R:R + N], low[:, t, None, R + N:]
            state = torch.exp(s[:, t, :, None] * a) * state + (s * xc)[:, t, :, None] * b
            ys.append((state * c).sum(2) + of(flat, i, "d") * xc[:, t])
        y = torch.stack(ys, 1) * z * torch.sigmoid(z) * live[:, :, None]
        h = h + y @ of(flat, i, "out").t()
    return norm(None, h).reshape(-1, D)


@pytest.mark.parametrize("distil", [False, True])
@pytest.mark.parametrize("ragged", [False, True])
def test_gradients_of_the_model(ragged, distil):
    """float32 layers.  Every gradient is a chain of about two dozen sums of at most B T = 60 or 2 D = 48 terms with
    relative errors of at most 2^-22 a term (a few roundings each, the terms of a sum adding up like their roots in norm,
    2^-22 * 60 at worst): 24 * 60 * 2^-22 = 3.5e-4 of its norm."""
    B, T, V, K = 3, 20, 70, 6
    layout = E.Layout(2, 24, V, states=5, taps=3, rank=4)
    flat = layout.init(DEV, 1)
    gen = torch.Generator(device=DEV).manual_seed(2)
    draw = lambda *s: torch.randint(0, V, s, generator=gen, device=DEV)
    words, targets = draw(B, T), draw(B * T)
    lengths = torch.tensor([20, 0, 7], dtype=torch.int32, device=DEV) if ragged else None
    targets[::7] = -100
    ids, teacher = draw(B * T, K), torch.randn(B * T, K, generator=gen, device=DEV) * 2
    ids[::7] = -1
    model = E.Model(layout, B, T, torch.float32, DEV)
    grad = torch.zeros_like(flat)
    if distil:
        loss = model.distillation(flat, flat, words, ids, teacher, grad, 2.0, lengths)
    else:
        loss = model.cross_entropy(flat, flat, words, targets, grad, lengths)

    flat64 = flat.double().cpu().requires_grad_()
    logits = plain(layout, flat64, words.cpu(), lengths.cpu() if ragged else None) @ layout.of(flat64, None, "head").t()
    if distil:
        on, p = ids.cpu() >= 0, torch.softmax(teacher.double().cpu() / 2.0, 1)
        logq = torch.gather(torch.log_softmax(logits / 2.0, 1), 1, ids.cpu().clamp(min=0))
        want = (p * (torch.log(p) - logq) * on).sum(1)
    else:
        want = torch.nn.functional.cross_entropy(logits, targets.cpu(), ignore_index=-100, reduction="none")
    (want.sum() / (B * T)).backward()
    assert float((loss.double().cpu() - want.detach()).norm()) <= 3.5e-4 * float(want.detach().norm())
    for i, name in layout.place:
        a, b = layout.of(grad, i, name).double().cpu(), layout.of(flat64.grad, i, name)
        assert float((a - b).norm()) <= 3.5e-4 * float(b.norm()), (i, name)


def test_decoding_word_by_word():
    """The logits behind every word: the same from one call and from the states, within the chain's roundings (as
    above, without the gradients: 12 * 48 * 2^-22 = 1.4e-4 of their norm)."""
    B, T, P = 2, 17, 9
    layout = E.Layout(2, 24, 70, states=5, taps=3, rank=4)
    flat = layout.init(DEV, 3)
    words = torch.randint(0, 70, (B, T), generator=torch.Generator(device=DEV).manual_seed(4), device=DEV)
    hidden = E.Model(layout, B, T, torch.float32, DEV).hidden(flat, flat, words)
    want = (hidden.double() @ layout.of(flat, None, "head").double().t()).view(B, T, -1)
    decoder = E.Decoder(layout, B, torch.float32, DEV)
    got = [decoder.step(flat, flat, words[:, :P], E.Model(layout, B, P, torch.float32, DEV, training=False))]
    got += [decoder.step(flat, flat, words[:, t:t + 1]) for t in range(P, T)]
    for t, g in enumerate(got):
        w = want[:, P - 1 + t]
        assert float((g.double() - w).norm()) <= 1.4e-4 * float(w.norm()), t


def test_training_runs():
    run = lambda n: E.train(layers=1, width=32, words=120, batch=4, length=24, learners=2, steps=n, picks=8,
                            log=lambda s: print(s, flush=True))
    losses, weights = run(6)
    assert all(x == x for x in losses) and torch.isfinite(weights).all()
    assert run(4)[0] == losses[:4]          # the same bits


class Step:
    """One pass through every operator on buffers of its own, whose inputs can change."""

    def __init__(self, seed):
        self.layout = E.Layout(1, 32, 3000, states=16)
        self.flat = self.layout.init(DEV, seed)
        self.work = self.flat.bfloat16()
        self.model = E.Model(self.layout, 3, 150, torch.bfloat16, DEV)
        self.words = torch.randint(0, 3000, (3, 150), device=DEV)
        self.targets = torch.randint(0, 3000, (450,), device=DEV)
        self.ids = torch.randint(0, 3000, (450, 5), device=DEV)
        self.teacher = torch.randn(450, 5, device=DEV)
        self.grads = [torch.zeros_like(self.flat) for _ in range(2)]

    def operators(self):
        """The calls of this library alone, from fixed activations (those of the last pass of run())."""
        m, L, k = self.model, self.layout, self.model.kept[0]
        Ei, N, R = L.inner, L.states, L.rank
        A.causal_conv(k["proj"][:, :, :Ei], L.of(self.flat, 0, "conv"), L.of(self.flat, 0, "conv_bias"), k["xc"])
        A.selective_scan(k["xc"], k["dt"], k["a"], k["low"][:, :, R:R + N], k["low"][:, :, R + N:], k["y"],
                         z=k["proj"][:, :, Ei:], states=k["states"], ws=m.scan_ws)
        g = lambda name: L.of(self.grads[0], 0, name)
        A.selective_scan_backward(k["y"], k["xc"], k["dt"], k["a"], k["low"][:, :, R:R + N], k["low"][:, :, R + N:],
                                  k["states"], m.dxc, m.ddt, g("rate"), m.dlow[:, :, R:R + N], m.dlow[:, :, R + N:],
                                  z=k["proj"][:, :, Ei:], dz=m.dproj[:, :, Ei:], ws=m.scan_ws)
        A.causal_conv_backward(m.dxc, k["proj"][:, :, :Ei], L.of(self.flat, 0, "conv"), L.of(self.flat, 0, "conv_bias"),
                               m.dproj[:, :, :Ei], g("conv"), g("conv_bias"), ws=m.conv_ws)
        hidden, head = m.last["norm"].view(-1, L.width), L.of(self.work, None, "head")
        A.linear_cross_entropy(hidden, head, self.targets, m.loss, m.lse, m.loss_ws)
        self.dloss = m.loss          # any numbers
        A.linear_cross_entropy_backward(hidden, head, self.targets, m.loss, m.lse, self.dloss,
                                        m.dnorm.view(hidden.shape), m.dhead, m.loss_ws)
        self.out = [k["xc"], k["y"], m.dxc, m.ddt, m.dlow[:, :, R:], m.dproj, g("rate"), g("conv"), g("conv_bias"), m.loss,
                    m.lse, m.dnorm, m.dhead]

    def run(self):
        self.model.cross_entropy(self.flat, self.work, self.words, self.targets, self.grads[0])
        self.model.distillation(self.flat, self.work, self.words, self.ids, self.teacher, self.grads[1])


def test_replays_of_a_captured_graph():
    """Captured once, replayed on new inputs with eager work and synchronisations between: each replay gives the
    eager call's bits."""
    s = Step(1)
    s.run()
    s.operators()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        s.operators()
    side.synchronize()
    with torch.cuda.graph(graph):
        s.operators()
    k = s.model.kept[0]
    for i in range(4):
        gen = torch.Generator(device=DEV).manual_seed(i)
        for t in (k["proj"], k["dt"], k["low"], s.model.last["norm"]):
            t.copy_(torch.randn(t.shape, generator=gen, device=DEV))
        s.targets.copy_(torch.randint(-5, 3000, (450,), generator=gen, device=DEV))
        s.operators()
        want = [t.clone() for t in s.out]
        for t in s.out:
            t.fill_(3.0)
        s.model.scan_ws.fill_(0xFF)
        s.model.loss_ws.fill_(0xFF)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, s.out)), i


def test_two_streams_at_once():
    """Two passes with buffers of their own on two streams, at once and one after the other: the same bits."""
    steps = [Step(5), Step(6)]
    for s in steps:
        s.run()
    want = [[g.clone() for g in s.grads] for s in steps]
    streams = [torch.cuda.Stream() for _ in steps]
    torch.cuda.synchronize()
    for _ in range(3):
        for s, stream in zip(steps, streams):
            with torch.cuda.stream(stream):
                for g in s.grads:
                    g.zero_()
                s.run()
        torch.cuda.synchronize()
        for s, w in zip(steps, want):
            for i, name in s.layout.place:
                assert all(torch.equal(s.layout.of(a, i, name), s.layout.of(b, i, name)) for a, b in zip(s.grads, w)), name
