"""Captured graphs of the distillation and of decoding steps: every replay, on new inputs and with eager work between,
gives the eager calls' bits."""
import pytest
import torch

import adaptive_residual_gradient_amd as A
import test_gpu_vocabulary_loss as losses

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def captured(calls):
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        calls()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    return graph


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("R,H,V,picks", [(50, 40, 300, 5), (700, 64, 5000, 70)])
def test_distillation(R, H, V, picks, dtype):
    c = losses.Case(R, H, V, TYPES[dtype], picks=picks, ignored=0.0, temperature=2.0)

    def calls():
        c.forward()
        c.backward()
    graph = captured(calls)
    gen = torch.Generator(device=DEV).manual_seed(0)
    out = (c.loss, c.lse, c.picked, c.dh, c.dw)
    for i in range(4):
        c.hidden.copy_(torch.randn(R, H, generator=gen, device=DEV))
        c.ids.copy_(torch.randint(-40, V, (R, picks), generator=gen, device=DEV))
        c.teacher.copy_(torch.randn(R, picks, generator=gen, device=DEV))
        c.teacher[i::7] = float("-inf")
        c.ids[i::5] = -1
        c.dloss.copy_(torch.randn(R, generator=gen, device=DEV))
        calls()
        want = [t.clone() for t in out]
        assert all(torch.isfinite(t).all() for t in want)
        for t in (*out, c.ws):
            t.fill_(3)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, out)), i


@pytest.mark.parametrize("dtype", TYPES)
def test_decoding(dtype):
    """A graph of two words' steps, whose states go from one pair of buffers to the other and back, replayed word pair by
    word pair: the bits of one eager call after the other."""
    B, C, N, K, words = 5, 70, 16, 4, 8
    gen = torch.Generator(device=DEV).manual_seed(3)
    normal = lambda *s: torch.randn(*s, generator=gen, device=DEV)
    t = TYPES[dtype]
    w, a, bias = normal(C, K), -torch.rand(C, N, generator=gen, device=DEV) - 0.1, normal(C)
    seq = [normal(words, B, 1, n).to(t) for n in (C, C, C, N, N)]
    now = [torch.empty_like(s[:2]) for s in seq]
    y = torch.empty(2, B, 1, C, dtype=t, device=DEV)
    mixed = torch.empty(B, 1, C, dtype=t, device=DEV)
    window = [torch.zeros(B, K - 1, C, dtype=t, device=DEV) for _ in range(2)]
    h = [torch.zeros(B, C, N, device=DEV) for _ in range(2)]
    ws = A.selective_scan_workspace(B, 1, C, N)

    def step(i, x, z, dt, b, c, out):
        A.causal_conv(x, w, bias, mixed, window[i % 2], window[(i + 1) % 2])
        A.selective_scan(mixed, dt, a, b, c, out, z=z, dt_bias=bias, h0=h[i % 2], h_last=h[(i + 1) % 2], ws=ws)

    def pair():
        for i in range(2):
            step(i, *(s[i] for s in now), y[i])
    graph = captured(pair)

    def clear():
        for s in (*window, *h):
            s.zero_()
    clear()
    want = torch.empty(words, B, 1, C, dtype=t, device=DEV)
    for i in range(words):
        step(i, *(s[i] for s in seq), want[i])
    ends = [s.clone() for s in (window[0], h[0])]
    clear()
    for i in range(0, words, 2):
        for s, v in zip(now, seq):
            s.copy_(v[i:i + 2])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want[i:i + 2]), i
    assert all(torch.equal(p, q) for p, q in zip(ends, (window[0], h[0])))
