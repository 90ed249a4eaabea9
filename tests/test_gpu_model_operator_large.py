"""The kernels of the convolution, the selective scan and the losses that only large calls take: long stretches of a
thread, stores past the cache, chunks of many steps, sequences of one chunk, and 256 x 256 tiles over many steps of
the inner axis.  Each case asserts the rule on sizes that chooses the kernel it is for."""
import pytest
import torch

import adaptive_residual_gradient_amd as A
import model_refs as M
import test_gpu_causal_conv as conv
import test_gpu_selective_scan as scan
import test_gpu_vocabulary_loss as losses

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


# ---- causal convolution ----

def steps_of_a_thread(B, T, C, size):
    """The first of 32, 12 and 4 that leaves 131072 threads of 8 bytes of channels."""
    lanes = -(-C // (8 // size))
    return next((r for r in (32, 12) if B * lanes * -(-T // r) >= 131072), 4)


def conv_check(c, steps, past, lengths=None):
    B, T, C = c.x.shape
    size = c.x.element_size()
    assert steps_of_a_thread(B, T, C, size) == steps and (B * T * C * size > 96 << 20) == past
    c.forward()
    c.backward()
    # some channels, the first and last among them, against 64 bits; a filter's channels do not meet
    n = None if c.lengths is None else c.lengths.cpu()
    for at in (slice(0, 5), slice(C // 2 - 3, C // 2 + 4), slice(C - 6, C)):
        part = lambda t: M.f64(t[..., at])
        want = M.conv(part(c.x), M.f64(c.w[at]), M.f64(c.bias[at]), part(c.state), n, c.silu, part(c.dy))
        for got, what in ((c.y[..., at], "y"), (c.state_out[..., at], "state_out"), (c.dx[..., at], "dx"),
                          (c.dw[at], "dweight"), (c.db[at], "dbias"), (c.dstate[..., at], "dstate")):
            M.assert_within(got, want[what], what)
    # and all of them against calls on parts, in 4 steps a thread: the same bits but for the sums
    wide = 96
    assert steps_of_a_thread(B, T, wide, size) == 4
    ws = A.causal_conv_workspace(B, T, wide, c.K, DEV)
    for at in (slice(k, min(k + wide, C)) for k in range(0, C, wide)):
        small = lambda t: t[..., at].contiguous()
        y, dx, w, bias, state = torch.empty_like(small(c.y)), torch.empty_like(small(c.dx)), c.w[at].contiguous(), \
            c.bias[at].contiguous(), small(c.state)
        out, dstate, dw, db = torch.empty_like(state), torch.empty_like(state), torch.empty_like(w), torch.empty_like(bias)
        A.causal_conv(c.x[..., at], w, bias, y, state, out, c.lengths, silu=c.silu)
        A.causal_conv_backward(c.dy[..., at], c.x[..., at], w, bias, dx, dw, db, state, dstate, c.lengths, silu=c.silu, ws=ws)
        for a, b, what in ((y, c.y, "y"), (out, c.state_out, "state_out"), (dx, c.dx, "dx"), (dstate, c.dstate, "dstate")):
            assert torch.equal(a, small(b)), (what, at)


@pytest.mark.parametrize("dtype,B,T,C,K,steps,past", [
    ("bf16", 8, 1000, 2048, 4, 32, False), ("f16", 9, 1111, 2050, 7, 32, False), ("bf16", 70, 130, 2048, 2, 32, False),
    ("f32", 8, 513, 2047, 3, 32, False),
    ("bf16", 4, 1000, 2048, 4, 12, False), ("f16", 5, 770, 2051, 8, 12, False), ("f32", 3, 600, 1999, 1, 12, False),
    ("bf16", 8, 3100, 2048, 4, 32, True), ("f16", 9, 3000, 2045, 5, 32, True), ("f32", 13, 2003, 1001, 3, 32, True)])
@pytest.mark.parametrize("ragged", [False, True])
def test_convolution(dtype, B, T, C, K, steps, past, ragged):
    lengths = [(0, T, T - 1, 1, 33, T // 2, 31, T + 7, T - 40, 64, 2, 65, 12)[b % 13] for b in range(B)] if ragged else None
    conv_check(conv.Case(B, T, C, K, TYPES[dtype], silu=K != 8, lengths=lengths, seed=T), steps, past)


# ---- selective scan ----

def chunks_of(B, T, C, N):
    """(chunks, steps of one): for 4096 wavefronts of 64 channels and up to 16 states, of 32 steps or more; where these
    leave less than half, for 2048, of 16; where these leave less than half, for 1024, of 8."""
    nb = 8 if N <= 8 else 16
    padded = -(-N // nb) * nb
    waves, chunks = B * -(-C // 64) * (padded // nb), 1
    for least in (32, 16, 8):
        want = 128 * least
        chunks = max(min(-(-want // waves), -(-T // least)), chunks)
        if chunks * waves >= want // 2:
            break
    steps = -(-(-(-T // chunks)) // 8) * 8
    chunks = -(-T // steps)
    # the rule as the library has it: its workspace is b and c in rows and, of several chunks, their ends, sums and s
    up = lambda floats: (4 * floats + 255) // 256 * 256
    bytes_ = up(B * T * 2 * padded)
    if chunks > 1:
        bytes_ += up(B * chunks * padded * C) + up(B * chunks * C) + up(B * T * C)
    assert A.selective_scan_workspace(B, T, C, N, device="cpu").numel() == bytes_
    return chunks, steps


@pytest.mark.parametrize("dtype,B,T,C,N,chunks,steps", [
    # sequences of one chunk: blocks of 8 states, 16, two of 16 and four
    ("f32", 4096, 21, 3, 8, 1, 24), ("bf16", 4100, 40, 2, 5, 1, 40), ("f32", 4096, 27, 3, 16, 1, 32),
    ("f16", 2100, 19, 65, 9, 1, 24), ("bf16", 2048, 33, 3, 24, 1, 40), ("f32", 1024, 26, 5, 64, 1, 32),
    ("f16", 1400, 17, 4, 48, 1, 24),
    # chunks of many steps
    ("f32", 1024, 200, 5, 16, 4, 56), ("bf16", 1500, 130, 3, 16, 3, 48), ("f16", 1024, 150, 5, 7, 4, 40),
    ("f32", 512, 170, 6, 32, 4, 48), ("bf16", 300, 190, 6, 64, 4, 48), ("f16", 700, 100, 70, 12, 3, 40),
    ("f32", 180, 110, 130, 40, 3, 40)])
@pytest.mark.parametrize("ragged", [False, True])
def test_scan(dtype, B, T, C, N, chunks, steps, ragged):
    assert chunks_of(B, T, C, N) == (chunks, steps)
    ends = (0, T, T - 1, 1, 8, 9, steps - 1, steps, steps + 1, steps + 8, T // 2, T + 5, T - 8, 15, -1)
    lengths = [ends[b % len(ends)] for b in range(B)] if ragged else None
    scan.Case(B, T, C, N, TYPES[dtype], gated=not ragged or N % 2 == 0, lengths=lengths, seed=T + N).check()


# ---- losses over a vocabulary ----

def tiles(m, n):
    """256 x 256 tiles of a product; it takes them from 192 on, if neither side is 64 or less."""
    return -(-m // 256) * -(-n // 256)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("R,H,V,picks", [(512, 200, 24576, 0), (700, 328, 16640, 0), (515, 136, 16500, 6)])
def test_logits_of_large_tiles(R, H, V, picks, dtype):
    """Several steps of 64 of the width, in the loss and in dz.  The loss of float32 takes 16384 words at a time, which
    are enough from 513 rows on."""
    assert tiles(V, R) >= 192 and H > 128 and (R <= 512 or tiles(16384, R) >= 192)
    losses.Case(R, H, V, TYPES[dtype], picks=picks, seed=R).check()


@pytest.mark.parametrize("dtype", TYPES)
def test_weight_gradients_of_large_tiles(dtype):
    """Several steps of 64 of the rows: 11."""
    R, H, V = 700, 16, 50000
    assert tiles(V, H) >= 192
    losses.Case(R, H, V, TYPES[dtype], seed=1).check()


@pytest.mark.parametrize("dtype", TYPES)
def test_hidden_gradients_of_large_tiles(dtype):
    """Four shares of the words, of 5 steps of 64."""
    R, H, V = 6000, 520, 1100
    assert 64 <= tiles(H, R) < 192 <= 4 * tiles(H, R)
    losses.Case(R, H, V, TYPES[dtype], seed=2).check()
