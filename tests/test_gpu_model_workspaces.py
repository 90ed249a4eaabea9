"""Workspaces and kept states at any 16 bytes, of the exact size, with other calls' bytes in them and around them."""
import pytest
import torch

import test_gpu_causal_conv as conv
import test_gpu_selective_scan as scan
import test_gpu_vocabulary_loss as losses

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


class Shifted:
    """A buffer of t's size `shift` bytes into a larger one, whose other bytes stay as they are."""

    def __init__(self, t, shift):
        n = t.numel() * t.element_size()
        self.room = torch.full((n + 512,), 0x5A, dtype=torch.uint8, device=DEV)
        assert self.room.data_ptr() % 256 == 0
        self.t = self.room[shift:shift + n].view(t.dtype)
        self.ends = (slice(0, shift), slice(shift + n, None))

    def check(self):
        assert all((self.room[s] == 0x5A).all() for s in self.ends)


@pytest.mark.parametrize("shift", [16, 48, 80, 240])
@pytest.mark.parametrize("dtype", TYPES)
def test_any_16_bytes(dtype, shift):
    t = TYPES[dtype]
    c = conv.Case(5, 70, 37, 4, t)
    ws = Shifted(c.ws, shift)
    c.ws = ws.t
    c.check()
    ws.check()
    for B, T, C, N in ((2, 100, 70, 16), (2, 40, 33, 24), (3, 20, 65, 5)):
        s = scan.Case(B, T, C, N, t)
        ws, kept = Shifted(s.ws, shift), Shifted(s.kept, shift)
        s.ws, s.kept = ws.t, kept.t
        s.check()
        ws.check()
        kept.check()
    for R, H, V, picks in ((100, 40, 700, 0), (70, 72, 300, 5), (600, 64, 1000, 0)):
        k = losses.Case(R, H, V, t, picks=picks)
        ws = Shifted(k.ws, shift)
        k.ws = ws.t
        k.check()
        ws.check()
