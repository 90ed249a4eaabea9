"""Data-parallel training of gated recurrent layers with compressed gradients.

One layer is  y = x + scan(gate, input) @ out^T,  gate and input the halves of
layer_norm(x) @ in^T, the scan a gated linear recurrence along the sequence.
Each learner computes its gradient on its own batch and compresses it into a
message; the messages are decoded into one flat gradient, which the clipped
AdamW step applies with its moments in 8 bits:

    layer_norm, gated_scan                        forward
    gated_scan_backward, layer_norm_backward      backward
    compress, decode_accumulate                   the exchange
    grad_norm, adamw_packed                       the step

The learners take turns on one GPU.  They learn the outputs of a fixed model
of the same form on random sequences.

    python examples/train_gated_layers.py --steps 60
"""
import argparse
import pathlib
import sys

import torch

sys.path.insert(0, str(pathlib.Path(__file__).resolve().parent.parent))
import adaptive_residual_gradient_amd as A  # noqa: E402

EPS = 1e-5


class Layout:
    """The layers' parameters in flat buffers, offsets multiples of 4 elements."""

    def __init__(self, layers, width):
        self.layers, self.width = layers, width
        self.place, self.tensors, self.segments, at = {}, [], [], 0
        for i in range(layers):
            # matrices are decayed and travel in bins of 500, vectors are not and take short bins
            for name, shape, decay, bin_length in (("in", (2 * width, width), 0.01, 500),
                                                   ("out", (width, width), 0.01, 500),
                                                   ("weight", (width,), 0.0, 50), ("bias", (width,), 0.0, 50)):
                n = torch.Size(shape).numel()
                self.place[i, name] = (at, shape)
                self.tensors.append((at, n, decay, 1.0))
                self.segments.append((at, n, bin_length))
                at += (n + 3) // 4 * 4
        self.span = at

    def of(self, flat, i, name):
        """Parameter `name` of layer i as a view of a flat buffer."""
        at, shape = self.place[i, name]
        return flat[at:at + torch.Size(shape).numel()].view(shape)

    def init(self, device, seed):
        gen = torch.Generator(device=device).manual_seed(seed)
        flat = torch.zeros(self.span, device=device)
        for i in range(self.layers):
            for name in ("in", "out"):
                w = self.of(flat, i, name)
                w.copy_(torch.randn(w.shape, generator=gen, device=device) * self.width ** -0.5)
            self.of(flat, i, "weight").fill_(1.0)
        return flat


class Model:
    """Forward and backward of the layers on [batch, length, width] activations of one type.  Keeps the
    buffers of one shape for its calls."""

    def __init__(self, layout, batch, length, dtype, device):
        self.layout, self.dtype = layout, dtype
        D, rows = layout.width, batch * length
        new = lambda *shape, t=dtype: torch.empty(shape, dtype=t, device=device)
        f32 = torch.float32
        self.kept = [dict(norm=new(batch, length, D), mean=new(rows, t=f32), rstd=new(rows, t=f32),
                          h=new(batch, length, D)) for _ in range(layout.layers)]
        self.dproj = new(batch, length, 2 * D)
        self.dnorm_x = new(batch, length, D)
        self.scan_ws = A.gated_scan_workspace(batch, length, D, device)
        self.norm_ws = A.layer_norm_workspace(rows, D, device)

    def forward(self, params, work, x, lengths=None):
        """params: the flat float32 parameters (layer norm's); work: their copy in the model's type."""
        L, D = self.layout, self.layout.width
        for i, k in enumerate(self.kept):
            k["x"] = x
            A.layer_norm(x, L.of(params, i, "weight"), L.of(params, i, "bias"), k["norm"], k["mean"], k["rstd"], eps=EPS)
            k["proj"] = k["norm"].view(-1, D).mm(L.of(work, i, "in").t()).view(*x.shape[:2], 2 * D)
            A.gated_scan(k["proj"][:, :, :D], k["proj"][:, :, D:], k["h"], lengths=lengths, ws=self.scan_ws)
            x = torch.addmm(x.reshape(-1, D), k["h"].view(-1, D), L.of(work, i, "out").t()).view(x.shape)
        return x

    def backward(self, params, work, dy, grad, lengths=None):
        """Gradients of every parameter into the flat float32 buffer `grad`; returns the input's."""
        L, D = self.layout, self.layout.width
        for i in reversed(range(L.layers)):
            k = self.kept[i]
            flat = dy.view(-1, D)
            L.of(grad, i, "out").copy_(flat.t().mm(k["h"].view(-1, D)))
            dh = flat.mm(L.of(work, i, "out")).view(dy.shape)
            A.gated_scan_backward(k["proj"][:, :, :D], k["proj"][:, :, D:], k["h"], dh, self.dproj[:, :, :D],
                                  self.dproj[:, :, D:], lengths=lengths, ws=self.scan_ws)
            flat = self.dproj.view(-1, 2 * D)
            L.of(grad, i, "in").copy_(flat.t().mm(k["norm"].view(-1, D)))
            dnorm = flat.mm(L.of(work, i, "in")).view(dy.shape)
            A.layer_norm_backward(dnorm, k["x"], L.of(params, i, "weight"), k["mean"], k["rstd"], self.dnorm_x,
                                  L.of(grad, i, "weight"), L.of(grad, i, "bias"), self.norm_ws)
            dy = dy + self.dnorm_x
        return dy


def train(layers=2, width=256, batch=8, length=128, learners=4, steps=60, lr=8e-3, seed=0, device="cuda", log=print):
    """Returns the loss of every step."""
    layout = Layout(layers, width)
    model = Model(layout, batch, length, torch.bfloat16, device)
    teacher = layout.init(device, seed + 1)
    teacher_work = teacher.bfloat16()
    weights = layout.init(device, seed)
    work = weights.bfloat16()

    opt = A.Optimizer(layout.tensors)
    m, v = (torch.zeros(layout.span, dtype=torch.float8_e4m3fn, device=device) for _ in range(2))
    scales, clip, norm_ws = opt.moment_scales(device), torch.zeros(2, device=device), opt.norm_workspace(device)

    plan = A.Plan(layout.segments)
    grad, total = (torch.zeros(int(plan.info.span) + 4, device=device) for _ in range(2))
    residues = [torch.zeros_like(grad) for _ in range(learners)]
    messages = [plan.message_buffer(device) for _ in range(learners)]
    compress_ws, decode_ws = plan.compress_workspace(device), plan.decode_workspace(learners, device)

    gen = torch.Generator(device=device).manual_seed(seed + 2)
    losses = []
    for step in range(1, steps + 1):
        loss = 0.0
        for residue, message in zip(residues, messages):
            x = torch.randn(batch, length, width, generator=gen, device=device).bfloat16()
            target = model.forward(teacher, teacher_work, x)
            error = (model.forward(weights, work, x) - target).float()
            loss = loss + error.square().mean() / learners
            model.backward(weights, work, (error * (2.0 / error.numel())).bfloat16(), grad)
            A.compress(plan, residue, grad, message, compress_ws)
        A.decode_accumulate(plan, messages, total, False, decode_ws)
        A.grad_norm(opt, total, clip, norm_ws, max_norm=1.0, scale=1.0 / learners)
        A.adamw_packed(opt, weights, total, m, v, scales, lr=lr, step=step, scale=1.0 / learners, seed=seed, clip=clip,
                       weights_bf16=work)
        losses.append(float(loss))
        if step == 1 or step % 10 == 0:
            log(f"step {step}: loss {losses[-1]:.5f}, gradient norm {float(clip[0]):.4f}")
    return losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--layers", type=int, default=2)
    ap.add_argument("--width", type=int, default=256)
    ap.add_argument("--batch", type=int, default=8)
    ap.add_argument("--length", type=int, default=128)
    ap.add_argument("--learners", type=int, default=4)
    ap.add_argument("--lr", type=float, default=8e-3)
    train(**vars(ap.parse_args()))
