"""Data-parallel training of a small state space language model with compressed
gradients, and decoding from it token by token.

One layer is  h + scan(conv(x), dt, b, c, gate z) @ out^T  with x and z the halves
of layer_norm(h) @ in^T, and dt, b and c projections of the convolution's
result.  A student learns from a fixed model of the same form: the cross
entropy of words drawn from it, and the distillation from its top logits.  Each
learner computes its gradient on its own batch and compresses it into a
message; the messages are decoded into one flat gradient, which the clipped
AdamW step applies with its moments in 8 bits:

    layer_norm, causal_conv, selective_scan                 forward
    linear_cross_entropy, linear_distillation               the losses, without the logits
    their gradients, back to the embedding                  backward
    compress, decode_accumulate                             the exchange
    grad_norm, adamw_packed                                 the step
    causal_conv, selective_scan with their states           decoding

    python examples/train_state_space.py --steps 40
"""
import argparse
import pathlib
import sys

import torch

sys.path.insert(0, str(pathlib.Path(__file__).resolve().parent.parent))
import adaptive_residual_gradient_amd as A  # noqa: E402

EPS = 1e-5


class Layout:
    """The parameters in flat buffers, offsets multiples of 4 elements."""

    def __init__(self, layers, width, words, states=16, taps=4, rank=8):
        self.layers, self.width, self.words, self.states, self.taps, self.rank = layers, width, words, states, taps, rank
        self.inner = E = 2 * width
        D, N = width, states
        self.place, self.tensors, self.segments, at = {}, [], [], 0
        shapes = [(None, "embed", (words, D), 0.0)]
        for i in range(layers):
            shapes += [(i, "weight", (D,), 0.0), (i, "bias", (D,), 0.0), (i, "in", (2 * E, D), 0.01),
                       (i, "conv", (E, taps), 0.0), (i, "conv_bias", (E,), 0.0), (i, "low", (rank + 2 * N, E), 0.01),
                       (i, "dt", (E, rank), 0.01), (i, "dt_bias", (E,), 0.0), (i, "rate", (E, N), 0.0), (i, "d", (E,), 0.0),
                       (i, "out", (D, E), 0.01)]
        shapes += [(None, "weight", (D,), 0.0), (None, "bias", (D,), 0.0), (None, "head", (words, D), 0.01)]
        for i, name, shape, decay in shapes:
            n = torch.Size(shape).numel()
            self.place[i, name] = (at, shape)
            self.tensors.append((at, n, decay, 1.0))
            self.segments.append((at, n, 500 if len(shape) == 2 else 50))
            at += (n + 7) // 8 * 8          # 16-byte aligned in every type
        self.span = at

    def of(self, flat, i, name):
        """Parameter `name` of layer i (None: the model's own) as a view of a flat buffer."""
        at, shape = self.place[i, name]
        return flat[at:at + torch.Size(shape).numel()].view(shape)

    def init(self, device, seed, sharp=1.0):
        """sharp: spread of the head's logits."""
        gen = torch.Generator(device=device).manual_seed(seed)
        normal = lambda w: torch.randn(w.shape, generator=gen, device=device)
        flat = torch.zeros(self.span, device=device)
        self.of(flat, None, "embed").copy_(normal(self.of(flat, None, "embed")))
        self.of(flat, None, "head").copy_(normal(self.of(flat, None, "head")) * sharp * self.width ** -0.5)
        self.of(flat, None, "weight").fill_(1.0)
        for i in range(self.layers):
            for name in ("in", "conv", "low", "dt", "out"):
                w = self.of(flat, i, name)
                w.copy_(normal(w) * w.shape[1] ** -0.5)
            self.of(flat, i, "weight").fill_(1.0)
            self.of(flat, i, "d").fill_(1.0)
            self.of(flat, i, "dt_bias").uniform_(-5.0, -2.0, generator=gen)      # steps of about 0.01 to 0.1
            rate = self.of(flat, i, "rate")
            rate.copy_(torch.log(torch.arange(1, self.states + 1, device=device)).expand(rate.shape))
        return flat


class Model:
    """Forward and backward on [batch, length] words, activations of one type.  Keeps the buffers of one shape for
    its calls.  params: the flat float32 parameters; work: their copy in the model's type."""

    def __init__(self, layout, batch, length, dtype, device, training=True):
        L, D, E, N = layout, layout.width, layout.inner, layout.states
        self.layout, self.dtype, self.rows = layout, dtype, batch * length
        new = lambda *shape, t=dtype: torch.empty(shape, dtype=t, device=device)
        f32, B, T = torch.float32, batch, length
        norm = lambda: dict(norm=new(B, T, D), mean=new(B * T, t=f32), rstd=new(B * T, t=f32))
        self.kept = [dict(norm(), xc=new(B, T, E), y=new(B, T, E), dt=new(B, T, E),
                          states=A.selective_scan_states(B, T, E, N, device) if training else None)
                     for _ in range(layout.layers)]
        self.last = norm()
        self.scan_ws = A.selective_scan_workspace(B, T, E, N, training, device)
        self.loss, self.lse = new(B * T, t=f32), new(B * T, t=f32)
        self.loss_ws = A.linear_loss_workspace(B * T, D, L.words, dtype, backward=training, device=device)
        if training:
            self.dproj, self.dlow = new(B, T, 2 * E), new(B, T, L.rank + 2 * N)
            self.dxc, self.ddt, self.dnorm, self.dhead = new(B, T, E), new(B, T, E), new(B, T, D), new(L.words, D)
            self.conv_ws = A.causal_conv_workspace(B, T, E, L.taps, device)
            self.norm_ws = A.layer_norm_workspace(B * T, D, device)

    def _norm(self, params, i, x, k):
        L = self.layout
        A.layer_norm(x, L.of(params, i, "weight"), L.of(params, i, "bias"), k["norm"], k["mean"], k["rstd"], eps=EPS)
        return k["norm"].view(-1, L.width)

    def hidden(self, params, work, words, lengths=None, states=None, new_states=None):
        """The last layer's normed states.  states: (convolution's, scan's) of each layer before the first word;
        new_states take those behind the last."""
        L, E, N = self.layout, self.layout.inner, self.layout.states
        h = L.of(work, None, "embed")[words]
        self.words, self.lengths, self.states = words, lengths, states
        for i, k in enumerate(self.kept):
            k["h"] = h
            k["proj"] = self._norm(params, i, h, k).mm(L.of(work, i, "in").t()).view(*words.shape, 2 * E)
            before, after = (s[i] if s is not None else (None, None) for s in (states, new_states))
            A.causal_conv(k["proj"][:, :, :E], L.of(params, i, "conv"), L.of(params, i, "conv_bias"), k["xc"], before[0],
                          after[0], lengths)
            k["low"] = k["xc"].view(-1, E).mm(L.of(work, i, "low").t()).view(*words.shape, -1)
            torch.mm(k["low"].view(-1, L.rank + 2 * N)[:, :L.rank], L.of(work, i, "dt").t(), out=k["dt"].view(-1, E))
            k["a"] = -torch.exp(L.of(params, i, "rate"))
            A.selective_scan(k["xc"], k["dt"], k["a"], k["low"][:, :, L.rank:L.rank + N], k["low"][:, :, L.rank + N:], k["y"],
                             d=L.of(params, i, "d"), z=k["proj"][:, :, E:], dt_bias=L.of(params, i, "dt_bias"), h0=before[1],
                             h_last=after[1], states=k["states"], lengths=lengths, ws=self.scan_ws)
            h = torch.addmm(h.reshape(-1, L.width), k["y"].view(-1, E), L.of(work, i, "out").t()).view(h.shape)
        self.last["h"] = h
        return self._norm(params, None, h, self.last)

    def cross_entropy(self, params, work, words, targets, grad, lengths=None):
        """Losses [rows]; the mean's gradient into the flat float32 buffer `grad`.  Targets below 0 do not count."""
        hidden, head = self.hidden(params, work, words, lengths), self.layout.of(work, None, "head")
        A.linear_cross_entropy(hidden, head, targets, self.loss, self.lse, self.loss_ws)
        dloss = torch.full_like(self.loss, 1.0 / self.rows)
        A.linear_cross_entropy_backward(hidden, head, targets, self.loss, self.lse, dloss, self.dnorm.view(hidden.shape),
                                        self.dhead, self.loss_ws)
        self._backward(params, work, grad)
        return self.loss

    def distillation(self, params, work, words, ids, teacher, grad, temperature=1.0, lengths=None):
        """The same for the distillation from a teacher's top logits [rows, picks]."""
        hidden, head = self.hidden(params, work, words, lengths), self.layout.of(work, None, "head")
        picked, dloss = torch.empty_like(teacher), torch.full_like(self.loss, 1.0 / self.rows)
        A.linear_distillation(hidden, head, ids, teacher, self.loss, self.lse, picked, self.loss_ws, temperature=temperature)
        A.linear_distillation_backward(hidden, head, ids, teacher, self.lse, picked, dloss, self.dnorm.view(hidden.shape),
                                       self.dhead, self.loss_ws, temperature=temperature)
        self._backward(params, work, grad)
        return self.loss

    def _norm_back(self, params, grad, i, k):
        L = self.layout
        dh = torch.empty_like(self.dnorm)
        A.layer_norm_backward(self.dnorm, k["h"], L.of(params, i, "weight"), k["mean"], k["rstd"], dh, L.of(grad, i, "weight"),
                              L.of(grad, i, "bias"), self.norm_ws)
        return dh

    def _backward(self, params, work, grad):
        """From dnorm, the gradient of what `hidden` returned, and dhead."""
        L, E, N, R = self.layout, self.layout.inner, self.layout.states, self.layout.rank
        L.of(grad, None, "head").copy_(self.dhead)
        dh = self._norm_back(params, grad, None, self.last)
        for i in reversed(range(L.layers)):
            k, g = self.kept[i], lambda name: L.of(grad, i, name)
            flat = dh.view(-1, L.width)
            g("out").copy_(flat.t().mm(k["y"].view(-1, E)))
            dy = flat.mm(L.of(work, i, "out")).view(k["y"].shape)
            low, dlow = k["low"], self.dlow
            A.selective_scan_backward(dy, k["xc"], k["dt"], k["a"], low[:, :, R:R + N], low[:, :, R + N:], k["states"], self.dxc,
                                      self.ddt, g("rate"), dlow[:, :, R:R + N], dlow[:, :, R + N:], d=L.of(params, i, "d"),
                                      z=k["proj"][:, :, E:], dt_bias=L.of(params, i, "dt_bias"), dz=self.dproj[:, :, E:],
                                      dd=g("d"), ddt_bias=g("dt_bias"), lengths=self.lengths, ws=self.scan_ws)
            g("rate").mul_(k["a"])          # the rates are -exp of the parameters
            ddt, flow, fdlow = self.ddt.view(-1, E), low.view(-1, R + 2 * N), dlow.view(-1, R + 2 * N)
            g("dt").copy_(ddt.t().mm(flow[:, :R]))
            fdlow[:, :R] = ddt.mm(L.of(work, i, "dt"))
            g("low").copy_(fdlow.t().mm(k["xc"].view(-1, E)))
            dxc = self.dxc.view(-1, E).addmm_(fdlow, L.of(work, i, "low")).view(k["xc"].shape)
            A.causal_conv_backward(dxc, k["proj"][:, :, :E], L.of(params, i, "conv"), L.of(params, i, "conv_bias"),
                                   self.dproj[:, :, :E], g("conv"), g("conv_bias"), lengths=self.lengths, ws=self.conv_ws)
            flat = self.dproj.view(-1, 2 * E)
            g("in").copy_(flat.t().mm(k["norm"].view(-1, L.width)))
            torch.mm(flat, L.of(work, i, "in"), out=self.dnorm.view(-1, L.width))
            dh = dh + self._norm_back(params, grad, i, k)
        # equal words' gradients in a fixed order
        L.of(grad, None, "embed").zero_().index_put_((self.words.reshape(-1),), dh.view(-1, L.width).float(), accumulate=True)


class Decoder:
    """Words one by one from the states of the layers."""

    def __init__(self, layout, batch, dtype, device):
        self.layout, self.one = layout, Model(layout, batch, 1, dtype, device, training=False)
        L, E = layout, layout.inner
        fresh = lambda: [(torch.zeros(batch, L.taps - 1, E, dtype=dtype, device=device),
                          torch.zeros(batch, E, L.states, device=device)) for _ in range(L.layers)]
        self.states, self.spare = fresh(), fresh()

    def step(self, params, work, words, model=None):
        """Logits behind words [batch, length]; model: one of that shape, for prompts."""
        out = (model or self.one).hidden(params, work, words, states=self.states, new_states=self.spare)
        self.states, self.spare = self.spare, self.states
        last = out.view(*words.shape, -1)[:, -1]
        return last.float().mm(self.layout.of(work, None, "head").float().t())

    def generate(self, params, work, prompt, count):
        """The `count` most likely words behind a prompt [batch, length]."""
        model = Model(self.layout, *prompt.shape, self.one.dtype, prompt.device, training=False)
        words, out = prompt, []
        for i in range(count):
            words = self.step(params, work, words, model if i == 0 else None).argmax(1, keepdim=True)
            out.append(words)
        return torch.cat(out, 1)


def train(layers=2, width=64, words=500, batch=8, length=64, learners=2, steps=40, picks=16, lr=5e-3, seed=0, device="cuda",
          log=print):
    """Returns the loss of every step (cross entropy and distillation in turn) and the trained flat parameters."""
    layout = Layout(layers, width, words)
    teacher = layout.init(device, seed + 1, sharp=3.0)
    teacher_work = teacher.bfloat16()
    reader = Model(layout, batch, length, torch.bfloat16, device, training=False)
    model = Model(layout, batch, length, torch.bfloat16, device)
    weights = layout.init(device, seed)
    work = weights.bfloat16()

    opt = A.Optimizer(layout.tensors)
    m, v = (torch.zeros(layout.span, dtype=torch.float8_e4m3fn, device=device) for _ in range(2))
    scales, clip, norm_ws = opt.moment_scales(device), torch.zeros(2, device=device), opt.norm_workspace(device)
    plan = A.Plan(layout.segments)
    grad, total = (torch.zeros(int(plan.info.span) + 8, device=device) for _ in range(2))
    residues = [torch.zeros_like(grad) for _ in range(learners)]
    messages = [plan.message_buffer(device) for _ in range(learners)]
    compress_ws, decode_ws = plan.compress_workspace(device), plan.decode_workspace(learners, device)

    gen = torch.Generator(device=device).manual_seed(seed + 2)
    losses = []
    for step in range(1, steps + 1):
        loss = 0.0
        for residue, message in zip(residues, messages):
            x = torch.randint(0, words, (batch, length), generator=gen, device=device)
            logits = reader.hidden(teacher, teacher_work, x).float().mm(layout.of(teacher_work, None, "head").float().t())
            if step % 2:
                drawn = torch.multinomial(torch.softmax(logits, 1), 1, generator=gen)[:, 0]
                loss = loss + model.cross_entropy(weights, work, x, drawn, grad).mean() / learners
            else:
                best = logits.topk(picks, 1)
                loss = loss + model.distillation(weights, work, x, best.indices, best.values, grad).mean() / learners
            A.compress(plan, residue, grad, message, compress_ws)
        A.decode_accumulate(plan, messages, total, False, decode_ws)
        A.grad_norm(opt, total, clip, norm_ws, max_norm=1.0, scale=1.0 / learners)
        A.adamw_packed(opt, weights, total, m, v, scales, lr=lr, step=step, scale=1.0 / learners, seed=seed, clip=clip,
                       weights_bf16=work)
        losses.append(float(loss))
        if step <= 2 or step % 10 < 2:
            log(f"step {step}: {'cross entropy' if step % 2 else 'distillation'} {losses[-1]:.4f}, "
                f"gradient norm {float(clip[0]):.4f}")
    prompt = torch.randint(0, words, (2, 8), generator=gen, device=device)
    log("words behind two prompts: " + str(Decoder(layout, 2, torch.bfloat16, device).generate(weights, work, prompt, 8).tolist()))
    return losses, weights


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, default in (("steps", 40), ("layers", 2), ("width", 64), ("words", 500), ("batch", 8), ("length", 64),
                          ("learners", 2), ("picks", 16)):
        ap.add_argument("--" + name, type=int, default=default)
    ap.add_argument("--lr", type=float, default=5e-3)
    train(**vars(ap.parse_args()))
