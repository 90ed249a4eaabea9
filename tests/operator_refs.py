"""Plain 64-bit forms of the training-step operators, on the CPU, and the error
bounds that the float32 kernels have to meet.

u = 2^-24 is float32's half step.  A bound counts the roundings of a result:
each adds at most u of the value rounded (half a step of the output type for
the last one), carried through the formula's derivative.
"""
import numpy as np
import torch

U = 2.0 ** -24
BLOCK = 32
HALF_STEP = {t: torch.finfo(t).eps / 2 for t in (torch.float32, torch.bfloat16, torch.float16)}
# half a step of the subnormal numbers
TINY = {torch.float32: 2.0 ** -150, torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}
SUM = 48   # additions on any path of a row's sum: 16 a lane, 6 + 16 joins, and a few products


def rounded(value, err, dtype):
    """Bound of a result within err of value, rounded to dtype."""
    return err + (np.abs(value) + err) * HALF_STEP[dtype] + TINY[dtype]


def assert_within(got, want, bound, what):
    got = got.detach().double().cpu().numpy() if torch.is_tensor(got) else np.asarray(got, np.float64)
    assert got.shape == want.shape, (what, got.shape, want.shape)
    bad = ~(np.abs(got - want) <= bound)
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{what}: {bad.sum()} of {bad.size} off, first at {i}: got {got[i]!r}, "
                             f"want {want[i]!r}, bound {np.broadcast_to(bound, got.shape)[i]!r}")


def f64(t):
    return t.detach().double().cpu().numpy()


# ---- AdamW ----

def f32(x):
    return float(np.float32(x))


def fmix32(h):
    h = np.asarray(h, np.uint64)
    h = h ^ (h >> np.uint64(16))
    h = (h * np.uint64(0x85EBCA6B)) & np.uint64(0xFFFFFFFF)
    h = h ^ (h >> np.uint64(13))
    h = (h * np.uint64(0xC2B2AE35)) & np.uint64(0xFFFFFFFF)
    return h ^ (h >> np.uint64(16))


def random_bits(places, seed, step):
    key = fmix32(seed & 0xFFFFFFFF) ^ np.uint64(step)
    high = ((places >> np.uint64(32)) * np.uint64(0x9E3779B9)) & np.uint64(0xFFFFFFFF)
    return fmix32((places & np.uint64(0xFFFFFFFF)) ^ fmix32(key ^ high))


def moments(g, m, v, p):
    b1, b2 = f32(p["beta1"]), f32(p["beta2"])
    return b1 * m + (1.0 - b1) * g, b2 * v + (1.0 - b2) * (g * g)


def adamw_weights(w, m, v, p, decay, lr_scale):
    """(new weights, step size, denominator) from the new moments."""
    lr = f32(p["lr"]) * f32(lr_scale)
    denom = np.sqrt(v / (1.0 - f32(p["beta2"]) ** p["step"])) + f32(p["eps"])
    size = lr / (1.0 - f32(p["beta1"]) ** p["step"])
    return w * (1.0 - lr * f32(decay)) - size * m / denom, size, denom


def weight_bound(w, new, m, m_err, size, denom):
    # keep and the final rounding; the step's quotient, product and denominator (12 roundings)
    return U * (2 * np.abs(w) + np.abs(new)) + size * (m_err + 16 * U * np.abs(m)) / denom + TINY[torch.float32]


def quantise(x, random16, positive):
    """(e4m3 values without their scale, biased scale) of one tensor's moments, by value: each
    magnitude is a multiple of its code's step plus a remainder, and goes up when the remainder
    and the random part reach the next multiple."""
    n = x.size
    mag = np.abs(x)
    top = np.pad(mag, (0, -n % BLOCK)).reshape(-1, BLOCK).max(1)
    frac, exp = np.frexp(top)
    exp = np.where(top == 0, -1100, exp - 9 + (np.floor(frac * 2.0 ** 21) > 0.875 * 2 ** 21))
    scale = np.clip(exp + 127, 0, 254).astype(np.int64)
    u = np.ldexp(mag, -np.repeat(scale - 127, BLOCK)[:n])
    step = np.ldexp(1.0, np.maximum(np.frexp(u)[1] - 1, -6) - 3)
    # remainders count in multiples of step / 2^17
    part = np.floor(u / step * 2.0 ** 17)
    q = np.floor((part + 2.0 * random16 + 1.0) / 2.0 ** 17) * step
    if positive:
        q = np.where((x > 0) & (q == 0), 2.0 ** -9, q)
    return np.copysign(q, x) if not positive else q, scale


# ---- layer norm ----

def norm_forward(x, w, b, eps):
    mean = x.mean(1)
    d = x - mean[:, None]
    rstd = 1.0 / np.sqrt((d * d).mean(1) + eps)
    return d * rstd[:, None] * w + b, mean, rstd


def norm_forward_bounds(x, w, b, eps):
    y, mean, rstd = norm_forward(x, w, b, eps)
    e_mean = SUM * U * np.abs(x).mean(1) + U * np.abs(mean)
    d = np.abs(x - mean[:, None])
    e_d = (e_mean[:, None] + U * d)
    var = (d * d).mean(1)
    e_var = (2 * d * e_d + e_d * e_d).mean(1) + SUM * U * var
    # floats below float32's smallest normal number keep an absolute error of 2^-150 each
    r = 0.5 * e_var / np.maximum(var + eps - e_var, 1e-300) + 4 * U
    e_rstd = r * rstd
    e_y = (e_d * rstd[:, None] + d * e_rstd[:, None]) * np.abs(w) + 4 * U * (d * rstd[:, None] * np.abs(w) + np.abs(b))
    return (y, e_y), (mean, e_mean), (rstd, e_rstd)


def norm_backward(dy, x, w, mean, rstd):
    hat = (x - mean[:, None]) * rstd[:, None]
    g = dy * w
    c1, c2 = g.mean(1, keepdims=True), (g * hat).mean(1, keepdims=True)
    return rstd[:, None] * (g - c1 - hat * c2), (dy * hat).sum(0), dy.sum(0)


def norm_backward_bounds(dy, x, w, mean, rstd):
    dx, dw, db = norm_backward(dy, x, w, mean, rstd)
    hat = np.abs((x - mean[:, None]) * rstd[:, None])
    g = np.abs(dy * w)
    c1, c2 = g.mean(1, keepdims=True), (g * hat).mean(1, keepdims=True)   # of magnitudes
    e = rstd[:, None] * U * (6 * g + (SUM + 4) * c1 + (SUM + 8) * hat * c2)
    rows = x.shape[0]
    chain = rows / 256 + SUM       # additions in a row of one workgroup's share, then joins
    return (dx, e), (dw, chain * U * (np.abs(dy) * hat).sum(0)), (db, chain * U * np.abs(dy).sum(0))


# ---- gated scan ----

def gate_factors(z, sigmoid):
    if not sigmoid:
        return z, np.ones_like(z)
    return 1.0 / (1.0 + np.exp(-z)), 1.0 / (1.0 + np.exp(z))


def _gate_roundings(z, dtype, sigmoid):
    """Roundings of one step: the recurrence's own, the factors' (the hardware's exponential of 16-bit
    types adds those of its argument, 2 |z| of them)."""
    if not sigmoid:
        return 4.0
    return 10.0 if dtype == torch.float32 else 10.0 + 2.0 * np.abs(z).max(initial=0.0)


def scan_forward(z, x, h0, n, sigmoid, dtype=torch.float32):
    """h, h_last and their bounds before the last rounding; steps from n[b] on are not read."""
    B, T, D = z.shape
    live = np.arange(T)[None, :, None] < n[:, None, None]
    z, x = np.where(live, z, 0.0), np.where(live, x, 0.0)
    a, k = gate_factors(z, sigmoid)
    c = _gate_roundings(z, dtype, sigmoid) * U
    h, e = np.zeros((B, T, D)), np.zeros((B, T, D))
    s, size, err = h0.copy(), np.abs(h0), np.zeros((B, D))
    for t in range(T):
        on = live[:, t]
        size = np.where(on, np.abs(a[:, t]) * size + np.abs(k[:, t] * x[:, t]), size)
        err = np.where(on, np.abs(a[:, t]) * err + c * size, err)
        s = np.where(on, a[:, t] * s + k[:, t] * x[:, t], s)
        h[:, t], e[:, t] = np.where(on, s, 0.0), np.where(on, err, 0.0)
    return (h, e), (s, err)


def scan_backward(z, x, h, dh, h0, dh_last, n, sigmoid, dtype=torch.float32):
    B, T, D = z.shape
    live = np.arange(T)[None, :, None] < n[:, None, None]
    z, dh = np.where(live, z, 0.0), np.where(live, dh, 0.0)
    x = np.where(live, x, 0.0) if x is not None else np.zeros_like(z)
    h = np.where(live, h, 0.0)
    a, k = gate_factors(z, sigmoid)
    c = _gate_roundings(z, dtype, sigmoid) * U
    out = [np.zeros((B, T, D)) for _ in range(4)]
    carry, size, err = dh_last.copy(), np.abs(dh_last), np.zeros((B, D))
    for t in range(T - 1, -1, -1):
        on = live[:, t]
        before = h[:, t - 1] if t else h0
        slope = (before - x[:, t]) * a[:, t] * k[:, t] if sigmoid else before
        l, ls = dh[:, t] + carry, np.abs(dh[:, t]) + size
        le = err + U * ls
        for o, v in zip(out, (l * slope, l * k[:, t], (le + 4 * c * ls) * np.abs(slope),
                              (le + 2 * c * ls) * np.abs(k[:, t]))):
            o[:, t] = np.where(on, v, 0.0)
        carry = np.where(on, a[:, t] * l, carry)
        err = np.where(on, np.abs(a[:, t]) * (le + c * ls), err)
        size = np.where(on, np.abs(a[:, t]) * ls, size)
    return (out[0], out[2]), (out[1], out[3]), (carry, err)
