"""Plain 64-bit forms of the causal convolution, the selective scan and the losses
over a vocabulary, on the CPU in torch, and the error bounds of the float32
kernels.

u = 2^-24 is float32's half step.  Every form returns values with a bound of what
float32 arithmetic may be off before the last rounding: a bound counts the
roundings of a result, each at most u of the value rounded, carried through the
formula's derivatives with absolute values in place of the terms.
"""
import torch

from operator_refs import HALF_STEP, TINY, U

GATE = 10    # roundings of the logistic function and a product with it


def f64(t):
    return None if t is None else t.detach().double().cpu()


def rounded(value, err, dtype):
    return err + (value.abs() + err) * HALF_STEP[dtype] + TINY[dtype]


def assert_within(got, pair, what, dtype=None):
    """got against (value, bound before the last rounding); an infinite bound takes anything."""
    want, err = pair
    bound = rounded(want, err, dtype or got.dtype)
    got = f64(got)
    assert got.shape == want.shape, (what, got.shape, want.shape)
    bad = ~((got - want).abs() <= bound) & ~torch.isinf(bound)
    if bad.any():
        i = tuple(torch.nonzero(bad)[0].tolist())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {i}: got {got[i]!r}, want "
                             f"{want[i]!r}, bound {bound[i]!r}")


def live_steps(lengths, B, T):
    """[B, T, 1]"""
    n = torch.full((B,), T) if lengths is None else torch.as_tensor(lengths).clamp(0, T)
    return (torch.arange(T) < n[:, None])[:, :, None], n


# ---- causal convolution ----

def conv(x, w, bias, state, lengths, silu, dy=None):
    """Dict of (value, bound): y, state_out, and with dy the gradients.  Everything 64-bit."""
    B, T, C = x.shape
    K = w.shape[1]
    live, n = live_steps(lengths, B, T)
    x = torch.where(live, x, torch.zeros(()).double())
    front = state if state is not None else torch.zeros(B, K - 1, C).double()
    rows = torch.cat([front, x], 1)
    bias = bias if bias is not None else torch.zeros(C).double()
    terms = [w[:, k] * rows[:, k:k + T] for k in range(K)]
    p = bias + sum(terms)
    ep = (K + 1) * U * (bias.abs() + sum(t.abs() for t in terms))
    zero = torch.zeros(()).double()
    q = torch.sigmoid(p)
    y, ey = (p * q, 1.1 * ep + GATE * U * (p * q).abs() + 1e-35) if silu else (p, ep)
    at = n[:, None] + torch.arange(K - 1)
    out = {"y": (torch.where(live, y, zero), torch.where(live, ey, zero)),
           "state_out": (torch.gather(rows, 1, at[:, :, None].expand(-1, -1, C)), zero)}
    if dy is None:
        return out
    dy = torch.where(live, dy, zero)
    if silu:
        slope, flat = q + p * q * (1 - q), q + (p * q * (1 - q)).abs()
        g, eg = dy * slope, dy.abs() * (0.51 * ep + (GATE + 6) * U * flat)     # |second derivative| <= 1/2
    else:
        g, eg = dy, zero * dy
    path = T + 260      # additions on the way of a term: along a stretch, over a workgroup's stretches
    total = lambda v: v.sum((0, 1))
    out["dweight"] = tuple(torch.stack(v, 1) for v in zip(*[
        (total(g * rows[:, k:k + T]), total(eg * rows[:, k:k + T].abs()) + path * U * total((g * rows[:, k:k + T]).abs()))
        for k in range(K)]))
    out["dbias"] = (total(g), total(eg) + path * U * total(g.abs()))
    d, e = torch.zeros_like(rows), torch.zeros_like(rows)
    for k in range(K):
        d[:, k:k + T] += w[:, k] * g
        e[:, k:k + T] += w[:, k].abs() * (eg + (K + 1) * U * g.abs())
    out["dx"], out["dstate"] = (d[:, K - 1:], e[:, K - 1:]), (d[:, :K - 1], e[:, :K - 1])
    return out


# ---- selective scan ----

def scan(x, dt, a, b, c, d=None, z=None, dt_bias=None, h0=None, lengths=None, softplus=True, dy=None, dh_last=None):
    """Dict of (value, bound): y, h_last, and with dy the gradients.  A channel whose states (or what is carried
    back) pass 2^126 on their way, where float32 ends, is bound by nothing, and nothing that it is a part of."""
    B, T, C = x.shape
    N = a.shape[1]
    top = torch.zeros(B, C).double()
    size = lambda v: torch.nan_to_num(v.abs(), nan=2.0 ** 200)
    far = lambda *vs: torch.stack([top] + [size(v).amax(2) if v.dim() == 3 else size(v) for v in vs]).amax(0)

    def unbound(out, keys):
        over = top > 2.0 ** 126
        if not over.any():
            return
        open_ = {"y": over[:, None, :], "h_last": over[:, :, None], "dx": over[:, None, :], "ddt": over[:, None, :],
                 "dz": over[:, None, :], "dh0": over[:, :, None], "db": over.any(1)[:, None, None],
                 "dc": over.any(1)[:, None, None], "da": over.any(0)[:, None], "dd": over.any(0), "ddt_bias": over.any(0)}
        for k in keys:
            v, e = out[k]
            out[k] = (v, torch.where(open_[k], torch.full((), float("inf")).double(), e))

    zero = torch.zeros(()).double()
    live, n = live_steps(lengths, B, T)
    cut = lambda v: torch.where(live, v, zero)
    x, dt, b, c = cut(x), cut(dt), cut(b), cut(c)
    d = d if d is not None else torch.zeros(C).double()
    raw = dt + (dt_bias if dt_bias is not None else 0.0)
    s = torch.logaddexp(raw, zero) if softplus else raw
    es = U * raw.abs() * torch.sigmoid(raw) + 12 * U * s if softplus else U * raw.abs()
    s, es = cut(s), cut(es)
    u, eu = s * x, es * x.abs() + 2 * U * (s * x).abs()
    h = h0 if h0 is not None else torch.zeros(B, C, N).double()
    eh = torch.zeros_like(h)
    # a chunk's decay goes by its steps' sum, one rounding a step more
    turns = min(T, 4096) + 6
    hs, es_h, decay, ed = [h], [eh], [], []
    y, ey = torch.zeros(B, T, C).double(), torch.zeros(B, T, C).double()
    for t in range(T):
        st, on = s[:, t, :, None], live[:, t, :, None]
        e = torch.exp(st * a)
        rel = a.abs() * es[:, t, :, None] + turns * U * (st * a).abs() + 6 * U
        ub = u[:, t, :, None] * b[:, t, None, :]
        new = e * h + ub
        enew = e * (1 + rel) * eh + rel * (e * h).abs() + eu[:, t, :, None] * b[:, t, None, :].abs() + 2 * U * (
            ub.abs() + (e * h).abs())
        h, eh = torch.where(on, new, h), torch.where(on, enew, eh)
        decay.append(torch.where(on, e, torch.ones(()).double()))
        ed.append(torch.where(on, rel, zero))
        hs.append(h)
        es_h.append(eh)
        ch = h * c[:, t, None, :]
        y[:, t] = ch.sum(2)
        ey[:, t] = (eh * c[:, t, None, :].abs()).sum(2) + (N + 6) * U * ch.abs().sum(2)
        top = far(h, ch.abs().sum(2))
    sums = y + d * x
    esums = ey + 3 * U * (d * x).abs() + U * y.abs()
    gate, slope, flat = torch.ones(()).double(), None, None
    if z is not None:
        z = cut(z)
        q = torch.sigmoid(z)
        gate, slope, flat = z * q, q + z * q * (1 - q), q + (z * q * (1 - q)).abs()
    y = cut(sums * gate)
    ey = cut(esums * gate.abs() + (GATE * U * y.abs() + 1e-35 * sums.abs() if z is not None else 0.0))
    out = {"y": (y, ey), "h_last": (h, eh)}
    if dy is None:
        unbound(out, out)
        return out
    dy = cut(dy)
    r, er = dy * gate, GATE * U * (dy * gate).abs() + (1e-35 * dy.abs() if z is not None else 0.0)
    if z is not None:
        out["dz"] = (dy * sums * slope, dy.abs() * (esums * slope.abs() + (GATE + 8) * U * sums.abs() * flat))
    f = dh_last if dh_last is not None else torch.zeros(B, C, N).double()
    ef = torch.zeros_like(f)
    du, edu, ds, eds = (torch.zeros(B, T, C).double() for _ in range(4))
    db, edb, dc, edc = (torch.zeros(B, T, N).double() for _ in range(4))
    da, eda = torch.zeros(C, N).double(), torch.zeros(C, N).double()
    lanes = 40 + C // 64      # additions over the channels
    path = T + 16             # and along a chunk
    for t in reversed(range(T)):
        on = live[:, t, :, None]
        rc = r[:, t, :, None] * c[:, t, None, :]
        l = f + rc
        el = ef + er[:, t, :, None] * c[:, t, None, :].abs() + 2 * U * (f.abs() + rc.abs())
        ut, bt = u[:, t, :, None], b[:, t, None, :]
        rh = r[:, t, :, None] * hs[t + 1]
        dc[:, t] = rh.sum(1)
        edc[:, t] = (er[:, t, :, None] * hs[t + 1].abs() + r[:, t, :, None].abs() * es_h[t + 1] + lanes * U * rh.abs()).sum(1)
        lu = l * ut
        db[:, t] = lu.sum(1)
        edb[:, t] = (el * ut.abs() + l.abs() * eu[:, t, :, None] + lanes * U * lu.abs()).sum(1)
        du[:, t] = (l * bt).sum(2)
        edu[:, t] = (el * bt.abs() + (N + 4) * U * (l * bt).abs()).sum(2)
        nf = decay[t] * l
        enf = decay[t] * (1 + ed[t]) * el + (ed[t] + U) * nf.abs()
        q = nf * hs[t]
        eq = enf * hs[t].abs() + nf.abs() * es_h[t] + U * q.abs()
        ds[:, t] = (q * a).sum(2)
        eds[:, t] = (eq * a.abs() + (N + 8) * U * (q * a).abs()).sum(2)
        st = s[:, t, :, None]
        da += (q * st).sum(0)
        eda += (eq * st.abs() + q.abs() * es[:, t, :, None] + path * U * (q * st).abs()).sum(0)
        f, ef = torch.where(on, nf, f), torch.where(on, enf, ef)
        top = far(l, q * (1 + a.abs()))
    v = ds + du * x
    ev = eds + edu * x.abs() + 4 * U * (ds.abs() + (du * x).abs())
    q = torch.sigmoid(raw) if softplus else torch.ones(()).double()
    dv = cut(v * q)
    edv = cut(ev * q + (GATE * U + U * raw.abs() if softplus else 0.0) * (v * q).abs())
    total = lambda t: t.sum((0, 1))
    out.update(
        dx=(cut(du * s + d * r), cut(edu * s.abs() + du.abs() * es + d.abs() * er + 4 * U * ((du * s).abs() + (d * r).abs()))),
        ddt=(dv, edv), db=(cut(db), cut(edb)), dc=(cut(dc), cut(edc)), da=(da, eda),
        dd=(total(r * x), total(er * x.abs()) + path * U * total((r * x).abs())),
        ddt_bias=(total(dv), total(edv) + path * U * total(dv.abs())), dh0=(f, ef))
    unbound(out, out)
    return out


# ---- losses over a vocabulary ----

def loss(hidden, weight, ids, teacher=None, temperature=1.0, dloss=None, dtype=torch.float32):
    """ids [rows, picks]; dtype: that of the matrices.  Dict of (value, bound): loss, lse, picked, and with dloss
    dhidden, dweight."""
    R, H = hidden.shape
    V = weight.shape[0]
    word = (ids >= 0) & (ids < V)
    used = word.any(1)
    # a matrix core's sum of H products may round each twice; planes leave out 2^-22 of a product
    planes = dtype == torch.float32
    terms = lambda k: 2 * k * U + (2.0 ** -22 if planes else 0.0)
    x = torch.where(used[:, None], hidden, torch.zeros(()).double())
    every = torch.nan_to_num(hidden, nan=0.0, posinf=0.0, neginf=0.0)   # rows that do not count may hold anything
    size = every.abs() @ weight.abs().t()
    z = every @ weight.t() / temperature
    ez = (terms(H) * size) / temperature + 3 * U * z.abs()
    lse = torch.logsumexp(z, 1)
    else_ = ez.max(1).values + 2 * U * (90 + lse.abs() + (z.max(1).values[:, None] - z).clamp(max=90).max(1).values)
    at = ids.clamp(0, V - 1)
    zk, ezk = torch.gather(z, 1, at), torch.gather(ez, 1, at)
    zero = torch.zeros(()).double()
    if teacher is None:
        p = word.double()
        terms_k, eterms = lse[:, None] - zk, else_[:, None] + ezk + U * (lse[:, None] - zk).abs()
        ep = zero * p
    else:
        logits = torch.where(word, teacher / temperature, torch.full((), -float("inf")).double())
        top = logits.max(1, keepdim=True).values
        top = torch.where(used[:, None], top, zero)
        far = (top - logits).clamp(max=110)
        e = torch.exp(logits - top)
        p = torch.where(used[:, None], e / e.sum(1, keepdim=True).clamp(min=1e-300), zero)
        logp = torch.where(p > 0, torch.log(p.clamp(min=1e-300)), zero)
        elogp = U * (4 * (top.abs() + far) + 12 + ids.shape[1] + logp.abs())
        ep = p * (elogp + 4 * U)
        inner = logp + lse[:, None] - zk
        terms_k = torch.where(p > 0, inner, zero)
        eterms = else_[:, None] + ezk + elogp + 3 * U * (logp.abs() + lse[:, None].abs() + zk.abs())
    out = {"loss": (torch.where(word, p * terms_k, zero).sum(1),
                    torch.where(word, p * eterms + (ep + (ids.shape[1] + 4) * U * p) * terms_k.abs(), zero).sum(1)),
           "lse": (lse, else_), "picked": (torch.where(word, zk, zero), torch.where(word, ezk, zero))}
    if dloss is None:
        return out
    f = torch.where(used, dloss / temperature, zero)
    q = torch.exp(z - lse[:, None])
    eq = q * (ez + else_[:, None] + 12 * U + U * (lse[:, None] - z).abs())
    dz = q.scatter_add(1, at, torch.where(word, -p, zero))
    edz = eq.scatter_add(1, at, torch.where(word, ep + (2 + ids.shape[1]) * U * p, zero))
    half = 2.0 ** -23 if planes else HALF_STEP[dtype]
    edz = edz + (dz.abs() + edz) * half + 4 * U * dz.abs()
    dz = dz * f[:, None]
    # what is below the smallest number of the scaled dz
    most = f.abs().max()
    edz = edz * f.abs()[:, None] + (most * 2.0 ** -38 if dtype == torch.float16 else 0.0)
    # and of float32's: an exponential below 2^-126 may be taken for 0, which leaves out |f| 2^-126 of dz; so may the
    # planes of dz, and the products and sums of terms, which are formed of dz / most 2^14, so 2^-126 2^-14 most each
    tiny = most * 2.0 ** -140
    edz = edz + f.abs()[:, None] * 2.0 ** -126 + 3 * tiny
    edz = torch.where(used[:, None], edz, zero)
    out["dhidden"] = (dz @ weight, edz @ weight.abs() + (terms(V) + 20 * U) * (dz.abs() @ weight.abs()) + 12 * V * tiny)
    out["dweight"] = (dz.t() @ x, edz.t() @ x.abs() + (terms(R) + 20 * U) * (dz.abs().t() @ x.abs()) + 12 * R * tiny)
    return out
