"""Host side of the causal convolution, the selective scan and the losses over a
vocabulary (no GPU needed): sizes, refusals of the C ABI before any device call,
and the 64-bit forms that the GPU tests compare with, against differences and
automatic derivatives."""
import ctypes

import pytest
import torch

import adaptive_residual_gradient_amd as A
import model_refs as M

OK, INVALID, MISALIGNED, CAPACITY, TOO_LARGE = 0, -1, -3, -5, -7


@pytest.fixture(scope="module", autouse=True)
def _lib_built():
    if not A.LIB_PATH.exists():
        from adaptive_residual_gradient_amd import _build
        _build.build()


def view(at, d, width):
    """(address[, batch stride, time stride]) or None."""
    if at is None:
        return A._View(None, 0, 0)
    at = at if isinstance(at, tuple) else (at, d["T"] * width, width)
    return A._View(*at)


# ---- causal convolution ----

CONV = dict(B=2, T=30, C=64, K=4, type=0, silu=1, x=0x100000, dy=0x200000, y=0x300000, weight=0x400000, bias=0x410000,
            state=0x420000, out=0x430000, dw=0x440000, db=0x450000, lengths=0x460000, ws=0x500000, nws=1 << 20)


def conv_call(change, back=False):
    d = dict(CONV, **change)
    s = A._ConvShape(d["T"], d["B"], d["C"], d["K"], d["type"], d["silu"])
    v = {k: ctypes.byref(view(d[k], d, d["C"])) if d[k] is not None else None for k in ("x", "dy", "y")}
    if back:
        return A.lib().adacomp_causal_conv_backward(ctypes.byref(s), v["dy"], v["x"], d["weight"], d["bias"], v["y"],
                                                    d["dw"], d["db"], d["state"], d["out"], d["lengths"], d["ws"], d["nws"],
                                                    None)
    return A.lib().adacomp_causal_conv(ctypes.byref(s), v["x"], d["weight"], d["bias"], v["y"], d["state"], d["out"],
                                       d["lengths"], None)


CONV_BOTH = [
    (dict(x=None), INVALID), (dict(y=None), INVALID), (dict(weight=None), INVALID), (dict(type=3), INVALID),
    (dict(silu=2), INVALID), (dict(C=0), INVALID), (dict(K=0), INVALID), (dict(K=9), INVALID),
    (dict(x=0x100002), MISALIGNED), (dict(type=1, x=0x100001), MISALIGNED), (dict(weight=0x400002), MISALIGNED),
    (dict(bias=0x410001), MISALIGNED), (dict(state=0x420002), MISALIGNED), (dict(out=0x430001), MISALIGNED),
    (dict(lengths=0x460002), MISALIGNED), (dict(y=0x100000), INVALID), (dict(y=0x100000 + 128), INVALID),
    (dict(out=0x420000), INVALID), (dict(y=0x400000), INVALID), (dict(out=0x100000), INVALID),
    (dict(x=(0x100000, 30 * 64, 63)), INVALID), (dict(y=(0x300000, 64, 64)), INVALID), (dict(T=1 << 31), TOO_LARGE),
    (dict(C=1 << 24), TOO_LARGE), (dict(B=1 << 24), TOO_LARGE), (dict(B=1 << 20, C=1 << 11), TOO_LARGE),
    (dict(T=(1 << 31) - 1, B=64, x=(0x100000, 1 << 38, 64)), TOO_LARGE),
    (dict(x=(0x100000, 1 << 40, 64)), TOO_LARGE), (dict(x=(0x100000, 64, 1 << 32)), TOO_LARGE),
]


@pytest.mark.parametrize("change,status", CONV_BOTH + [(dict(B=0), OK)])
def test_causal_conv_refused_before_any_device_call(change, status):
    assert conv_call(change) == status


@pytest.mark.parametrize("change,status", CONV_BOTH + [
    (dict(dy=None), INVALID), (dict(dw=None), INVALID), (dict(ws=None), INVALID), (dict(nws=64), CAPACITY),
    (dict(ws=0x500008), MISALIGNED), (dict(dw=0x440002), MISALIGNED), (dict(db=0x440000), INVALID),
    (dict(dw=0x400000), INVALID), (dict(ws=0x100000), INVALID), (dict(y=0x200000), INVALID),
])
def test_causal_conv_backward_refused_before_any_device_call(change, status):
    assert conv_call(change, back=True) == status


def test_causal_conv_workspace_bytes():
    n, L = ctypes.c_uint64(), A.lib()
    s = A._ConvShape(30, 2, 64, 4, 0, 1)
    assert L.adacomp_causal_conv_workspace_bytes(ctypes.byref(s), None) == INVALID
    assert L.adacomp_causal_conv_workspace_bytes(None, ctypes.byref(n)) == INVALID
    assert L.adacomp_causal_conv_workspace_bytes(ctypes.byref(s), ctypes.byref(n)) == OK
    assert n.value == 5 * 64 * 4          # 2 stretches of one workgroup
    for C, B, T in ((1, 1, 1), (7, 3, 100000), (2048, 8, 4096), (100000, 2, 7)):
        L.adacomp_causal_conv_workspace_bytes(ctypes.byref(A._ConvShape(T, B, C, 4, 1, 1)), ctypes.byref(n))
        assert n.value % (5 * C * 4) == 0 and 1 <= n.value // (5 * C * 4) <= 385


# ---- selective scan ----

SSM = dict(B=2, T=30, C=64, N=16, type=0, softplus=1, x=0x100000, dt=0x110000, b=0x120000, c=0x130000, z=0x140000,
           y=0x150000, a=0x160000, d=0x170000, bias=0x180000, lengths=0x190000, h0=0x1A0000, last=0x1B0000, kept=0x200000,
           ws=0x1000000, nws=1 << 24, dx=0x300000, ddt=0x310000, db=0x320000, dc=0x330000, dz=0x340000, da=0x350000,
           dd=0x360000, dbias=0x370000)


def ssm_call(change, back=False):
    d = dict(SSM, **change)
    s = A._SsmShape(d["T"], d["B"], d["C"], d["N"], d["type"], d["softplus"])
    width = lambda k: d["N"] if k[-1] in "bc" else d["C"]
    i = A._SsmInputs(*[view(d[k], d, width(k)) for k in ("x", "dt", "b", "c", "z")], d["a"], d["d"], d["bias"], d["lengths"])
    y = ctypes.byref(view(d["y"], d, d["C"])) if d["y"] is not None else None
    if back:
        g = A._SsmGradients(*[view(d[k], d, width(k)) for k in ("dx", "ddt", "db", "dc", "dz")], d["da"], d["dd"],
                            d["dbias"], d["last"])
        return A.lib().adacomp_selective_scan_backward(ctypes.byref(s), ctypes.byref(i), y, d["kept"], d["h0"],
                                                       ctypes.byref(g), d["ws"], d["nws"], None)
    return A.lib().adacomp_selective_scan(ctypes.byref(s), ctypes.byref(i), y, d["h0"], d["last"], d["kept"], d["ws"],
                                          d["nws"], None)


SSM_BOTH = [
    (dict(x=None), INVALID), (dict(dt=None), INVALID), (dict(b=None), INVALID), (dict(c=None), INVALID),
    (dict(y=None), INVALID), (dict(a=None), INVALID), (dict(ws=None), INVALID), (dict(type=-1), INVALID),
    (dict(softplus=2), INVALID), (dict(C=0), INVALID), (dict(N=0), INVALID), (dict(N=65), TOO_LARGE),
    (dict(x=0x100001), MISALIGNED), (dict(b=0x120002), MISALIGNED), (dict(a=0x160002), MISALIGNED),
    (dict(d=0x170001), MISALIGNED), (dict(bias=0x180002), MISALIGNED), (dict(lengths=0x190002), MISALIGNED),
    (dict(h0=0x1A0002), MISALIGNED), (dict(last=0x1B0002), MISALIGNED), (dict(kept=0x200004), MISALIGNED),
    (dict(ws=0x1000008), MISALIGNED), (dict(nws=256), CAPACITY), (dict(last=0x1A0000), INVALID),
    (dict(ws=0x100000), INVALID), (dict(b=(0x120000, 30 * 16, 15)), INVALID), (dict(T=1 << 31), TOO_LARGE),
    (dict(T=1 << 30, x=(0x100000, 1 << 36, 64)), TOO_LARGE), (dict(c=(0x130000, 1 << 40, 16)), TOO_LARGE),
    (dict(B=1 << 20, C=1 << 11), TOO_LARGE),
]


@pytest.mark.parametrize("change,status", SSM_BOTH + [
    (dict(B=0), OK), (dict(y=0x100000), INVALID), (dict(y=0x140000), INVALID), (dict(y=0x120000 + 64), INVALID),
    (dict(last=0x160000), INVALID), (dict(kept=0x100000), INVALID), (dict(y=(0x150000, 64, 64)), INVALID),
])
def test_selective_scan_refused_before_any_device_call(change, status):
    assert ssm_call(change) == status


PROJECTION = dict(dx=(0x300000, 30 * 160, 160), dz=(0x300000 + 4 * 64, 30 * 160, 160), db=(0x300000 + 4 * 128, 30 * 160, 160))


@pytest.mark.parametrize("change,status", SSM_BOTH + [
    (dict(dx=None), INVALID), (dict(ddt=None), INVALID), (dict(db=None), INVALID), (dict(dc=None), INVALID),
    (dict(da=None), INVALID), (dict(dz=None), INVALID), (dict(z=None), INVALID), (dict(kept=None), INVALID),
    (dict(dx=0x100000), INVALID), (dict(ddt=0x300000), INVALID), (dict(db=0x330000), INVALID), (dict(dd=0x370000), INVALID),
    (dict(da=0x360000), INVALID), (dict(dc=(0x330000, 16, 16)), INVALID), (dict(dbias=0x370002), MISALIGNED),
    # parts of one projection of different widths; the last ones share an element with another part
    (dict(PROJECTION, dc=(0x300000 + 4 * 144, 30 * 160, 160), nws=0), CAPACITY),
    (dict(PROJECTION, dc=(0x300000 + 4 * 143, 30 * 160, 160)), INVALID),
    (dict(PROJECTION, dc=(0x300000 + 4 * 145, 30 * 160, 160)), INVALID),
    (dict(PROJECTION, ddt=(0x300000 + 4 * 100, 30 * 160, 160)), INVALID),
])
def test_selective_scan_backward_refused_before_any_device_call(change, status):
    assert ssm_call(change, back=True) == status


def test_selective_scan_sizes():
    n, m, L = ctypes.c_uint64(), ctypes.c_uint64(), A.lib()
    s = A._SsmShape(30, 2, 64, 16, 0, 1)
    assert L.adacomp_selective_scan_workspace_bytes(ctypes.byref(s), 2, ctypes.byref(n)) == INVALID
    assert L.adacomp_selective_scan_workspace_bytes(ctypes.byref(s), 0, None) == INVALID
    assert L.adacomp_selective_scan_kept_bytes(None, ctypes.byref(n)) == INVALID
    assert L.adacomp_selective_scan_kept_bytes(ctypes.byref(s), ctypes.byref(n)) == OK
    assert n.value == 4 * 2 * 4 * 16 * 64       # a state of every 8 steps
    for T, B, C, N in ((1, 1, 1, 1), (5000, 3, 100, 16), (2048, 8, 2048, 64), (0, 2, 5, 3)):
        s = A._SsmShape(T, B, C, N, 1, 1)
        assert L.adacomp_selective_scan_workspace_bytes(ctypes.byref(s), 0, ctypes.byref(n)) == OK
        assert L.adacomp_selective_scan_workspace_bytes(ctypes.byref(s), 1, ctypes.byref(m)) == OK
        assert m.value >= n.value
        if T:
            assert n.value >= 4 * 2 * B * T * N


# ---- losses over a vocabulary ----

HEAD = dict(R=10, H=64, V=300, type=0, hs=64, ws_=64, hidden=0x100000, weight=0x200000, ids=0x300000, teacher=0x310000,
            picks=4, t=2.0, loss=0x320000, lse=0x330000, picked=0x340000, dloss=0x350000, dh=0x360000, dhs=64, dw=0x400000,
            dws=64, ws=0x1000000, nws=1 << 26)


def head_call(change, back=False, distil=False):
    d = dict(HEAD, **change)
    h = A._Head(d["R"], d["H"], d["V"], d["type"], d["hs"], d["ws_"], d["hidden"], d["weight"])
    L, h = A.lib(), ctypes.byref(h)
    grads = (d["dloss"], d["dh"], d["dhs"], d["dw"], d["dws"], d["ws"], d["nws"], None)
    if distil and back:
        return L.adacomp_linear_distillation_backward(h, d["ids"], d["teacher"], d["picks"], d["t"], d["lse"], d["picked"],
                                                      *grads)
    if distil:
        return L.adacomp_linear_distillation(h, d["ids"], d["teacher"], d["picks"], d["t"], d["loss"], d["lse"],
                                             d["picked"], d["ws"], d["nws"], None)
    if back:
        return L.adacomp_linear_cross_entropy_backward(h, d["ids"], d["loss"], d["lse"], *grads)
    return L.adacomp_linear_cross_entropy(h, d["ids"], d["loss"], d["lse"], d["ws"], d["nws"], None)


HEAD_ALL = [
    (dict(type=3), INVALID), (dict(H=0), INVALID), (dict(V=0), INVALID), (dict(hidden=None), INVALID),
    (dict(weight=None), INVALID), (dict(ids=None), INVALID), (dict(lse=None), INVALID), (dict(ws=None), INVALID),
    (dict(hs=63), INVALID), (dict(ws_=63), INVALID), (dict(hidden=0x100002), MISALIGNED),
    (dict(type=1, weight=0x200001), MISALIGNED), (dict(ids=0x300004), MISALIGNED), (dict(lse=0x330002), MISALIGNED),
    (dict(ws=0x1000008), MISALIGNED), (dict(nws=1 << 12), CAPACITY), (dict(R=1 << 24), TOO_LARGE),
    (dict(V=1 << 24), TOO_LARGE), (dict(H=65537, hs=65537, ws_=65537), TOO_LARGE), (dict(ws_=1 << 24), TOO_LARGE),
    (dict(ws=0x100000), INVALID), (dict(ws=0x200000), INVALID),
]


@pytest.mark.parametrize("distil", [False, True])
@pytest.mark.parametrize("change,status", HEAD_ALL + [
    (dict(loss=None), INVALID), (dict(loss=0x320001), MISALIGNED), (dict(loss=0x330000), INVALID),
    (dict(loss=0x100000), INVALID), (dict(lse=0x200000), INVALID),
])
def test_losses_refused_before_any_device_call(change, status, distil):
    assert head_call(change, distil=distil) == status


@pytest.mark.parametrize("distil", [False, True])
@pytest.mark.parametrize("change,status", HEAD_ALL + [
    (dict(dloss=None), INVALID), (dict(dhs=63), INVALID), (dict(dws=63), INVALID), (dict(dh=0x360002), MISALIGNED),
    (dict(dw=0x400002), MISALIGNED), (dict(dh=0x100000), INVALID), (dict(dw=0x200000), INVALID), (dict(dw=0x360000), INVALID),
    (dict(dh=0x350000), INVALID), (dict(dloss=0x350001), MISALIGNED), (dict(ws=0x350000), INVALID),
])
def test_gradients_of_losses_refused_before_any_device_call(change, status, distil):
    assert head_call(change, back=True, distil=distil) == status


@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("change,status", [
    (dict(picks=0), INVALID), (dict(picks=1025), TOO_LARGE), (dict(t=0.0), INVALID), (dict(t=-1.0), INVALID),
    (dict(t=float("nan")), INVALID), (dict(t=float("inf")), INVALID), (dict(t=1e-39), INVALID), (dict(teacher=None), INVALID),
    (dict(picked=None), INVALID), (dict(teacher=0x310002), MISALIGNED),
])
def test_distillation_refused_before_any_device_call(change, status, back):
    assert head_call(change, back=back, distil=True) == status


def test_no_rows_are_no_work():
    assert head_call(dict(R=0)) == OK and head_call(dict(R=0), distil=True) == OK
    assert head_call(dict(R=0, dw=None), back=True) == OK


def test_head_workspace_bytes():
    n, m, L = ctypes.c_uint64(), ctypes.c_uint64(), A.lib()
    head = lambda R, H, V, t: ctypes.byref(A._Head(R, H, V, t, H, H, None, None))
    assert L.adacomp_head_workspace_bytes(None, 1, 0, ctypes.byref(n)) == INVALID
    assert L.adacomp_head_workspace_bytes(head(1, 1, 1, 0), 1, 2, ctypes.byref(n)) == INVALID
    assert L.adacomp_head_workspace_bytes(head(1, 1, 1, 0), 0, 0, ctypes.byref(n)) == INVALID
    for R, H, V in ((1, 1, 1), (300, 256, 5000), (8192, 2048, 50000), (1, 4096, 131072), (100000, 64, 70000)):
        for t in range(3):
            assert L.adacomp_head_workspace_bytes(head(R, H, V, t), 1, 0, ctypes.byref(n)) == OK
            assert L.adacomp_head_workspace_bytes(head(R, H, V, t), 1, 1, ctypes.byref(m)) == OK
            assert m.value >= n.value
            # never the logits of everything: a piece, and what a small vocabulary is rounded up to
            assert m.value < 6 * (2 ** 30 + 2 * R * 2048) + R * (40 * H + 1000) + 6 * 65536 * (H + 8) + 256 * R * H


# ---- the 64-bit forms themselves ----

def gradients_of(f, ins, want):
    for v in ins.values():
        v.requires_grad_()
    f(**ins).backward()
    for k, v in ins.items():
        assert torch.allclose(want[k], v.grad, rtol=1e-10, atol=1e-12), k
    with torch.no_grad():
        gen = torch.Generator().manual_seed(9)
        for k, v in ins.items():
            u = torch.randn(v.shape, generator=gen, dtype=torch.float64)
            step = lambda e: f(**{n: (t + e * u if n == k else t) for n, t in ins.items()})
            assert abs(float((step(1e-6) - step(-1e-6)) / 2e-6 - (want[k] * u).sum())) < 1e-6, k


def normal(seed):
    gen = torch.Generator().manual_seed(seed)
    return lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)


@pytest.mark.parametrize("silu", [True, False])
@pytest.mark.parametrize("K", [1, 3, 4])
def test_conv_gradient(K, silu):
    r = normal(K)
    ins = dict(x=r(3, 6, 4), w=r(4, K), bias=r(4), state=r(3, K - 1, 4))
    dy, lengths = r(3, 6, 4), [6, 0, 2]
    want = M.conv(**ins, lengths=lengths, silu=silu, dy=dy)
    gradients_of(lambda **i: (M.conv(**i, lengths=lengths, silu=silu)["y"][0] * dy).sum(), ins,
                 dict(x=want["dx"][0], w=want["dweight"][0], bias=want["dbias"][0], state=want["dstate"][0]))


@pytest.mark.parametrize("softplus", [True, False])
@pytest.mark.parametrize("gated", [True, False])
def test_scan_gradient(gated, softplus):
    r = normal(5)
    B, T, C, N = 3, 6, 4, 5
    ins = dict(x=r(B, T, C), dt=r(B, T, C), a=-torch.rand(C, N, dtype=torch.float64) - 0.2, b=r(B, T, N), c=r(B, T, N), d=r(C),
               dt_bias=r(C), h0=r(B, C, N))
    if gated:
        ins["z"] = r(B, T, C)
    dy, dl, lengths = r(B, T, C), r(B, C, N), [6, 0, 2]
    want = M.scan(**ins, lengths=lengths, softplus=softplus, dy=dy, dh_last=dl)

    def f(**i):
        out = M.scan(**i, lengths=lengths, softplus=softplus)
        return (out["y"][0] * dy).sum() + (out["h_last"][0] * dl).sum()
    gradients_of(f, ins, {k: want["d" + k][0] for k in ins})


@pytest.mark.parametrize("picks", [0, 5])
def test_loss_gradient(picks):
    r = normal(7)
    R, H, V = 6, 5, 9
    ins = dict(hidden=r(R, H), weight=r(V, H))
    ids = torch.randint(0, V, (R, max(picks, 1)), generator=torch.Generator().manual_seed(1))
    ids[2] = -1
    if picks:
        ids[1, 3] = V
    kw = dict(ids=ids, teacher=r(R, picks) if picks else None, temperature=1.5 if picks else 1.0)
    g = r(R)
    want = M.loss(**ins, **kw, dloss=g)
    gradients_of(lambda **i: (M.loss(**i, **kw)["loss"][0] * g).sum(), ins,
                 dict(hidden=want["dhidden"][0], weight=want["dweight"][0]))


def test_type_and_shape_checks_of_the_binding():
    x, w = torch.zeros(1, 2, 3), torch.zeros(3, 4)
    with pytest.raises(TypeError):
        A.causal_conv(x, w, None, x.clone())          # CPU tensors
    with pytest.raises(TypeError):
        A.selective_scan(x, x, w, x, x, x.clone())
    with pytest.raises(TypeError):
        A.linear_cross_entropy(w, w, torch.zeros(3, dtype=torch.int64), w, w, None)
    with pytest.raises(TypeError):
        A.linear_distillation(w, w, torch.zeros(3, 2, dtype=torch.int64), w, w, w, w, None)
    with pytest.raises(TypeError):
        A.linear_loss_workspace(1, 1, 1, torch.float64)
