"""Host side of the training-step operators (no GPU needed): tables, sizes,
refusals of the C ABI before any device call, and the 64-bit forms that the GPU
tests compare with, checked against differences and by hand."""
import ctypes

import numpy as np
import pytest
import torch

import adaptive_residual_gradient_amd as A
import operator_refs as R

OK, INVALID, MISALIGNED, OVERLAP, CAPACITY, TOO_LARGE = 0, -1, -3, -4, -5, -7


@pytest.fixture(scope="module", autouse=True)
def _lib_built():
    if not A.LIB_PATH.exists():
        from adaptive_residual_gradient_amd import _build
        _build.build()


# ---- optimizer tables ----

@pytest.mark.parametrize("table,status", [
    ([], INVALID),
    ([(0, 0, 0.0, 1.0)], INVALID),
    ([(0, 10, float("nan"), 1.0)], INVALID),
    ([(0, 10, 0.0, float("inf"))], INVALID),
    ([(2, 10, 0.0, 1.0)], MISALIGNED),
    ([(0, 100, 0.0, 1.0), (96, 10, 0.0, 1.0)], OVERLAP),
    ([(100, 10, 0.0, 1.0), (0, 101, 0.0, 1.0)], OVERLAP),
    ([(0, 1 << 40, 0.0, 1.0)], TOO_LARGE),
    ([(0, 1 << 39, 0.0, 1.0)], TOO_LARGE),
])
def test_optimizer_table_refused(table, status):
    with pytest.raises(A.AdaCompError) as e:
        A.optimizer_query(table)
    assert e.value.status == status


def test_optimizer_info():
    info = A.optimizer_query([(8, 33, 0.1, 1.0), (0, 5, 0.0, 0.5), (44, 8193, 0.0, 1.0)])
    assert info.as_dict() == {"ntensors": 3, "total_numel": 33 + 5 + 8193, "span": 8240,
                              "nblocks": 2 + 1 + 257, "norm_workspace_bytes": 8 * (1 + 1 + 9)}
    # more work tiles than the norm's first pass has workgroups
    assert A.optimizer_query([(0, 1 << 30, 0.0, 1.0)]).norm_workspace_bytes == 8 * 2048


def test_optimizer_null_arguments():
    L = A.lib()
    p = A.AdamW(1e-3, 0.9, 0.999, 1e-8, 1.0, 1)
    assert L.adacomp_optimizer_create(None, 0, None) == INVALID
    assert L.adacomp_optimizer_destroy(None) == INVALID
    assert L.adacomp_optimizer_get_info(None, None) == INVALID
    assert L.adacomp_grad_norm(None, 16, 0, 0, 1.0, 1.0, 16, 16, 8, None) == INVALID
    assert L.adacomp_adamw_step(None, 16, 32, 0, 48, 64, None, 4, ctypes.byref(p), None, None) == INVALID
    assert L.adacomp_adamw_packed_step(None, 16, 32, 0, 48, 64, 80, None, 4, ctypes.byref(p), 0, None,
                                       None) == INVALID


# ---- layer norm ----

def norm_call(x=0x10000, xs=64, w=0x20000, b=0x21000, y=0x30000, ys=64, mean=0x40000, rstd=0x41000, rows=4,
              cols=64, type=0, eps=1e-5):
    return A.lib().adacomp_layer_norm(x, xs, w, b, y, ys, mean, rstd, rows, cols, type, eps, None)


@pytest.mark.parametrize("change,status", [
    (dict(x=None), INVALID), (dict(y=None), INVALID), (dict(type=3), INVALID), (dict(type=-1), INVALID),
    (dict(cols=0), INVALID), (dict(cols=65537, xs=65537, ys=65537), TOO_LARGE), (dict(rows=1 << 32), TOO_LARGE),
    (dict(xs=63), INVALID), (dict(ys=63), INVALID), (dict(xs=1 << 40), TOO_LARGE),
    (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID),
    (dict(x=0x10002), MISALIGNED), (dict(type=1, y=0x30001), MISALIGNED), (dict(w=0x20002), MISALIGNED),
    (dict(y=0x10000), INVALID), (dict(y=0x10000 + 4 * 64 * 4 - 4), INVALID), (dict(mean=0x41004), INVALID),
    (dict(y=0x20000 - 16), INVALID), (dict(rstd=0x21000), INVALID),
    (dict(rows=0, x=None, y=None), OK),
])
def test_layer_norm_refused_before_any_device_call(change, status):
    assert norm_call(**change) == status


def norm_back(dy=0x10000, ds=64, x=0x20000, xs=64, w=0x30000, mean=0x31000, rstd=0x32000, dx=0x40000, dxs=64,
              dw=0x50000, db=0x51000, rows=4, cols=64, type=0, ws=0x60000, nws=1 << 16):
    return A.lib().adacomp_layer_norm_backward(dy, ds, x, xs, w, mean, rstd, dx, dxs, dw, db, rows, cols, type, ws,
                                               nws, None)


@pytest.mark.parametrize("change,status", [
    (dict(dy=None), INVALID), (dict(x=None), INVALID), (dict(dx=None), INVALID), (dict(mean=None), INVALID),
    (dict(rstd=None), INVALID), (dict(dw=None), INVALID), (dict(db=None), INVALID), (dict(ws=None), INVALID),
    (dict(nws=4 * 2 * 64 * 4 - 1), CAPACITY), (dict(ws=0x60008), MISALIGNED), (dict(dx=0x10000), INVALID),
    (dict(dw=0x51000 - 4), INVALID), (dict(dxs=10), INVALID), (dict(type=7), INVALID),
    (dict(ws=0x40000), INVALID), (dict(cols=1 << 17), TOO_LARGE),
    (dict(rows=0, dw=None, db=None), OK),
])
def test_layer_norm_backward_refused_before_any_device_call(change, status):
    assert norm_back(**change) == status


def test_layer_norm_workspace_bytes():
    n = ctypes.c_uint64()
    L = A.lib()
    assert L.adacomp_layer_norm_workspace_bytes(4, 64, None) == INVALID
    assert L.adacomp_layer_norm_workspace_bytes(4, 0, ctypes.byref(n)) == INVALID
    assert L.adacomp_layer_norm_workspace_bytes(4, 64, ctypes.byref(n)) == OK and n.value == 4 * 2 * 64 * 4


# ---- gated scan ----

def scan_call(change, back=False):
    d = dict(B=2, T=300, D=64, type=0, sigmoid=1, ts=64, bs=300 * 64, h0=0x900000, last=0x910000, dlast=0x920000,
             lengths=0x930000, ws=0xA00000, nws=1 << 24)
    views = dict(gate=0x100000, x=0x200000, h=0x300000, dh=0x400000, dgate=0x500000, dx=0x600000)
    d.update({k: v for k, v in change.items() if k in d})
    shape = A._ScanShape(d["T"], d["B"], d["D"], d["type"], d["sigmoid"])
    p = {}
    for k, at in views.items():
        at = change.get(k, at)
        if at is None:
            p[k] = None
        else:
            at = at if isinstance(at, tuple) else (at, d["bs"], d["ts"])
            p[k] = ctypes.byref(A._View(*at))
    L = A.lib()
    if back:
        return L.adacomp_gated_scan_backward(ctypes.byref(shape), p["gate"], p["x"], p["h"], p["dh"], p["dgate"],
                                             p["dx"], d["h0"], d["dlast"], d["last"], d["lengths"], d["ws"],
                                             d["nws"], None)
    return L.adacomp_gated_scan(ctypes.byref(shape), p["gate"], p["x"], p["h"], d["h0"], d["last"], d["lengths"],
                                d["ws"], d["nws"], None)


SCAN_BOTH = [
    (dict(gate=None), INVALID), (dict(x=None), INVALID), (dict(h=None), INVALID), (dict(type=3), INVALID),
    (dict(sigmoid=2), INVALID), (dict(D=0), INVALID), (dict(ts=63), INVALID), (dict(gate=0x100002), MISALIGNED),
    (dict(type=1, gate=0x100001), MISALIGNED), (dict(nws=16), CAPACITY), (dict(ws=None), INVALID),
    (dict(ws=0xA00008), MISALIGNED), (dict(h0=0x900002), MISALIGNED), (dict(lengths=0x930002), MISALIGNED),
    (dict(last=0x900000), INVALID), (dict(last=0x930000), INVALID), (dict(T=1 << 31), TOO_LARGE),
    (dict(ws=0x100000), INVALID), (dict(B=0), OK),
    (dict(D=1 << 20, B=1 << 20, ts=1 << 20), TOO_LARGE),
]


@pytest.mark.parametrize("change,status", SCAN_BOTH + [
    (dict(h=0x100000), INVALID), (dict(h=0x200000 + 64), INVALID),
    # two sequences of the output in the same rows
    (dict(h=(0x300000, 64, 64)), INVALID),
])
def test_gated_scan_refused_before_any_device_call(change, status):
    assert scan_call(change) == status


@pytest.mark.parametrize("change,status", SCAN_BOTH + [
    (dict(dh=None), INVALID), (dict(dgate=None), INVALID), (dict(dx=None), INVALID),
    (dict(dgate=0x600000), INVALID), (dict(dgate=0x100000), INVALID), (dict(dx=0x300000), INVALID),
    (dict(dgate=(0x500000, 0, 64)), INVALID),
    # parts of one row that share channels
    (dict(dgate=(0x500000, 300 * 100, 100), dx=(0x500000 + 4 * 63, 300 * 100, 100)), INVALID),
    (dict(dgate=(0x500000, 300 * 128, 128), dx=(0x500000 + 4 * 65, 300 * 128, 128)), INVALID),
])
def test_gated_scan_backward_refused_before_any_device_call(change, status):
    assert scan_call(change, back=True) == status


def test_gated_scan_workspace_bytes():
    n = ctypes.c_uint64()
    L = A.lib()
    s = A._ScanShape(1, 4, 64, 1, 1)
    assert L.adacomp_gated_scan_workspace_bytes(ctypes.byref(s), None) == INVALID
    assert L.adacomp_gated_scan_workspace_bytes(None, ctypes.byref(n)) == INVALID
    assert L.adacomp_gated_scan_workspace_bytes(ctypes.byref(s), ctypes.byref(n)) == OK
    assert n.value == 0          # one step: nothing to carry between chunks


# ---- the 64-bit forms themselves ----

def directional(f, at, direction, eps):
    return (f(at + eps * direction) - f(at - eps * direction)) / (2 * eps)


def test_norm_gradient_against_differences():
    rng = np.random.default_rng(0)
    x, dy = rng.standard_normal((5, 9)), rng.standard_normal((5, 9))
    w, b = 1 + 0.2 * rng.standard_normal(9), rng.standard_normal(9)
    _, mean, rstd = R.norm_forward(x, w, b, 1e-5)
    dx, dw, db = R.norm_backward(dy, x, w, mean, rstd)
    u, uw = rng.standard_normal((5, 9)), rng.standard_normal(9)
    loss = lambda x_, w_, b_: (R.norm_forward(x_, w_, b_, 1e-5)[0] * dy).sum()
    assert abs(directional(lambda t: loss(t, w, b), x, u, 1e-6) - (dx * u).sum()) < 1e-7
    assert abs(directional(lambda t: loss(x, t, b), w, uw, 1e-6) - (dw * uw).sum()) < 1e-7
    assert abs(directional(lambda t: loss(x, w, t), b, uw, 1e-6) - (db * uw).sum()) < 1e-7


@pytest.mark.parametrize("sigmoid", [True, False])
def test_scan_gradient_against_differences(sigmoid):
    rng = np.random.default_rng(1)
    B, T, D = 3, 7, 4
    z = rng.standard_normal((B, T, D)) * (1.0 if sigmoid else 0.5)
    x, dh = rng.standard_normal((B, T, D)), rng.standard_normal((B, T, D))
    h0, dl = rng.standard_normal((B, D)), rng.standard_normal((B, D))
    n = np.array([7, 0, 4])
    def loss(z_, x_, h0_):
        (h, _), (last, _) = R.scan_forward(z_, x_, h0_, n, sigmoid)
        return (h * dh).sum() + (last * dl).sum()
    (h, _), _ = R.scan_forward(z, x, h0, n, sigmoid)
    (dz, _), (dx, _), (dh0, _) = R.scan_backward(z, x, h, dh, h0, dl, n, sigmoid)
    u, u0 = rng.standard_normal((B, T, D)), rng.standard_normal((B, D))
    assert abs(directional(lambda t: loss(t, x, h0), z, u, 1e-6) - (dz * u).sum()) < 1e-7
    assert abs(directional(lambda t: loss(z, t, h0), x, u, 1e-6) - (dx * u).sum()) < 1e-7
    assert abs(directional(lambda t: loss(z, x, t), h0, u0, 1e-6) - (dh0 * u0).sum()) < 1e-7


def test_quantise_by_hand():
    # block maximum 448: scale 0 (biased 127); 300 lies between 288 and 320 (step 32): remainder 12/32
    x = np.array([448.0, 300.0, -0.001, 0.0])
    lo, scale = R.quantise(x, np.zeros(4), False)
    hi, _ = R.quantise(x, np.full(4, 65535.0), False)
    assert scale.tolist() == [127]
    assert lo.tolist() == [448.0, 288.0, -0.0, 0.0] and hi.tolist() == [448.0, 320.0, -2.0 ** -9, 0.0]
    # the remainder is the probability of the upper value
    up = [R.quantise(x, np.full(4, r), False)[0][1] == 320.0 for r in np.arange(0, 65536, 64)]
    assert abs(np.mean(up) - 12 / 32) < 2e-3
    # a second moment above zero stays above; the scale follows the largest
    q, scale = R.quantise(np.array([2.0 ** 20, 1e-9]), np.zeros(2), True)
    assert scale.tolist() == [127 + 20 - 8] and q[0] == 256.0 and q[1] == 2.0 ** -9
    assert R.quantise(np.array([449.0]), np.zeros(1), True)[1].tolist() == [128]
    assert R.quantise(np.zeros(3), np.zeros(3), True)[1].tolist() == [0]
    assert torch.tensor(q, dtype=torch.float32).to(torch.float8_e4m3fn).float().tolist() == q.tolist()


def test_type_and_shape_checks_of_the_binding():
    x = torch.zeros(4, 8)
    with pytest.raises(TypeError):
        A.layer_norm(x, None, None, x.clone())          # CPU tensors
    with pytest.raises(TypeError):
        A.gated_scan(torch.zeros(1, 2, 3), torch.zeros(1, 2, 3), torch.zeros(1, 2, 3))
    with pytest.raises(TypeError):
        A._grad(torch.zeros(4))
