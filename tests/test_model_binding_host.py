"""The entry points of the convolution, the selective scan and the losses without a GPU: tensors that only claim a device, and
the C ABI replaced by functions that report how they were called.  Each case runs in a process of its own."""
import pathlib
import subprocess
import sys

import pytest

ROOT = pathlib.Path(__file__).resolve().parent.parent

STUB = """
extern int PyGILState_Check(void);
#define REPORT(name) int name() { return 100 + PyGILState_Check(); }
REPORT(adacomp_causal_conv) REPORT(adacomp_causal_conv_backward)
REPORT(adacomp_selective_scan) REPORT(adacomp_selective_scan_backward)
REPORT(adacomp_linear_cross_entropy) REPORT(adacomp_linear_cross_entropy_backward)
REPORT(adacomp_linear_distillation) REPORT(adacomp_linear_distillation_backward)
"""

SETUP = """
import ctypes, sys, warnings
warnings.simplefilter("ignore")
import torch
from torch._subclasses.fake_tensor import FakeTensorMode
torch._C._cuda_getDevice = lambda: 0
torch._C._cuda_getCurrentRawStream = lambda device: 0
ctypes.CDLL(sys.argv[1], mode=ctypes.RTLD_GLOBAL)     # before the entry points: theirs are these functions
import adaptive_residual_gradient_amd as A
ops = A._operators()
def new(*shape, t=torch.float32, device=0):
    with FakeTensorMode():
        return torch.empty(shape, dtype=t, device=f"cuda:{device}")
u8, i32, i64 = torch.uint8, torch.int32, torch.int64
B, T, C, N, K, R, H, V, P = 2, 20, 8, 5, 4, 6, 16, 30, 3
v = lambda: new(B, T, C)
n = lambda: new(B, T, N)
ch = lambda: new(C)
st = lambda: new(B, K - 1, C)
h = lambda: new(B, C, N)
ln = lambda: new(B, t=i32)
ws = lambda: new(64, t=u8)
kept = lambda: new(B * 3 * 8 * C)
hid, wt, row = lambda: new(R, H), lambda: new(V, H), lambda: new(R)
tg, ids, pk = lambda: new(R, t=i64), lambda: new(R, P, t=i64), lambda: new(R, P)
# the arguments of every entry point; callables make a tensor
CALLS = {
    "causal_conv": [v, lambda: new(C, K), ch, v, st, st, ln, True, None],
    "causal_conv_backward": [v, v, lambda: new(C, K), ch, v, lambda: new(C, K), ch, st, st, ln, True, ws, None],
    "selective_scan": [v, v, lambda: new(C, N), n, n, v, ch, v, ch, h, h, kept, ln, True, ws, None],
    "selective_scan_backward": [v, v, v, lambda: new(C, N), n, n, kept, v, v, lambda: new(C, N), n, n, ch, v, ch, v, ch, ch, h,
                                h, ln, True, ws, None],
    "linear_cross_entropy": [hid, wt, tg, row, row, ws, None],
    "linear_cross_entropy_backward": [hid, wt, tg, row, row, row, hid, wt, ws, None],
    "linear_distillation": [hid, wt, ids, pk, row, row, pk, ws, 2.0, None],
    "linear_distillation_backward": [hid, wt, ids, pk, row, pk, row, hid, wt, ws, 2.0, None],
}
def call(name, other=None, change=None):
    args = []
    for i, a in enumerate(CALLS[name]):
        a = a() if callable(a) else a
        if i == other:
            a = change(a) if change else new(*a.shape, t=a.dtype, device=1)
        args.append(a)
    return getattr(ops, name)(*args)
"""


@pytest.fixture(scope="module")
def stub(tmp_path_factory):
    import adaptive_residual_gradient_amd as A
    if not A.LIB_PATH.exists():
        from adaptive_residual_gradient_amd import _build
        _build.build()
    at = tmp_path_factory.mktemp("stub")
    (at / "stub.c").write_text(STUB)
    subprocess.run(["gcc", "-shared", "-fPIC", "-w", "-o", str(at / "stub.so"), str(at / "stub.c")], check=True)
    return at / "stub.so"


def run(stub, body):
    r = subprocess.run([sys.executable, "-c", SETUP + body, str(stub)], capture_output=True, text=True, cwd=ROOT)
    assert r.returncode == 0, r.stdout + r.stderr[-3000:]


def test_tensors_of_another_device_are_refused(stub):
    run(stub, """
for name, args in CALLS.items():
    assert call(name) >= 100, name
    for i, a in enumerate(args):
        if not callable(a):
            continue
        try:
            call(name, other=i)
        except ValueError as e:
            assert "current device" in str(e), (name, i, e)
        else:
            raise AssertionError(f"{name}: argument {i} of another device was taken")
""")


def test_other_sizes_and_types_are_refused(stub):
    """One more place along an axis, and another type, of any tensor but a workspace and the kept states, whose
    size the C ABI checks or which may be larger."""
    run(stub, """
for name, args in CALLS.items():
    for i, a in enumerate(args):
        if not callable(a) or a in (ws, kept):
            continue
        def longer(t):
            return new(*[s + (k == 0) for k, s in enumerate(t.shape)], t=t.dtype)
        def other(t):
            return new(*t.shape, t=torch.float64)
        for change in (longer, other):
            if change is longer and (name, i) in {("linear_cross_entropy", 1), ("linear_distillation", 1)}:
                continue        # any number of words
            try:
                call(name, other=i, change=change)
            except (ValueError, TypeError):
                continue
            raise AssertionError((name, i, change.__name__))
""")


def test_calls_are_made_without_the_interpreter_lock(stub):
    run(stub, """
for name in CALLS:
    assert call(name) == 100, name
""")
