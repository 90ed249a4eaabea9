"""The operators' entry points without a GPU: tensors that only claim a device, and the C ABI
replaced by functions that report how they were called.  Each case runs in a process of its own,
in which torch names device 0 as the current one."""
import pathlib
import subprocess
import sys

import pytest

ROOT = pathlib.Path(__file__).resolve().parent.parent

STUB = """
extern int PyGILState_Check(void);
#define REPORT(name) int name() { return 100 + PyGILState_Check(); }
REPORT(adacomp_grad_norm) REPORT(adacomp_adamw_step) REPORT(adacomp_adamw_packed_step)
REPORT(adacomp_layer_norm) REPORT(adacomp_layer_norm_backward)
REPORT(adacomp_gated_scan) REPORT(adacomp_gated_scan_backward)
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
u8, bf = torch.uint8, torch.bfloat16
f = lambda: new(64)
v = lambda: new(2, 20, 8)
s = lambda: new(2, 8)
# the arguments of every entry point; callables make a tensor
CALLS = {
    "grad_norm": [16, f, lambda: new(2), lambda: new(64, t=u8), 1.0, 1.0, None],
    "adamw": [16, 64, 2, f, f, f, f, None, 1e-3, 0.9, 0.999, 1e-8, 1, 1.0, 0, lambda: new(2), lambda: new(64, t=bf), None],
    "adamw packed": [16, 64, 2, f, f, lambda: new(64, t=u8), lambda: new(64, t=u8), lambda: new(4, t=u8), 1e-3, 0.9, 0.999,
                     1e-8, 1, 1.0, 0, lambda: new(2), lambda: new(64, t=bf), None],
    "layer_norm": [lambda: new(4, 64), f, f, lambda: new(4, 64), lambda: new(4), lambda: new(4), 1e-5, None],
    "layer_norm_backward": [lambda: new(4, 64), lambda: new(4, 64), f, lambda: new(4), lambda: new(4), lambda: new(4, 64),
                            f, f, lambda: new(64, t=u8), None],
    "gated_scan": [v, v, v, s, s, lambda: new(2, t=torch.int32), True, lambda: new(64, t=u8), None],
    "gated_scan_backward": [v, v, v, v, v, v, s, s, s, lambda: new(2, t=torch.int32), True, lambda: new(64, t=u8), None],
}
def call(name, other=None):
    args = []
    for i, a in enumerate(CALLS[name]):
        a = a() if callable(a) else a
        if i == other:
            a = new(*a.shape, t=a.dtype, device=1)
        args.append(a)
    return getattr(ops, name.split()[0])(*args)
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
    """Whichever tensor it is; and all of them, when another device is the current one."""
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
for t in (new(64, t=torch.float32, device=1), new(3, device=1)):
    try:
        ops.layer_norm(t, None, None, t, None, None, 1e-5, None)
    except ValueError as e:
        assert "current device" in str(e), e
    else:
        raise AssertionError("taken")
""")


def test_calls_are_made_without_the_interpreter_lock(stub):
    run(stub, """
for name in CALLS:
    assert call(name) == 100, name
""")
