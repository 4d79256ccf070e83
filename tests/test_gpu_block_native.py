"""The native marshalling of the block operators' calls with the C ABI behind it
replaced: a small library, preloaded into a process of its own, takes the
module's calls (the step-by-step calls of block.py still reach the real one),
counts them and answers with the code that the test sets."""
import os
import shutil
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

STUB = """
int PyGILState_Check(void);
int stub_code, stub_calls, stub_locked;
static int answer(void) { ++stub_calls; stub_locked += PyGILState_Check(); return stub_code; }
int moe_layer_norm_fwd() { return answer(); }
int moe_layer_norm_bwd() { return answer(); }
int moe_layer() { return answer(); }
int moe_experts() { return answer(); }
int moe_grad_norm() { return answer(); }
int moe_clip_grads() { return answer(); }
"""

HEAD = """
import ctypes, sys
import torch
import padded_permute_combine_gb300 as p
stub = ctypes.CDLL(sys.argv[1])
code, calls, locked = (ctypes.c_int.in_dll(stub, "stub_" + n) for n in ("code", "calls", "locked"))
r = lambda *s: torch.randn(*s, device="cuda")
x, w, row = r(4, 64), r(64), r(4)
router, gate_up, down = r(4, 64), r(4, 32, 64), r(4, 64, 16)
top, share = torch.zeros(4, 2, dtype=torch.int32, device="cuda"), r(4, 2)
grads = p.moe_grad_set([r(1000)])
every = {
    "moe_layer_norm_fwd": lambda: p.moe_layer_norm_fwd(x, w, w),
    "moe_layer_norm_bwd": lambda: p.moe_layer_norm_bwd(x, x, w, row, row),
    "moe_layer": lambda: p.moe_layer(x, router, gate_up, down, 2),
    "moe_experts": lambda: p.moe_experts(x, top, share, gate_up, down),
    "moe_grad_norm": lambda: p.moe_grad_norm(grads),
    "moe_clip_grads": lambda: p.moe_clip_grads(grads, 0.5),
}
"""


def run_with_stub(tmp_path, body):
    gcc = shutil.which("gcc")
    if gcc is None or not torch.cuda.is_available():
        pytest.skip("needs gcc and a CUDA device")
    (tmp_path / "stub.c").write_text(STUB)
    lib = str(tmp_path / "libstub.so")
    subprocess.run([gcc, "-shared", "-fPIC", "-o", lib, str(tmp_path / "stub.c")], check=True)
    env = dict(os.environ, PYTHONPATH=ROOT + os.pathsep + os.environ.get("PYTHONPATH", ""))
    # Preloaded by the interpreter alone, not by what it may start.
    script = "import os; os.environ.pop('LD_PRELOAD')\n" + HEAD + body
    res = subprocess.run([sys.executable, "-c", script, lib], env=dict(env, LD_PRELOAD=lib), capture_output=True, text=True,
                         timeout=300)
    assert res.returncode == 0, res.stdout + res.stderr


def test_a_failed_call_is_reported_and_not_repeated(tmp_path):
    """Only refused arguments are left to the step-by-step call: after a CUDA
    error part of the work may be enqueued, and a second call would do it again."""
    run_with_stub(tmp_path, """
before = grads.grads[0].clone()
for name, call in every.items():
    code.value, calls.value = 3, 0
    try:
        call()
    except p.MoeError as e:
        assert e.code == 3 and name in str(e) and "CUDA" in str(e), e
    else:
        raise AssertionError(name + " repeated the call")
    assert calls.value == 1, name
assert torch.equal(grads.grads[0], before)  # nobody clipped
for name, call in every.items():
    for refused in (1, 2):
        code.value, calls.value = refused, 0
        assert call() is not None and calls.value == 1, name
code.value = 0
assert float(grads.grads[0].norm()) < 0.51
""")


def test_calls_leave_the_interpreter_to_other_threads(tmp_path):
    """As ctypes' calls do: a launch that waits for room in a full queue must
    not hold up the process's other Python threads."""
    run_with_stub(tmp_path, """
code.value = 0
for name, call in every.items():
    calls.value = locked.value = 0
    call()
    assert calls.value == 1 and locked.value == 0, name
""")


def test_calls_make_the_tensors_device_current(monkeypatch):
    """A C call works on the current device, so another one that is current has
    to give way for its length (there is one GPU here: which device is current
    is faked, and the step-by-step calls' guard is seen to be entered)."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import padded_permute_combine_gb300 as p

    x, w, row = torch.randn(4, 64, device="cuda"), torch.randn(64, device="cuda"), torch.ones(4, device="cuda")
    out, norm = torch.empty_like(x), torch.empty((), device="cuda")
    router, gate_up, down = (torch.randn(*s, device="cuda") for s in ((4, 64), (4, 32, 64), (4, 64, 16)))
    top, share = torch.zeros(4, 2, dtype=torch.int32, device="cuda"), torch.randn(4, 2, device="cuda")
    grads = p.moe_grad_set([torch.randn(100, device="cuda")])
    calls = [lambda: p.moe_layer_norm_fwd(x, w, w, out=out), lambda: p.moe_layer_norm_bwd(x, x, w, row, row, out=out),
             lambda: p.moe_layer(x, router, gate_up, down, 2, out=out), lambda: p.moe_experts(x, top, share, gate_up, down, out=out),
             lambda: p.moe_grad_norm(grads, norm=norm), lambda: p.moe_clip_grads(grads, 1.0, norm=norm)]
    entered = []

    class Device:
        def __init__(self, device):
            self.device = device

        def __enter__(self):
            entered.append(self.device)

        def __exit__(self, *_):
            entered.append(None)

    monkeypatch.setattr(torch.cuda, "device", Device)
    for call in calls:  # the tensors' device is current already
        call()
    assert entered == []
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    for call in calls:
        entered.clear()
        call()
        assert entered == [x.device, None]


def test_errors_of_torch_inside_a_call_are_exceptions():
    """A tensor without memory raises: refused as a null pointer, or by torch while the interpreter's lock is given back."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import padded_permute_combine_gb300 as p
    from torch._subclasses.fake_tensor import FakeTensorMode

    real = torch.randn(4, 64, device="cuda")
    with FakeTensorMode():
        fake = torch.empty(4, 64, device="cuda")
    for call in (lambda: p.moe_layer_norm_fwd(fake), lambda: p.moe_layer_norm_bwd(fake, fake, None, real[:, 0].clone(), real[:, 0].clone())):
        with pytest.raises(RuntimeError):
            call()
    y, mean, _ = p.moe_layer_norm_fwd(real)
    assert torch.isfinite(y).all() and torch.isfinite(mean).all()
