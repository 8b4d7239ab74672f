"""The binding's outputs on the device: torch's own memory also in a process whose first call was given
a fake tensor, seen by a dispatch mode, and filled where torch is told to fill what it allocates."""
import ctypes
import os
import subprocess
import sys

import pytest

from tests.gpu_util import note

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# runs in a process of its own, whose first call of the binding is the one with a fake tensor
FAKE_FIRST = """
import torch
from torch._subclasses import FakeTensorMode
import scaled_fp8_linear_amd as m
with FakeTensorMode():
    x = torch.empty(128, 256, device="cuda", dtype=torch.bfloat16)
    try:
        m.fp8_layernorm_fwd(x)
    except Exception as e:
        print("refused:", type(e).__name__, flush=True)
try:
    m.fp8_moe_route(x, 2)
except Exception as e:
    print("refused:", type(e).__name__, flush=True)
x = torch.randn(128, 256, device="cuda", dtype=torch.bfloat16)
y, mean, rstd = m.fp8_layernorm_fwd(x)
assert y.data_ptr() and mean.data_ptr() and rstd.data_ptr()
torch.testing.assert_close(y.float(), torch.nn.functional.layer_norm(x.float(), (256,)), atol=0.05,
                           rtol=0.02)
r = m.fp8_moe_route(x, 2)
assert torch.equal(r[0], x.float().sort(dim=1, descending=True, stable=True)[1][:, :2].int())
hq, hs = m.fp8_act_quantize(x, "relu", False)[4:]
dh = m.fp8_act_quantize_bwd(x, hq, hs, "relu", False, want_q=False, want_q_t=False, want_dh=True)[4]
assert dh.data_ptr() and torch.equal(dh, torch.where(hq.view(torch.float8_e4m3fn).float() > 0, x, 0))
print("done", flush=True)
"""


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import scaled_fp8_linear_amd as m
    m.load()
    return m


def test_a_fake_tensor_first(lib):
    note("a fake tensor in the first call of a process")
    r = subprocess.run([sys.executable, "-c", FAKE_FIRST], cwd=ROOT, capture_output=True, text=True,
                       timeout=100)
    assert r.returncode == 0 and r.stdout.split()[-1] == "done", r.stdout + r.stderr
    assert r.stdout.count("refused: ") == 2, r.stdout


def test_a_mode_sees_the_outputs(lib):
    from torch.utils._python_dispatch import TorchDispatchMode

    class Seen(TorchDispatchMode):
        def __torch_dispatch__(self, func, types, args=(), kwargs=None):
            out = func(*args, **(kwargs or {}))
            self.given.append((func, out))
            return out

    note("outputs under a dispatch mode")
    x = torch.randn(70, 128, device="cuda")
    want = lib.fp8_layernorm_fwd(x) + lib.fp8_moe_route(x, 3)
    mode = Seen()
    mode.given = []
    with mode:
        got = lib.fp8_layernorm_fwd(x) + lib.fp8_moe_route(x, 3)
    made = {t.data_ptr() for f, t in mode.given if f is torch.ops.aten.empty.memory_format}
    assert all(t.data_ptr() in made for t in got)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_filled_where_torch_fills(lib):
    """Entry points that launch nothing leave what the allocation left."""
    note("outputs where allocated memory is filled")
    entry = ctypes.CFUNCTYPE(ctypes.c_int)(lambda: 0)
    at = {n: ctypes.cast(entry, ctypes.c_void_p).value for n in lib._abi.EXPORTS}
    x = torch.zeros(5, 64, device="cuda")
    native = lib._abi._native()
    was = torch.are_deterministic_algorithms_enabled()
    try:
        native.bind(at, lib._abi._new, lib._abi._check, lambda: 0, lambda d: 0)
        torch.use_deterministic_algorithms(True)
        outs = native.layernorm_fwd(x, None, None, 1e-5, None, None, None, True, None)
        outs += native.moe_route(x, 2, None, True, *[None] * 7)[1:3]
    finally:
        torch.use_deterministic_algorithms(was)
        lib._abi._bind(lib.load())
    assert all(torch.isnan(t).all() for t in outs)
    y, _, _ = lib.fp8_layernorm_fwd(x + torch.arange(64, device="cuda"))     # the real ones are back
    assert torch.isfinite(y).all()
