"""Where the binding's outputs come from, without a GPU: torch allocates them in the call itself, so a
dispatch mode sees every allocation, and what one call found (a fake tensor among its operands)
does not stay for the next. The C entry points are stand-ins that launch nothing."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

from torch._subclasses import FakeTensorMode  # noqa: E402
from torch.utils._python_dispatch import TorchDispatchMode  # noqa: E402

import scaled_fp8_linear_amd as m  # noqa: E402

BF = torch.bfloat16


class Operand(torch.Tensor):
    """A tensor that says it is on the first device and has no memory."""

    @staticmethod
    def __new__(cls, shape, dtype=BF):
        return torch.Tensor._make_wrapper_subclass(cls, shape, dtype=dtype, device="cuda:0")

    def __torch_dispatch__(self, func, types, args=(), kwargs=None):
        raise AssertionError(f"{func} on an operand")


class OnHost(TorchDispatchMode):
    """Gives host memory for device memory and keeps what it gave."""

    def __enter__(self):
        self.given = []
        return super().__enter__()

    def __torch_dispatch__(self, func, types, args=(), kwargs=None):
        assert func is torch.ops.aten.empty.memory_format, func
        assert kwargs.pop("device").type == "cuda"
        self.given.append(torch.empty(args[0], dtype=kwargs.get("dtype")))
        return self.given[-1]


@pytest.fixture
def native():
    """The binding on entry points that do nothing and on a device 0 that is current."""
    m.load()
    native = m._abi._native()
    entry = ctypes.CFUNCTYPE(ctypes.c_int)(lambda: 0)
    at = {n: ctypes.cast(entry, ctypes.c_void_p).value for n in m._abi.EXPORTS}
    native.bind(at, m._abi._new, m._abi._check, lambda: 0, lambda d: 0)
    yield native
    m._abi._bind(m.load())


def norm(native):
    return native.layernorm_fwd(Operand((5, 64)), None, None, 1e-5, None, None, None, True, None)


def route(native):
    return native.moe_route(Operand((5, 16)), 2, None, True, None, None, None, None, None, None, None)


def act_bwd(native):
    """dh alone."""
    return native.act_quantize_bwd(Operand((128, 128)), Operand((128, 128), torch.uint8),
                                   Operand((128, 1), torch.float32), 1, False, None, None, None, None,
                                   None, None, False, False, True, None)


def check(native):
    with OnHost() as mode:
        y, mean, rstd = norm(native)
    # each output is what torch gave
    assert [t.data_ptr() for t in (y, mean, rstd)] == [t.data_ptr() for t in mode.given]
    assert y.dtype == BF and y.shape == (5, 64) and mean.shape == rstd.shape == (5,)
    with OnHost() as mode:
        outs = route(native)
    kept = {t.data_ptr() for t in mode.given}
    assert len(outs) == 5 and all(t.data_ptr() in kept for t in outs)
    with OnHost() as mode:
        outs = act_bwd(native)
    assert outs[:4] == (None,) * 4 and outs[4].data_ptr() == mode.given[-1].data_ptr()
    assert outs[4].shape == (128, 128) and outs[4].dtype == BF


def test_after_a_fake_tensor(native):
    with FakeTensorMode() as fake:
        x = fake.from_tensor(torch.empty(5, 64, dtype=BF)).to("cuda:0")
        for call in (lambda: native.layernorm_fwd(x, None, None, 1e-5, None, None, None, True, None),
                     lambda: native.moe_route(x, 2, None, True, *[None] * 7)):
            try:            # the address of a fake tensor is null, which a real entry point refuses
                call()
            except RuntimeError:
                pass
    check(native)


def test_torch_allocates_every_output(native):
    check(native)
    check(native)
