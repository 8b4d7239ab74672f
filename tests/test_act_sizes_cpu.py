"""The activation entry points refuse what one launch cannot hold (2^32 threads), before anything of it
is launched. Made-up addresses; every call here is refused."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

import scaled_fp8_linear_amd as m  # noqa: E402

pytestmark = pytest.mark.skipif(torch.cuda.device_count() > 0, reason="passes made-up addresses")

FAR = 1 << 42


@pytest.mark.parametrize("rows,cols", [((1 << 23) - 1, (1 << 14)), ((1 << 22) + 1, 1 << 15),
                                       ((1 << 23) - 128, (1 << 17) - 128)])
def test_too_many_tiles(rows, cols):
    lib = m.load()
    at = [ctypes.c_void_p((i + 1) * FAR) for i in range(6)]
    rc = lib.fp8_act_quantize(at[0], 2 * cols, rows, 1, cols, 1, 1, 0, at[1], at[2], None, None, None, None,
                              None)
    assert rc == 4 and "tiles" in m.fp8_last_error()
    rc = lib.fp8_act_quantize_bwd(at[0], cols, at[1], at[2], rows, 1, cols, 1, 1, 0, at[3], at[4], None,
                                  None, None, None)
    assert rc == 4 and "tiles" in m.fp8_last_error()


def test_the_largest_are_not_refused_for_it():
    """2^23 - 64 tiles: refused for another reason here (the codes lie on h)."""
    lib = m.load()
    rows, cols = 1 << 22, (1 << 15) - 128
    assert rows // 128 * (cols // 128) <= (1 << 23) - 64
    rc = lib.fp8_act_quantize(ctypes.c_void_p(FAR), 2 * cols, rows, 1, cols, 1, 1, 0, ctypes.c_void_p(FAR),
                              ctypes.c_void_p(2 * FAR), None, None, None, None, None)
    assert rc == 4 and "shares memory" in m.fp8_last_error()
