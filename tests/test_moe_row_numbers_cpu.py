"""The expert sort's row arithmetic at the end of 32 bits, without a GPU: csrc/moe_rows.h, which the
kernel uses, compiled for the host and held against Python's integers. fp8_moe_rows lets through
every buffer of less than 2^31 rows, so an expert's padded count may be as large as that."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

import scaled_fp8_linear_amd as m
from scaled_fp8_linear_amd import build

SOURCE = r"""
#include "moe_rows.h"
extern "C" int32_t padded(int32_t n, int32_t multiple) { return fp8lin::padded_count(n, multiple); }
// the lane's rows into out, `room` of them at most; returns how many there would be (to 4 room)
extern "C" int32_t padding_rows(int32_t from, int32_t to, int32_t lane, int32_t* out, int32_t room) {
  int32_t n = 0;
  struct Enough {};
  try {
    fp8lin::each_padding_row(from, to, lane, [&](int32_t r) {
      if (n < room) out[n] = r;
      if (++n >= 4 * room) throw Enough();
    });
  } catch (const Enough&) {
  }
  return n;
}
"""
LAST = 2 ** 31 - 1


@pytest.fixture(scope="module")
def rows(tmp_path_factory):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no g++")
    d = tmp_path_factory.mktemp("moe_rows")
    (d / "rows.cpp").write_text(SOURCE)
    so = str(d / "rows.so")
    # -fwrapv: an overflow shows as a wrong number rather than as anything
    subprocess.run([cxx, "-std=c++17", "-O1", "-fwrapv", "-fPIC", "-shared", f"-I{build.CSRC}",
                    str(d / "rows.cpp"), "-o", so], check=True)
    return ctypes.CDLL(so)


@pytest.mark.parametrize("n,multiple", [
    (0, 1), (0, 16), (0, LAST), (1, 16), (16, 16), (17, 16), (5, 3), (LAST, 1), (LAST - 15, 16),
    (LAST - 30, 16), (2147483600, 100), (2147483501, 100), (600_000_000, 1_610_000_000),
    (1, LAST), (2, LAST), (LAST - 1, LAST), (LAST, LAST), ((1 << 30) + 1, (1 << 30) + 1)])
def test_padded_count(rows, n, multiple):
    want = -(-n // multiple) * multiple
    assert want <= LAST
    assert rows.padded(n, multiple) == want


@pytest.mark.parametrize("start,end", [(0, 0), (0, 1), (0, 15), (3, 40), (LAST, LAST),
                                       (LAST - 1, LAST), (LAST - 99, LAST), (LAST - 100, LAST - 5),
                                       (LAST - 47, LAST - 15)])
def test_padding_rows_are_each_named_once(rows, start, end):
    room = 16
    out = np.zeros(room, np.int32)
    got = []
    for lane in range(16):
        n = rows.padding_rows(start, end, lane, out.ctypes.data_as(ctypes.c_void_p), room)
        assert n <= room, "goes on past the rows"
        got += out[:n].tolist()
    assert sorted(got) == list(range(start, end))


def test_such_buffers_are_let_through():
    if not os.path.exists(build.LIB):
        pytest.skip("libfp8lin.so not built (python -m scaled_fp8_linear_amd.build)")
    assert m.fp8_moe_rows(2147483600, 1, 1, 100) == 2147483600
    assert m.fp8_moe_rows(600_000_000, 1, 1, 1_610_000_000) == 1_610_000_000
    assert m.fp8_moe_rows(1, 2, 1, LAST) == LAST
