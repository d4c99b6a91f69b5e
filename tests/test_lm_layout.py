"""Shared memory of the 8-bit product: what the kernels lay out lies inside what their launches ask for, wherever the
dynamic shared memory begins (host arithmetic, no GPU needed)."""

import os
import shutil
import subprocess

import pytest

from kronecker_factored_second_gb300 import build

PROGRAM = r"""
#include <stdio.h>
#include "okls_fp8_layout.h"
using namespace okls;
// bytes from the rounded-up base to the end of the barriers and the TMEM address
template <int BN>
long one_cta() {
  typedef Tile<BN> T;
  const long bars = 2L * T::kRing + 2L * T::kSlots + 2L * Buffers<BN>::kCount + 1;
  return T::kRing * (long)T::kBytes + T::kSlots * (long)T::kScaleBytes + 8 * bars + 4;
}
int main() {
  const long pair_bars = 2L * kPairRing + 2L * kPairSlots + 2L * Buffers<kPN>::kCount + 2;
  const long pair = kPairRing * (long)kPairStage + 8L * kOutWarp + kPairSlots * (long)kPairScaleBytes + 8 * pair_bars + 4;
  printf("%ld %ld %ld %ld %ld %ld\n", one_cta<64>(), (long)Tile<64>::kSmem, one_cta<128>(), (long)Tile<128>::kSmem, pair,
         (long)kPairSmem);
}
"""


def test_barriers_lie_inside_the_launch(tmp_path):
    cxx = os.environ.get("CXX") or shutil.which("g++")
    if not cxx:
        pytest.skip("no host compiler")
    src, exe = tmp_path / "layout.cpp", tmp_path / "layout"
    src.write_text(PROGRAM)
    cuda = os.path.dirname(os.path.dirname(build.nvcc()))
    subprocess.run([cxx, "-std=c++17", "-I" + build.CSRC, "-I" + os.path.join(cuda, "include"), str(src), "-o", str(exe)],
                   check=True)
    v = [int(t) for t in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()]
    for used, given in zip(v[::2], v[1::2]):
        # dynamic shared memory is aligned to 16 bytes at least; the kernels round its start up to 1024
        assert used + 1024 - 16 <= given <= 227 * 1024, (used, given)
