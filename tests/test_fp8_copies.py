"""Where the LDS-tiled 8-bit product's copies read, walked on the CPU: the
offsets come from the header that the kernel takes them from
(``csrc/fp8_copies.h``), compiled into a small host program.

Weights: every lane's 16 bytes of every copy of a tile lie inside the matrix,
also where N ends inside the tile.  Scales: the vector offset alone is the
distance from the base, so that the buffer bound, which is compared with it,
covers it."""

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = r"""
#include <cstdio>
#include <initializer_list>
#include "fp8_copies.h"
using namespace lmoe;

static int fail(const char* what, long a, long b) {
  std::printf("%s: %ld, %ld\n", what, a, b);
  return 1;
}

// tiles of bn weight rows, eight waves, two halves of bh rows in nih copies
static int weights(int bn, long N, long K) {
  const int bh = bn / 2, nih = bh / 64;
  for (long n0 = 0; n0 < N; n0 += bn)
    for (int h = 0; h < 2; ++h)
      for (int w = 0; w < 8; ++w)
        for (int j = 0; j < nih; ++j)
          for (int kb : {0L, K / 128 - 1})
            for (int lane = 0; lane < 64; ++lane) {
              const int row = h * bh + (w + 8 * j) * 8;
              const int left = (int)(N - n0);
              const long s = fp8_weight_scalar(row, left, kb, (int)K);
              const long at = n0 * K + s + fp8_weight_lane(lane, (lane & 7) * 16, (uint32_t)K);
              if (at < 0 || at + 16 > N * K) return fail("weights past the matrix", at, N * K);
              // rows that are stored are read from their own place
              if (row + 7 < left && s != kb * 128 + row * K) return fail("moved", row, left);
            }
  return 0;
}

static int scales(int KB) {
  for (int g = 0; g <= KB / 8 + 1; ++g)
    for (int i = 0; i < 32; ++i)
      for (int lane = 0; lane < 64; ++lane) {
        // place lane % 8 of row 8 i + lane / 8 holds block (lane % 8) ^ 4 (i % 2)
        const long want = 1000L * KB * 4 + (8L * g + ((lane & 7) ^ (4 * (i & 1)))) * 4;
        if (fp8_xscale_lane(1000u * KB * 4, lane, i, g) != want) return fail("token scale", g, lane);
      }
  for (int b = 0; b < 2; ++b)
    for (int i = 0; i < 4; ++i)
      for (int lane = 0; lane < 64; ++lane)
        if (fp8_wscale_lane(lane, b, i, KB) != (b * KB + i * 64L + lane) * 4)
          return fail("weight scale", b, lane);
  return 0;
}

int main() {
  for (int bn : {128, 256})
    for (long N : {16, 32, 48, 112, 128, 144, 240, 256, 272, 400, 784, 1040, 10256})
      for (long K : {128, 384, 8192})
        if (weights(bn, N, K)) return 1;
  // the largest: offsets stay within 31 bits
  if (weights(256, 16, 65536) || weights(256, 256, 65536) || weights(256, 496, 65536)) return 1;
  for (int KB : {1, 3, 8, 9, 64, 256, 512})
    if (scales(KB)) return 1;
  return 0;
}
"""


def test_copies_stay_inside_their_arrays(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host C++ compiler")
    src, exe = tmp_path / "copies.cpp", tmp_path / "copies"
    src.write_text(PROGRAM)
    inc = os.path.join(ROOT, "sparse_moe_layer_latentmoe_amd", "csrc")
    subprocess.run([cxx, "-std=c++17", "-O1", "-Wall", "-I", inc, str(src), "-o", str(exe)],
                   check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout
