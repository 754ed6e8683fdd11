"""Offsets of the products' loads to shared memory, on the CPU: compiled from
the header that the kernels use.  No load may reach past the operand, whatever
the hardware's range check makes of the scalar offset."""
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "nonlinear_rnn_evaluation_newton_amd",
                    "csrc")

DRIVER = r"""
#include <cstdint>
#include <cstdio>
#include <initializer_list>
#include "direct_rows.h"
// Every load of every lane of a tile with `rows` rows of the operand, each of
// `k` bytes, `ld` bytes apart.  The vector offset alone must be outside the
// resource (rows * ld bytes) or the 16 bytes must be k0 + chunk of a row that exists.
int main() {
  long inside = 0;
  for (int tile : {128, 256})
    for (int rows = 1; rows <= tile; rows += rows < 20 ? 1 : 13)
      for (unsigned k : {16u, 112u, 128u, 272u, 2064u})
        for (unsigned ld : {k, k + 16, k + 4096}) {
          for (int u = 0; u < tile / 8; u++)
            for (int lane = 0; lane < 64; lane++) {
              const unsigned off = pr::direct_offset(u, lane, rows, ld);
              const int c = pr::direct_chunk(u, lane), row = u * 8 + lane / 8;
              if (c < 0 || c > 112 || c % 16) return printf("chunk %d\n", c), 1;
              for (unsigned k0 = 0; k0 < k; k0 += 128) {
                const unsigned v = k0 + c < k ? off : pr::DIRECT_OOB;
                if (v >= (unsigned)rows * ld) {  // nothing is read, with or without the scalar offset
                  if (v < 0x7fffffffu || (row < rows && k0 + c < k)) return printf("row %d of %d left out\n", row, rows), 1;
                  continue;
                }
                const uint64_t at = (uint64_t)v + k0;
                if (row >= rows || at != (uint64_t)row * ld + k0 + c || k0 + c + 16 > k)
                  return printf("tile %d rows %d ld %u k %u: load %d lane %d reads byte %llu\n", tile, rows, ld, k, u,
                                lane, (unsigned long long)at), 1;
                if (k0 >= (unsigned)rows * ld) return printf("scalar offset past the resource\n"), 1;
                inside++;
              }
            }
        }
  // the chunks of a row are fetched once each
  for (int u = 0; u < 32; u++)
    for (int r = 0; r < 8; r++) {
      unsigned seen = 0;
      for (int q = 0; q < 8; q++) seen |= 1u << (pr::direct_chunk(u, r * 8 + q) / 16);
      if (seen != 255) return printf("row %d of load %d: chunks %x\n", r, u, seen), 1;
    }
  printf("ok %ld\n", inside);
  return 0;
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_direct_loads_stay_in_their_rows(tmp_path):
    src, exe = tmp_path / "driver.cpp", tmp_path / "driver"
    src.write_text(DRIVER)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and r.stdout.startswith("ok"), r.stdout


@pytest.mark.parametrize("kernel", ["k_gemm.hip", "k_gemm_i8.hip"])
def test_kernels_take_their_offsets_from_it(kernel):
    text = open(os.path.join(CSRC, kernel)).read()
    loads = text.count("__builtin_amdgcn_raw_ptr_buffer_load_lds(")
    assert loads > 0 and text.count("direct_offset(") == loads
