"""The FP8 GEMM's copies into LDS: every lane's address, on the CPU.

A buffer load adds a lane offset and a wave offset to its descriptor's base.
What the range check does with the wave offset is taken in every way that it
could be: left out, added, or subtracted from the size (modulo 2^32).  In each,
a row of the operand has to be read from its own place and a row past it has to
be out of range; the same after the last stage, where the size is zero."""
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "w4a4_integer_gemm_amd", "csrc")

SRC = r"""
#include <cstdint>
#include <cstdio>
#include "fq_fp8_copy.h"

// out of range under any reading of the check / in range under every one
static bool out_by(int rule, uint32_t lane, uint32_t common, uint32_t size) {
    if (rule == 0) return lane >= size;
    if (rule == 1) return uint64_t(lane) + common >= size;
    return lane >= size - common;
}

int main() {
    long checked = 0, bad_row = 0, bad_past = 0, bad_end = 0;
    const int tile_rows[] = {64, 96, 128, 160, 192, 256}, Ks[] = {128, 384, 3584, 65536};
    const int left[] = {1, 7, 8, 9, 63, 64, 71, 120, 129, 250, 256, 1000};  // rows from the tile's first on
    for (int K : Ks)
        for (int tile : tile_rows)
            for (int l : left) {
                const int rows = l < tile ? l : tile, nu = K / 128;
                const uint32_t size = uint32_t(rows) * uint32_t(K);
                for (int row0 = 0; row0 < tile; row0 += 8)
                    for (int lane = 0; lane < 64; ++lane) {
                        const uint32_t part = fq::fp8_copy_lane(lane, (row0 / 8) & 1, K);
                        const int row = row0 + lane / 8, chunk = (lane & 7) ^ fq::fp8_swizzle(row);
                        const int units[] = {0, 1 < nu ? 1 : 0, nu / 2, nu - 1};
                        for (int u : units) {
                            const fq::Fp8CopyOffset at = fq::fp8_copy_at(part, row0, u, K);
                            const uint64_t want = uint64_t(row) * K + 128 * u + 16 * chunk;
                            for (int rule = 0; rule < 3; ++rule, ++checked) {
                                const bool out = out_by(rule, at.lane, at.common, size);
                                if (row < rows)
                                    bad_row += out || uint64_t(at.lane) + at.common != want;
                                else
                                    bad_past += !out;
                            }
                        }
                        const fq::Fp8CopyOffset end = fq::fp8_copy_at(part, row0, 0, K);  // (past the last stage)
                        for (int rule = 0; rule < 3; ++rule) bad_end += !out_by(rule, end.lane, end.common, 0);
                    }
            }
    printf("%ld %ld %ld %ld\n", checked, bad_row, bad_past, bad_end);
    return 0;
}
"""


def test_rows_past_an_operand_are_out_of_range_whatever_the_check_counts(tmp_path):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no g++")
    src, exe = tmp_path / "copy.cpp", tmp_path / "copy"
    src.write_text(SRC)
    subprocess.run([cxx, "-std=c++17", "-O1", "-Wall", f"-I{CSRC}", str(src), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()
    checked, bad_row, bad_past, bad_end = (int(v) for v in out)
    assert checked > 1_000_000
    assert (bad_row, bad_past, bad_end) == (0, 0, 0)

