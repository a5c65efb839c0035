"""The bounds of what the join of the shared-prefix attention reads (csrc/prefix_join.h), compiled for the
host: for every entry that a workspace may hold, the slots, rows and dimensions that the kernel
derives from it lie within the partials, and an entry that the attention kernel wrote is kept as it is."""
from __future__ import annotations

import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "mixed_precision_kv_arkv_b200", "csrc")

HARNESS = r"""
#include <climits>
#include <cstdio>
#include <initializer_list>
#include "prefix_join.h"
using namespace arkv;
int main() {
    const int kRows = 128, kBatch = 5;
    long long checked = 0;
    for (int slots : {1, 2, 193, 200, 5000})
        for (int row_tiles = 1; row_tiles <= 2; ++row_tiles)
            for (int G = 1; G <= 4; ++G) {
                const int n = row_tiles * kRows;
                const int any[] = {INT_MIN, INT_MIN + 1, -1 << 24, -129, -128, -5, -4, -3, -2, -1, 0, 1, 2, 3, 4, 5, 63, 124, 125, 126, 127,
                                   128, 129, 191, 192, 193, 199, 200, 252, 253, 254, 255, 256, 257, 4999, 5000, 5001, 0x3f800000,
                                   0x7f800000, (int)0xff800000, 0x7fffffc0, INT_MAX - 20, INT_MAX - 3, INT_MAX - 1, INT_MAX};
                for (int x : any)
                    for (int y : any)
                        for (int z : any) {
                            const JoinSpan s = join_span(x, y, z, slots, row_tiles, kRows, G);
                            const bool good = x >= 0 && y >= x && y < slots && z >= 0 && z <= n - G;
                            if (good && (s.first != x || s.last != y || s.row != z)) return std::printf("changed %d %d %d\n", x, y, z), 1;
                            if (y < x && s.last >= s.first)
                                return std::printf("not empty %d %d\n", x, y), 1;
                            if (s.first < 0 || s.first > slots || s.last >= slots || s.row < 0)
                                return std::printf("span %d %d %d\n", x, y, z), 1;
                            if (s.last < s.first) continue;
                            // the largest place of part_ml, and of part_o's [slot][tile][D / 4][row], that a thread reads
                            for (int d4 : {16, 32})
                                for (int q = 0; q < G; ++q) {
                                    const long long ml = ((long long)s.last * row_tiles + s.row / kRows) * kRows + s.row % kRows + q;
                                    const long long o = (((long long)s.last * row_tiles + s.row / kRows) * d4 + d4 - 1) * kRows + s.row % kRows + q;
                                    if (ml >= (long long)slots * n || o >= (long long)slots * n * d4) return std::printf("past %d %d %d\n", x, y, z), 1;
                                    ++checked;
                                }
                            // the loop's last step: c + 4 * kBatch stays an int
                            if ((long long)s.last + 3 + 4 * kBatch > INT_MAX) return std::printf("loop %d\n", s.last), 1;
                        }
            }
    std::printf(checked > 100000 ? "ok\n" : "few\n");
    return 0;
}
"""


def test_join_reads_stay_within_the_workspace(tmp_path):
    src, exe = tmp_path / "join_check.cpp", tmp_path / "join_check"
    src.write_text(HARNESS)
    subprocess.run([os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert out.returncode == 0 and out.stdout.strip() == "ok", out.stdout + out.stderr
