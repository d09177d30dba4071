"""The 4-bit products' choice of tile, split and grid (mx_fp4_choice.h, host code) on devices of any number of SMs."""
from __future__ import annotations

import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# The kernel joins the partial sums of one unit to a cluster: fewer clusters than units would leave some unwritten.
SOURCE = r"""
#include "mx_fp4_choice.h"
#include <cstdio>
using namespace mx::fp4;
int main()
{
    const int rows[] = {1, 2, 16, 17, 31, 64, 65, 128, 200, 449, 1000, 5000}, stages[] = {1, 8, 15, 16, 17, 18, 40, 4096};
    long bad = 0, eights = 0, fours = 0;
    for (int sms = 1; sms <= 160; ++sms)
        for (int r : rows)
            for (int KB : stages)
                for (int FT = 1; FT <= 64; ++FT) {
                    const Choice c = choose(r, false, 1, FT, KB, sms);
                    const long units = (long)((r + c.nt - 1) / c.nt) * FT;
                    const bool ok = c.grid >= 1 && c.grid <= sms && c.grid % c.cl == 0 && (c.cl == 1 || c.grid / c.cl == units);
                    if (!ok && bad++ < 5)
                        std::printf("%d SMs, %d rows, %d tiles, %d stages: tile %d, cluster %d, grid %d\n", sms, r, FT, KB, c.nt,
                                    c.cl, c.grid);
                    if (sms == 152)
                        eights += c.cl == 8, fours += c.cl == 4;
                    // (the split of eight where its clusters have room)
                    if (units <= 8 && KB >= 16 && 8 * units <= sms && c.cl != 8 && bad++ < 5)
                        std::printf("%d SMs, %d rows, %d tiles, %d stages: cluster %d\n", sms, r, FT, KB, c.cl);
                    const Choice g = choose(r, true, FT, FT, KB, sms);
                    if ((g.cl != 1 || g.grid < 1 || g.grid > sms) && bad++ < 5)
                        std::printf("grouped: %d SMs, %d rows: cluster %d, grid %d\n", sms, r, g.cl, g.grid);
                }
    std::printf("%ld %ld %ld\n", bad, eights, fours);
    return 0;
}
"""


def test_a_cluster_has_one_unit_on_any_device(tmp_path):
    src, exe = tmp_path / "choice.cpp", tmp_path / "choice"
    src.write_text(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-I", os.path.join(ROOT, "expert_ffn_gb300", "csrc"),
                    str(src), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout
    bad, eights, fours = map(int, out.splitlines()[-1].split())
    assert bad == 0, out
    assert eights and fours
