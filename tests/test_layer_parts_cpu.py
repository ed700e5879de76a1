"""The parts that a dense layer's sum is cut into (csrc/parts.hpp), compiled for the host: together they are the sum,
each tile once and in order, and no part, an empty one neither, starts outside of the sum's segments."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = r"""
#include <cstdio>
#include "parts.hpp"
using gnnmb::part_of_sum;
int main() {
    for (int64_t seg_tiles = 0; seg_tiles <= 40; ++seg_tiles)
        for (int segs = 1; segs <= 4; ++segs)
            for (int64_t parts = 1; parts <= 64; ++parts) {
                int64_t next = 0;
                for (int64_t part = 0; part < parts; ++part) {
                    const auto p = part_of_sum(seg_tiles, segs, parts, part);
                    const bool placed = p.seg >= 0 && p.seg < segs && p.tile >= 0 && (p.tile < seg_tiles || seg_tiles == 0);
                    const bool follows = p.steps >= 0 && p.first == next &&
                                         (p.steps == 0 || p.seg * seg_tiles + p.tile == p.first);
                    if (!placed || !follows) {
                        std::printf("%d tiles x %d, part %d of %d: first %d, steps %d, segment %d, tile %d\n", (int)seg_tiles,
                                    segs, (int)part, (int)parts, (int)p.first, (int)p.steps, (int)p.seg, (int)p.tile);
                        return 1;
                    }
                    next += p.steps;
                }
                if (next != seg_tiles * segs) return 2;
            }
    return 0;
}
"""


def test_parts_of_a_sum(tmp_path):
    src, exe = tmp_path / "parts.cpp", tmp_path / "parts"
    src.write_text(PROGRAM)
    subprocess.check_call(["g++", "-std=c++17", "-Wall", "-Werror", "-I",
                           os.path.join(ROOT, "graph_mini_pipeline_amd", "csrc"), str(src), "-o", str(exe)])
    run = subprocess.run([str(exe)], stdout=subprocess.PIPE, text=True)
    assert run.returncode == 0, run.stdout
