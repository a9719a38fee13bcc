"""How the sort of routed entries is split over blocks and threads, without a GPU: the header
that holds it has no CUDA in it."""
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "muon_newton_schulz_step_gb300", "csrc")

PROGRAM = """
#include <cstdio>
#include "sort_split.h"
using namespace muon;
int main() {
    for (long long n = 0; n <= 300000; n += n < 5000 ? 1 : 997) {
        const int blocks = sort_blocks(n);
        if ((blocks == 0) != (n <= kSortAlone) || blocks > kSortMaxBlocks) return std::printf("blocks of %lld\\n", n), 1;
        for (int buckets = 2; blocks > 0 && buckets <= 1025; ++buckets) {
            const int parts = sort_parts(blocks, buckets);
            if (parts < 1 || parts > blocks || (parts > 1 && parts * buckets > kSortThreads))
                return std::printf("%d parts, %d blocks, %d buckets\\n", parts, blocks, buckets), 1;
            int all = 0;
            for (int part = 0; part < parts; ++part) {
                const int rows = sort_part_rows(blocks, parts, part);   // the kernel takes the block's number modulo this
                if (rows < 1 || part + (rows - 1) * parts >= blocks)
                    return std::printf("%d rows of part %d of %d, %d blocks\\n", rows, part, parts, blocks), 1;
                all += rows;
            }
            if (all != blocks) return std::printf("%d of %d rows\\n", all, blocks), 1;
        }
    }
    return 0;
}
"""


def test_every_part_of_the_table_has_rows(tmp_path):
    compiler = shutil.which("g++") or shutil.which("c++")
    if compiler is None:
        pytest.skip("no host compiler")
    source, program = tmp_path / "split.cpp", tmp_path / "split"
    source.write_text(PROGRAM)
    subprocess.run([compiler, "-std=c++17", "-I", CSRC, str(source), "-o", str(program)], check=True, timeout=120)
    r = subprocess.run([str(program)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout
