"""How the order by expert shares its work out (csrc/sort_layout.h), checked on the host: every count of
every block is added up once, whatever the numbers of experts and blocks, with no division by zero."""

import os
import shutil
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = r"""
#include <stdio.h>
#include <vector>
#include "sort_layout.h"
using namespace dlrm;

static int check(bool ok, const char* what, int a, int b)
{
    if (!ok) printf("%s: %d, %d\n", what, a, b);
    return !ok;
}

int main()
{
    // few experts and few blocks: more parts than blocks; 256 experts: a part of every thread but some
    for (int E : {1, 2, 3, 7, 16, 33, 64, 100, 170, 171, 255, 256})
        for (int blocks = 2; blocks <= kSortBlocks; blocks += blocks < 40 ? 1 : 11)
            for (int block = 0; block < blocks; block += 1 + blocks / 5) {
                const int bins = E + 1;
                std::vector<int> seen((size_t)blocks * bins);
                for (int t = 0; t < kSortThreads; ++t) {
                    const CountShare s = count_share(t, bins, blocks, block);
                    for (int i = 0; i < s.rows; ++i) {
                        const int b = s.block(i);
                        if (check(b >= 0 && b < blocks && s.bin >= 0 && s.bin < bins, "outside", E, blocks)) return 1;
                        ++seen[(size_t)b * bins + s.bin];
                    }
                }
                for (int n : seen)
                    if (check(n == 1, "not once", E, blocks)) return 1;
            }
    // the blocks' chunks hold the choices, in whole parts of the warps
    for (int64_t n : {(int64_t)0, (int64_t)1, (int64_t)511, (int64_t)4096, (int64_t)4097, (int64_t)6144, (int64_t)262144,
                      (int64_t)262145, (int64_t)1 << 30, (int64_t)2147483647 - (1 << 20)}) {
        const SortShape z = sort_shape(n);
        if (check(z.blocks >= 1 && z.blocks <= kSortBlocks && z.chunk % kSortThreads == 0, "shape", (int)n, z.blocks)) return 1;
        if (check(z.blocks * z.chunk >= n && (z.blocks - 1) * z.chunk <= n, "chunks", (int)n, z.blocks)) return 1;
        if (check((z.blocks == 1) == (n <= kSortOne), "one block", (int)n, z.blocks)) return 1;
    }
    puts("ok");
    return 0;
}
"""


def test_every_count_is_added_up_once(tmp_path):
    (tmp_path / "l.cpp").write_text(SOURCE)
    # a division by zero ends the program, on machines whose division does not, too
    subprocess.run([shutil.which("g++") or "c++", "-std=c++17", "-O1", "-fsanitize=integer-divide-by-zero",
                    "-fsanitize-undefined-trap-on-error", "-I", os.path.join(ROOT, "dlrm_embeddings_dot_gb300", "csrc"), "-o",
                    str(tmp_path / "l"), str(tmp_path / "l.cpp")], check=True)
    r = subprocess.run([str(tmp_path / "l")], capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.strip() == "ok", (r.returncode, r.stdout)
