"""Rows of a launch: no launch of the log probabilities' backward asks for more work
items than a dispatch counts (32 bits).  The arithmetic is compiled for the host."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "quantized_fine_tuning_nf4_amd", "csrc")

MAIN = r"""
#include <cstdio>
#include <cstdlib>
#include "launch_rows.h"
int main(int, char** a) {
  std::printf("%lld", (long long)qn::rows_per_launch(std::atoll(a[1]), std::atoll(a[2])));
}
"""


def test_a_launch_counts_its_work_items(tmp_path):
    src, exe = tmp_path / "m.cpp", tmp_path / "m"
    src.write_text(MAIN)
    subprocess.run(["g++", "-std=c++17", "-I", CSRC, str(src), "-o", str(exe)], check=True)

    def rows(chunks, threads=256):
        return int(subprocess.run([str(exe), str(chunks), str(threads)], check=True,
                                  capture_output=True, text=True).stdout)

    for threads in (64, 256, 1024):
        for chunks in (1, 2, 3, 7, 1000, 65536, (1 << 22) - 1):
            n = rows(chunks, threads)
            assert n >= 1
            assert n == 1 or n * chunks * threads < 1 << 32
            assert n * chunks < 1 << 31
            # and no fewer than fit
            assert (n + 1) * chunks * threads >= 1 << 32 or (n + 1) * chunks >= 1 << 31
    # 2^23 rows of 8193 bf16 or 4097 fp32 logits: two workgroups a row, 2^24 in all
    assert 1 << 22 < rows(2) < 1 << 23
    # the most logits a row may hold: 2^28, by 4 vectors of 4 fp32 for 256 threads
    assert rows((1 << 28) // (256 * 16)) * (1 << 16) * 256 < 1 << 32


def test_the_backward_uses_it():
    body = open(os.path.join(CSRC, "logprob.hip")).read().split("hipError_t launch_logprobs_bwd")[1]
    assert "rows_per_launch(chunks, kThreads)" in body
