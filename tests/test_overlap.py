"""The host's check of overlapping arguments (ndq_overlap.h) against sets of
bytes: pieces and rows of every small layout, with one stride or two."""
import os
import shutil
import subprocess

import pytest

import quantized_weight_block_gb300 as ndq

SOURCE = """
#include <cstdio>
#include <cstring>
#include "ndq_overlap.h"
static unsigned seed = 1;
static int below(int n) { seed = seed * 1664525u + 1013904223u; return static_cast<int>((seed >> 8) % static_cast<unsigned>(n)); }
int main() {
    static char bytes[4096];
    long yes = 0, n = 400000;
    for (long c = 0; c < n; ++c) {
        ndq::Rows r[2];
        const int shared = below(40) + 1;
        for (auto& x : r) {
            x.rows = below(5) == 0 ? 1 : below(9);
            x.bytes = below(14);
            x.stride = (below(2) ? shared : below(40) + 1) + 0;
            if (x.stride < x.bytes) x.stride = x.bytes;
            x.p = bytes + below(400);
        }
        bool mark[4096] = {}, want = false;
        for (int i = 0; i < r[0].rows; ++i)
            for (int e = 0; e < r[0].bytes; ++e) mark[static_cast<const char*>(r[0].p) - bytes + i * r[0].stride + e] = true;
        for (int i = 0; i < r[1].rows; ++i)
            for (int e = 0; e < r[1].bytes; ++e) want = want || mark[static_cast<const char*>(r[1].p) - bytes + i * r[1].stride + e];
        yes += want;
        if (overlap(r[0], r[1]) != want || overlap(r[1], r[0]) != want) {
            for (auto& x : r) std::printf("at %ld, %ld rows of %ld every %ld\\n", static_cast<long>(static_cast<const char*>(x.p) - bytes), static_cast<long>(x.rows), static_cast<long>(x.bytes), static_cast<long>(x.stride));
            std::printf("case %ld: want %d\\n", c, want);
            return 1;
        }
    }
    // the largest rows and strides of a call
    const ndq::Rows far{reinterpret_cast<const void*>(uintptr_t(1) << 40), 8192, INT64_C(2147483647), INT64_C(1) << 42};
    const ndq::Rows near{reinterpret_cast<const void*>((uintptr_t(1) << 40) + 8192), 1024, INT64_C(2147483647), INT64_C(1) << 42};
    if (overlap(far, near) || !overlap(far, far)) return 2;
    std::printf("%ld of %ld overlap\\n", yes, n);
    return yes > n / 10 && yes < n - n / 10 ? 0 : 3;
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_against_sets_of_bytes(tmp_path):
    src, exe = tmp_path / "overlap.cpp", tmp_path / "overlap"
    src.write_text(SOURCE)
    csrc = os.path.join(os.path.dirname(ndq.__file__), "csrc")
    subprocess.run(["g++", "-O2", "-std=c++17", "-Wall", "-Wextra", "-I", csrc, str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout
