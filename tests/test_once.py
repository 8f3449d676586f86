"""What the launchers ask of a device once (ndq_once.h), by many threads at a
time, under the thread sanitizer: two words written one after the other, as a
plain pair of fields, are reported as a race there."""
import os
import shutil
import subprocess

import pytest

import quantized_weight_block_gb300 as ndq

ONCE = """
#include "ndq_once.h"
static ndq::Once cached[64];
static int resident(int i) {
    int v = 0;
    return cached[i].get([&](int* n) { *n = 152 * (i + 1); return 0; }, &v) == 0 ? v : -1;
}
"""
PAIR = """
struct { int sms = 0, ctas = 0; } cached[64];
static int resident(int i) {
    if (cached[i].ctas == 0) {
        cached[i].sms = 152;
        cached[i].ctas = i + 1;
    }
    return cached[i].sms * cached[i].ctas;
}
"""
MAIN = """
#include <atomic>
#include <thread>
#include <vector>
int main() {
    std::atomic<int> waiting{8}, bad{0};
    std::vector<std::thread> threads;
    for (int t = 0; t < 8; ++t)
        threads.emplace_back([&] {
            for (--waiting; waiting > 0;) {}
            for (int i = 0; i < 64; ++i) bad += resident(i) != 152 * (i + 1);
        });
    for (auto& t : threads) t.join();
    return bad != 0;
}
"""


def run(code, tmp_path, name):
    src, exe = tmp_path / f"{name}.cpp", tmp_path / name
    src.write_text(code + MAIN)
    csrc = os.path.join(os.path.dirname(ndq.__file__), "csrc")
    flags = ["-O1", "-g", "-std=c++17", "-fsanitize=thread", "-pthread", "-I", csrc]
    if subprocess.run(["g++", *flags, str(src), "-o", str(exe)], capture_output=True).returncode:
        return None
    return subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_many_threads_at_once(tmp_path):
    pair = run(PAIR, tmp_path, "pair")
    if pair is None or "data race" not in pair.stderr:
        pytest.skip("no working thread sanitizer")
    once = run(ONCE, tmp_path, "once")
    assert once is not None and once.returncode == 0, once and once.stderr


def test_a_failure_is_passed_on_and_asked_again(tmp_path):
    src, exe = tmp_path / "fail.cpp", tmp_path / "fail"
    src.write_text("""
#include "ndq_once.h"
int main() {
    ndq::Once o;
    int v = 7, asked = 0;
    if (o.get([&](int*) { ++asked; return 3; }, &v) != 3 || v != 7) return 1;
    for (int i = 0; i < 2; ++i)
        if (o.get([&](int* n) { ++asked; *n = 5; return 0; }, &v) != 0 || v != 5) return 2;
    return asked == 2 ? 0 : 3;
}
""")
    csrc = os.path.join(os.path.dirname(ndq.__file__), "csrc")
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Wextra", "-I", csrc, str(src), "-o", str(exe)], check=True)
    assert subprocess.run([str(exe)]).returncode == 0
