"""What the launchers keep per device is shared by host threads: csrc/device_figure.h under the compiler's race detector
(no GPU needed), and its use by the launchers."""
import os
import re
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "rht_bit_block_gb300", "csrc")
PROGRAM = r"""
#include <cstdio>
#include <thread>
#include <vector>
#include "device_figure.h"
int main() {
    int wrong[8] = {};
    for (int round = 0; round < 200; ++round) {
        static ufp4::DeviceFigure figures[200];
        std::vector<std::thread> threads;
        for (int i = 0; i < 8; ++i)
            threads.emplace_back([&, i] {
                for (int d = -1; d <= 64; ++d) {
                    const bool inside = d >= 0 && d < 64;
                    if (figures[round].get(d, [&] { return d + 1; }) != (inside ? d + 1 : 0)) ++wrong[i];
                    if (inside && figures[round].get(d, [] { return -5; }) != d + 1) ++wrong[i];   // kept
                }
            });
        for (auto& t : threads) t.join();
    }
    ufp4::DeviceFigure failing;
    int bad = failing.get(0, [] { return 0; }) + failing.get(0, [] { return -1; });
    bad += failing.get(0, [] { return 7; }) != 7;                                               // a failure is not kept
    for (int w : wrong) bad += w;
    std::printf("%d wrong\n", bad);
    return bad != 0;
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="no host compiler")
def test_threads_that_ask_at_once(tmp_path):
    source, program = tmp_path / "figure.cpp", tmp_path / "figure"
    source.write_text(PROGRAM)
    command = ["g++", "-std=c++17", "-O1", "-pthread", "-I", CSRC, str(source), "-o", str(program)]
    detector = subprocess.run([*command, "-fsanitize=thread"], capture_output=True, text=True)
    if detector.returncode:
        subprocess.run(command, check=True)
    run = subprocess.run([str(program)], capture_output=True, text=True, timeout=120)
    if "FATAL: ThreadSanitizer" in run.stderr:  # the detector does not start on this kernel's memory layout
        subprocess.run(command, check=True)
        run = subprocess.run([str(program)], capture_output=True, text=True, timeout=120)
    assert run.returncode == 0, run.stdout + run.stderr


def test_launchers_keep_no_bare_static_numbers():
    """A function's static that is not constant, a lock, or one of the above is written by every thread that calls it."""
    found = []
    for name in sorted(os.listdir(CSRC)):
        text = open(os.path.join(CSRC, name)).read()
        found += [(name, m.group(0).strip()) for m in
                  re.finditer(r"^[ \t]+static (?!const|inline|__device__|std::mutex|std::atomic|DeviceFigure)[\w:]+[ *]+"
                              r"\w+(?:\[[^\]]*\])?\s*(?:=[^;(]*)?;", text, re.M)]
    assert found == [("api.cu", "static bool done[64];")], found   # under ensure_loaded's lock
