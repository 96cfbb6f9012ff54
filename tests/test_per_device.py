"""What the launchers keep from a first launch is safe for several host threads.
CPU only."""
import os
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "fp8_linear_layer_gb300", "csrc")

PROGRAM = r"""
#include <thread>
#include <vector>
#include "per_device.h"

static fp8ll::PerDevice value;

int main() {
    std::vector<std::thread> threads;
    std::atomic<int> wrong{0};
    for (int t = 0; t < 8; ++t)
        threads.emplace_back([&wrong] {
            for (int i = 0; i < 2000; ++i)
                for (int d = 0; d < 64; ++d)
                    if (value.get(d, [d] { return d; }) != d) ++wrong;  // never another value, 0 for one not there yet
        });
    for (auto& t : threads) t.join();
    if (wrong.load() != 0) return 1;
    static fp8ll::PerDevice late;
    if (late.get(3, [] { return -3; }) != -3) return 2;  // an error is not kept
    if (late.get(3, [] { return 5; }) != 5 || late.get(3, [] { return 6; }) != 5) return 3;
    if (late.get(64, [] { return 5; }) >= 0 || late.get(-1, [] { return 5; }) >= 0) return 4;
    return 0;
}
"""


def compiled(tmp_path, text, *flags):
    src, exe = tmp_path / "program.cpp", tmp_path / "program"
    src.write_text(text)
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-pthread", *flags, "-I", CSRC, "-o", str(exe), str(src)],
                       capture_output=True, text=True)
    return r, exe


@pytest.mark.parametrize("flags", [(), ("-fsanitize=thread",)], ids=["plain", "race checks"])
def test_first_use_by_several_threads(tmp_path, flags):
    if flags:  # where the checker is installed and starts
        r, exe = compiled(tmp_path, "int main() { return 0; }", *flags)
        if r.returncode != 0 or subprocess.run([str(exe)]).returncode != 0:
            pytest.skip("no thread sanitizer here")
    r, exe = compiled(tmp_path, PROGRAM, *flags)
    assert r.returncode == 0, r.stderr
    ran = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert ran.returncode == 0, ran.stderr[-2000:]


def test_no_plain_word_is_kept_between_launches():
    plain = re.compile(r"^\s*static\s+(?!const|std::)(?:unsigned|signed|int|long|bool|char|size_t|u?int\d+_t)\b[^(]*;")
    found = []
    for name in sorted(os.listdir(CSRC)):
        with open(os.path.join(CSRC, name)) as f:
            found += ["%s:%d: %s" % (name, i, line.strip()) for i, line in enumerate(f, 1) if plain.match(line)]
    assert not found
