"""The wait of a block for its own copies and products before it ends (csrc/wait.h), compiled for the host."""
import glob
import os
import re
import subprocess

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "differentiable_gaussian_splatting_gs_gb300", "csrc")

PROGRAM = """
#include "wait.h"
#include <cstdio>
#include <initializer_list>
int main() {
    for (unsigned ready : {0u, 1u, 1024u, 5000u, gs::kDrainLimit - 1, gs::kDrainLimit}) {
        unsigned polls = 0;
        const bool ok = gs::poll_drain([&] { return polls++ == ready; });
        std::printf("%u %d %u\\n", ready, (int)ok, polls);
    }
}
"""


def test_a_drain_ends_with_its_barrier_or_at_its_limit_alone(tmp_path):
    src, exe = tmp_path / "drain.cpp", tmp_path / "drain"
    src.write_text(PROGRAM)
    subprocess.run([os.environ.get("CXX") or "g++", "-std=c++17", "-O1", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    got = [tuple(map(int, line.split())) for line in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.splitlines()]
    limit = 1 << 22
    assert got == [(r, 1, r + 1) for r in (0, 1, 1024, 5000, limit - 1)] + [(limit, 0, limit)]


def test_every_drain_is_one():
    # a wait that looks at the error word ends after 1024 polls once any wait has given up: none of a fixed, large bound is left
    for path in glob.glob(os.path.join(CSRC, "*.cu*")):
        with open(path) as f:
            text = f.read()
        assert "kDrainLimit" not in text, path
        for call in re.findall(r"mbar_wait_bounded\([^;]*;", text):
            assert "<<" not in call, (path, call)
