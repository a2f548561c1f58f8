"""The end of the copies of the 8-bit product's pairs of blocks (csrc/pair_ring.h), compiled for the host with a model of the barriers.

The two blocks run in every order that their waits allow, and stop after every number of turns. The model fails on what the
hardware leaves undefined or what a block may not leave behind: an arrival beyond the count of a barrier's phase, a drain
that ends before the copies of its phase have landed, or never, a copy under way at the end."""
import os
import subprocess

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "differentiable_gaussian_splatting_gs_gb300", "csrc")

PROGRAM = """
#include <cstdio>
#include <cstdlib>
#include <vector>
#include "pair_ring.h"
constexpr int S = 4, kHalf = 100;
[[noreturn]] static void wrong(const char* what, int t0, int t1, int c) { std::printf("%s: %d %d turns, %d multiplied\\n", what, t0, t1, c), std::exit(1); }
struct Bar { int arrived = 0, tx = 0, phase = 0; };
static int T0, T1, C;
struct Model {
    Bar bar[S];
    std::vector<int> under_way[S];  // the turns of copies that have not landed
    bool now;                       // copies land at once, or where a drain waits for them
    void end(int s) { if (bar[s].arrived == 1 && bar[s].tx == 0) bar[s].arrived = 0, ++bar[s].phase; }
    void expect_bytes(int s, int n) {
        if (bar[s].arrived++) wrong("a second arrival", T0, T1, C);
        bar[s].tx += n;
        end(s);
    }
    void land(int s) {
        for (int i : under_way[s]) {
            if (i / S != bar[s].phase) wrong("bytes in another turn's phase", T0, T1, C);
            bar[s].tx -= kHalf;
        }
        under_way[s].clear();
        end(s);
    }
    void copy(int i) { under_way[i % S].push_back(i); if (now) land(i % S); }
    // what end_copies asks for
    void expect(int s) { expect_bytes(s, kHalf); }
    void complete(int s) { bar[s].tx -= kHalf; end(s); }
    void drain(int s, unsigned parity) {
        if ((unsigned)(bar[s].phase & 1) != parity && under_way[s].empty()) return;
        if (!under_way[s].empty() && (unsigned)(bar[s].phase & 1) != parity) wrong("a phase ended before its copies", T0, T1, C);
        land(s);
        if ((unsigned)(bar[s].phase & 1) == parity) wrong("a phase that never ends", T0, T1, C);
    }
};
int main() {
    int n = 0;
    for (C = 0; C <= 11; ++C)  // turns multiplied, each of both blocks'
        for (T0 = C; T0 <= C + S; ++T0)
            for (T1 = C; T1 <= C + S; ++T1)
                for (int order = 0; order < 2; ++order)
                    for (bool now : std::vector<bool>{false, true}) {
                        Model m;
                        m.now = now;
                        // a turn is multiplied (its copies have landed) before the one S later is asked for
                        for (int i = 0; i < C + S; ++i) {
                            if (i >= S) m.land(i % S);
                            for (int b = 0; b < 2; ++b) {
                                const int block = b ^ order;
                                if (block == 0 && i < T0) m.expect_bytes(i % S, 2 * kHalf), m.copy(i);
                                if (block == 1 && i < T1) m.copy(i);
                            }
                        }
                        gs::end_copies<S>(T0, T1, m);
                        for (int s = 0; s < S; ++s)
                            if (!m.under_way[s].empty() || m.bar[s].tx || m.bar[s].arrived) wrong("something under way at the end", T0, T1, C);
                        ++n;
                    }
    std::printf("%d\\n", n);
}
"""


def _run(tmp_path, program):
    src, exe = tmp_path / "pair.cpp", tmp_path / "pair"
    src.write_text(program)
    subprocess.run([os.environ.get("CXX") or "g++", "-std=c++17", "-O1", "-w", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    return subprocess.run([str(exe)], capture_output=True, text=True)


def test_wherever_the_blocks_stop_all_copies_land_and_all_phases_end(tmp_path):
    r = _run(tmp_path, PROGRAM)
    assert r.returncode == 0, r.stdout
    assert int(r.stdout) == 12 * 5 * 5 * 4


def test_the_model_sees_the_first_blocks_turns_alone_drained(tmp_path):
    r = _run(tmp_path, PROGRAM.replace("gs::end_copies<S>(T0, T1, m)", "gs::end_copies<S>(T0, T0, m)"))
    assert r.returncode == 1, r.stdout


def test_the_product_ends_its_copies_so():
    with open(os.path.join(CSRC, "matmul_fp8.cu")) as f:
        text = f.read()
    assert "end_copies<kStages>(turns, others" in text and text.count("tile_load2<kPair>(") == 2
