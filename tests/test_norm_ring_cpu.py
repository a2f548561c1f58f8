"""The layer norm kernels' ring of row copies (csrc/norm_ring.cuh), compiled for the host with a model of the barriers.

The model fails on what the hardware leaves undefined: an arrival beyond the count of a barrier's phase. Copies land when
the program says so. A wait gives up when its copy is not there."""
import os
import subprocess

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "differentiable_gaussian_splatting_gs_gb300", "csrc")

PROGRAM = """
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <map>
#define __device__
#define __host__
#define __forceinline__ inline
static struct { int x; } threadIdx;
namespace gs {
struct Bar { int arrivals = 0, phase = 0; unsigned pending = 0; };
static std::map<uint64_t*, Bar> bars;
static int waits = 0, late = -1, drained = 0, asked = 0;  // late: the wait whose copies have not landed
static void land(uint64_t* bar) {
    Bar& b = bars[bar];
    if (b.arrivals) b.pending = 0, b.arrivals = 0, ++b.phase;
}
static void mbar_arrive_expect_tx(uint64_t* bar, unsigned n) {
    if (bars[bar].arrivals++) std::printf("undefined: a second arrival\\n"), std::exit(1);
    bars[bar].pending += n, ++asked;
}
static void bulk_copy_g2s(void*, const void*, unsigned, uint64_t*) {}
static bool mbar_wait_bounded(uint64_t* bar, unsigned parity, unsigned, unsigned*) {
    if (waits++ != late) land(bar);
    return (unsigned)(bars[bar].phase & 1) != parity;
}
static void mbar_drain(uint64_t* bar, unsigned parity, unsigned*) {
    if (bars[bar].arrivals) ++drained;
    land(bar);
    if ((unsigned)(bars[bar].phase & 1) == parity) std::printf("a drain of a phase that never ends\\n"), std::exit(1);
}
}
#include "norm_ring.cuh"
int main() {
    for (int rows : {1, 2, 3, 4, 7, 20})
        for (int late = -1; late < rows; ++late) {
            gs::bars.clear();
            gs::waits = gs::drained = gs::asked = 0;
            gs::late = late;
            gs::NormRing<2, 32, 3> ring;
            ring.src[0] = ring.src[1] = nullptr;
            ring.stride[0] = ring.stride[1] = 16;
            uint64_t bars[3];
            unsigned char room[1];
            ring.start(room, bars, 8, 2, 0, rows, 1, 1, nullptr);
            for (int r = 0; r < rows; ++r) { ring.wait(); ring.next(); }
            ring.finish();
            for (auto& b : gs::bars) if (b.second.arrivals) std::printf("a copy on its way at the end\\n"), std::exit(1);
            std::printf("%d %d %d %d\\n", rows, late, gs::asked, gs::drained);
        }
}
"""


def test_after_a_wait_that_gave_up_nothing_more_is_copied_and_all_copies_land(tmp_path):
    src, exe = tmp_path / "ring.cpp", tmp_path / "ring"
    src.write_text(PROGRAM.replace("#include <map>", "#include <initializer_list>\n#include <map>"))
    subprocess.run([os.environ.get("CXX") or "g++", "-std=c++17", "-O1", "-w", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout.splitlines()[-1]
    for line in r.stdout.splitlines():
        rows, late, asked, drained = map(int, line.split())
        if late < 0:
            assert (asked, drained) == (rows, 0)
        else:  # three ahead from the start, one more after each wait before the one that gave up
            assert asked == min(rows, 3 + late) and 1 <= drained <= 3, line
