// The end of the 8-bit product's copies, apart from what it does to barriers, so that it also compiles for the host.
#pragma once

#include "wait.h"

namespace gs {

// Two blocks copy the halves of each stage's tiles; one barrier of the first counts both, with the first's arrival, which expects both
// halves' bytes. Each block asks for its half of a turn once the products of the turn STAGES before are over, and stops where that
// wait gives up, so that one may stop up to STAGES turns before the other. The first block ends the phases that then lack
// something, and waits for the copies under way in either block's shared memory:
//   bar.expect(stage): the arrival that the first left out, for the other's bytes alone;
//   bar.complete(stage): the bytes that the other left out;
//   bar.drain(stage, parity): a phase's end.
// Where one block has all tiles, it has as many turns as itself.
template <int STAGES, class Bar>
GS_HOST_DEVICE void end_copies(int turns, int others, Bar&& bar) {
    for (int i = turns; i < others; ++i) bar.expect(i % STAGES);
    for (int i = others; i < turns; ++i) bar.complete(i % STAGES);
    const int most = turns > others ? turns : others;
    for (int i = most > STAGES ? most - STAGES : 0; i < most; ++i) bar.drain(i % STAGES, (unsigned)(i / STAGES) & 1u);
}

}  // namespace gs
