// Which of a call's n workgroups gets to a point last, by one count in memory that is 0 between calls.
#pragma once

#include <stdint.h>

namespace ga {

// What workgroup i of n adds: the first 1 - n, the others 1.  Their sum is 0, and no part of them that lacks one is: the
// workgroup whose addition leaves 0 is the last.  Nothing is reset, so that calls that overlapped, whose results are lost,
// leave the count as they found it.
constexpr uint32_t arrival(uint32_t i, uint32_t n) { return i == 0 ? 1u - n : 1u; }

}  // namespace ga
