// Which tokens a piece [s0, s1) of the packed stream takes from the sequence of
// tokens [first, last). Plain arithmetic, the same on the host and in the
// kernels: whatever the offsets hold, a run that these functions give lies
// inside its piece and has a token at least.
#pragma once

#include <cstdint>

namespace ssd {

// The run that reaches the piece's end and goes on behind it: from r0 to s1.
// (Before the first offset a piece has no such run: the search for the sequence
// of its last token gives the first sequence there, which begins behind it.)
constexpr bool passing_run(int64_t first, int64_t last, int64_t s0, int64_t s1, int64_t& r0) {
  if (last <= s1 || first >= s1) return false;
  r0 = first > s0 ? first : s0;
  return true;
}

// The next run of a piece whose tokens before pos are done: tokens r0 to r1.
// (It begins behind pos where tokens before the first sequence lie between.)
constexpr bool next_run(int64_t first, int64_t last, int64_t pos, int64_t s1, int64_t& r0, int64_t& r1) {
  r0 = first > pos ? first : pos;
  r1 = last < s1 ? last : s1;
  return r0 < r1;
}

}  // namespace ssd
