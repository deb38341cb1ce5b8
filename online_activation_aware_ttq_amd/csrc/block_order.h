// The order in which blocks of 256 query rows of a K/V head are taken, for up to 64
// sequences, one a lane of a wave.  No GPU code: `Wave` is a wave, or on the host a
// loop over its lanes.
#pragma once

#include <cstdint>

namespace ttq {

// A lane's sequence: its query rows (tokens * G), the position of its first token and
// the keys that it holds.
struct LaneSeq {
  int64_t rows, shift, len;
};

// Its blocks that see more than 256 x keys: its last ones, for the last row sees all
// `len` (none of a sequence without rows in this step, however many keys it holds)
constexpr int blocks_above(const LaneSeq& s, int G, int x) {
  const int blocks = (int)((s.rows + 255) >> 8);
  if (x == 0 || blocks == 0) return blocks;
  if (s.len <= (int64_t)x << 8) return 0;
  const int64_t key = ((int64_t)x << 8) - s.shift, from = key > 0 ? key * G >> 8 : 0;
  return from < blocks ? blocks - (int)from : 1;
}

// Block b in the order of the most keys (to within 256) first: the lane of its
// sequence and its first row; false: there are not so many.  Wave:
//   total(f)          the sum over the lanes of f(its sequence)
//   owner(f, i, at)   the lane in whose range of the running sum of f place i is, and
//                     in `at` which place of the range
//   of(lane, f)       f of that lane's sequence
template <class Wave>
constexpr bool long_block(const Wave& w, int b, int64_t max_len, int G, int& lane, int64_t& r0) {
  auto count = [&](int x) { return w.total([=](const LaneSeq& s) { return blocks_above(s, G, x); }); };
  if (b < 0 || b >= count(0)) return false;
  int top = 0;  // 2^(top + 1) is more than any block is asked for
  while (max_len >> 8 >> (top + 1)) ++top;
  int x = 0;  // the largest that more than b blocks exceed
  for (int i = top; i >= 0; --i)
    if (count(x | 1 << i) > b) x |= 1 << i;
  const bool last = (x + 1) >> (top + 1);
  auto above = [=](const LaneSeq& s) { return last ? 0 : blocks_above(s, G, x + 1); };
  int at = 0;
  lane = w.owner([=](const LaneSeq& s) { return blocks_above(s, G, x) - above(s); }, b - w.total(above), at);
  r0 = (int64_t)(w.of(lane, [=](const LaneSeq& s) { return blocks_above(s, G, 0) - blocks_above(s, G, x); }) + at) << 8;
  return r0 >= 0 && r0 < w.of(lane, [](const LaneSeq& s) { return (int)s.rows; });
}

}  // namespace ttq
