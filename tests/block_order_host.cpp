// The block order of the kernel of prompts (csrc/block_order.h) on the host: a wave is a
// loop over its lanes.
#include "block_order.h"

namespace {
struct HostWave {
  ttq::LaneSeq own[64] = {};
  template <class F>
  int total(F f) const {
    int sum = 0;
    for (const auto& s : own) sum += f(s);
    return sum;
  }
  template <class F>
  int owner(F f, int i, int& at) const {
    for (int lane = 0; lane < 64; ++lane) {
      at = i;
      if ((i -= f(own[lane])) < 0) return lane;
    }
    return -1;
  }
  template <class F>
  int of(int lane, F f) const {
    return lane < 0 ? 0 : f(own[lane]);
  }
};
}  // namespace

// blocks 0 .. tiles - 1 of n sequences: lane[b] (-1: none) and r0[b]
extern "C" void block_order(int n, const int64_t* rows, const int64_t* shift, const int64_t* len, int G,
                            int64_t max_len, int tiles, int32_t* lane, int64_t* r0) {
  HostWave w;
  for (int i = 0; i < n; ++i) w.own[i] = {rows[i], shift[i], len[i]};
  for (int b = 0; b < tiles; ++b) {
    int l = -1;
    if (!ttq::long_block(w, b, max_len, G, l, r0[b])) l = -1;
    lane[b] = l;
  }
}
