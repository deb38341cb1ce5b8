// Loads of stored packed codes in the quarter order of a group, shared by the
// kernels that contract them on the matrix cores.
#pragma once

#include "ttq_internal.h"

namespace ttq {

// A lane's codes of one group: its contiguous quarter of the group, NB =
// GS/32 * CB bytes, fetched with the widest loads that tile it.
template <int CB, int GS>
struct GroupCodes {
  static constexpr int NB = GS / 32 * CB;
  unsigned w[NB >= 4 ? NB / 4 : 1];
};

template <int CB, int GS>
__device__ __forceinline__ void load_codes(GroupCodes<CB, GS>& c,
                                           __amdgpu_buffer_rsrc_t r,
                                           uint32_t voff, uint32_t soff) {
  constexpr int NB = GroupCodes<CB, GS>::NB;
  if constexpr (NB >= 16) {
#pragma unroll
    for (int i = 0; i < NB / 16; ++i) {
      const u32x4 v = buf_load16(r, voff + i * 16, soff);
      c.w[4 * i] = v.x; c.w[4 * i + 1] = v.y; c.w[4 * i + 2] = v.z; c.w[4 * i + 3] = v.w;
    }
  } else if constexpr (NB == 8) {
    const auto v = __builtin_amdgcn_raw_buffer_load_b64(r, voff, soff, 0);
    c.w[0] = v[0];
    c.w[1] = v[1];
  } else if constexpr (NB == 4) {
    c.w[0] = __builtin_amdgcn_raw_buffer_load_b32(r, voff, soff, 0);
  } else if constexpr (NB == 2) {
    c.w[0] = __builtin_amdgcn_raw_buffer_load_b16(r, voff, soff, 0);
  } else {
    c.w[0] = __builtin_amdgcn_raw_buffer_load_b8(r, voff, soff, 0);
  }
}

// the 8 codes (CB bytes) of MFMA step k, low bits first
template <int CB, int GS>
__device__ __forceinline__ u32x2 step_codes(const GroupCodes<CB, GS>& c, int k) {
  if (CB == 8) return u32x2{c.w[2 * k], c.w[2 * k + 1]};
  if (CB == 4) return u32x2{c.w[k], 0u};
  if (CB == 2) return u32x2{(c.w[k / 2] >> (16 * (k % 2))) & 0xFFFFu, 0u};
  return u32x2{(c.w[k / 4] >> (8 * (k % 4))) & 0xFFu, 0u};
}

}  // namespace ttq
