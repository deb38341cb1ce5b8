// One wave's part of a cache row, quantized: shared by the kernels that write
// rows into a cache.
#pragma once

#include "ttq_internal.h"

namespace ttq {

// min and max over the LPG consecutive lanes of a group, and whether any of
// them saw a value that is not finite
template <int LPG>
__device__ __forceinline__ void group_range(float& mn, float& mx, int& bad) {
#pragma unroll
  for (int off = 1; off < LPG; off <<= 1) {
    mn = fminf(mn, __shfl_xor(mn, off));
    mx = fmaxf(mx, __shfl_xor(mx, off));
    bad |= __shfl_xor(bad, off);
  }
}

// what the scale of a format is a fixed part of
template <int QF>
__device__ __forceinline__ float qrange(float mn, float mx) {
  if constexpr (QF == QF_ASYM) return mx - mn;
  else if constexpr (QF == QF_INTZP) return fmaxf(mx, 0.f) - fminf(mn, 0.f);
  else return fmaxf(-mn, mx);
}

// 8 channels a lane from channel c0 of cache row `slot` on: a group is GS / 8
// adjacent lanes; the lanes behind the last channel are not live.
//
// The code decision is that of the weight quantizer (qgroup_si / qlevels8:
// float32, no fused operations) except that the scale is the range times rN, the
// float32 nearest to 1/N (1/Z, 1/448), instead of the range divided by N: the
// bits of the same steps in elementary torch operations on the GPU, which divide
// by a number so.  It is no matter of speed (2047 float32 rows of 8192 channels:
// 18.4 us, 18.7 with the quotient).  A group that holds a value that is not
// finite, or whose range overflows, gets a NaN scale and offset, and so reads
// back as NaN; a scale below float32's normal range (whose reciprocal may
// overflow) counts as 0.
template <int GS, int QF>
__device__ __forceinline__ void quantize8(const float (&u)[8], bool live, int64_t slot,
                                          int64_t c0, int64_t C, int64_t row_bytes,
                                          float Nf, float rN, int cb, uint8_t* codes,
                                          float* scales, float* mins) {
  constexpr int LPG = GS / 8;
  float mn = u[0], mx = u[0];
  int bad = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    mn = fminf(mn, u[j]);
    mx = fmaxf(mx, u[j]);
    bad |= !(__builtin_fabsf(u[j]) <= 3.402823466e38f);
  }
  group_range<LPG>(mn, mx, bad);
  float s = qrange<QF>(mn, mx) * rN;
  bad |= !(s <= 3.402823466e38f);
  if (s < 1.17549435e-38f) s = 0.f;
  QGroup g = qgroup_si<QF>(mn, s, s > 0.f ? 1.0f / s : 0.f, Nf);
  if (bad) g.s = g.off = __builtin_nanf("");
  float L[8];
  qlevels8<QF>(g, u, L);
  if (!live) return;
  unsigned q[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) q[j] = bad ? 0u : qcode<QF>(g, L[j]);
  uint8_t* dst = codes + slot * row_bytes + c0 * cb / 8;
  if (cb == 8) {
    *(u32x2*)dst = u32x2{q[0] | (q[1] << 8) | (q[2] << 16) | (q[3] << 24),
                         q[4] | (q[5] << 8) | (q[6] << 16) | (q[7] << 24)};
  } else {
    unsigned c = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) c |= q[j] << (j * cb);
    if (cb == 4) *(unsigned*)dst = c;
    else if (cb == 2) *(uint16_t*)dst = (uint16_t)c;
    else *dst = (uint8_t)c;
  }
  if ((threadIdx.x & 63) % LPG == 0) {
    const int64_t o = slot * (C / GS) + c0 / GS;
    scales[o] = g.s;
    mins[o] = g.off;
  }
}

}  // namespace ttq
