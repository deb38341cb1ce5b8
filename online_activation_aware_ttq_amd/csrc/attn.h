// Pieces shared by the attention kernels: stored codes as fp16 operands of the
// matrix cores, and where a block of query rows and its keys lie.
//
// A stored code is an exact fp16 value as it stands: an integer code c of up to 10
// bits is the pattern of the subnormal c 2^-24, which the matrix cores multiply
// exactly; so a mask leaves two operands of a register's halves, with no
// conversion, and a nibble taken in place counts 16-fold, which the other operand
// or the result makes up for.  E4M3 codes become fp16 by gfx950's conversion, two
// an instruction.
#pragma once

#include "ttq_internal.h"

namespace ttq {

typedef __attribute__((ext_vector_type(2))) _Float16 f16x2;

// what a code's operand is to be multiplied with to be the code: 2^kUnit
template <bool F8>
constexpr int kUnit = F8 ? 0 : 24;

// (times a power of two)
__device__ __forceinline__ unsigned e4m3_pair(unsigned w, bool hi, float times = 1.f) {
  return __builtin_bit_cast(unsigned, hi ? __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, times, true)
                                         : __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, times, false));
}

// Workgroups of a launch, which has fewer than 2^32 threads along x; some of the last row
// are too many.  (A multiple of 8 in a row, for the dies.  Fewer than 2^31 of them: blocks
// of a K/V head times K/V heads are T heads / 16 and n_seq kv_heads at most, 2^27 + 2^30.)
inline dim3 attn_grid(int64_t n) {
  const int64_t x = int64_t(1) << 21;
  return n <= x ? dim3((unsigned)n) : dim3((unsigned)x, (unsigned)((n + x - 1) / x));
}
__device__ __forceinline__ unsigned attn_group() { return blockIdx.y * gridDim.x + blockIdx.x; }

// A maximum of scores (log2) from which on its rounding is no small part of an exponent
constexpr float kFarScore = 0x1p18f;

__device__ __forceinline__ int64_t uniform64(int64_t v) {
  const unsigned lo = __builtin_amdgcn_readfirstlane((int)v), hi = __builtin_amdgcn_readfirstlane((int)(v >> 32));
  return (int64_t)((uint64_t)hi << 32 | lo);
}

// A scale and offset that are not both finite count as NaN
__device__ __forceinline__ void finite_or_nan(float& s, float& m) {
  if (!((__builtin_fabsf(s) <= 3.402823466e38f) & (__builtin_fabsf(m) <= 3.402823466e38f))) s = m = __builtin_nanf("");
}

// Eight codes of one row (CB bytes, low bits first) as an operand.  4 bits: slots
// (2i, 2i + 1) are codes (i, i + 4), 16-fold where i is odd (slot_code,
// slot_shift); 8 bits: in order.
template <int CB, bool F8>
__device__ __forceinline__ f16x8 codes8(unsigned w0, unsigned w1) {
  u32x4 r;
  if constexpr (F8) {
    r = u32x4{e4m3_pair(w0, false), e4m3_pair(w0, true), e4m3_pair(w1, false), e4m3_pair(w1, true)};
  } else if constexpr (CB == 8) {
    r = u32x4{__builtin_amdgcn_perm(0u, w0, 0x0c010c00u), __builtin_amdgcn_perm(0u, w0, 0x0c030c02u),
              __builtin_amdgcn_perm(0u, w1, 0x0c010c00u), __builtin_amdgcn_perm(0u, w1, 0x0c030c02u)};
  } else {
    const unsigned h = w0 >> 8;
    r = u32x4{w0 & 0x000f000fu, w0 & 0x00f000f0u, h & 0x000f000fu, h & 0x00f000f0u};
  }
  return __builtin_bit_cast(f16x8, r);
}
template <int CB>
__device__ __forceinline__ constexpr int slot_code(int slot) {
  return CB == 4 ? slot / 2 + 4 * (slot & 1) : slot;
}
template <int CB>
__device__ __forceinline__ constexpr int slot_shift(int slot) {
  return CB == 4 && (slot / 2) & 1 ? 4 : 0;
}

// The same as normal fp16 values, which a scale can make as small as fp16 goes: codes as
// 16 + c / 64 (k = k16; nibbles above others: 16 + c / 4), E4M3 as 2^-8 of what they are.
constexpr unsigned k16 = 0x4c004c00u;
template <int CB, bool F8>
__device__ __forceinline__ u32x4 codes8_normal(unsigned w0, unsigned w1, unsigned k) {
  if constexpr (F8) {
    return u32x4{e4m3_pair(w0, false, 0x1p-8f), e4m3_pair(w0, true, 0x1p-8f), e4m3_pair(w1, false, 0x1p-8f),
                 e4m3_pair(w1, true, 0x1p-8f)};
  } else if constexpr (CB == 8) {
    return u32x4{__builtin_amdgcn_perm(k | k >> 8, w0, 0x04010400u), __builtin_amdgcn_perm(k | k >> 8, w0, 0x04030402u),
                 __builtin_amdgcn_perm(k | k >> 8, w1, 0x04010400u), __builtin_amdgcn_perm(k | k >> 8, w1, 0x04030402u)};
  } else {
    const unsigned h = w0 >> 8;
    return u32x4{(w0 & 0x000f000fu) | k, (w0 & 0x00f000f0u) | k, (h & 0x000f000fu) | k, (h & 0x00f000f0u) | k};
  }
}

// Channels 4 i .. 4 i + 3 of two keys a and b as pairs (a, b), one a channel; 4 bits:
// 16-fold where the channel is odd.  Integers with k (0, or k16 as above) beside them.
template <int CB, bool F8>
__device__ __forceinline__ void key_pairs(const unsigned* a, const unsigned* b, int i, unsigned k, unsigned (&out)[4]) {
  if constexpr (F8) {
    const unsigned lo = __builtin_amdgcn_perm(b[i], a[i], 0x05010400u);
    const unsigned hi = __builtin_amdgcn_perm(b[i], a[i], 0x07030602u);
    out[0] = e4m3_pair(lo, false);
    out[1] = e4m3_pair(lo, true);
    out[2] = e4m3_pair(hi, false);
    out[3] = e4m3_pair(hi, true);
  } else if constexpr (CB == 8) {
    out[0] = __builtin_amdgcn_perm(b[i], a[i], 0x0c040c00u) | k;
    out[1] = __builtin_amdgcn_perm(b[i], a[i], 0x0c050c01u) | k;
    out[2] = __builtin_amdgcn_perm(b[i], a[i], 0x0c060c02u) | k;
    out[3] = __builtin_amdgcn_perm(b[i], a[i], 0x0c070c03u) | k;
  } else {
    const unsigned x = __builtin_amdgcn_perm(b[i / 2], a[i / 2], i % 2 ? 0x07060302u : 0x05040100u);
    const unsigned h = x >> 8;
    out[0] = (x & 0x000f000fu) | k;
    out[1] = (x & 0x00f000f0u) | k;
    out[2] = (h & 0x000f000fu) | k;
    out[3] = (h & 0x00f000f0u) | k;
  }
}

// The rows of a sequence, and which keys they may see.  A query row r of a K/V
// head is (token r / G, head r % G) of its sequence.
struct SeqRows {
  int64_t first;   // row of its first token
  int rows;        // tokens * G
  int64_t shift;   // position of token j: shift + j
  int64_t len;     // keys that the pages hold
};

// The block b of SZ query rows of a K/V head: its sequence and first row.  Sequence
// i's blocks begin at offsets[i] G / SZ + i, which leaves each enough, so no table
// of them is needed; a block past its sequence's last has no rows (false).
template <int SZ>
__device__ __forceinline__ bool find_block(const AttnArgs& a, int64_t b, int64_t& seq, SeqRows& s,
                                           int64_t& r0) {
  int64_t begin, tokens = 1;
  if (a.offsets) {
    auto off = [&](int64_t i) __attribute__((always_inline)) { return min(max((int64_t)a.offsets[i], (int64_t)0), a.T); };
    int64_t lo = 0, hi = a.n_seq;
    while (hi - lo > 1) {
      const int64_t mid = (lo + hi) >> 1;
      if (off(mid) * a.G / SZ + mid <= b) lo = mid;
      else hi = mid;
    }
    seq = lo;
    s.first = off(lo);
    tokens = max(off(lo + 1) - s.first, (int64_t)0);
    s.rows = (int)(tokens * a.G);
    begin = s.first * a.G / SZ + lo;
  } else {
    const int64_t per = (a.G + SZ - 1) / SZ;
    seq = b / per;
    s.first = seq;
    s.rows = a.G;
    begin = seq * per;
  }
  r0 = (b - begin) * SZ;
  if (r0 < 0 || r0 >= s.rows) return false;
  const int64_t n = max(a.lens[seq], 0);
  s.shift = n - tokens;
  s.len = min(min(n, a.max_len), a.max_pages << a.pshift);
  return true;
}

}  // namespace ttq
