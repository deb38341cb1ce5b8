// Low-rank adapters of many requests beside a shared projection: row t of a
// batch adds the pair its request names,
//
//   Y[t] = base[t] + c_e B_e (A_e x_t),   e = index[t]
//
// (rows that name no pair: Y[t] = base[t]).  The pages' static low-rank term
// B (A X) has one pair per projection; here A is [n][rank][d], B
// [n][d_out][rank].
//
// Two launches.  k_ad_shrink forms S = A_e x_t in float32 (bf16 products are
// exact), as partial sums over ranges of channels; k_ad_expand adds the
// partials in range order and contracts with B_e.  S enters that second
// product as three bf16 planes that sum to it exactly (split24), so the result
// is as exact as float32 products would be, on the matrix cores.
//
// Both work on tiles of 16 consecutive tokens.  A tile's distinct pairs are
// found by ballots over its 16 indices, and each workgroup takes the tile's
// j-th pair: the rows that name another one are not loaded, and their columns
// of the product not stored.  So every pair is read once per tile that uses
// it, whatever the order of the requests, with no sorting pass, and a tile of
// one request's prompt is one ordinary matrix product.
#include "ttq_internal.h"

namespace ttq {

namespace {

constexpr int AW = 4;  // waves per workgroup

struct TilePair {
  int e;              // the j-th distinct pair of the tile, -1: it has fewer
  unsigned rows;      // the tile's rows that name it
  unsigned none;      // the tile's rows that name no pair
};

// (uniform over the wave: every lane looks at token l & 15)
__device__ __forceinline__ TilePair tile_pair(const int32_t* index, int64_t T, int64_t n,
                                              int64_t t0, int j) {
  const int lr = threadIdx.x & 15;
  const int64_t t = t0 + lr;
  const int idx = t < T ? index[t] : -1;
  const bool ok = idx >= 0 && idx < n;
  unsigned left = (unsigned)__ballot(ok) & 0xffffu;
  const unsigned in = t0 + 16 <= T ? 0xffffu : (1u << (int)(T - t0)) - 1u;
  TilePair p{-1, 0u, in & ~left};
  while (left) {
    const int e = __builtin_amdgcn_readlane(idx, __builtin_ctz(left));
    const unsigned same = (unsigned)__ballot(ok && idx == e) & 0xffffu;
    if (j-- == 0) {
      p.e = e;
      p.rows = same;
      break;
    }
    left &= ~same;
  }
  return p;
}

// S partials: workgroup (tile, j, range) of AW waves, which take the range's
// 32-channel steps in turn and add up in LDS in wave order.  NR: 16-row
// blocks of A_e.
template <int NR>
__global__ __launch_bounds__(AW * 64) void k_ad_shrink(AdaptersArgs a) {
  __shared__ f32x4 red[AW - 1][NR][64];
  const int l = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int lr = l & 15, q = l >> 4;
  const int64_t t0 = (int64_t)blockIdx.x * 16;
  const int ks = blockIdx.z;
  const int64_t k0 = ks * a.kc, k1 = min(a.d, k0 + a.kc);
  for (int j = blockIdx.y; j < 16; j += gridDim.y) {
    const TilePair p = tile_pair(a.index, a.T, a.n, t0, j);
    if (p.e < 0) break;  // uniform over the workgroup
    const __amdgpu_buffer_rsrc_t ar =
        make_rsrc(a.A + (int64_t)p.e * a.rank * a.d, (uint32_t)(a.rank * a.d * 2));
    const __amdgpu_buffer_rsrc_t xr =
        make_rsrc(a.X + t0 * a.d, (uint32_t)(min((int64_t)16, a.T - t0) * a.d * 2));
    const uint32_t xoff = (p.rows >> lr & 1u) ? (uint32_t)(lr * a.d * 2) : kOutOfRange;
    f32x4 acc[NR];
#pragma unroll
    for (int n = 0; n < NR; ++n) acc[n] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll 2
    for (int64_t k = k0 + w * 32; k < k1; k += AW * 32) {
      // channels past the range (a multiple of 8 wide) read zeros
      const uint32_t c = k + q * 8 < k1 ? (uint32_t)(k + q * 8) * 2 : kOutOfRange;
      const u32x4 xv = buf_load16(xr, min(xoff + c, kOutOfRange), 0);
#pragma unroll
      for (int n = 0; n < NR; ++n) {
        const uint32_t row = (uint32_t)((n * 16 + lr) * a.d * 2);
        const u32x4 av = buf_load16(ar, min(row + c, kOutOfRange), 0);
        acc[n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
            __builtin_bit_cast(bf16x8, xv), __builtin_bit_cast(bf16x8, av), acc[n], 0, 0, 0);
      }
    }
    if (w > 0) {
#pragma unroll
      for (int n = 0; n < NR; ++n) red[w - 1][n][l] = acc[n];
    }
    __syncthreads();
    if (w == 0) {
      // lane l of a 16 x 16 product holds column l & 15 and rows 4 (l >> 4) + i
#pragma unroll
      for (int n = 0; n < NR; ++n) {
#pragma unroll
        for (int ww = 0; ww < AW - 1; ++ww) acc[n] += red[ww][n][l];
        const int col = n * 16 + lr;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (col < a.rank && (p.rows >> (q * 4 + i) & 1u))
            a.S[((int64_t)ks * a.T + t0 + q * 4 + i) * a.rank + col] = acc[n][i];
      }
    }
    __syncthreads();
  }
}

// Y: workgroup (tile, j, block of 16 * OT outputs per wave).  NK: 32-column
// steps of the rank.
constexpr int OT = 4;

template <int NK>
__global__ __launch_bounds__(AW * 64) void k_ad_expand(AdaptersArgs a) {
  const int l = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int lr = l & 15, q = l >> 4;
  const int64_t t0 = (int64_t)blockIdx.x * 16, t = t0 + lr;
  const int64_t o0 = ((int64_t)blockIdx.z * AW + w) * (OT * 16);
  if (o0 >= a.d_out) return;
  for (int j = blockIdx.y; j < 16; j += gridDim.y) {
    const TilePair p = tile_pair(a.index, a.T, a.n, t0, j);
    // rows that name no pair go with the first one
    const unsigned rows = j == 0 ? p.rows | p.none : p.rows;
    if (!rows) break;
    const bool mine = rows >> lr & 1u, live = p.rows >> lr & 1u;
    f32x4 acc[OT];
#pragma unroll
    for (int o = 0; o < OT; ++o) acc[o] = f32x4{0.f, 0.f, 0.f, 0.f};
    float c = 0.f;
    if (p.e >= 0) {
      c = a.scale ? a.scale[p.e] : 1.f;
      const __amdgpu_buffer_rsrc_t br =
          make_rsrc(a.B + (int64_t)p.e * a.d_out * a.rank, (uint32_t)(a.d_out * a.rank * 2));
      u32x4 bv[OT][NK];
#pragma unroll
      for (int o = 0; o < OT; ++o)
#pragma unroll
        for (int k = 0; k < NK; ++k) {
          const int64_t row = o0 + o * 16 + lr;
          const int col = k * 32 + q * 8;
          bv[o][k] = buf_load16(br, row < a.d_out && col < a.rank
                                        ? (uint32_t)((row * a.rank + col) * 2) : kOutOfRange, 0);
        }
#pragma unroll
      for (int k = 0; k < NK; ++k) {
        const int col = k * 32 + q * 8;
        float s[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) s[i] = 0.f;
        if (live && col < a.rank) {
          for (int ks = 0; ks < a.nks; ++ks) {
            const float* sp = a.S + ((int64_t)ks * a.T + t) * a.rank + col;
            const f32x4 s0 = *(const f32x4*)sp, s1 = *(const f32x4*)(sp + 4);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              s[i] += s0[i];
              s[4 + i] += s1[i];
            }
          }
        }
        u32x4 pl[3];
        split24<true>(s, pl);
#pragma unroll
        for (int o = 0; o < OT; ++o)
#pragma unroll
          for (int i = 0; i < 3; ++i)
            acc[o] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, bv[o][k]),
                                                            __builtin_bit_cast(bf16x8, pl[i]),
                                                            acc[o], 0, 0, 0);
      }
    }
    // lane l holds token l & 15, outputs 4 (l >> 4) + i of each block
    if (mine) {
#pragma unroll
      for (int o = 0; o < OT; ++o) {
        const int64_t col = o0 + o * 16 + q * 4;
        const float* bp = a.base ? a.base + t * a.d_out + col : nullptr;
        float* yp = a.Y + t * a.d_out + col;
        if (a.vec && col < a.d_out) {
          f32x4 b = {0.f, 0.f, 0.f, 0.f};
          if (bp) b = *(const f32x4*)bp;
#pragma unroll
          for (int i = 0; i < 4; ++i) b[i] = live ? fmaf(c, acc[o][i], b[i]) : b[i];
          *(f32x4*)yp = b;
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (col + i < a.d_out) {
              const float b = bp ? bp[i] : 0.f;
              yp[i] = live ? fmaf(c, acc[o][i], b) : b;
            }
        }
      }
    }
  }
}

}  // namespace

hipError_t launch_ad_shrink(const AdaptersArgs& a, int slots, const Launch& L) {
  const int64_t tiles = (a.T + 15) / 16;
  if (tiles == 0 || a.n == 0) return hipSuccess;
  const dim3 grid((unsigned)tiles, (unsigned)slots, (unsigned)a.nks), blk(AW * 64);
  switch ((a.rank + 15) / 16) {
    case 1: return ext_launch(k_ad_shrink<1>, grid, blk, 0, L, a);
    case 2: return ext_launch(k_ad_shrink<2>, grid, blk, 0, L, a);
    case 3: return ext_launch(k_ad_shrink<3>, grid, blk, 0, L, a);
    case 4: return ext_launch(k_ad_shrink<4>, grid, blk, 0, L, a);
    case 5: case 6: return ext_launch(k_ad_shrink<6>, grid, blk, 0, L, a);
    case 7: case 8: return ext_launch(k_ad_shrink<8>, grid, blk, 0, L, a);
    default: return hipErrorInvalidValue;
  }
}

hipError_t launch_ad_expand(const AdaptersArgs& a, int slots, const Launch& L) {
  const int64_t tiles = (a.T + 15) / 16;
  const int64_t blocks = (a.d_out + AW * OT * 16 - 1) / (AW * OT * 16);
  if (tiles == 0 || blocks == 0) return hipSuccess;
  const dim3 grid((unsigned)tiles, (unsigned)slots, (unsigned)blocks), blk(AW * 64);
  switch ((a.rank + 31) / 32) {
    case 0:  // no pairs at all
    case 1: return ext_launch(k_ad_expand<1>, grid, blk, 0, L, a);
    case 2: return ext_launch(k_ad_expand<2>, grid, blk, 0, L, a);
    case 3: return ext_launch(k_ad_expand<3>, grid, blk, 0, L, a);
    case 4: return ext_launch(k_ad_expand<4>, grid, blk, 0, L, a);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace ttq
