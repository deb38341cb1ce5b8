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
// is as exact as float32 products would be, on the matrix cores.  Small decode
// steps do both in one launch (k_ad_step).
//
// Both work on tiles of consecutive tokens (128 of a decode batch, 64 of
// prompts).  A tile's distinct pairs are found by ballots over its indices, and
// a workgroup gathers the rows that name the j-th of them, 16 to a matrix
// instruction: every pair is read once per tile that uses it, whatever the
// order of the requests and with no sorting pass, and a tile of one request's
// prompt is one ordinary matrix product.
//
// Bound by memory: a decode step by the pairs it reads, prompts by X, base and
// Y.  128 rows with 64 pairs of rank 64 on 4096 -> 11008: 13.3 us for 34 MB of
// A, 30 us for 90 MB of B and 11 MB of base and Y.  4096 rows of eight prompts,
// rank 64 on 4096 -> 4096: 15 us for 34 MB of X, 36 us for 134 MB of base and Y
// (a plain copy of those: 26 us).
#include <algorithm>
#include <type_traits>

#include "ttq_internal.h"

namespace ttq {

namespace {

constexpr int AW = 4;  // waves per workgroup

// Prompts: workgroups go to the eight dies in turn, each of which has its own L2,
// and the tiles of one prompt share a pair, so a die gets tiles in a row (8 per).
__device__ __forceinline__ int64_t prompt_tile() {
  return (int64_t)(blockIdx.x % 8) * (gridDim.x / 8) + blockIdx.x / 8;
}

// The distinct pairs of the tile at t0 (TC * 64 tokens) that a workgroup takes,
// one after another, and the rows that name them.  A decode step (TC = 2): the
// pair of row blockIdx.y, counted from row `turn` on, if no earlier row names
// it.  (Workgroups go to the eight dies in turn, in the order of their numbers:
// with turn = blockIdx.z a pair's workgroups, of which few rows have any, are
// spread over them whatever the number of rows.)  Prompts, whose tiles
// have few: every gridDim.y-th distinct one.  The rows that name no pair go
// with the first workgroup.  Uniform; every wave writes the same list of rows,
// so none waits for another: list[0, n) name pair e, list[n, all) none.
template <int TC>
struct TilePairs {
  int idx[TC];
  uint64_t left[TC], none[TC];  // rows not yet taken, rows that name no pair
  int e, n, all;

  __device__ __forceinline__ TilePairs(const AdaptersArgs& a, int64_t t0, int turn) {
    const int l = threadIdx.x & 63;
    int j = blockIdx.y;
    if (TC > 1) j = (j + turn) % (int)gridDim.y;
#pragma unroll
    for (int c = 0; c < TC; ++c) {
      const int64_t t = t0 + c * 64 + l;
      const int i = t < a.T ? a.index[t] : -1;
      idx[c] = i < a.n ? i : -1;
      left[c] = __ballot(idx[c] >= 0);
      none[c] = __ballot(t < a.T && idx[c] < 0);
    }
    if (TC == 1) {
      for (int i = 0; i < j; ++i) skip();
    } else {  // only the rows that name what row j does, if it is their first
      uint64_t same[TC];
      const int pick = lane_index(j);
      int first = -1;
#pragma unroll
      for (int c = TC - 1; c >= 0; --c) {
        same[c] = __ballot(idx[c] == pick);
        if (same[c]) first = c * 64 + __builtin_ctzll(same[c]);
      }
#pragma unroll
      for (int c = 0; c < TC; ++c) left[c] = pick >= 0 && first == j ? same[c] : 0;
    }
    if (j != 0) {
#pragma unroll
      for (int c = 0; c < TC; ++c) none[c] = 0;
    }
  }
  __device__ __forceinline__ int lane_index(int row) const {
    int i = 0;
#pragma unroll
    for (int c = 0; c < TC; ++c)
      if (row / 64 == c) i = __builtin_amdgcn_readlane(idx[c], row % 64);
    return i;
  }
  // the next pair's rows leave left[]; returns them in same[]
  __device__ __forceinline__ int skip(uint64_t* rows = nullptr) {
    int i = -1;
#pragma unroll
    for (int c = TC - 1; c >= 0; --c)
      if (left[c]) i = __builtin_amdgcn_readlane(idx[c], __builtin_ctzll(left[c]));
#pragma unroll
    for (int c = 0; c < TC; ++c) {
      const uint64_t same = i < 0 ? 0 : __ballot(idx[c] == i);
      left[c] &= ~same;
      if (rows) rows[c] = same;
    }
    return i;
  }
  // false: nothing is left
  __device__ __forceinline__ bool next(uint8_t* list, bool with_none) {
    const int l = threadIdx.x & 63;
    const uint64_t below = (1ull << l) - 1ull;
    uint64_t same[TC];
    e = skip(same);
    n = 0;
#pragma unroll
    for (int c = 0; c < TC; ++c) {
      if (same[c] >> l & 1u) list[n + __builtin_popcountll(same[c] & below)] = (uint8_t)(c * 64 + l);
      n += __builtin_popcountll(same[c]);
    }
    all = n;
    if (with_none) {
#pragma unroll
      for (int c = 0; c < TC; ++c) {
        if (none[c] >> l & 1u) list[all + __builtin_popcountll(none[c] & below)] = (uint8_t)(c * 64 + l);
        all += __builtin_popcountll(none[c]);
        none[c] = 0;
      }
    }
    for (int i = 1; i < (TC == 1 ? (int)gridDim.y : 1); ++i) skip();  // the other workgroups'
    return all > 0;
  }
};

// S partials: workgroup (tile, its pairs, range) of AW waves, which take the range's
// 32-channel steps in turn and add up in LDS in wave order.  NR: 16-row blocks
// of A_e; NB: 16-token blocks of a pass over the range.
template <int TC, int NR, int NB>
__global__ __launch_bounds__(AW * 64) void k_ad_shrink(AdaptersArgs a) {
  __shared__ __attribute__((aligned(16))) float red[AW][16][NR * 16 + 4];
  __shared__ uint8_t list[TC * 64];
  const int l = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int lr = l & 15, q = l >> 4;
  const int64_t t0 = TC == 1 ? prompt_tile() * 64 : 0;
  if (t0 >= a.T) return;
  const int64_t k0 = blockIdx.z * a.kc, k1 = min(a.d, k0 + a.kc);
  TilePairs<TC> r(a, t0, blockIdx.z);
  while (r.next(list, false)) {  // uniform over the workgroup
    const __amdgpu_buffer_rsrc_t ar =
        make_rsrc(a.A + (int64_t)r.e * a.rank * a.d, (uint32_t)(a.rank * a.d * 2));
    const __amdgpu_buffer_rsrc_t xr =
        make_rsrc(a.X + t0 * a.d, (uint32_t)(min((int64_t)TC * 64, a.T - t0) * a.d * 2));
    for (int b0 = 0; b0 < r.n; b0 += NB * 16) {
      uint32_t xoff[NB];
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const int i = b0 + b * 16 + lr;
        xoff[b] = i < r.n ? (uint32_t)(list[i] * a.d * 2) : kOutOfRange;
      }
      f32x4 acc[NB][NR];
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int n = 0; n < NR; ++n) acc[b][n] = f32x4{0.f, 0.f, 0.f, 0.f};
      // U steps' loads at a time, the next ones in flight while these multiply
      constexpr int U = NR * NB > 4 ? 1 : 2;
      u32x4 xv[2][U][NB], av[2][U][NR];
      auto load = [&](int s, int64_t k) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
          // channels past the range (a multiple of 8 wide) read zeros
          const int64_t kk = k + u * (AW * 32) + q * 8;
          const uint32_t c = kk < k1 ? (uint32_t)kk * 2 : kOutOfRange;
#pragma unroll
          for (int n = 0; n < NR; ++n)
            av[s][u][n] = buf_load16(ar, min((uint32_t)((n * 16 + lr) * a.d * 2) + c, kOutOfRange), 0);
#pragma unroll
          for (int b = 0; b < NB; ++b) xv[s][u][b] = buf_load16(xr, min(xoff[b] + c, kOutOfRange), 0);
        }
      };
      auto use = [&](int s) {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int n = 0; n < NR; ++n)
              acc[b][n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                  __builtin_bit_cast(bf16x8, xv[s][u][b]), __builtin_bit_cast(bf16x8, av[s][u][n]),
                  acc[b][n], 0, 0, 0);
      };
      constexpr int64_t STEP = U * AW * 32;
      int64_t k = k0 + w * 32;
      load(0, k);
      __builtin_amdgcn_sched_barrier(0);
      for (; k < k1; k += 2 * STEP) {
        load(1, k + STEP);
        __builtin_amdgcn_sched_barrier(0);
        use(0);
        __builtin_amdgcn_sched_barrier(0);
        load(0, k + 2 * STEP);
        __builtin_amdgcn_sched_barrier(0);
        use(1);  // (past the range: zeros)
        __builtin_amdgcn_sched_barrier(0);
      }
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        if (b0 + b * 16 >= r.n) break;  // uniform
        // lane l of a 16 x 16 product holds column l & 15 and rows 4 (l >> 4) + i
#pragma unroll
        for (int n = 0; n < NR; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) red[w][q * 4 + i][n * 16 + lr] = acc[b][n][i];
        __syncthreads();
        // a thread adds up, and stores, 4 columns of a row
        for (int i = threadIdx.x; i < NR * 64; i += AW * 64) {
          const int at = b0 + b * 16 + i / (NR * 4), col = i % (NR * 4) * 4;
          if (at >= r.n || col >= a.rank) continue;
          f32x4 v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int ww = 0; ww < AW; ++ww) v += *(const f32x4*)&red[ww][i / (NR * 4)][col];
          *(f32x4*)(a.S + ((int64_t)blockIdx.z * a.T + t0 + list[at]) * a.rank + col) = v;
        }
        __syncthreads();
      }
    }
  }
}

// sum of the partials of 8 columns of S, in range order
__device__ __forceinline__ void sum_parts(const AdaptersArgs& a, const float* sp, float (&s)[8]) {
  f32x4 v[4][2];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float* p = sp + (int64_t)min(i, a.nks - 1) * a.T * a.rank;
    v[i][0] = *(const f32x4*)p;
    v[i][1] = *(const f32x4*)(p + 4);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (i >= a.nks) break;
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      s[x] += v[i][0][x];
      s[4 + x] += v[i][1][x];
    }
  }
}

// Four outputs of a row of base, and of Y, by bounded buffers: what lies past the
// rows or the outputs reads zeros and is not written, with no branch.  (A wait
// after a branch is for every load in flight: with tests around the accesses the
// loads that were sent ahead hid nothing, and 4096 rows of 4096 outputs took 47 us,
// not 40.)  VEC: in one access.
constexpr uint32_t kNoRow = 0x80000000u;  // past any 128 rows of outputs

template <bool VEC>
__device__ __forceinline__ f32x4 load_y(__amdgpu_buffer_rsrc_t r, uint32_t row, int64_t col, int64_t d_out) {
  if constexpr (VEC) {
    return __builtin_bit_cast(f32x4, buf_load16(r, col < d_out ? row + (uint32_t)col * 4 : kNoRow, 0));
  } else {
    f32x4 y;
#pragma unroll
    for (int x = 0; x < 4; ++x)
      y[x] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(
          r, col + x < d_out ? row + (uint32_t)(col + x) * 4 : kNoRow, 0, 0));
    return y;
  }
}
template <bool VEC>
__device__ __forceinline__ void store_y(f32x4 y, __amdgpu_buffer_rsrc_t r, uint32_t row, int64_t col,
                                        int64_t d_out) {
  if constexpr (VEC) {
    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, y), r,
                                           col < d_out ? row + (uint32_t)col * 4 : kNoRow, 0, 0);
  } else {
#pragma unroll
    for (int x = 0; x < 4; ++x)
      __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(y[x]), r,
                                            col + x < d_out ? row + (uint32_t)(col + x) * 4 : kNoRow, 0, 0);
  }
}
// `rows` rows of base (none: zeros) or Y from row t0 on
__device__ __forceinline__ __amdgpu_buffer_rsrc_t y_rows(const AdaptersArgs& a, const float* y, int64_t t0,
                                                         int64_t rows) {
  const int64_t n = min(rows, a.T - t0);
  return make_rsrc(y ? y + t0 * a.d_out : a.Y, y ? (uint32_t)(n * a.d_out * 4) : 0u);
}

// Y of a decode step: workgroup (pair, outputs).  Its waves share the planes of
// 16 of the pair's rows and take 16 * OT outputs each at a time, B_e and base of
// the next ones in flight while these multiply.  (One turn per workgroup spent
// most of its time on the way to its first loads: 61 us for 64 pairs of rank
// 64 on 4096 -> 11008.)  NK: 32-column steps of the rank.
constexpr int OT = 2;

template <int NK, bool VEC>
__global__ __launch_bounds__(AW * 64, NK <= 2 ? 2 : 1) void k_ad_expand_step(AdaptersArgs a) {
  __shared__ u32x4 planes[NK][3][64];
  __shared__ uint8_t list[128];
  const int tid = threadIdx.x, l = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lr = l & 15, q = l >> 4;
  TilePairs<2> r(a, 0, blockIdx.z);
  if (!r.next(list, true)) return;  // uniform over the workgroup
  const bool pair = r.e >= 0;
  const __amdgpu_buffer_rsrc_t br =
      make_rsrc(a.B + (int64_t)max(r.e, 0) * a.d_out * a.rank,
                pair ? (uint32_t)(a.d_out * a.rank * 2) : 0u);
  const __amdgpu_buffer_rsrc_t yin = y_rows(a, a.base, 0, 128), yout = y_rows(a, a.Y, 0, 128);
  const float c = !pair ? 0.f : a.scale ? a.scale[r.e] : 1.f;
  const int64_t o0 = ((int64_t)blockIdx.z * AW + w) * (OT * 16);
  const int64_t ostep = (int64_t)gridDim.z * AW * (OT * 16);
  for (int b0 = 0; b0 < r.all; b0 += 16) {
    const int at = b0 + lr;
    const bool live = at < r.n;
    const uint32_t yrow = at < r.all ? (uint32_t)(list[min(at, r.all - 1)] * a.d_out * 4) : kNoRow;
    struct Turn {
      u32x4 b[OT][NK];
      f32x4 y[OT];  // lane l holds token l & 15 and outputs 4 (l >> 4) + i of each 16
    };
    auto load = [&](Turn& u, int64_t o) {
#pragma unroll
      for (int i = 0; i < OT; ++i) {
#pragma unroll
        for (int k = 0; k < NK; ++k) {
          const int64_t row = o + i * 16 + lr;
          const int col = k * 32 + q * 8;
          u.b[i][k] = buf_load16(br, ((row < a.d_out) & (col < a.rank))
                                         ? (uint32_t)((row * a.rank + col) * 2) : kOutOfRange, 0);
        }
        u.y[i] = load_y<VEC>(yin, yrow, o + i * 16 + q * 4, a.d_out);
      }
    };
    auto use = [&](Turn& u, int64_t o) {
      f32x4 acc[OT];
#pragma unroll
      for (int i = 0; i < OT; ++i) acc[i] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int k = 0; k < NK; ++k)
#pragma unroll
        for (int x = 0; x < 3; ++x) {
          const u32x4 pl = planes[k][x][l];
#pragma unroll
          for (int i = 0; i < OT; ++i)
            acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, u.b[i][k]),
                                                            __builtin_bit_cast(bf16x8, pl), acc[i],
                                                            0, 0, 0);
        }
#pragma unroll
      for (int i = 0; i < OT; ++i) {
#pragma unroll
        for (int x = 0; x < 4; ++x) u.y[i][x] = live ? fmaf(c, acc[i][x], u.y[i][x]) : u.y[i][x];
        store_y<VEC>(u.y[i], yout, yrow, o + i * 16 + q * 4, a.d_out);
      }
    };
    Turn u0, u1;
    load(u0, o0);
    // a thread sums the partials of 4 columns of a row
    if (b0 > 0) __syncthreads();
    for (int i = tid; i < NK * 128; i += AW * 64) {
      const int sr = i / (NK * 8), sc = i % (NK * 8) * 4;
      f32x4 s = {0.f, 0.f, 0.f, 0.f};
      if (b0 + sr < r.n && sc < a.rank) {
        const float* sp = a.S + (int64_t)list[b0 + sr] * a.rank + sc;
        f32x4 v[8];
#pragma unroll
        for (int p = 0; p < 8; ++p) v[p] = *(const f32x4*)(sp + (int64_t)min(p, a.nks - 1) * a.T * a.rank);
#pragma unroll
        for (int p = 0; p < 8; ++p)
          if (p < a.nks) s += v[p];
      }
      const float s8[8] = {s.x, s.y, s.z, s.w, 0.f, 0.f, 0.f, 0.f};
      u32x4 pl[3];
      split24<true>(s8, pl);
#pragma unroll
      for (int x = 0; x < 3; ++x)
        reinterpret_cast<u32x2*>(&planes[sc / 32][x][sc % 32 / 8 * 16 + sr])[sc / 4 % 2] =
            u32x2{pl[x].x, pl[x].y};
    }
    __syncthreads();
    for (int64_t o = o0; o < a.d_out; o += 2 * ostep) {  // (past the outputs: nothing)
      load(u1, o + ostep);
      use(u0, o);
      load(u0, o + 2 * ostep);
      use(u1, o + ostep);
    }
  }
}

// Both products of a small decode step in one launch: workgroup (pair, outputs)
// forms its pair's S itself, from A_e in L2.  That costs every workgroup the
// whole of A_e, and saves a launch and the way of S through memory; see
// ad_one_launch for where it pays.
constexpr int SW = 8;        // waves
constexpr int ST = 2;        // turns of 16 * OT outputs a wave

template <int NK>
__global__ __launch_bounds__(SW * 64) void k_ad_step(AdaptersArgs a) {
  constexpr int NR = 2 * NK, PITCH = 32 * NK + 4;
  __shared__ float part[SW][16][PITCH];
  __shared__ u32x4 planes[NK][3][64];
  __shared__ uint8_t list[128];
  const int tid = threadIdx.x, l = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lr = l & 15, q = l >> 4;
  TilePairs<2> r(a, 0, 0);
  if (!r.next(list, true)) return;  // uniform over the workgroup
  const bool pair = r.e >= 0;
  const __amdgpu_buffer_rsrc_t br =
      make_rsrc(a.B + (int64_t)max(r.e, 0) * a.d_out * a.rank,
                pair ? (uint32_t)(a.d_out * a.rank * 2) : 0u);
  const __amdgpu_buffer_rsrc_t ar =
      make_rsrc(a.A + (int64_t)max(r.e, 0) * a.rank * a.d, pair ? (uint32_t)(a.rank * a.d * 2) : 0u);
  const __amdgpu_buffer_rsrc_t xr = make_rsrc(a.X, (uint32_t)(a.T * a.d * 2));
  const int64_t o0 = ((int64_t)blockIdx.z * SW + w) * (ST * OT * 16);
  u32x4 bv[ST * OT][NK];
#pragma unroll
  for (int i = 0; i < ST * OT; ++i)
#pragma unroll
    for (int k = 0; k < NK; ++k) {
      const int64_t row = o0 + i * 16 + lr;
      const int col = k * 32 + q * 8;
      bv[i][k] = buf_load16(br, row < a.d_out && col < a.rank
                                    ? (uint32_t)((row * a.rank + col) * 2) : kOutOfRange, 0);
    }
  const float c = !pair ? 0.f : a.scale ? a.scale[r.e] : 1.f;
  for (int b0 = 0; b0 < r.all; b0 += 16) {
    const int at = b0 + lr;
    const bool mine = at < r.all, live = at < r.n;
    const int64_t t = list[min(at, r.all - 1)];
    // S: the waves take 32-channel steps in turn, four steps' loads at a time
    const uint32_t xoff = live ? (uint32_t)(t * a.d * 2) : kOutOfRange;
    f32x4 acc[NR];
#pragma unroll
    for (int n = 0; n < NR; ++n) acc[n] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int64_t k = w * 32; k < a.d; k += 4 * SW * 32) {
      u32x4 xv[4], av[4][NR];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int64_t kk = k + u * (SW * 32) + q * 8;
        const uint32_t cc = kk < a.d ? (uint32_t)kk * 2 : kOutOfRange;
        xv[u] = buf_load16(xr, min(xoff + cc, kOutOfRange), 0);
#pragma unroll
        for (int n = 0; n < NR; ++n)
          av[u][n] = buf_load16(ar, min((uint32_t)((n * 16 + lr) * a.d * 2) + cc, kOutOfRange), 0);
      }
#pragma unroll
      for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int n = 0; n < NR; ++n)
          acc[n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, xv[u]),
                                                          __builtin_bit_cast(bf16x8, av[u][n]),
                                                          acc[n], 0, 0, 0);
    }
    // lane l of a 16 x 16 product holds column l & 15 and rows 4 (l >> 4) + i
#pragma unroll
    for (int n = 0; n < NR; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) part[w][q * 4 + i][n * 16 + lr] = acc[n][i];
    // base is on its way while the waves meet
    const float* bp = a.base ? a.base + t * a.d_out + q * 4 : nullptr;
    float* yp = a.Y + t * a.d_out + q * 4;
    f32x4 y[ST * OT];
#pragma unroll
    for (int i = 0; i < ST * OT; ++i) {
      y[i] = f32x4{0.f, 0.f, 0.f, 0.f};
      const int64_t col = o0 + i * 16 + q * 4;
      if (!bp || !mine) continue;
      if (a.vec) {
        if (col < a.d_out) y[i] = *(const f32x4*)(bp + o0 + i * 16);
      } else {
#pragma unroll
        for (int x = 0; x < 4; ++x)
          if (col + x < a.d_out) y[i][x] = bp[o0 + i * 16 + x];
      }
    }
    __syncthreads();
    if (tid < NK * 128) {
      const int sr = tid / (NK * 8), sc = tid % (NK * 8) * 4;
      f32x4 s = {0.f, 0.f, 0.f, 0.f};
      // (columns past the rank: the zeros read for A_e times an infinite x)
      if (sc < a.rank) {
#pragma unroll
        for (int ww = 0; ww < SW; ++ww) s += *(const f32x4*)&part[ww][sr][sc];
      }
      const float s8[8] = {s.x, s.y, s.z, s.w, 0.f, 0.f, 0.f, 0.f};
      u32x4 pl[3];
      split24<true>(s8, pl);
#pragma unroll
      for (int x = 0; x < 3; ++x)
        reinterpret_cast<u32x2*>(&planes[sc / 32][x][sc % 32 / 8 * 16 + sr])[sc / 4 % 2] =
            u32x2{pl[x].x, pl[x].y};
    }
    __syncthreads();
    f32x4 d[ST * OT];
#pragma unroll
    for (int i = 0; i < ST * OT; ++i) d[i] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < NK; ++k)
#pragma unroll
      for (int x = 0; x < 3; ++x) {
        const u32x4 pl = planes[k][x][l];
#pragma unroll
        for (int i = 0; i < ST * OT; ++i)
          d[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, bv[i][k]),
                                                        __builtin_bit_cast(bf16x8, pl), d[i], 0, 0, 0);
      }
    if (!mine) continue;
#pragma unroll
    for (int i = 0; i < ST * OT; ++i) {
      const int64_t col = o0 + i * 16 + q * 4;
      if (live) {
#pragma unroll
        for (int x = 0; x < 4; ++x) y[i][x] = fmaf(c, d[i][x], y[i][x]);
      }
      if (a.vec) {
        if (col < a.d_out) *(f32x4*)(yp + o0 + i * 16) = y[i];
      } else {
#pragma unroll
        for (int x = 0; x < 4; ++x)
          if (col + x < a.d_out) yp[o0 + i * 16 + x] = y[i][x];
      }
    }
  }
}

// Y of prompts: workgroup (tile, its pairs, outputs).  The planes of up to 64
// gathered rows' S go to LDS, once for the workgroup's four waves, which take
// 16 * OT outputs at a time against 16 rows after another.
template <int NK, bool VEC>
__global__ __launch_bounds__(AW * 64, NK <= 2 ? 2 : 1) void k_ad_expand(AdaptersArgs a) {
  // [block of 16 rows][step][plane][lane]: a wave's read is 1 KiB in a row
  __shared__ u32x4 planes[4][NK][3][64];
  __shared__ uint8_t list[64];
  const int tid = threadIdx.x, l = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lr = l & 15, q = l >> 4;
  const int64_t t0 = prompt_tile() * 64;
  if (t0 >= a.T) return;
  const __amdgpu_buffer_rsrc_t yin = y_rows(a, a.base, t0, 64), yout = y_rows(a, a.Y, t0, 64);
  constexpr int64_t ostep = AW * (OT * 16);
  // a range of outputs in a row, turn by turn
  const int64_t range = ((a.d_out + ostep - 1) / ostep + gridDim.z - 1) / gridDim.z * ostep;
  const int64_t o0 = blockIdx.z * range + w * (OT * 16), o1 = min(a.d_out, (blockIdx.z + 1) * range);
  TilePairs<1> r(a, t0, 0);
  while (r.next(list, true)) {  // uniform over the workgroup
    const float c = r.e < 0 ? 0.f : a.scale ? a.scale[r.e] : 1.f;
    const __amdgpu_buffer_rsrc_t br =
        make_rsrc(a.B + (int64_t)max(r.e, 0) * a.d_out * a.rank,
                  r.e < 0 ? 0u : (uint32_t)(a.d_out * a.rank * 2));
    // NB blocks of 16 rows; the next outputs' factors and base are in flight
    // while these are computed
    auto turns = [&](auto blocks) {
      constexpr int NB = decltype(blocks)::value;
      uint32_t row[NB];
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const int at = b * 16 + lr;
        row[b] = at < r.all ? (uint32_t)(list[min(at, r.all - 1)] * a.d_out * 4) : kNoRow;
      }
      struct Turn {
        u32x4 b[OT][NK];
        f32x4 y[NB][OT];  // lane l holds token l & 15 and outputs 4 (l >> 4) + i of each 16
      };
      auto load = [&](Turn& u, int64_t o) {
#pragma unroll
        for (int i = 0; i < OT; ++i) {
#pragma unroll
          for (int k = 0; k < NK; ++k) {
            const int64_t br_row = o + i * 16 + lr;
            const int col = k * 32 + q * 8;
            u.b[i][k] = buf_load16(br, ((br_row < o1) & (col < a.rank))
                                           ? (uint32_t)((br_row * a.rank + col) * 2) : kOutOfRange, 0);
          }
        }
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int i = 0; i < OT; ++i) u.y[b][i] = load_y<VEC>(yin, row[b], o + i * 16 + q * 4, o1);
      };
      auto use = [&](Turn& u, int64_t o) {
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          const bool live = b * 16 + lr < r.n;
          f32x4 acc[OT];
#pragma unroll
          for (int i = 0; i < OT; ++i) acc[i] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int k = 0; k < NK; ++k)
#pragma unroll
            for (int x = 0; x < 3; ++x) {
              const u32x4 pl = planes[b][k][x][l];
#pragma unroll
              for (int i = 0; i < OT; ++i)
                acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, u.b[i][k]),
                                                                __builtin_bit_cast(bf16x8, pl), acc[i],
                                                                0, 0, 0);
            }
#pragma unroll
          for (int i = 0; i < OT; ++i) {
#pragma unroll
            for (int x = 0; x < 4; ++x) u.y[b][i][x] = live ? fmaf(c, acc[i][x], u.y[b][i][x]) : u.y[b][i][x];
            store_y<VEC>(u.y[b][i], yout, row[b], o + i * 16 + q * 4, o1);
          }
        }
      };
      Turn u0, u1;
      load(u0, o0);
      // S: wave w takes rows 16 w ..
      if (w < NB) {
        const int at = w * 16 + lr;
        const int64_t t = t0 + list[min(at, r.all - 1)];
#pragma unroll
        for (int k = 0; k < NK; ++k) {
          const int col = k * 32 + q * 8;
          float s[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) s[i] = 0.f;
          if (at < r.n && col < a.rank) sum_parts(a, a.S + t * a.rank + col, s);
          u32x4 pl[3];
          split24<true>(s, pl);
#pragma unroll
          for (int i = 0; i < 3; ++i) planes[w][k][i][l] = pl[i];
        }
      }
      __syncthreads();
      for (int64_t o = o0; o < o1; o += 2 * ostep) {  // (past the outputs: nothing)
        load(u1, o + ostep);
        use(u0, o);
        load(u0, o + 2 * ostep);
        use(u1, o + ostep);
      }
    };
    if (r.all <= 16) turns(std::integral_constant<int, 1>{});
    else turns(std::integral_constant<int, 4>{});
    __syncthreads();
  }
}

}  // namespace

hipError_t launch_ad_step(const AdaptersArgs& a, const Launch& L) {
  const int64_t per = SW * ST * OT * 16, blocks = (a.d_out + per - 1) / per;
  const dim3 grid(1, (unsigned)a.T, (unsigned)blocks), blk(SW * 64);
  switch ((a.rank + 31) / 32) {
    case 1: return ext_launch(k_ad_step<1>, grid, blk, 0, L, a);
    case 2: return ext_launch(k_ad_step<2>, grid, blk, 0, L, a);
    default: return hipErrorInvalidValue;
  }
}

hipError_t launch_ad_shrink(const AdaptersArgs& a, int slots, const Launch& L) {
  const bool step = a.T <= kAdStepTokens;
  const int64_t tiles = (a.T + (step ? 127 : 63)) / (step ? 128 : 64);
  if (tiles == 0 || a.n == 0) return hipSuccess;
  const dim3 grid(step ? 1u : (unsigned)((tiles + 7) / 8 * 8), (unsigned)slots, (unsigned)a.nks);
  const dim3 blk(AW * 64);
#define TTQ_AD_SHRINK(NR)                                                         \
  return step ? ext_launch(k_ad_shrink<2, NR, 1>, grid, blk, 0, L, a)             \
              : ext_launch(k_ad_shrink<1, NR, NR <= 4 ? 4 : 2>, grid, blk, 0, L, a);
  switch ((a.rank + 15) / 16) {
    case 1: TTQ_AD_SHRINK(1)
    case 2: TTQ_AD_SHRINK(2)
    case 3: case 4: TTQ_AD_SHRINK(4)
    case 5: case 6: TTQ_AD_SHRINK(6)
    case 7: case 8: TTQ_AD_SHRINK(8)
    default: return hipErrorInvalidValue;
  }
#undef TTQ_AD_SHRINK
}

hipError_t launch_ad_expand(const AdaptersArgs& a, int slots, const Launch& L) {
  const bool step = a.T <= kAdStepTokens;
  const int64_t tiles = (a.T + (step ? 127 : 63)) / (step ? 128 : 64);
  const int64_t per = AW * OT * 16;
  int64_t blocks = (a.d_out + per - 1) / per;
  if (tiles == 0 || blocks == 0) return hipSuccess;
  // several blocks of outputs a workgroup, while that leaves enough of them for
  // the chip: two per compute unit for prompts (4096 rows: 36.5 us; one 37.9, four
  // 40.4), eight for decode steps, where some find no pair
  blocks = std::max<int64_t>(1, std::min(blocks, step ? 2048 / a.T : 512 / tiles));
  // and workgroups of their own for a tile's further pairs, of which most find
  // none, only where the others leave compute units idle (557 rows of four prompts,
  // rank 24 on 3904 -> 3076: 20.0 us, 25.7 with four for every tile)
  if (!step) slots = (int)std::max<int64_t>(1, std::min<int64_t>(slots, 256 / (tiles * blocks)));
  const dim3 grid(step ? 1u : (unsigned)((tiles + 7) / 8 * 8), (unsigned)slots, (unsigned)blocks);
  const dim3 blk(AW * 64);
#define TTQ_AD_EXPAND(NK)                                                          \
  if (step)                                                                        \
    return a.vec ? ext_launch(k_ad_expand_step<NK, true>, grid, blk, 0, L, a)      \
                 : ext_launch(k_ad_expand_step<NK, false>, grid, blk, 0, L, a);    \
  return a.vec ? ext_launch(k_ad_expand<NK, true>, grid, blk, 0, L, a)             \
               : ext_launch(k_ad_expand<NK, false>, grid, blk, 0, L, a);
  switch ((a.rank + 31) / 32) {
    case 1: TTQ_AD_EXPAND(1)
    case 2: TTQ_AD_EXPAND(2)
    case 3: TTQ_AD_EXPAND(3)
    case 4: TTQ_AD_EXPAND(4)
    default: return hipErrorInvalidValue;
  }
#undef TTQ_AD_EXPAND
}

}  // namespace ttq
