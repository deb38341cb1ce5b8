// A mixture-of-experts layer for a few tokens, from stored codes: the experts'
// gate, up and down projections are kept as ttq_quantize leaves them and
// contracted with the tokens that choose them.
//
//   l_e = W_r[e] . x              scores, in float64 (a near tie has one answer)
//   chosen: the k largest l_e, equal ones by the lower index, NaN last
//   w_j = exp(l_j - max) / sum    over the chosen (renorm) or all experts
//   h   = silu(G x') * (U x'),    y = sum_j w_j D_j h'
//
// where a product with stored codes is, per group g of a row,
//   s_g sum_{i in g} q_i x'_i + m_g sum_{i in g} x'_i,   x' = x D^{-1/2}.
//
// The codes are exact in bf16, and x' is the sum of three bf16 planes
// (split24), so float32 accumulation on the matrix cores is as exact as
// float32 products.  The planes are COLUMNS of the products: an expert that n
// tokens chose has 3 n of them, 16 to a matrix instruction, and a token's three
// results are added at the end.  One token then costs one instruction per 32
// channels and 16 rows, not three, and 5 tokens no more than one.
//
// Bound by the codes and scales it reads while tokens are few: one token, 2 of 8
// experts of 4096 / 11008, 4 bits in groups of 128: 25 us for 101 MB of gate and
// up, 18 us for 51 MB of down (4.1 and 2.8 TB/s; codes alone stream in 18 and
// 11).  16 tokens, 8 of 64 experts of 2048 / 1408: 47 us for 184 MB, 27 for 92.
// Where they are many, bound by waiting: 97 tokens, 4 of 16 2-bit experts of 4096
// / 2816, take 177 and 85 us, with the vector units busy 35 and 27 % of it, the
// matrix ones 20 and 15 %, and 1.3 and 1.1 waves a SIMD, which wait (barriers,
// loads) two fifths of their time.
#include <algorithm>
#include <cmath>

#include "codes.h"
#include "ttq_internal.h"

namespace ttq {

namespace {

// The order in which the expansion of 8 codes leaves their channels: that of
// the bytes which hold them (1: 4-bit containers, even codes first; 2: 2-bit
// containers, channel i beside i + 4; 0: as they are).
__host__ __device__ constexpr int order_of(int cb, bool f8) {
  return f8 ? 0 : cb == 4 ? 1 : cb == 2 ? 2 : 0;
}
__host__ __device__ constexpr int code_order(int order, int i) {
  return order == 1 ? (i < 4 ? 2 * i : 2 * (i - 4) + 1) : order == 2 ? i / 2 + 4 * (i % 2) : i;
}

// ------------------------------------------------------------- routing
// does expert a (score la) come before expert b?
__device__ __forceinline__ bool before(double la, int a, double lb, int b) {
  const bool na = la != la, nb = lb != lb;
  if (na || nb) return na == nb ? a < b : nb;
  return la > lb || (la == lb && a < b);
}

// one wave's part of a score: channels c0 + 8 l + step i, below d
__device__ __forceinline__ double score_part(const bf16_t* x, const bf16_t* r, int64_t c0,
                                             int64_t step, int64_t d) {
  double s0 = 0.0, s1 = 0.0;
  // four steps' loads at a time (past the end: the same channels, not added)
  for (int64_t c = c0; c < d; c += 4 * step) {
    u32x4 xv[4], rv[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t ci = c + i * step < d ? c + i * step : c;
      xv[i] = *(const u32x4*)(x + ci);
      rv[i] = *(const u32x4*)(r + ci);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (c + i * step >= d) break;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        // (in float64: exact also where the product leaves float32's range)
        s0 = fma((double)bf16lo(xv[i][j]), (double)bf16lo(rv[i][j]), s0);
        s1 = fma((double)bf16hi(xv[i][j]), (double)bf16hi(rv[i][j]), s1);
      }
    }
  }
  return s0 + s1;
}
__device__ __forceinline__ double wave_sum(double s) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) s += __shfl_xor(s, off);
  return s;
}

// scores of many experts: a wave per (token, expert)
__global__ __launch_bounds__(256) void k_moe_score(MoeArgs a) {
  const int l = threadIdx.x & 63, e = blockIdx.x * 4 + (threadIdx.x >> 6);
  const int64_t t = blockIdx.y;
  if (e >= a.E) return;
  const double s = wave_sum(score_part(a.X + t * a.d, a.router + (int64_t)e * a.d, l * 8, 512, a.d));
  if (l == 0) a.score[t * a.E + e] = s;
}

// Where piece (of 8 channels) c / 8 of a row of planes lies, and in which
// order its channels: a lane of the products holds a contiguous quarter of a
// group's codes, 8 for each matrix instruction, in the order their expansion
// leaves them in (code_order).  Rows are [group][plane][GS].
__host__ __device__ constexpr int64_t plane_piece(int64_t c, int gs) {
  const int64_t g = c / gs, i = c % gs, q = i / (gs / 4), k = i % (gs / 4) / 8;
  return g * 3 * gs + k * 32 + q * 8;
}

// The scores of a token (its own, when few), every expert's rank by counting
// those before it, the weights, and x' of the chosen ones as planes.  Several
// workgroups a token, each of which finds the chosen experts and writes a part of
// the planes (16 tokens, 8 experts of 2048 channels each: 6.4 us with two, 7.9 with
// one).
template <int ORDER>
__global__ __launch_bounds__(1024) void k_moe_route(MoeArgs a) {
  __shared__ double score[kMoeMaxE];
  __shared__ double part[16];
  __shared__ int rank[kMoeMaxE];
  __shared__ int chosen[kMoeMaxK];
  const int tid = threadIdx.x, l = tid & 63, w = tid >> 6;
  const int64_t t = blockIdx.x;
  const bf16_t* x = a.X + t * a.d;
  if (a.score) {
    if (tid < a.E) score[tid] = a.score[t * a.E + tid];
  } else if (a.E <= 8) {  // two waves an expert
    const int e = w >> 1;
    if (e < a.E) {
      const double s = wave_sum(score_part(x, a.router + (int64_t)e * a.d, (w & 1) * 512 + l * 8, 1024, a.d));
      if (l == 0) part[w] = s;
    }
    __syncthreads();
    if (tid < a.E) score[tid] = part[2 * tid] + part[2 * tid + 1];
  } else {
    for (int e = w; e < a.E; e += 16) {
      const double s = wave_sum(score_part(x, a.router + (int64_t)e * a.d, l * 8, 512, a.d));
      if (l == 0) score[e] = s;
    }
  }
  if (tid < a.E) rank[tid] = 0;
  __syncthreads();
  for (int i = tid; i < a.E * a.E; i += 1024) {
    const int e = i / a.E, o = i % a.E;
    if (o != e && before(score[o], o, score[e], e)) atomicAdd(&rank[e], 1);
  }
  __syncthreads();
  if (tid < a.E && rank[tid] < a.k) chosen[rank[tid]] = tid;
  __syncthreads();
  if (blockIdx.y == 0 && tid < a.k) {
    const int e = chosen[tid];
    const double top = score[chosen[0]];
    float sum = 0.f;
    if (a.renorm)
      for (int j = 0; j < a.k; ++j) sum += expf((float)(score[chosen[j]] - top));
    else
      for (int j = 0; j < a.E; ++j) sum += expf((float)(score[j] - top));
    a.ids[t * a.k + tid] = e;
    a.w[t * a.k + tid] = expf((float)(score[e] - top)) / sum;
  }
  const int np = (int)(a.d / 8);
  for (int i = blockIdx.y * 1024 + tid; i < a.k * np; i += gridDim.y * 1024) {
    const int j = i / np;
    const int64_t c = (int64_t)(i % np) * 8;
    const u32x4 xv = *(const u32x4*)(x + c);
    const float* dhi = a.gu_dhi + (int64_t)chosen[j] * a.d + c;
    const f32x4 h0 = *(const f32x4*)dhi, h1 = *(const f32x4*)(dhi + 4);
    const float v[8] = {bf16lo(xv.x) * h0.x, bf16hi(xv.x) * h0.y, bf16lo(xv.y) * h0.z,
                        bf16hi(xv.y) * h0.w, bf16lo(xv.z) * h1.x, bf16hi(xv.z) * h1.y,
                        bf16lo(xv.w) * h1.z, bf16hi(xv.w) * h1.w};
    float u[8];
#pragma unroll
    for (int b = 0; b < 8; ++b) u[b] = v[code_order(ORDER, b)];
    u32x4 pl[3];
    split24(u, pl);
    bf16_t* dst = a.Xp + (t * a.k + j) * 3 * a.d + plane_piece(c, a.gs);
#pragma unroll
    for (int b = 0; b < 3; ++b) *(u32x4*)(dst + b * a.gs) = pl[b];
  }
}

// ------------------------------------------------------------ products
// 8 codes -> 4 bf16 pairs, exactly.  A code of up to 4 bits, read as an E4M3
// pattern, is code * 2^-9 (0..7 are its subnormals, 8..15 its first binade),
// so the E4M3 conversion with a scale of 2^9 expands two codes at once.  The
// pairs come in the order of the bytes that hold the codes; see code_order.
template <int CB, int GS, bool F8>
__device__ __forceinline__ u32x4 codes_bf16(const GroupCodes<CB, GS>& gc, int k) {
  const u32x2 raw = CB == 2 ? u32x2{gc.w[k / 2], 0u} : step_codes<CB, GS>(gc, k);
  auto pair = [](unsigned w, bool hi, float sc) {
    return hi ? __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, sc, true))
              : __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, sc, false));
  };
  if constexpr (F8) {
    return u32x4{pair(raw.x, false, 1.f), pair(raw.x, true, 1.f), pair(raw.y, false, 1.f),
                 pair(raw.y, true, 1.f)};
  } else if constexpr (CB == 8) {
    float f[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[i] = (float)((raw.x >> (8 * i)) & 0xFFu);
      f[4 + i] = (float)((raw.y >> (8 * i)) & 0xFFu);
    }
    u32x4 r;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      r[i] = __builtin_amdgcn_perm(__float_as_uint(f[2 * i + 1]), __float_as_uint(f[2 * i]), 0x07060302u);
    return r;
  } else if constexpr (CB == 4) {
    const unsigned lo = raw.x & 0x0F0F0F0Fu, hi = (raw.x >> 4) & 0x0F0F0F0Fu;
    return u32x4{pair(lo, false, 512.f), pair(lo, true, 512.f), pair(hi, false, 512.f),
                 pair(hi, true, 512.f)};
  } else if constexpr (CB == 2) {
    // codes 0 4 | 1 5 | 2 6 | 3 7 (the two bytes of the step's 16 bits; two
    // steps share a word, whose masks the compiler forms once)
    const unsigned a = raw.x & 0x03030303u, b = (raw.x >> 2) & 0x03030303u;
    const unsigned c = (raw.x >> 4) & 0x03030303u, d = (raw.x >> 6) & 0x03030303u;
    const bool hi = k % 2;
    return u32x4{pair(a, hi, 512.f), pair(b, hi, 512.f), pair(c, hi, 512.f), pair(d, hi, 512.f)};
  } else {
    unsigned p[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      p[i] = ((raw.x >> (2 * i)) & 1u) * 0x3F80u + ((raw.x >> (2 * i + 1)) & 1u) * 0x3F800000u;
    return u32x4{p[0], p[1], p[2], p[3]};
  }
}

// The expert of blockIdx.y and the choices (pairs) that name it, in order, in
// list[]: n of them (0: none).  Up to 64 choices: the blockIdx.y-th distinct
// expert of them in order of appearance; more: expert blockIdx.y itself.  Every
// wave finds them for itself and writes the same list, so no barrier is needed.
struct Mine {
  int e, n;
};
__host__ inline int expert_slots(int64_t P, int E) {
  return P <= 64 ? (int)std::min(P, (int64_t)E) : E;
}
__device__ __forceinline__ Mine my_expert(const MoeArgs& a, int16_t* list) {
  const int l = threadIdx.x & 63;
  const int P = (int)a.T * a.k, slot = blockIdx.y;
  const uint64_t below = (1ull << l) - 1ull;
  if (P <= 64) {
    const int id = l < P ? a.ids[l] : -1;
    uint64_t left = __ballot(l < P);
    int e = 0;
    uint64_t same = 0;
    for (int i = 0; i <= slot; ++i) {
      if (!left) return Mine{0, 0};
      e = __builtin_amdgcn_readlane(id, __builtin_ctzll(left));
      same = __ballot(id == e);
      left &= ~same;
    }
    if (id == e) list[__builtin_popcountll(same & below)] = (int16_t)l;
    return Mine{e, (int)__builtin_popcountll(same)};
  }
  int n = 0;
  for (int i0 = 0; i0 < P; i0 += 256) {
    int id[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int at = i0 + i * 64 + l;
      id[i] = at < P ? a.ids[at] : -1;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint64_t m = __ballot(id[i] == slot);
      if (id[i] == slot) list[n + __builtin_popcountll(m & below)] = (int16_t)(i0 + i * 64 + l);
      n += __builtin_popcountll(m);
    }
  }
  return Mine{slot, n};
}

// The rows of one kind of projection of one expert as the products read them.
struct Rows {
  __amdgpu_buffer_rsrc_t c0, c1;  // codes of the first and second kind of row
};
template <int RB, bool UP>
__device__ __forceinline__ Rows expert_rows(const MoeArgs& a, int e, int64_t row0) {
  const int64_t N = UP ? a.ff : a.d, rb = UP ? a.gu_rb : a.dn_rb;
  const int64_t nrow = max((int64_t)0, min((int64_t)RB * 16, N - row0));
  const int64_t erow = (int64_t)e * (UP ? 2 * a.ff : a.d) + min(row0, N - 1);
  const uint8_t* codes = UP ? a.gu : a.dn;
  Rows r;
  // bounded buffers: rows past the last read zeros
  r.c0 = make_rsrc(codes + erow * rb, (uint32_t)(nrow * rb));
  r.c1 = UP ? make_rsrc(codes + (erow + a.ff) * rb, (uint32_t)(nrow * rb)) : r.c0;
  return r;
}

// The scales and offsets of `rows` rows of one kind from row0 on, scale groups
// [g0, g0 + ng), to LDS as sm[row][group] (an odd pitch: 16 rows of a read in
// 16 banks): rows are contiguous in memory, so each is fetched once.  Groups
// up to `full` (of a last slot that the rows do not fill) count nothing.
__device__ __forceinline__ void stage_scales(float2* sm, int pitch, const float* s, const float* m,
                                             int64_t row0, int rows, int64_t nrow, int64_t Gs,
                                             int64_t g0, int ng, int full) {
  const int sh = 32 - __builtin_clz(full - 1 | 1);  // lanes of a row: a power of two
  // four elements' loads at a time (past the end: the last one again)
  for (int i0 = threadIdx.x; i0 < rows << sh; i0 += 4 * blockDim.x) {
    float2 v[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int i = min(i0 + u * (int)blockDim.x, (rows << sh) - 1);
      const int r = i >> sh, g = i & ((1 << sh) - 1);
      const int64_t at = (row0 + min((int64_t)r, nrow - 1)) * Gs + g0 + min(g, ng - 1);
      v[u] = float2{s[at], m[at]};
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int i = i0 + u * (int)blockDim.x;
      const int r = i >> sh, g = i & ((1 << sh) - 1);
      if (r < rows && g < full) sm[r * pitch + g] = g < ng ? v[u] : float2{0.f, 0.f};
    }
  }
}

// The codes come in slots of SB bytes of each row: a wave loads whole lines of
// its RT * 16 rows (16 bytes a lane, SB / 16 lanes a row) into registers, and
// puts them in its own part of LDS, from where the products read the pieces
// their lanes need.  (Read in place, a lane's piece of a group makes 64-byte
// requests, and with those the kernel stayed at 3.4 TB/s whatever its tiles.)
// In LDS the 16-byte pieces of row r are swapped by r / 2, which puts the 16
// rows of a read on all banks.
template <int CB, int GS, bool HALF>
struct Slot {
  // HALF lines, while they hold 128 channels, take half the LDS, and more
  // workgroups share a compute unit: 46 + 27 us for 16 tokens over 64 experts of
  // 2048 / 1408, where whole lines took 53 + 33.  (The down product of one token,
  // which a few workgroups do: 20.7 us with half lines, 17.9 with whole ones.)
  static constexpr int SB = CB == 1 || (HALF && CB <= 4) ? 64 : 128;
  static constexpr int SG = SB * 8 / CB / GS;   // groups
  static constexpr int LPR = SB / 16;           // lanes a row
  static constexpr int RPI = 64 / LPR;          // rows a load
};
template <int CB, int GS, int RT, bool HALF>
struct Stage {
  u32x4 c[RT * 16 / Slot<CB, GS, HALF>::RPI];
};
template <int CB, int GS, int RT, int RB, bool HALF>
__device__ __forceinline__ void load_codes_of(Stage<CB, GS, RT, HALF>& st, const Rows& r, int64_t rb,
                                              int slot, int end, int l) {
  // (a slot at or past the end: nothing is read)
  const uint32_t at = slot < end ? (uint32_t)(slot * Slot<CB, GS, HALF>::SB) : kOutOfRange;
  using S = Slot<CB, GS, HALF>;
  constexpr int PER = RB * 16 / S::RPI;  // loads of one kind of row
  // Behind a row's end lie the next row's codes, and zeros are put in their place:
  // the scales of those groups are 0, but 0 times an E4M3 NaN is not.
  const uint32_t col = l % S::LPR * 16;
  const uint32_t off = slot * S::SB + col < (uint32_t)rb ? l / S::LPR * (uint32_t)rb + col : kOutOfRange;
#pragma unroll
  for (int i = 0; i < RT * 16 / S::RPI; ++i)
    st.c[i] = buf_load16(i < PER ? r.c0 : r.c1, off + (uint32_t)((i % PER) * S::RPI * rb), at);
}
template <int CB, int GS, int RT, bool HALF>
__device__ __forceinline__ void put_codes(const Stage<CB, GS, RT, HALF>& st, uint8_t* lds, int l) {
  using S = Slot<CB, GS, HALF>;
#pragma unroll
  for (int i = 0; i < RT * 16 / S::RPI; ++i) {
    const int row = i * S::RPI + l / S::LPR;
    *(u32x4*)(lds + row * S::SB + ((l % S::LPR) ^ (row >> 1 & (S::LPR - 1))) * 16) = st.c[i];
  }
}
// the lane's quarter of group j of a slot, row block r
template <int CB, int GS, bool HALF>
__device__ __forceinline__ GroupCodes<CB, GS> get_codes(const uint8_t* lds, int r, int j, int lr, int q) {
  using S = Slot<CB, GS, HALF>;
  constexpr int NB = GroupCodes<CB, GS>::NB;
  const int row = r * 16 + lr, at = j * (GS * CB / 8) + q * NB;
  const int swz = row >> 1 & (S::LPR - 1);
  const uint8_t* base = lds + row * S::SB;
  GroupCodes<CB, GS> c;
  if constexpr (NB >= 16) {
#pragma unroll
    for (int i = 0; i < NB / 16; ++i) {
      const u32x4 v = *(const u32x4*)(base + ((at / 16 + i) ^ swz) * 16);
      c.w[4 * i] = v.x; c.w[4 * i + 1] = v.y; c.w[4 * i + 2] = v.z; c.w[4 * i + 3] = v.w;
    }
  } else {
    const uint8_t* p = base + ((at / 16) ^ swz) * 16 + at % 16;
    if constexpr (NB == 8) {
      const u32x2 v = *(const u32x2*)p;
      c.w[0] = v.x;
      c.w[1] = v.y;
    } else if constexpr (NB == 4) {
      c.w[0] = *(const unsigned*)p;
    } else if constexpr (NB == 2) {
      c.w[0] = *(const uint16_t*)p;
    } else {
      c.w[0] = *p;
    }
  }
  return c;
}

// group j of a slot: RT row blocks against NB * 16 columns of planes x
template <int CB, bool F8, int GS, int RT, int NB, bool HALF>
__device__ __forceinline__ void use_group(const uint8_t* lds, int j, const u32x4 (&x)[GS / 32][NB],
                                          const float2* sm, int pitch, int lr, int q,
                                          f32x4 (&acc)[RT][NB]) {
  const u32x4 ones = {0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u};
  f32x4 sx[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    sx[b] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < GS / 32; ++k)
      sx[b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, x[k][b]),
                                                     __builtin_bit_cast(bf16x8, ones), sx[b], 0, 0, 0);
  }
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    const float2 sc = sm[r * 16 * pitch];
    const GroupCodes<CB, GS> c = get_codes<CB, GS, HALF>(lds, r, j, lr, q);
    f32x4 p[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) p[b] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < GS / 32; ++k) {
      const u32x4 cq = codes_bf16<CB, GS, F8>(c, k);
#pragma unroll
      for (int b = 0; b < NB; ++b)
        p[b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, x[k][b]),
                                                      __builtin_bit_cast(bf16x8, cq), p[b], 0, 0, 0);
    }
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        acc[r][b][i] = fmaf(sc.x, p[b][i], fmaf(sc.y, sx[b][i], acc[r][b][i]));
  }
}

// slots s0, s0 + step, ... below s1 (groups below G), the next one's loads in
// flight while one is contracted; sm: the lane's row of the staged scales,
// whose first group is gs0.  stage() puts them there while the first codes are
// on their way.
template <int CB, bool F8, int GS, int RT, int RB, int NB, bool HALF, class F>
__device__ __forceinline__ void contract(const Rows& r, const bf16_t* const (&col)[NB], int64_t rb,
                                         int s0, int s1, int step, int G, uint8_t* lds,
                                         const float2* sm, int pitch, int gs0, int gdiv, int l,
                                         f32x4 (&acc)[RT][NB], F&& stage) {
  using S = Slot<CB, GS, HALF>;
  constexpr int NKS = GS / 32;
  const int lr = l & 15, q = l >> 4;
  // planes of XG groups at a time, those of a slot's first groups asked for
  // before its codes are waited for
  constexpr int XG = S::SG * NKS * NB <= 12 ? S::SG : S::SG * NKS * NB <= 24 ? S::SG / 2 : 1;
  u32x4 x[XG][NKS][NB];
  auto planes = [&](int slot, int j) {
    const int gg = min(slot * S::SG + j, G - 1);  // (a group past the end is not used)
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int k = 0; k < NKS; ++k)
        x[j % XG][k][b] = *(const u32x4*)(col[b] + (int64_t)gg * 3 * GS + k * 32 + q * 8);
  };
  Stage<CB, GS, RT, HALF> st;
  load_codes_of<CB, GS, RT, RB, HALF>(st, r, rb, s0, s1, l);
#pragma unroll
  for (int j = 0; j < XG; ++j) planes(s0, j);
  __builtin_amdgcn_sched_barrier(0);
  stage();
  for (int s = s0; s < s1; s += step) {
    put_codes<CB, GS, RT, HALF>(st, lds, l);
    load_codes_of<CB, GS, RT, RB, HALF>(st, r, rb, s + step, s1, l);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int j = 0; j < S::SG; ++j) {
      if (j > 0 && j % XG == 0) {
#pragma unroll
        for (int i = 0; i < XG; ++i) planes(s, j + i);
      }
      use_group<CB, F8, GS, RT, NB, HALF>(lds, j, x[j % XG], sm + (((s * S::SG + j) >> gdiv) - gs0), pitch,
                                    lr, q, acc);
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int j = 0; j < XG; ++j) planes(s + step, j);
  }
}

// silu(g) u D^{-1/2} as the planes of the down product
template <int ORDER>
__device__ __forceinline__ void store_hidden(const MoeArgs& a, int64_t p, int64_t row, float gate,
                                             float up, float dhi) {
  const float h = gate / (1.f + expf(-gate)) * up * dhi;
  const unsigned hi = __float_as_uint(h) & 0xffff0000u;
  const float r1 = h - __uint_as_float(hi);
  const unsigned mid = __float_as_uint(r1) & 0xffff0000u;
  const unsigned lo = __float_as_uint(r1 - __uint_as_float(mid));
  int at = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (code_order(ORDER, j) == (int)(row & 7)) at = j;
  bf16_t* dst = a.H + p * 3 * a.ff + plane_piece(row & ~(int64_t)7, a.gs) + at;
  dst[0] = (bf16_t)(hi >> 16);
  dst[a.gs] = (bf16_t)(mid >> 16);
  dst[2 * a.gs] = (bf16_t)(lo >> 16);
}

// One expert's rows against the tokens that chose it, NB * 16 columns at a
// time: every pass reads the codes again.  The W waves are KS ranges of groups (taken in turn) by W / KS blocks
// of rows.  UP: a block is RT/2 * 16 gate rows and the up rows beside them, and
// the result goes to H; else RT * 16 down rows, and the weighted result to Yp.
template <int CB, bool F8, int GS, int RT, int NB, int W, int KS, bool UP>
__global__ __launch_bounds__(W * 64, 4) void k_moe_proj(MoeArgs a) {
  constexpr int RB = UP ? RT / 2 : RT;
  constexpr int ORDER = order_of(CB, F8);
  __shared__ int16_t list[kMoeMaxT];
  // the waves' slots of codes and the staged scales, then (in their place) the
  // products [column][row]
  extern __shared__ __attribute__((aligned(16))) float dyn[];
  float(*red)[RT][NB][16][17] = reinterpret_cast<float(*)[RT][NB][16][17]>(dyn);
  const int tid = threadIdx.x, l = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lr = l & 15, q = l >> 4;
  const Mine mine = my_expert(a, list);
  const int n = mine.n, e = mine.e;
  if (n == 0) return;  // uniform

  const int64_t N = UP ? a.ff : a.d, rb = UP ? a.gu_rb : a.dn_rb;
  const int G = (int)((UP ? a.d : a.ff) / GS);
  const int gdiv = a.gshift - __builtin_ctz((unsigned)GS);
  const int64_t row0 = ((int64_t)blockIdx.x * (W / KS) + w / KS) * (RB * 16);
  const Rows rows = expert_rows<RB, UP>(a, e, row0);
  const bf16_t* xp = UP ? a.Xp : a.H;
  const int64_t K3 = 3 * (UP ? a.d : a.ff);
  constexpr int WR = RB * 16 * (W / KS);  // rows (of one kind) of the workgroup
  const int64_t wrow0 = (int64_t)blockIdx.x * WR, wn = min((int64_t)WR, N - wrow0);
  const int64_t erow = (int64_t)e * (UP ? 2 * a.ff : a.d) + wrow0;
  const int64_t Gs = (UP ? a.d : a.ff) >> a.gshift;
  const float* ss = UP ? a.gu_s : a.dn_s;
  const float* mm = UP ? a.gu_m : a.dn_m;
  // scale groups staged at a time; the lane's first row there: its row block's
  // rows (of both kinds) are 16 RT rows one after another
  const int pitch = a.pitch;
  constexpr int SLOT = RT * 16 * Slot<CB, GS, true>::SB;
  uint8_t* slot = reinterpret_cast<uint8_t*>(dyn) + w * SLOT;
  float2* sm = reinterpret_cast<float2*>(reinterpret_cast<uint8_t*>(dyn) + W * SLOT);
  const float2* sml = sm + ((w / KS) * RT * 16 + lr) * pitch;

  // a thread's row is the same in every turn of the last loop below; its factor
  // is asked for ahead of the codes
  static_assert(W * 64 % WR == 0, "rows of a workgroup");
  const int rr = tid % WR;
  const int64_t row = wrow0 + rr;
  const float dhi = UP && row < N ? a.dn_dhi[(int64_t)e * a.ff + row] : 0.f;

  // tokens of a pass: their columns are 3 j, 3 j + 1, 3 j + 2
  constexpr int TP = NB * 16 / 3;
  for (int t0 = 0; t0 < n; t0 += TP) {
    const int here = min(TP, n - t0);
    const bf16_t* col[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      // columns past the last repeat the first (never stored)
      const int c = b * 16 + lr < 3 * here ? b * 16 + lr : 0;
      col[b] = xp + (int64_t)list[t0 + c / 3] * K3 + (c % 3) * GS;
    }
    f32x4 acc[RT][NB];
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int b = 0; b < NB; ++b) acc[r][b] = f32x4{0.f, 0.f, 0.f, 0.f};
    constexpr int SG = Slot<CB, GS, true>::SG;
    for (int gs0 = 0; gs0 < Gs; gs0 += a.ngs) {
      const int ng = min(a.ngs, (int)Gs - gs0);
      const int g1 = min(G, (gs0 + ng) << gdiv);
      const int full = ((g1 + SG - 1) / SG * SG >> gdiv) - gs0;
      contract<CB, F8, GS, RT, RB, NB, true>(
          rows, col, rb, (gs0 << gdiv) / SG + w % KS, (g1 + SG - 1) / SG, KS, g1, slot, sml, pitch,
          gs0, gdiv, l, acc, [&] {
            if (gs0 > 0) __syncthreads();
            for (int b = 0; b < W / KS; ++b)
              for (int kind = 0; kind < (UP ? 2 : 1); ++kind)
                stage_scales(sm + (b * RT + kind * RB) * 16 * pitch, pitch, ss, mm,
                             erow + kind * a.ff + min((int64_t)b * RB * 16, wn - 1), RB * 16,
                             max((int64_t)1, wn - b * RB * 16), Gs, gs0, ng, full);
            __syncthreads();
          });
    }
    // lane l of a product holds row l & 15 and columns 4 (l >> 4) + i
    __syncthreads();
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int i = 0; i < 4; ++i) red[w][r][b][q * 4 + i][lr] = acc[r][b][i];
    __syncthreads();
    for (int i = tid; i < here * WR; i += W * 64) {
      const int j = i / WR;
      const int wb = rr / (RB * 16), ri = rr % (RB * 16);
      if (row >= N) continue;
      auto value = [&](int r) {
        float v = 0.f;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks)
#pragma unroll
          for (int pl = 0; pl < 3; ++pl) {
            const int c = 3 * j + pl;
            v += red[wb * KS + ks][r][c >> 4][c & 15][ri & 15];
          }
        return v;
      };
      const int64_t p = list[t0 + j];
      if constexpr (UP)
        store_hidden<ORDER>(a, p, row, value(ri >> 4), value(RB + (ri >> 4)), dhi);
      else
        a.Yp[p * a.d + row] = a.w[p] * value(ri >> 4);
    }
    __syncthreads();
  }
}

// The same for experts that many tokens chose, where the planes, not the codes,
// are what the products read most of: they go through LDS, once for the four
// waves of a workgroup, each of which has RT row blocks of its own and all
// channels.  A step is XC channels of NB * 16 columns; the next step's planes,
// and with a slot's first step the next slot's codes and scales, are in flight
// while it is contracted.  (Planes from L2 by every wave: 256 + 115 us for 97
// tokens over 16 2-bit experts of 4096 / 2816, against 177 + 85.)
template <int CB, bool F8, int GS, int NB, bool UP>
__global__ __launch_bounds__(256, 2) void k_moe_wide(MoeArgs a) {
  constexpr int RT = 4, W = 4, RB = UP ? RT / 2 : RT, NKS = GS / 32;
  constexpr int ORDER = order_of(CB, F8);
  using S = Slot<CB, GS, true>;
  constexpr int XC = 128, XG = XC / GS, XK = XC / 32;
  constexpr int NC = S::SB * 8 / CB / XC;           // steps of a slot
  static_assert(NC >= 1 && NC * XG == S::SG, "a slot is whole steps");
  constexpr int NX = (XK * NB + W - 1) / W;         // fragments of a step a wave brings
  constexpr int SLOT = RT * 16 * S::SB, PITCH = S::SG | 1;
  constexpr int WR = RB * 16 * W;                   // rows (of one kind) of the workgroup
  constexpr int PR = UP ? 2 : 1;                    // row blocks of a turn of the epilogue
  constexpr size_t WORK = W * SLOT + W * RT * 16 * PITCH * 8 + XK * NB * 1024;
  constexpr size_t PROD = (size_t)W * PR * NB * 16 * 17 * 4;
  __shared__ __attribute__((aligned(16))) uint8_t dyn[WORK > PROD ? WORK : PROD];
  __shared__ int16_t list[kMoeMaxT];
  const int tid = threadIdx.x, l = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lr = l & 15, q = l >> 4;
  const Mine mine = my_expert(a, list);
  const int n = mine.n, e = mine.e;
  if (n == 0) return;  // uniform

  uint8_t* slot = dyn + w * SLOT;
  float2* sm = reinterpret_cast<float2*>(dyn + W * SLOT);
  u32x4* xl = reinterpret_cast<u32x4*>(dyn + W * SLOT + W * RT * 16 * PITCH * 8);
  float(*red)[PR][NB][16][17] = reinterpret_cast<float(*)[PR][NB][16][17]>(dyn);

  const int64_t N = UP ? a.ff : a.d, rb = UP ? a.gu_rb : a.dn_rb;
  const int G = (int)((UP ? a.d : a.ff) / GS);
  const int gdiv = a.gshift - __builtin_ctz((unsigned)GS);
  const int64_t Gs = (UP ? a.d : a.ff) >> a.gshift;
  const int64_t wrow0 = (int64_t)blockIdx.x * WR, row0 = wrow0 + w * (RB * 16);
  const Rows rows = expert_rows<RB, UP>(a, e, row0);
  const bf16_t* xp = UP ? a.Xp : a.H;
  const int64_t K3 = 3 * (UP ? a.d : a.ff);
  const int ns = (G + S::SG - 1) / S::SG;
  // the row whose scales this thread stages
  const int64_t mine_row = (int64_t)e * (UP ? 2 * a.ff : a.d) + (UP && l >= 32 ? a.ff : 0) +
                           min(row0 + (UP ? l % 32 : l), N - 1);
  const float* sp = (UP ? a.gu_s : a.dn_s) + mine_row * Gs;
  const float* mp = (UP ? a.gu_m : a.dn_m) + mine_row * Gs;
  const u32x4 ones = {0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u};

  constexpr int TP = NB * 16 / 3;
  for (int t0 = blockIdx.z * TP; t0 < n; t0 += TP * gridDim.z) {
    const int here = min(TP, n - t0);
    // a wave brings fragments f = w, w + W, ..: step f / NB, columns f % NB
    const bf16_t* src[NX];
#pragma unroll
    for (int i = 0; i < NX; ++i) {
      const int f = w + i * W;
      const int c0 = (f % NB) * 16 + lr;
      const int c = c0 < 3 * here ? c0 : 0;  // columns past the last: never stored
      src[i] = xp + (int64_t)list[t0 + c / 3] * K3 + (c % 3) * GS + (f / NB) % NKS * 32 + q * 8;
    }
    u32x4 xr[NX];
    float2 sr[S::SG];
    Stage<CB, GS, RT, true> st;
    auto load_x = [&](int step) {
#pragma unroll
      for (int i = 0; i < NX; ++i) {
        const int g = step * XG + (w + i * W) / NB / NKS;
        xr[i] = *(const u32x4*)(src[i] + (int64_t)min(g, G - 1) * 3 * GS);
      }
    };
    auto load_scales = [&](int sl) {
      // (four at a time where they are all the row's own: every lane has a row
      // of its own, and a load costs as many requests as it has lanes)
      typedef __attribute__((ext_vector_type(4), aligned(4))) float f32x4u;
      if (S::SG % 4 == 0 && gdiv == 0 && (int64_t)(sl + 1) * S::SG <= Gs) {
#pragma unroll
        for (int j = 0; j < S::SG; j += 4) {
          const f32x4u sv = *(const f32x4u*)(sp + sl * S::SG + j);
          const f32x4u mv = *(const f32x4u*)(mp + sl * S::SG + j);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (j + i < S::SG) sr[j + i] = float2{sv[i], mv[i]};
        }
      } else {
#pragma unroll
        for (int j = 0; j < S::SG; ++j) {
          // (groups past the end count nothing: their codes are another row's)
          const int g = min(sl * S::SG + j, G - 1) >> gdiv;
          const float2 v = {sp[g], mp[g]};
          sr[j] = sl * S::SG + j < G ? v : float2{0.f, 0.f};
        }
      }
    };
    f32x4 acc[RT][NB];
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int b = 0; b < NB; ++b) acc[r][b] = f32x4{0.f, 0.f, 0.f, 0.f};
    load_codes_of<CB, GS, RT, RB, true>(st, rows, rb, 0, ns, l);
    load_scales(0);
    load_x(0);
    for (int s = 0; s < ns; ++s) {
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const int step = s * NC + c;
        if (c > 0 && step * XG >= G) break;  // uniform
        __syncthreads();
        if (c == 0) {
          put_codes<CB, GS, RT, true>(st, slot, l);
#pragma unroll
          for (int j = 0; j < S::SG; ++j) sm[tid * PITCH + j] = sr[j];
        }
#pragma unroll
        for (int i = 0; i < NX; ++i) {
          const int f = w + i * W;
          if (f < XK * NB) xl[f * 64 + l] = xr[i];
        }
        __syncthreads();
        load_x(step + 1);
        if (c == 0) {
          load_codes_of<CB, GS, RT, RB, true>(st, rows, rb, s + 1, ns, l);
          load_scales(s + 1);
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int j = 0; j < XG; ++j) {
          const int sj = c * XG + j;  // the group's place in the slot
          f32x4 sx[NB];
          u32x4 x[NKS][NB];
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            sx[b] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int k = 0; k < NKS; ++k) {
              x[k][b] = xl[((j * NKS + k) * NB + b) * 64 + l];
              sx[b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, x[k][b]),
                                                             __builtin_bit_cast(bf16x8, ones), sx[b],
                                                             0, 0, 0);
            }
          }
#pragma unroll
          for (int r = 0; r < RT; ++r) {
            const float2 sc = sm[(w * RT * 16 + r * 16 + lr) * PITCH + sj];
            const GroupCodes<CB, GS> gc = get_codes<CB, GS, true>(slot, r, sj, lr, q);
            u32x4 cq[NKS];
#pragma unroll
            for (int k = 0; k < NKS; ++k) cq[k] = codes_bf16<CB, GS, F8>(gc, k);
#pragma unroll
            for (int b = 0; b < NB; ++b) {
              f32x4 p = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
              for (int k = 0; k < NKS; ++k)
                p = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, x[k][b]),
                                                           __builtin_bit_cast(bf16x8, cq[k]), p, 0, 0, 0);
#pragma unroll
              for (int i = 0; i < 4; ++i)
                acc[r][b][i] = fmaf(sc.x, p[i], fmaf(sc.y, sx[b][i], acc[r][b][i]));
            }
          }
        }
      }
    }
    // lane l of a product holds row l & 15 and columns 4 (l >> 4) + i; PR row
    // blocks of every wave at a time
#pragma unroll
    for (int r = 0; r < RB; ++r) {
      __syncthreads();
#pragma unroll
      for (int pr = 0; pr < PR; ++pr)
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int i = 0; i < 4; ++i) red[w][pr][b][q * 4 + i][lr] = acc[r + pr * RB][b][i];
      __syncthreads();
      // thread: a row of a wave, and every fourth token
      const int wb = tid >> 4 & 3, ri = tid & 15;
      const int64_t row = wrow0 + wb * (RB * 16) + r * 16 + ri;
      if (row < N) {
        const float dhi = UP ? a.dn_dhi[(int64_t)e * a.ff + row] : 0.f;
        for (int j = tid >> 6; j < here; j += 4) {
          auto value = [&](int pr) {
            float v = 0.f;
#pragma unroll
            for (int pl = 0; pl < 3; ++pl) {
              const int c = 3 * j + pl;
              v += red[wb][pr][c >> 4][c & 15][ri];
            }
            return v;
          };
          const int64_t p = list[t0 + j];
          if constexpr (UP) store_hidden<ORDER>(a, p, row, value(0), value(1), dhi);
          else a.Yp[p * a.d + row] = a.w[p] * value(0);
        }
      }
    }
    __syncthreads();
  }
}

// The down products and their weighted sum of ONE token: a workgroup owns 16
// rows of all its k experts, the waves being experts by ranges of groups.
template <int CB, bool F8, int GS, int W>
__global__ __launch_bounds__(W * 64) void k_moe_down_one(MoeArgs a) {
  __shared__ float red[W][3][17];
  extern __shared__ __attribute__((aligned(16))) float dyn[];
  const int l = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  constexpr int SG = Slot<CB, GS, false>::SG, SLOT = 16 * Slot<CB, GS, false>::SB;
  uint8_t* slot = reinterpret_cast<uint8_t*>(dyn) + w * SLOT;
  float2* sm = reinterpret_cast<float2*>(reinterpret_cast<uint8_t*>(dyn) + W * SLOT);
  const int lr = l & 15, q = l >> 4;
  const int64_t row0 = (int64_t)blockIdx.x * 16;
  const int G = (int)(a.ff / GS);
  const int gdiv = a.gshift - __builtin_ctz((unsigned)GS);
  const int64_t Gs = a.ff >> a.gshift;
  const int KS = max(1, W / a.k);  // waves an expert
  const int EP = W / KS;           // experts at a time
  const int pitch = a.pitch;
  f32x4 sum = {0.f, 0.f, 0.f, 0.f};
  for (int j0 = 0; j0 < a.k; j0 += EP) {
    const int j = j0 + w / KS;
    const bool live = j < a.k;
    f32x4 acc[1][1] = {{{0.f, 0.f, 0.f, 0.f}}};
    for (int gs0 = 0; gs0 < Gs; gs0 += a.ngs) {
      const int ng = min(a.ngs, (int)Gs - gs0);
      const int g1 = min(G, (gs0 + ng) << gdiv);
      const int full = ((g1 + SG - 1) / SG * SG >> gdiv) - gs0;
      // (waves with no expert of their own in this turn go along with the last)
      const int jj = min(j, a.k - 1);
      const Rows rows = expert_rows<1, false>(a, a.ids[jj], row0);
      const bf16_t* const col[1] = {a.H + (int64_t)jj * 3 * a.ff + (lr < 3 ? lr : 0) * GS};
      contract<CB, F8, GS, 1, 1, 1, false>(
          rows, col, a.dn_rb, (gs0 << gdiv) / SG + w % KS, live ? (g1 + SG - 1) / SG : 0, KS, g1, slot,
          sm + ((w / KS) % EP * 16 + lr) * pitch, pitch, gs0, gdiv, l, acc, [&] {
            if (j0 > 0 || gs0 > 0) __syncthreads();
            for (int b = 0; b < EP && j0 + b < a.k; ++b)
              stage_scales(sm + b * 16 * pitch, pitch, a.dn_s, a.dn_m,
                           (int64_t)a.ids[j0 + b] * a.d + row0, 16, a.d - row0, Gs, gs0, ng, full);
            __syncthreads();
          });
    }
    if (live) {
      const float wj = a.w[j];
#pragma unroll
      for (int i = 0; i < 4; ++i) sum[i] = fmaf(wj, acc[0][0][i], sum[i]);
    }
  }
  if (q == 0) {
#pragma unroll
    for (int i = 0; i < 3; ++i) red[w][i][lr] = sum[i];
  }
  __syncthreads();
  if (threadIdx.x < 16 && row0 + threadIdx.x < a.d) {
    float y = 0.f;
#pragma unroll
    for (int ww = 0; ww < W; ++ww)
#pragma unroll
      for (int i = 0; i < 3; ++i) y += red[ww][i][threadIdx.x];
    a.Y[row0 + threadIdx.x] = y;
  }
}

__global__ __launch_bounds__(256) void k_moe_sum(MoeArgs a) {
  const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;  // d is a multiple of 32
  if (i >= a.T * a.d) return;
  const int64_t t = i / a.d, c = i % a.d;
  f32x4 y = {0.f, 0.f, 0.f, 0.f};
  for (int j0 = 0; j0 < a.k; j0 += 8) {
    f32x4 v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = *(const f32x4*)(a.Yp + (t * a.k + min(j0 + j, a.k - 1)) * a.d + c);
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j0 + j < a.k) y += v[j];
  }
  *(f32x4*)(a.Y + i) = y;
}

template <int CB, bool F8, int GS, bool UP>
hipError_t launch_proj(const MoeArgs& a, const Launch& L) {
  const int64_t N = UP ? a.ff : a.d;
  const int slots = expert_slots(a.T * a.k, a.E);
  const int64_t Gs = (UP ? a.d : a.ff) >> a.gshift;
  // LDS: the waves' slots, and `rows` rows of staged scales, up to kStage bytes
  // of them at a time (an odd number of float2 a row, whole slots' groups); the
  // products later, in their place.  More than 64 KiB of dynamic LDS would have to
  // be allowed per kernel.  16 slots of 64-byte rows leave 48 KiB for the scales;
  // those of 8-bit codes, of 128-byte rows, leave 32, of which 24 are used: 48
  // groups, which are whole turns of the 4 waves, so the sums keep their order.
  constexpr int kStage = 40 * 1024, kStage8 = 24 * 1024;
  constexpr uint32_t kMoeLds = 64 * 1024;
  MoeArgs b = a;
  auto lds = [&](auto slot, int rows, int slots, size_t products) {
    using S = decltype(slot);
    const int64_t stage = CB == 8 && slots == 16 ? kStage8 : kStage;
    b.ngs = (int)(std::min(Gs + S::SG - 1, stage / (rows * 8)) / S::SG * S::SG);
    b.pitch = b.ngs | 1;
    return (uint32_t)std::max((size_t)slots * 16 * S::SB + (size_t)rows * b.pitch * 8, products);
  };
  auto go = [&](auto kernel, int RT, int NB, int W, int KS) {
    const int rows = RT * 16 * (W / KS), per = UP ? rows / 2 : rows;
    const uint32_t bytes = lds(Slot<CB, GS, true>{}, rows, W * RT, (size_t)W * RT * NB * 16 * 17 * 4);
    if (bytes > kMoeLds) return hipErrorInvalidValue;
    return ext_launch(kernel, dim3((unsigned)((N + per - 1) / per), (unsigned)slots), dim3(W * 64),
                      bytes, L, b);
  };
  if (!UP && a.T == 1) {
    constexpr int W = 8;
    const uint32_t bytes = lds(Slot<CB, GS, false>{}, 16 * (W / std::max(1, W / a.k)), W, 0);
    if (bytes > kMoeLds) return hipErrorInvalidValue;
    return ext_launch(k_moe_down_one<CB, F8, GS, W>, dim3((unsigned)((N + 15) / 16)),
                      dim3(W * 64), bytes, L, b);
  }
  // Few tokens an expert (5 are 16 columns): every pass over them reads the
  // codes again, but its small workgroups fill the chip also where experts are
  // few.  Measured, a whole call: 64 experts of 2048 / 1408, top 8, at a mean of 6
  // tokens 152 us and 170 with shared planes, of 8 183 and 186, of 10 214 and 197;
  // 8 experts of 4096 / 2816, top 2, at 10 tokens 116 and 140, at 16 153 and 142.
  const int64_t wide = (N + (UP ? 127 : 255)) / (UP ? 128 : 256) * slots;
  if (a.T * a.k <= (wide < 512 ? 13 : 8) * (int64_t)a.E)
    return go(k_moe_proj<CB, F8, GS, 4, 1, 4, 4, UP>, 4, 1, 4, 4);
  // many tokens an expert: passes of 16 tokens side by side, as many as a
  // mean and three of its deviations need (more take turns)
  constexpr int NB = 3;
  const int per = UP ? 128 : 256;
  const double mean = (double)a.T * a.k / a.E;
  const unsigned passes = (unsigned)std::min((double)(a.T + 15) / 16, (mean + 3 * std::sqrt(mean) + 15) / 16);
  return ext_launch(k_moe_wide<CB, F8, GS, NB, UP>,
                    dim3((unsigned)((N + per - 1) / per), (unsigned)slots, std::max(1u, passes)),
                    dim3(256), 0, L, b);
}

template <bool UP>
hipError_t launch_cb(const MoeArgs& a, int cb, const Launch& L) {
#define TTQ_MOE_GS(CBV, F8)                                       \
  switch (a.gs) {                                                 \
    case 32: return launch_proj<CBV, F8, 32, UP>(a, L);           \
    case 64: return launch_proj<CBV, F8, 64, UP>(a, L);           \
    case 128: return launch_proj<CBV, F8, 128, UP>(a, L);         \
    default: return hipErrorInvalidValue;                         \
  }
  if (a.qf == QF_FP8) {
    if (cb != 8) return hipErrorInvalidValue;
    TTQ_MOE_GS(8, true)
  }
  switch (cb) {
    case 1: TTQ_MOE_GS(1, false)
    case 2: TTQ_MOE_GS(2, false)
    case 4: TTQ_MOE_GS(4, false)
    case 8: TTQ_MOE_GS(8, false)
    default: return hipErrorInvalidValue;
  }
#undef TTQ_MOE_GS
}

}  // namespace

hipError_t launch_moe_score(const MoeArgs& a, const Launch& L) {
  return ext_launch(k_moe_score, dim3((unsigned)((a.E + 3) / 4), (unsigned)a.T), dim3(256), 0, L, a);
}
hipError_t launch_moe_route(const MoeArgs& a, int cb, const Launch& L) {
  const int64_t parts = std::min<int64_t>(256 / a.T, (a.k * (a.d / 8) + 1023) / 1024);
  const dim3 grid((unsigned)a.T, (unsigned)std::max<int64_t>(1, parts)), blk(1024);
  switch (order_of(cb, a.qf == QF_FP8)) {
    case 1: return ext_launch(k_moe_route<1>, grid, blk, 0, L, a);
    case 2: return ext_launch(k_moe_route<2>, grid, blk, 0, L, a);
    default: return ext_launch(k_moe_route<0>, grid, blk, 0, L, a);
  }
}
hipError_t launch_moe_up(const MoeArgs& a, int cb, const Launch& L) {
  return launch_cb<true>(a, cb, L);
}
hipError_t launch_moe_down(const MoeArgs& a, int cb, const Launch& L) {
  return launch_cb<false>(a, cb, L);
}
hipError_t launch_moe_sum(const MoeArgs& a, const Launch& L) {
  return ext_launch(k_moe_sum, dim3((unsigned)((a.T * a.d / 4 + 255) / 256)), dim3(256), 0, L, a);
}

}  // namespace ttq
