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
// The codes are exact in bf16 and x' enters as three bf16 planes that sum to
// it (split24), so the products are as exact as float32 ones, on the matrix
// cores; the group sums of x' come from the same planes against ones.
#include "codes.h"
#include "ttq_internal.h"

namespace ttq {

namespace {

// ------------------------------------------------------------- routing
// does expert a (score la) come before expert b?
__device__ __forceinline__ bool before(double la, int a, double lb, int b) {
  const bool na = la != la, nb = lb != lb;
  if (na || nb) return na == nb ? a < b : nb;
  return la > lb || (la == lb && a < b);
}

// One workgroup per token: 16 waves take the experts in turn, then every
// expert's rank is counted against all others.
__global__ __launch_bounds__(1024) void k_moe_route(MoeArgs a) {
  __shared__ double score[kMoeMaxE];
  __shared__ int rank[kMoeMaxE];
  __shared__ int chosen[kMoeMaxK];
  const int tid = threadIdx.x, l = tid & 63, w = tid >> 6;
  const int64_t t = blockIdx.x;
  const bf16_t* x = a.X + t * a.d;
  for (int e = w; e < a.E; e += 16) {
    const bf16_t* r = a.router + (int64_t)e * a.d;
    double s = 0.0;
    for (int64_t c = l * 8; c < a.d; c += 512) {
      const u32x4 xv = *(const u32x4*)(x + c), rv = *(const u32x4*)(r + c);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        s += (double)(bf16lo(xv[i]) * bf16lo(rv[i]));
        s += (double)(bf16hi(xv[i]) * bf16hi(rv[i]));
      }
    }
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) s += __shfl_xor(s, off);
    if (l == 0) score[e] = s;
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
  if (tid < a.k) {
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
}

// ------------------------------------------------------------ products
// 8 codes -> 4 bf16 pairs, exactly.  A code of up to 4 bits, read as an E4M3
// pattern, is code * 2^-9 (0..7 are its subnormals, 8..15 its first binade),
// so the E4M3 conversion with a scale of 2^9 expands two codes at once.  The
// pairs come in the order of the bytes that hold the codes; see code_order.
template <int CB, bool F8>
__device__ __forceinline__ u32x4 codes_bf16(u32x2 raw) {
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
    // codes 0 4 | 1 5 | 2 6 | 3 7 (the two bytes of the 16 bits)
    const unsigned a = raw.x & 0x0303u, b = (raw.x >> 2) & 0x0303u;
    const unsigned c = (raw.x >> 4) & 0x0303u, d = (raw.x >> 6) & 0x0303u;
    return u32x4{pair(a, false, 512.f), pair(b, false, 512.f), pair(c, false, 512.f),
                 pair(d, false, 512.f)};
  } else {
    unsigned p[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      p[i] = ((raw.x >> (2 * i)) & 1u) * 0x3F80u + ((raw.x >> (2 * i + 1)) & 1u) * 0x3F800000u;
    return u32x4{p[0], p[1], p[2], p[3]};
  }
}
// the channel (of 8) at place i of that operand
template <int CB, bool F8>
constexpr int code_order(int i) {
  if (!F8 && CB == 4) return i < 4 ? 2 * i : 2 * (i - 4) + 1;
  if (!F8 && CB == 2) return i / 2 + 4 * (i % 2);
  return i;
}

// One expert's rows against the tokens that chose it, 16 at a time.
// UP: rows are RT/2 blocks of 16 gate rows and the RT/2 up rows beside them,
// x' is formed from X, and the result is silu(g) u D^{-1/2} as planes; else
// RT blocks of down rows, x' is those planes, and the result is the expert's
// weighted output.  The four waves of a workgroup take the groups in turn and
// add up in LDS in wave order.
constexpr int MW = 4;

template <int CB, bool F8, int GS, int RT, bool UP>
__global__ __launch_bounds__(MW * 64) void k_moe_proj(MoeArgs a) {
  constexpr int NKS = GS / 32;
  __shared__ unsigned have[kMoeMaxE / 32];
  __shared__ int16_t list[kMoeMaxT];
  __shared__ int count;
  __shared__ f32x4 red[MW][RT][64];
  const int tid = threadIdx.x, l = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lr = l & 15, q = l >> 4;
  const int P = (int)a.T * a.k;

  // the blockIdx.y-th expert that any token chose, and the choices that name it
  if (tid < kMoeMaxE / 32) have[tid] = 0u;
  __syncthreads();
  for (int i = tid; i < P; i += MW * 64) atomicOr(&have[a.ids[i] >> 5], 1u << (a.ids[i] & 31));
  __syncthreads();
  int e = -1;
  for (int i = 0, left = blockIdx.y; i < kMoeMaxE / 32; ++i) {
    unsigned b = have[i];
    const int c = __builtin_popcount(b);
    if (left < c) {
      while (left--) b &= b - 1u;
      e = i * 32 + __builtin_ctz(b);
      break;
    }
    left -= c;
  }
  if (e < 0) return;  // uniform
  if (w == 0) {
    int n = 0;
    for (int i0 = 0; i0 < P; i0 += 64) {
      const bool mine = i0 + l < P && a.ids[i0 + l] == e;
      const uint64_t m = __ballot(mine);
      if (mine) list[n + __builtin_popcountll(m & ((1ull << l) - 1ull))] = (int16_t)(i0 + l);
      n += __builtin_popcountll(m);
    }
    if (l == 0) count = n;
  }
  __syncthreads();
  const int n = count;

  const int64_t K = UP ? a.d : a.ff, N = UP ? a.ff : a.d;  // channels, rows (of each kind)
  const int64_t rb = UP ? a.gu_rb : a.dn_rb;
  const int64_t Gs = K >> a.gshift;  // scales per row
  const int G = (int)(K / GS);
  constexpr int RB = UP ? RT / 2 : RT;  // row blocks of one kind
  const int64_t row0 = (int64_t)blockIdx.x * RB * 16;
  const int64_t nrow = min((int64_t)RB * 16, N - row0);
  const int64_t erow = (int64_t)e * (UP ? 2 * a.ff : a.d) + row0;  // first row among all experts'
  const uint8_t* codes = UP ? a.gu : a.dn;
  const float* sp = UP ? a.gu_s : a.dn_s;
  const float* mp = UP ? a.gu_m : a.dn_m;
  // one bounded buffer per kind of row: rows past the last read zeros
  const __amdgpu_buffer_rsrc_t c0 = make_rsrc(codes + erow * rb, (uint32_t)(nrow * rb));
  const __amdgpu_buffer_rsrc_t c1 = UP ? make_rsrc(codes + (erow + a.ff) * rb, (uint32_t)(nrow * rb)) : c0;
  int64_t srow[RT];
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    const int64_t in = (r % RB) * 16 + lr;
    srow[r] = (erow + (r / RB) * a.ff + min(in, nrow - 1)) * Gs;
  }
  const float* dhi = UP ? a.gu_dhi + (int64_t)e * a.d : nullptr;
  const int gsub = __builtin_ctz((unsigned)GS);

  for (int tb = 0; tb < n; tb += 16) {
    // columns past the last repeat the first (never stored)
    const int pick = list[tb + lr < n ? tb + lr : tb];
    const bf16_t* xsrc = UP ? a.X + (int64_t)(pick / a.k) * a.d : a.H + (int64_t)pick * 3 * a.ff;
    f32x4 acc[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r) acc[r] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int g = w; g < G; g += MW) {
      GroupCodes<CB, GS> cv[RT];
      float s[RT], m[RT];
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        load_codes<CB, GS>(cv[r], r < RB ? c0 : c1,
                           (uint32_t)(((r % RB) * 16 + lr) * rb + q * GroupCodes<CB, GS>::NB),
                           (uint32_t)((int64_t)g * GS * CB / 8));
        const int64_t gi = srow[r] + (((int64_t)g << gsub) >> a.gshift);
        s[r] = sp[gi];
        m[r] = mp[gi];
      }
      f32x4 Pr[RT], Sx = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int r = 0; r < RT; ++r) Pr[r] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int k = 0; k < NKS; ++k) {
        const int64_t c = (int64_t)g * GS + q * (GS / 4) + k * 8;
        u32x4 pl[3];
        if constexpr (UP) {
          const u32x4 xv = *(const u32x4*)(xsrc + c);
          const f32x4 h0 = *(const f32x4*)(dhi + c), h1 = *(const f32x4*)(dhi + c + 4);
          const float v[8] = {bf16lo(xv.x) * h0.x, bf16hi(xv.x) * h0.y, bf16lo(xv.y) * h0.z,
                              bf16hi(xv.y) * h0.w, bf16lo(xv.z) * h1.x, bf16hi(xv.z) * h1.y,
                              bf16lo(xv.w) * h1.z, bf16hi(xv.w) * h1.w};
          float u[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) u[i] = v[code_order<CB, F8>(i)];
          split24(u, pl);
        } else {
          // (the planes are stored in the operand's order)
#pragma unroll
          for (int i = 0; i < 3; ++i) pl[i] = *(const u32x4*)(xsrc + i * a.ff + c);
        }
        const u32x4 ones = {0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u};
#pragma unroll
        for (int i = 0; i < 3; ++i)
          Sx = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, pl[i]),
                                                      __builtin_bit_cast(bf16x8, ones), Sx, 0, 0, 0);
#pragma unroll
        for (int r = 0; r < RT; ++r) {
          const u32x4 cq = codes_bf16<CB, F8>(step_codes<CB, GS>(cv[r], k));
#pragma unroll
          for (int i = 0; i < 3; ++i)
            Pr[r] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, pl[i]),
                                                           __builtin_bit_cast(bf16x8, cq), Pr[r], 0, 0, 0);
        }
      }
#pragma unroll
      for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[r][i] = fmaf(s[r], Pr[r][i], fmaf(m[r], Sx[i], acc[r][i]));
    }
#pragma unroll
    for (int r = 0; r < RT; ++r) red[w][r][l] = acc[r];
    __syncthreads();
    // lane ll of block r holds row r * 16 + (ll & 15), columns 4 (ll >> 4) + i
    for (int i = tid; i < RB * 256; i += MW * 64) {
      const int r = i >> 8, ll = i & 63, c = (i >> 6) & 3;
      const int col = tb + (ll >> 4) * 4 + c;
      const int64_t row = row0 + r * 16 + (ll & 15);
      if (col >= n || row >= N) continue;
      auto sum = [&](int rr) {
        float v = red[0][rr][ll][c];
#pragma unroll
        for (int ww = 1; ww < MW; ++ww) v += red[ww][rr][ll][c];
        return v;
      };
      const int64_t p = list[col];
      if constexpr (UP) {
        const float gate = sum(r), up = sum(RB + r);
        const float h = gate / (1.f + expf(-gate)) * up * a.dn_dhi[(int64_t)e * a.ff + row];
        const unsigned hi = __float_as_uint(h) & 0xffff0000u;
        const float r1 = h - __uint_as_float(hi);
        const unsigned mid = __float_as_uint(r1) & 0xffff0000u;
        const unsigned lo = __float_as_uint(r1 - __uint_as_float(mid));
        // in the order of the down product's operand
        int at = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (code_order<CB, F8>(j) == (int)(row & 7)) at = j;
        bf16_t* dst = a.H + p * 3 * a.ff + (row & ~(int64_t)7) + at;
        dst[0] = (bf16_t)(hi >> 16);
        dst[a.ff] = (bf16_t)(mid >> 16);
        dst[2 * a.ff] = (bf16_t)(lo >> 16);
      } else {
        a.Yp[p * a.d + row] = a.w[p] * sum(r);
      }
    }
    __syncthreads();
  }
}

__global__ __launch_bounds__(256) void k_moe_sum(MoeArgs a) {
  const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;  // d is a multiple of 32
  if (i >= a.T * a.d) return;
  const int64_t t = i / a.d, c = i % a.d;
  f32x4 y = {0.f, 0.f, 0.f, 0.f};
  for (int j = 0; j < a.k; ++j) y += *(const f32x4*)(a.Yp + (t * a.k + j) * a.d + c);
  *(f32x4*)(a.Y + i) = y;
}

template <int CB, bool F8, bool UP>
hipError_t launch_proj(const MoeArgs& a, int group, const Launch& L) {
  constexpr int RT = 4;
  const int64_t N = UP ? a.ff : a.d;
  const int64_t per = 16 * (UP ? RT / 2 : RT);
  const int slots = (int)(a.T * a.k < a.E ? a.T * a.k : a.E);
  const dim3 grid((unsigned)((N + per - 1) / per), (unsigned)slots), blk(MW * 64);
  switch (group) {
    case 32: return ext_launch(k_moe_proj<CB, F8, 32, RT, UP>, grid, blk, 0, L, a);
    case 64: return ext_launch(k_moe_proj<CB, F8, 64, RT, UP>, grid, blk, 0, L, a);
    // a group of 256 is two halves with one scale
    case 128: case 256: return ext_launch(k_moe_proj<CB, F8, 128, RT, UP>, grid, blk, 0, L, a);
    default: return hipErrorInvalidValue;
  }
}

template <bool UP>
hipError_t launch_cb(const MoeArgs& a, int group, int cb, const Launch& L) {
  if (a.qf == QF_FP8) return cb == 8 ? launch_proj<8, true, UP>(a, group, L) : hipErrorInvalidValue;
  switch (cb) {
    case 1: return launch_proj<1, false, UP>(a, group, L);
    case 2: return launch_proj<2, false, UP>(a, group, L);
    case 4: return launch_proj<4, false, UP>(a, group, L);
    case 8: return launch_proj<8, false, UP>(a, group, L);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace

hipError_t launch_moe_route(const MoeArgs& a, const Launch& L) {
  return ext_launch(k_moe_route, dim3((unsigned)a.T), dim3(1024), 0, L, a);
}
hipError_t launch_moe_up(const MoeArgs& a, int group, int cb, const Launch& L) {
  return launch_cb<true>(a, group, cb, L);
}
hipError_t launch_moe_down(const MoeArgs& a, int group, int cb, const Launch& L) {
  return launch_cb<false>(a, group, cb, L);
}
hipError_t launch_moe_sum(const MoeArgs& a, const Launch& L) {
  return ext_launch(k_moe_sum, dim3((unsigned)((a.T * a.d / 4 + 255) / 256)), dim3(256), 0, L, a);
}

}  // namespace ttq
