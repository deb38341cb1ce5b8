// Attention over a cache of quantized rows, the keys of a row divided over waves.
//
// For a query row q (one head of one token) and the keys it sees,
//   t_j = scale q . k_j,  p_j = exp(t_j - max),  out = sum_j p_j v_j / sum_j p_j
// with k_j, v_j = (m + s c) D^{-1/2} by groups of channels.  The codes c enter the
// matrix cores as they are stored (attn.h), and what is common to a group comes
// out of the sum:
//   q . k_j = sum_g s_jg (sum_{i in g} q'_i c_ji) + m_jg (sum_{i in g} q'_i),  q' = q D^{-1/2}
// (float32), and V's scales multiply its codes as they become operands; its offsets
// are rows of a product of their own, sum_j p_j m_jg, beside a row of ones, which
// gives sum_j p_j of the very p_j (fp16) that weight the values.
//
// One wave takes 16 query rows of one K/V head (a token's G heads, or several
// tokens') and a range of its keys, 32 at a time:
//   S^T = K q'^T   two tiles of 16 keys x 16 rows.  Row 4a + i of tile b is key
//                  8a + 4b + i, so that a lane (row l % 16, a = l / 16) has the 8
//                  keys 8a .. 8a + 7 of its row,
//   O^T += V^T P^T which are what it gives as the operand of this one.  Nothing
//                  passes between lanes but the maximum.
// V's operand takes 8 keys of one channel from a lane: it reads HD / 16 adjacent
// channels of 8 keys and parts them in registers.
//
// fp16 holds q' (times a power of two, its largest value in [2^10, 2^11)), p <= 1 and
// V's scales and offsets (divided by 2^Y, Y the wave's so far): 11 bits each, one
// half unit of 2^-11, an eighth of what the bf16 result is rounded by.
//
// What the maxima and sums of the ranges are is kept in float32 and joined by
// k_attn_join; with one range the row is written at once.
#include <algorithm>

#include "attn.h"

namespace ttq {

namespace {

__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

template <int NB>
struct Words {
  unsigned w[NB >= 4 ? NB / 4 : 1];
};
template <int NB>
__device__ __forceinline__ void load_words(Words<NB>& d, const uint8_t* p) {
  if constexpr (NB >= 16) {
#pragma unroll
    for (int i = 0; i < NB / 16; ++i) {
      const u32x4 v = *(const u32x4*)(p + 16 * i);
      d.w[4 * i] = v.x; d.w[4 * i + 1] = v.y; d.w[4 * i + 2] = v.z; d.w[4 * i + 3] = v.w;
    }
  } else if constexpr (NB == 8) {
    const u32x2 v = *(const u32x2*)p;
    d.w[0] = v.x; d.w[1] = v.y;
  } else if constexpr (NB == 4) {
    d.w[0] = *(const unsigned*)p;
  } else {
    d.w[0] = *(const uint16_t*)p;
  }
}

__device__ __forceinline__ unsigned mul_pair(unsigned a, unsigned b) {
  return __builtin_bit_cast(unsigned, __builtin_bit_cast(f16x2, a) * __builtin_bit_cast(f16x2, b));
}

// HD channels a head; GSE = min(group, HD) of them a group; CB-bit codes
template <int HD, int GSE, int CB, bool F8>
__global__ __launch_bounds__(256) void k_attn_split(AttnArgs a) {
  constexpr int NG = HD / GSE;           // groups of a head
  constexpr int KB = GSE * CB / 32;      // bytes of a lane's quarter of a group of K
  constexpr int NC = HD / 16;            // channels of V of a lane
  constexpr int VB = NC * CB / 8;
  constexpr int U = kUnit<F8>;
  constexpr float kInf = __builtin_inff();
  // what S may reach before Y has to grow, and what it is set to reach
  constexpr float kSMax = F8 ? 128.f : 60000.f;
  constexpr int kSBits = F8 ? 5 : 13;
  __shared__ __align__(16) int sm_row[4][32];
  __shared__ __align__(16) float sm_k[4][2][NG][32];
  __shared__ __align__(16) _Float16 sm_v[4][2][NG][32];

  const int l = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int n = l & 15, c = l >> 4;
  // units: (block of rows, range of keys, K/V head), the heads of a range in
  // neighbouring waves: they read the same rows of the cache
  const int64_t unit = (int64_t)blockIdx.x * 4 + w;
  const int h = (int)(unit % a.KV);
  const int64_t bs = unit / a.KV;
  const int split = (int)(bs % a.nsplit);
  const int64_t block = bs / a.nsplit;
  if (block >= a.tiles) return;  // uniform over the wave, as all that follows
  int64_t seq, r0;
  SeqRows sr;
  if (!find_block<16>(a, block, seq, sr, r0)) return;

  // this lane's row
  const int r = (int)min(r0 + n, (int64_t)sr.rows - 1);
  const int tok = r / a.G, head = h * a.G + r % a.G;
  const int64_t pos = sr.shift + tok;
  const int64_t pos_lo = sr.shift + (int)r0 / a.G;
  const int64_t pos_hi = sr.shift + (int)min(r0 + 15, (int64_t)sr.rows - 1) / a.G;
  int64_t lo = a.window > 0 ? max(pos_lo - a.window + 1, (int64_t)0) & ~int64_t(31) : 0;
  const int64_t hi = min(sr.len, pos_hi + 1);
  const int64_t per = ((hi - lo + a.nsplit - 1) / a.nsplit + 31) & ~int64_t(31);
  lo += per * split;
  const int64_t end = min(lo + per, hi);
  const int64_t orow = ((sr.first + tok) * a.H + head) * a.nsplit + split;

  // q' of this lane's channels, by group and step, and its sums
  f16x8 q[HD / 32];
  float qs[NG], qm;
  {
    const bf16_t* src = a.Q + (sr.first + tok) * a.ldq + head * HD;
    float qf[HD / 4], top = 0.f;
#pragma unroll
    for (int i = 0; i < HD / 32; ++i) {
      const int ch = i / (GSE / 32) * GSE + c * (GSE / 4) + i % (GSE / 32) * 8;
      const u32x4 x = *(const u32x4*)(src + ch);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        qf[8 * i + 2 * j] = bf16lo(x[j]);
        qf[8 * i + 2 * j + 1] = bf16hi(x[j]);
      }
      if (a.kdhi) {
        const float* d = a.kdhi + a.k_first + h * HD + ch;
        const f32x4 d0 = *(const f32x4*)d, d1 = *(const f32x4*)(d + 4);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          qf[8 * i + j] *= d0[j];
          qf[8 * i + 4 + j] *= d1[j];
        }
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) top = fmaxf(top, __builtin_fabsf(qf[8 * i + j]));
    }
    top = fmaxf(top, __shfl_xor(top, 16));
    top = fmaxf(top, __shfl_xor(top, 32));
    const int e = (top > 0.f ? min(ilogbf(top), 127) : 0) - 10;
#pragma unroll
    for (int g = 0; g < NG; ++g) qs[g] = 0.f;
#pragma unroll
    for (int i = 0; i < HD / 32; ++i) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float v = ldexpf(qf[8 * i + slot_code<CB>(j)], -e);
        const _Float16 f = (_Float16)v;
        qs[i / (GSE / 32)] += (float)f;
        q[i][j] = (!F8 && slot_shift<CB>(j)) ? f * (_Float16)0.0625f : f;
      }
    }
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      qs[g] += __shfl_xor(qs[g], 16);
      qs[g] += __shfl_xor(qs[g], 32);
      qs[g] = ldexpf(qs[g], -U);
    }
    qm = ldexpf(a.scale2, e + U);
  }

  f32x4 o[NC], om = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < NC; ++i) o[i] = om;
  float mrun = -kInf;
  int Y = -200;
  unsigned nan_groups = 0;

  struct Block {
    Words<KB> k[2][NG];
    Words<VB> v[8];
    float s[NG], m[NG];
    bool seen;  // this lane's key is in the range and in the cache
  };
  const int32_t* table = a.pages + seq * a.max_pages;
  const int64_t pmask = (int64_t(1) << a.pshift) - 1;
  auto page_of = [&](int64_t k0) {
    const int64_t key = k0 + (l & 31);
    return key < end ? table[key >> a.pshift] : -1;
  };
  const int64_t ko = (a.k_first + h * HD) * CB / 8, vo = (a.v_first + h * HD) * CB / 8;
  const int64_t go = ((l < 32 ? a.k_first : a.v_first) + h * HD) >> a.gshift;
  const float* sp = (l < 32 ? a.ks : a.vs) + go;
  const float* mp = (l < 32 ? a.km : a.vm) + go;

  auto fetch = [&](Block& b, int64_t k0, int page) {
    const int64_t at = ((int64_t)page << a.pshift) + ((k0 + (l & 31)) & pmask);
    b.seen = page >= 0 && at < a.n_slots;
    const int row = b.seen ? (int)at : 0;  // (row 0 is there to be read)
    wave_sync();
    sm_row[w][l & 31] = row;
    wave_sync();
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const uint8_t* p = a.kc + (int64_t)sm_row[w][(n >> 2) * 8 + t * 4 + (n & 3)] * a.row_bytes + ko + c * KB;
#pragma unroll
      for (int g = 0; g < NG; ++g) load_words<KB>(b.k[t][g], p + g * (GSE * CB / 8));
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
      load_words<VB>(b.v[j], a.vc + (int64_t)sm_row[w][c * 8 + j] * a.row_bytes + vo + n * VB);
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      b.s[g] = sp[(int64_t)row * a.groups + g];
      b.m[g] = mp[(int64_t)row * a.groups + g];
    }
  };

  auto rescale = [&](float f) {
#pragma unroll
    for (int i = 0; i < NC; ++i) o[i] *= f;
    om *= f;
  };

  auto compute = [&](Block& b, int64_t k0) {
    // scales to where the lanes that need them find them
    bool grow = false, bad = false;
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      if (!b.seen) b.s[g] = b.m[g] = 0.f;
      if (l >= 32) {
        grow |= ldexpf(b.s[g], -Y) > kSMax || ldexpf(__builtin_fabsf(b.m[g]), -Y - U) > 30000.f;
        bad |= b.s[g] != b.s[g] || b.m[g] != b.m[g];
      }
    }
    if (__ballot(grow)) {
      int top = -1000;
      if (l >= 32)
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          if (b.s[g] > 0.f) top = max(top, ilogbf(b.s[g]));
          if (b.m[g] != 0.f && b.m[g] == b.m[g]) top = max(top, ilogbf(b.m[g]) - U);
        }
#pragma unroll
      for (int off = 1; off < 64; off <<= 1) top = max(top, __shfl_xor(top, off));
      const int y = max(Y, top + 1 - kSBits);
      rescale(ldexpf(1.f, Y - y));
      Y = y;
    }
    const bool any_bad = __ballot(bad) != 0;
    wave_sync();
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      if (l < 32) {
        sm_k[w][0][g][l] = b.s[g];
        sm_k[w][1][g][l] = b.m[g];
      } else {
        const bool x = b.s[g] != b.s[g] || b.m[g] != b.m[g];
        sm_v[w][0][g][l - 32] = x ? (_Float16)0.f : (_Float16)ldexpf(b.s[g], -Y);
        sm_v[w][1][g][l - 32] = x ? (_Float16)0.f : (_Float16)ldexpf(b.m[g], -Y - U);
      }
    }
    wave_sync();

    float t[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) t[i] = 0.f;
#pragma unroll
    for (int g = 0; g < NG; ++g) {
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = 0; s < GSE / 32; ++s) {
          const unsigned* kw = b.k[half][g].w;
          const f16x8 k = CB == 8 ? codes8<CB, F8>(kw[2 * s], kw[2 * s + 1]) : codes8<CB, F8>(kw[s], 0u);
          acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(k, q[g * (GSE / 32) + s], acc, 0, 0, 0);
        }
        const f32x4 s4 = *(const f32x4*)&sm_k[w][0][g][c * 8 + half * 4];
        const f32x4 m4 = *(const f32x4*)&sm_k[w][1][g][c * 8 + half * 4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          t[half * 4 + i] = fmaf(s4[i], acc[i], t[half * 4 + i]);
          if (!F8) t[half * 4 + i] = fmaf(m4[i], qs[g], t[half * 4 + i]);
        }
      }
    }
    // bit j: this lane's row sees its key j
    unsigned mask = 0xffu;
    const unsigned seen = (unsigned)__ballot(b.seen && l < 32);
    const bool whole = seen == 0xffffffffu && k0 + 31 <= pos_lo &&
                       (a.window <= 0 || k0 > pos_hi - a.window);
    if (!whole) {
      mask = (seen >> (c * 8)) & 0xffu;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int64_t key = k0 + c * 8 + i;
        if (key > pos || (a.window > 0 && key <= pos - a.window)) mask &= ~(1u << i);
      }
    }
    float mx = -kInf;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      t[i] = (mask >> i) & 1 ? t[i] * qm : -kInf;
      mx = fmaxf(mx, t[i]);
    }
    mx = fmaxf(mx, __shfl_xor(mx, 16));
    mx = fmaxf(mx, __shfl_xor(mx, 32));
    if (__ballot(mx > mrun)) {
      const float mnew = fmaxf(mrun, mx);
      rescale(mrun == -kInf ? 0.f : __builtin_amdgcn_exp2f(mrun - mnew));
      mrun = mnew;
    }
    const float base = mrun == -kInf ? 0.f : mrun;
    f16x8 p;
#pragma unroll
    for (int i = 0; i < 8; ++i) p[i] = (_Float16)__builtin_amdgcn_exp2f(t[i] - base);
    if (any_bad) {  // a scale of V that is NaN: its group, in the rows that see it
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        const unsigned keys = (unsigned)(__ballot(l >= 32 && (b.s[g] != b.s[g] || b.m[g] != b.m[g])) >> 32);
        if (mask & (keys >> (c * 8)) & 0xffu) nan_groups |= 1u << g;
      }
    }
    // V's operands
    const u32x4 sv = *(const u32x4*)&sm_v[w][0][n * NC / GSE][c * 8];
    unsigned vp[4][NC];
#pragma unroll
    for (int j = 0; j < 4; ++j) key_pairs<CB, F8, NC>(b.v[2 * j].w, b.v[2 * j + 1].w, vp[j]);
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const u32x4 v = {mul_pair(vp[0][i], sv.x), mul_pair(vp[1][i], sv.y), mul_pair(vp[2][i], sv.z),
                       mul_pair(vp[3][i], sv.w)};
      o[i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, v), p, o[i], 0, 0, 0);
    }
    u32x4 mv = {0u, 0u, 0u, 0u};
    if (n == 15) mv = u32x4{0x3c003c00u, 0x3c003c00u, 0x3c003c00u, 0x3c003c00u};  // ones
    else if (!F8 && n < NG) mv = *(const u32x4*)&sm_v[w][1][n][c * 8];
    om = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, mv), p, om, 0, 0, 0);
  };

  if (lo < end) {
    Block A, B;
    fetch(A, lo, page_of(lo));
    int page = page_of(lo + 32);
    for (int64_t k0 = lo;;) {
      if (k0 + 32 < end) {
        fetch(B, k0 + 32, page);
        page = page_of(k0 + 64);
      }
      compute(A, k0);
      if ((k0 += 32) >= end) break;
      if (k0 + 32 < end) {
        fetch(A, k0 + 32, page);
        page = page_of(k0 + 64);
      }
      compute(B, k0);
      if ((k0 += 32) >= end) break;
    }
  }

  // rows of O^T are channels c HD/4 + i NC + j of this lane's row
  nan_groups |= __shfl_xor(nan_groups, 16);
  nan_groups |= __shfl_xor(nan_groups, 32);
  const float sum = __shfl(om[3], 48 + n);
  const float inv = sum > 0.f || sum != sum ? 1.f / sum : 0.f;
  float off[NG];
#pragma unroll
  for (int g = 0; g < NG; ++g) {
    off[g] = __shfl(om[g & 3], (g >> 2) * 16 + n);
    if ((nan_groups >> g) & 1) off[g] = __builtin_nanf("");
  }
  if (r0 + n >= sr.rows) return;  // (no shuffles below)
  if (a.nsplit > 1 && c == 0) {
    a.ml[2 * orow] = mrun;
    a.ml[2 * orow + 1] = sum;
  }
  if (a.nsplit > 1 && !(sum > 0.f || sum != sum)) return;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float x[NC];
    const int ch = c * (HD / 4) + i * NC;
    float f = 0.f;
#pragma unroll
    for (int g = 0; g < NG; ++g) f = ch / GSE == g ? off[g] : f;
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      const float v = o[j][i] * (CB == 4 && (j & 1) ? 0.0625f : 1.f);
      x[j] = ldexpf((v + f) * inv, Y + U);
      if (a.vdhi) x[j] *= a.vdhi[a.v_first + h * HD + ch + j];
    }
    if (a.nsplit > 1) {
      float* dst = a.part + orow * HD + ch;
#pragma unroll
      for (int j = 0; j < NC; j += 4) *(f32x4*)(dst + j) = f32x4{x[j], x[j + 1], x[j + 2], x[j + 3]};
    } else {
      bf16_t* dst = a.out + ((sr.first + tok) * a.H + head) * HD + ch;
#pragma unroll
      for (int j = 0; j < NC; j += 4) *(u32x2*)(dst + j) = u32x2{pack_bf16(x[j], x[j + 1]), pack_bf16(x[j + 2], x[j + 3])};
    }
  }
}

// One workgroup joins the ranges of a row: out = sum_s w_s l_s o_s / sum_s w_s l_s,
// w_s = exp(m_s - max m), o_s the mean of range s; the ranges dealt to its waves.
template <int HD>
__global__ __launch_bounds__(256) void k_attn_join(AttnArgs a) {
  constexpr int NC = HD / 64;
  __shared__ float sm[4][HD], smw[4];
  const int l = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int64_t row = blockIdx.x, t = row / a.H;
  if (a.offsets && (t >= a.offsets[a.n_seq] || t < a.offsets[0])) return;  // uniform
  const float* ml = a.ml + row * a.nsplit * 2;
  float mx = -__builtin_inff();
  for (int s = l; s < a.nsplit; s += 64) mx = fmaxf(mx, ml[2 * s]);
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) mx = fmaxf(mx, __shfl_xor(mx, off));
  float acc[NC], sum = 0.f;
#pragma unroll
  for (int j = 0; j < NC; ++j) acc[j] = 0.f;
  for (int s = w; s < a.nsplit; s += 4) {
    const float lsum = ml[2 * s + 1];
    if (!(lsum > 0.f || lsum != lsum)) continue;  // no key, and no row written
    const float f = __builtin_amdgcn_exp2f(ml[2 * s] - mx) * lsum;
    sum += f;
    const float* p = a.part + (row * a.nsplit + s) * HD + l * NC;
#pragma unroll
    for (int j = 0; j < NC; ++j) acc[j] = fmaf(f, p[j], acc[j]);
  }
#pragma unroll
  for (int j = 0; j < NC; ++j) sm[w][l * NC + j] = acc[j];
  if (l == 0) smw[w] = sum;
  __syncthreads();
  const float total = smw[0] + smw[1] + smw[2] + smw[3];
  for (int i = threadIdx.x; i < HD / 2; i += 256) {
    float x[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      x[j] = sm[0][2 * i + j] + sm[1][2 * i + j] + sm[2][2 * i + j] + sm[3][2 * i + j];
      x[j] = total == 0.f ? 0.f : x[j] / total;
    }
    *(unsigned*)(a.out + row * HD + 2 * i) = pack_bf16(x[0], x[1]);
  }
}

}  // namespace

hipError_t launch_attn_split(const AttnArgs& a, int head_dim, int cb, int qf, int group,
                             const Launch& L) {
  const int64_t units = a.tiles * a.nsplit * a.KV;
  const dim3 grid((unsigned)((units + 3) / 4)), blk(256);
  const int gse = std::min(group, head_dim);
#define TTQ_AS(HDV, GSV)                                                                          \
  if (head_dim == HDV && gse == GSV) {                                                            \
    if (qf == QF_FP8) return ext_launch(k_attn_split<HDV, GSV, 8, true>, grid, blk, 0, L, a);     \
    if (cb == 8) return ext_launch(k_attn_split<HDV, GSV, 8, false>, grid, blk, 0, L, a);         \
    return ext_launch(k_attn_split<HDV, GSV, 4, false>, grid, blk, 0, L, a);                      \
  }
  TTQ_AS(64, 32)
  TTQ_AS(64, 64)
  TTQ_AS(128, 32)
  TTQ_AS(128, 64)
  TTQ_AS(128, 128)
  TTQ_AS(256, 32)
  TTQ_AS(256, 64)
  TTQ_AS(256, 128)
  TTQ_AS(256, 256)
#undef TTQ_AS
  return hipErrorInvalidValue;
}

hipError_t launch_attn_join(const AttnArgs& a, int head_dim, const Launch& L) {
  const dim3 grid((unsigned)(a.T * a.H)), blk(256);
  if (head_dim == 64) return ext_launch(k_attn_join<64>, grid, blk, 0, L, a);
  if (head_dim == 128) return ext_launch(k_attn_join<128>, grid, blk, 0, L, a);
  return ext_launch(k_attn_join<256>, grid, blk, 0, L, a);
}

}  // namespace ttq
