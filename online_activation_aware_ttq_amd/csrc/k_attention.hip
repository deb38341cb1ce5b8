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
// V's scales (divided by 2^Y, Y the wave's so far): 11 bits each, an eighth of what
// the bf16 result is rounded by.
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
// the same at byte lane + uniform of a buffer: no address arithmetic a lane
template <int NB>
__device__ __forceinline__ void load_words(Words<NB>& d, __amdgpu_buffer_rsrc_t r, unsigned lane,
                                           unsigned uniform) {
  if constexpr (NB >= 16) {
#pragma unroll
    for (int i = 0; i < NB / 16; ++i) {
      const u32x4 v = buf_load16(r, lane + 16 * i, uniform);
      d.w[4 * i] = v.x; d.w[4 * i + 1] = v.y; d.w[4 * i + 2] = v.z; d.w[4 * i + 3] = v.w;
    }
  } else if constexpr (NB == 8) {
    const auto v = __builtin_amdgcn_raw_buffer_load_b64(r, lane, uniform, 0);
    d.w[0] = v[0]; d.w[1] = v[1];
  } else if constexpr (NB == 4) {
    d.w[0] = __builtin_amdgcn_raw_buffer_load_b32(r, lane, uniform, 0);
  } else {
    d.w[0] = __builtin_amdgcn_raw_buffer_load_b16(r, lane, uniform, 0);
  }
}

__device__ __forceinline__ unsigned mul_pair(unsigned a, unsigned b) {
  return __builtin_bit_cast(unsigned, __builtin_bit_cast(f16x2, a) * __builtin_bit_cast(f16x2, b));
}

// HD channels a head; GSE = min(group, HD) of them a group; CB-bit codes
template <int HD, int GSE, int CB, bool F8, bool OCT>
__global__ __launch_bounds__(256, HD == 256 ? 1 : HD / GSE <= 2 ? 3 : 2) void k_attn_split(AttnArgs a) {
  constexpr int NG = HD / GSE;           // groups of a head
  constexpr int KB = GSE * CB / 32;      // bytes of a lane's quarter of a group of K
  constexpr int NC = HD / 16;            // channels of V of a lane
  constexpr int VB = NC * CB / 8;
  constexpr int U = kUnit<F8>;
  constexpr float kInf = __builtin_inff();
  constexpr bool kP = NG == 1;           // V's scales go into p, not into V
  // What a scale times 2^-Y may reach before Y has to grow, and what it is set to
  // reach: its product with a code (or with p, up to 2^kLazy) stays below 2^16.
  constexpr float kSMax = kP ? 200.f : F8 ? 128.f : 60000.f;
  constexpr int kSBits = kP ? 5 : F8 ? 5 : 13;
  constexpr int MU = F8 ? 0 : kP ? 20 : 10;  // V's offsets: 2^MU of O's unit
  constexpr int kMid = F8 ? 0 : 1 << (CB - 1);
  constexpr float kLazy = 8.f;
  __shared__ __align__(16) unsigned sm_row[4][32];
  __shared__ __align__(16) float sm_k[4][2][NG][32];
  __shared__ __align__(16) _Float16 sm_s[4][NG][32], sm_m[4][F8 ? 1 : 2 * NG][32];

  const int l = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
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
    const float sign = a.scale2 == 0.f ? 0.f : a.scale2 < 0.f ? -1.f : 1.f;
    float qf[HD / 4], top = 0.f;
#pragma unroll
    for (int i = 0; i < HD / 32; ++i) {
      const int ch = i / (GSE / 32) * GSE + c * (GSE / 4) + i % (GSE / 32) * 8;
      const u32x4 x = *(const u32x4*)(src + ch);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        qf[8 * i + 2 * j] = bf16lo(x[j]) * sign;
        qf[8 * i + 2 * j + 1] = bf16hi(x[j]) * sign;
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
    qm = sign == 0.f ? 1.f : fmaxf(ldexpf(__builtin_fabsf(a.scale2), e + U), 1.17549435e-38f);
  }

  f32x4 o[NC], om = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < NC; ++i) o[i] = om;
  float mrun = -kInf;
  int Y = -200;
  unsigned nan_groups = 0;

  // The keys in hand, 32 from k0 on; the next ones are asked for as each part has
  // been used.
  Words<KB> kw[2][NG];
  Words<VB> vw[8];
  float sc[NG], of[NG];   // scales and offsets of key l % 32: K's, or (l >= 32) V's
  bool seen;              // that key is in the range and in the cache

  const int32_t* table = a.pages + seq * a.max_pages;
  const int64_t pmask = (int64_t(1) << a.pshift) - 1;
  auto page_of = [&](int64_t k0) {
    const int64_t key = k0 + (l & 31);
    return key < end ? table[key >> a.pshift] : -1;
  };
  const uint8_t* kbase = a.kc + (a.k_first + h * HD) * CB / 8;
  const uint8_t* vbase = a.vc + (a.v_first + h * HD) * CB / 8;
  const int64_t go = ((l < 32 ? a.k_first : a.v_first) + h * HD) >> a.gshift;
  const float* sp = (l < 32 ? a.ks : a.vs) + go;
  const float* mp = (l < 32 ? a.km : a.vm) + go;
  const unsigned rb = (unsigned)a.row_bytes;
  // (up to 2^32 - 1 bytes from a head's first channel on: rows of 32-bit offsets)
  const int64_t room = std::min<int64_t>(a.n_slots * a.row_bytes, 0xffffffff);
  const auto kbuf = make_rsrc(kbase, (uint32_t)(room - (kbase - a.kc)));
  const auto vbuf = make_rsrc(vbase, (uint32_t)(room - (vbase - a.vc)));

  unsigned row;                 // of this lane's key of the next block
  unsigned ko = 0, vo = 0;      // OCT: where this lane's parts of it begin
  auto locate = [&](int64_t k0, int page) {
    const int64_t at = ((int64_t)page << a.pshift) + ((k0 + (l & 31)) & pmask);
    seen = page >= 0 && at < a.n_slots;
    row = seen ? (unsigned)at : 0u;  // (row 0 is there to be read)
    wave_sync();
    sm_row[w][l & 31] = OCT ? row * rb : row;
    wave_sync();
    if constexpr (OCT) {
      ko = sm_row[w][(n >> 2) * 8] + (n & 3) * rb + c * KB;
      vo = sm_row[w][c * 8] + n * VB;
    }
  };
  auto fetch_k = [&] {
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      if constexpr (OCT) {  // eight rows one after another, 32-bit offsets
#pragma unroll
        for (int g = 0; g < NG; ++g) load_words<KB>(kw[t][g], kbuf, ko + g * (GSE * CB / 8), t * 4 * rb);
      } else {
        const uint8_t* p = kbase + (int64_t)sm_row[w][(n >> 2) * 8 + t * 4 + (n & 3)] * a.row_bytes + c * KB;
#pragma unroll
        for (int g = 0; g < NG; ++g) load_words<KB>(kw[t][g], p + g * (GSE * CB / 8));
      }
    }
    const int64_t so = (int64_t)row * a.groups;
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      sc[g] = sp[so + g];
      of[g] = mp[so + g];
    }
  };
  auto fetch_v = [&] {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if constexpr (OCT) load_words<VB>(vw[j], vbuf, vo, j * rb);
      else load_words<VB>(vw[j], vbase + (int64_t)sm_row[w][c * 8 + j] * a.row_bytes + n * VB);
    }
  };

  auto rescale = [&](float f) {
#pragma unroll
    for (int i = 0; i < NC; ++i) o[i] *= f;
    om *= f;
  };

  int page = -1;
  if (lo < end) {
    locate(lo, page_of(lo));
    page = page_of(lo + 32);
    fetch_k();
    fetch_v();
  }
  for (int64_t k0 = lo; k0 < end; k0 += 32) {
    const bool now = seen;
    // scales to where the lanes that need them find them
    bool grow = false, bad = false;
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      if (!now) sc[g] = of[g] = 0.f;
      grow |= ldexpf(sc[g], -Y) > kSMax || (!F8 && ldexpf(__builtin_fabsf(of[g]), MU - U - Y) > 30000.f);
      bad |= sc[g] != sc[g] || of[g] != of[g];
    }
    if (__ballot(l >= 32 && grow)) {
      int top = -1000;
      if (l >= 32)
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          if (sc[g] > 0.f) top = max(top, ilogbf(sc[g]));
          if (of[g] != 0.f && of[g] == of[g]) top = max(top, ilogbf(of[g]) + MU - U + kSBits - 13);
        }
#pragma unroll
      for (int off = 1; off < 64; off <<= 1) top = max(top, __shfl_xor(top, off));
      const int y = max(Y, top + 1 - kSBits);
      rescale(ldexpf(1.f, Y - y));
      Y = y;
    }
    const bool any_bad = __ballot(l >= 32 && bad) != 0;
    unsigned bad_keys[NG];
    if (any_bad) {
#pragma unroll
      for (int g = 0; g < NG; ++g)
        bad_keys[g] = (unsigned)(__ballot(l >= 32 && (sc[g] != sc[g] || of[g] != of[g])) >> 32);
    }
    wave_sync();
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      if (l < 32) {
        sm_k[w][0][g][l] = sc[g];
        if (!F8) sm_k[w][1][g][l] = of[g];
      } else {
        // the scale in 11 bits; what it is off is made up for in the middle of the
        // codes by the offset, which is a sum of two fp16 values
        const bool x = sc[g] != sc[g] || of[g] != of[g];
        const float sv = x ? 0.f : ldexpf(sc[g], -Y);
        const _Float16 s16 = (_Float16)sv;
        sm_s[w][g][l - 32] = s16;
        if constexpr (!F8) {
          const float mv = x ? 0.f : fmaf(sv - (float)s16, ldexpf((float)kMid, MU - U), ldexpf(of[g], MU - U - Y));
          const _Float16 m16 = (_Float16)mv;
          sm_m[w][g][l - 32] = m16;
          sm_m[w][NG + g][l - 32] = (_Float16)(mv - (float)m16);
        }
      }
    }
    const unsigned seen_keys = (unsigned)__ballot(now && l < 32);
    const bool more = k0 + 32 < end;
    if (more) {
      locate(k0 + 32, page);
      page = page_of(k0 + 64);
    }
    wave_sync();

    float t[8];
#pragma unroll
    for (int g = 0; g < NG; ++g) {
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = 0; s < GSE / 32; ++s) {
          const unsigned* kx = kw[half][g].w;
          const f16x8 k = CB == 8 ? codes8<CB, F8>(kx[2 * s], kx[2 * s + 1]) : codes8<CB, F8>(kx[s], 0u);
          acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(k, q[g * (GSE / 32) + s], acc, 0, 0, 0);
        }
        const f32x4 s4 = *(const f32x4*)&sm_k[w][0][g][c * 8 + half * 4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          t[half * 4 + i] = g == 0 ? s4[i] * acc[i] : fmaf(s4[i], acc[i], t[half * 4 + i]);
        if constexpr (!F8) {
          const f32x4 m4 = *(const f32x4*)&sm_k[w][1][g][c * 8 + half * 4];
#pragma unroll
          for (int i = 0; i < 4; ++i) t[half * 4 + i] = fmaf(m4[i], qs[g], t[half * 4 + i]);
        }
      }
    }
    if (more) fetch_k();
    // where not all rows see all keys: bit j of mask, this lane's row sees its key j
    unsigned mask = 0xffu;
    if (seen_keys != 0xffffffffu || k0 + 31 > pos_lo || (a.window > 0 && k0 <= pos_hi - a.window)) {
      const int top = (int)max(min(pos - k0, (int64_t)64), (int64_t)-1);
      const int bottom = a.window > 0 ? (int)max(min(pos - a.window - k0, (int64_t)64), (int64_t)-1) : -1;
      mask = (seen_keys >> (c * 8)) & 0xffu;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int key = c * 8 + i;
        if (key > top || key <= bottom) mask &= ~(1u << i);
        if (!((mask >> i) & 1)) t[i] = -kInf;
      }
    }
    auto mx2 = [](float x, float y) { return __builtin_elementwise_maximum(x, y); };
    float mx = mx2(mx2(mx2(t[0], t[1]), mx2(t[2], t[3])), mx2(mx2(t[4], t[5]), mx2(t[6], t[7])));
    mx = mx2(mx, __shfl_xor(mx, 16));
    mx = mx2(mx, __shfl_xor(mx, 32)) * qm;
    if (__ballot(mx > mrun + kLazy)) {
      const float mnew = fmaxf(mrun, mx);
      rescale(mrun == -kInf ? 0.f : __builtin_amdgcn_exp2f(mrun - mnew));
      mrun = mnew;
    }
    const float base = mrun == -kInf ? 0.f : -mrun;
    f16x8 p;
#pragma unroll
    for (int i = 0; i < 8; ++i) p[i] = (_Float16)__builtin_amdgcn_exp2f(fmaf(t[i], qm, base));
    if (any_bad) {  // a scale of V that is NaN: its group, in the rows that see it
#pragma unroll
      for (int g = 0; g < NG; ++g)
        if (mask & (bad_keys[g] >> (c * 8)) & 0xffu) nan_groups |= 1u << g;
    }
    // V's operands, their scales (of this lane's channels: one group) in p or in V
    const u32x4 sv = *(const u32x4*)&sm_s[w][n * NC / GSE][c * 8];
    f16x8 ps = p;
    if constexpr (kP) ps = p * __builtin_bit_cast(f16x8, sv);
#pragma unroll
    for (int i = 0; i < NC / 4; ++i) {
      unsigned vp[4][4];
#pragma unroll
      for (int j = 0; j < 4; ++j) key_pairs<CB, F8>(vw[2 * j].w, vw[2 * j + 1].w, i, vp[j]);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const u32x4 v = kP ? u32x4{vp[0][k], vp[1][k], vp[2][k], vp[3][k]}
                           : u32x4{mul_pair(vp[0][k], sv.x), mul_pair(vp[1][k], sv.y),
                                   mul_pair(vp[2][k], sv.z), mul_pair(vp[3][k], sv.w)};
        o[4 * i + k] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, v), ps, o[4 * i + k], 0, 0, 0);
      }
    }
    if (more) fetch_v();
    // rows 0 .. NG - 1 of this product: V's offsets; 15: ones
    u32x4 mv = {0x3c003c00u, 0x3c003c00u, 0x3c003c00u, 0x3c003c00u};
    if (n < 15) mv = u32x4{0u, 0u, 0u, 0u};
    if (!F8 && n < NG) mv = *(const u32x4*)&sm_m[w][n][c * 8];
    om = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, mv), p, om, 0, 0, 0);
    if constexpr (!F8) {
      u32x4 ml = {0u, 0u, 0u, 0u};
      if (n < NG) ml = *(const u32x4*)&sm_m[w][NG + n][c * 8];
      om = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, ml), p, om, 0, 0, 0);
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
      x[j] = ldexpf((v + ldexpf(f, -MU)) * inv, Y + U);
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
// w_s = exp(m_s - max m), o_s the mean of range s.  The weights first, all at once;
// then HD / 4 lanes a range, 1024 / HD ranges side by side.
template <int HD>
__global__ __launch_bounds__(256) void k_attn_join(AttnArgs a) {
  constexpr int LN = HD / 4, SB = 256 / LN;
  __shared__ float sm_w[kAttnMaxSplit], sm_red[8];
  __shared__ __align__(16) float sm[SB][HD];
  const int tid = threadIdx.x, l = tid & 63, w = tid >> 6;
  const int64_t row = blockIdx.x, t = row / a.H;
  if (a.offsets && (t >= a.offsets[a.n_seq] || t < a.offsets[0])) return;  // uniform
  const float* ml = a.ml + row * a.nsplit * 2;
  float m = -__builtin_inff(), sum = 0.f;
  static_assert(kAttnMaxSplit <= 256);
  if (tid < a.nsplit) {
    m = ml[2 * tid];
    sum = ml[2 * tid + 1];
  }
  float mx = m;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) mx = fmaxf(mx, __shfl_xor(mx, off));
  if (l == 0) sm_red[w] = mx;
  __syncthreads();
  mx = fmaxf(fmaxf(sm_red[0], sm_red[1]), fmaxf(sm_red[2], sm_red[3]));
  // (a range without keys has no sum and has written no row)
  const float f = sum > 0.f || sum != sum ? __builtin_amdgcn_exp2f(m - mx) * sum : 0.f;
  sm_w[tid] = f;
  float total = f;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) total += __shfl_xor(total, off);
  if (l == 0) sm_red[4 + w] = total;
  __syncthreads();
  total = sm_red[4] + sm_red[5] + sm_red[6] + sm_red[7];
  const int c = tid % LN * 4, s0 = tid / LN;
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
  const float* p = a.part + row * a.nsplit * HD + c;
#pragma unroll 4
  for (int s = s0; s < a.nsplit; s += SB) {
    const float g = sm_w[s];
    if (g == 0.f) continue;
    const f32x4 v = *(const f32x4*)(p + (int64_t)s * HD);
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[j] = fmaf(g, v[j], acc[j]);
  }
  *(f32x4*)&sm[s0][c] = acc;
  __syncthreads();
  if (tid < HD / 2) {
    float x[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < SB; ++i) {
      x[0] += sm[i][2 * tid];
      x[1] += sm[i][2 * tid + 1];
    }
    const float inv = total == 0.f ? 0.f : 1.f / total;
    *(unsigned*)(a.out + row * HD + 2 * tid) = pack_bf16(x[0] * inv, x[1] * inv);
  }
}

}  // namespace

hipError_t launch_attn_split(const AttnArgs& a, int head_dim, int cb, int qf, int group,
                             const Launch& L) {
  const int64_t units = a.tiles * a.nsplit * a.KV;
  const dim3 grid((unsigned)((units + 3) / 4)), blk(256);
  const int gse = std::min(group, head_dim);
  auto go = [&](auto octets, auto rows) {
    return ext_launch(a.octets ? octets : rows, grid, blk, 0, L, a);
  };
#define TTQ_AS(HDV, GSV)                                                      \
  if (head_dim == HDV && gse == GSV) {                                        \
    if (qf == QF_FP8) return go(k_attn_split<HDV, GSV, 8, true, true>,        \
                                k_attn_split<HDV, GSV, 8, true, false>);      \
    if (cb == 8) return go(k_attn_split<HDV, GSV, 8, false, true>,            \
                           k_attn_split<HDV, GSV, 8, false, false>);          \
    return go(k_attn_split<HDV, GSV, 4, false, true>,                         \
              k_attn_split<HDV, GSV, 4, false, false>);                       \
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
