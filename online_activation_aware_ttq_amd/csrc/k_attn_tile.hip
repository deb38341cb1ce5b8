// Attention over a cache of quantized rows where many query rows share their keys
// (prompts and chunks of them): tiles of keys, decoded once for 256 rows.
//
// A workgroup takes 256 query rows of one K/V head (a token's G heads, then the next
// token's) and its keys, KT = 8192 / HD at a time.  Its eight waves decode a tile
// together, (s c + m) in fp16, K as rows and V as columns, into LDS, while they work
// on the tile before, each for 32 rows:
//   S^T = K q'^T   (32 keys x 32 rows an instruction block).  Key 16s + 8h + 4a + b
//                  of a block is row 16s + 8a + 4h + b, so that the lane of a row (h
//                  = lane / 32) ends with the 8 adjacent keys 16s + 8h ..  of it
//   O^T += V^T P^T that it has to give here: nothing passes between lanes but the
//                  maximum.
// The sums of p are those of the fp16 values that weight V (v_dot2).
//
// fp16's range is kept by powers of two: K and V are decoded as 2^-YK and 2^-YV of
// what they are, which the workgroup raises, with a tile decoded again, when a scale
// or offset would leave it; q' as in k_attention.hip.  The maximum of a row follows
// only steps of 2^8 (p and the sums may be as much larger), so O is seldom scaled.
//
// What bounds it, a tile of 64 keys and 128 channels: 32 matrix instructions a wave
// of 32 cycles each, 32 exponentials of 16, about as much other vector work, and 32
// KiB from LDS a wave (64 of whose rows' reads would halve that, for twice the
// registers).
#include <algorithm>

#include "attn.h"

namespace ttq {

namespace {

__device__ __forceinline__ f16x2 h2(unsigned v) { return __builtin_bit_cast(f16x2, v); }
__device__ __forceinline__ unsigned u2(f16x2 v) { return __builtin_bit_cast(unsigned, v); }

// a x + b of both halves, rounded once
__device__ __forceinline__ unsigned fma2(unsigned a, unsigned x, unsigned b) {
  return u2(__builtin_elementwise_fma(h2(a), h2(x), h2(b)));
}
__device__ __forceinline__ unsigned both(float a, float b) {
  return u2(f16x2{(_Float16)a, (_Float16)b});
}

template <int HD, int CB, bool F8>
__global__ __launch_bounds__(512, 2) void k_attn_tile(AttnArgs a) {
  constexpr int KT = 8192 / HD;      // keys of a tile
  constexpr int NKT = KT / 32;       // blocks of 32 keys
  constexpr int NCT = HD / 32;       // blocks of 32 channels
  constexpr int KS = HD / 16;        // steps of 16 channels
  constexpr int PS = KT / 16;        // steps of 16 keys
  constexpr int U = kUnit<F8>;
  constexpr float kInf = __builtin_inff();
  constexpr float kSMax = F8 ? 100.f : 50000.f;  // (k_attention.hip)
  constexpr int kSBits = F8 ? 4 : 12;
  constexpr float kLazy = 8.f;
  constexpr unsigned kOut = 1u << 31;  // the key is in no page of the cache
  __shared__ __align__(16) _Float16 sm_k[2][KT * HD];
  __shared__ __align__(16) _Float16 sm_v[2][HD * KT];
  __shared__ unsigned sm_bad[2][KT];  // of a key: groups of V that are NaN; kOut
  __shared__ int sm_flag[3], sm_y[2];

  const int tid = threadIdx.x, l = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int n = l & 31, hf = l >> 5;
  const int h = (int)(blockIdx.x % a.KV);
  const int64_t bs = blockIdx.x / a.KV;
  const int split = (int)(bs % a.nsplit);
  const int64_t block = a.tiles - 1 - bs / a.nsplit;  // long rows of a prompt first
  int64_t seq, r0;
  SeqRows sr;
  if (!find_block<256>(a, block, seq, sr, r0)) return;  // uniform over the workgroup

  // keys of the workgroup, and of this wave
  const int64_t last = sr.rows - 1;
  const int64_t wg_lo = sr.shift + r0 / a.G, wg_hi = sr.shift + min(r0 + 255, last) / a.G;
  int64_t lo = a.window > 0 ? max(wg_lo - a.window + 1, (int64_t)0) / KT * KT : 0;
  const int64_t hi = min(sr.len, wg_hi + 1);
  const int64_t per = ((hi - lo + a.nsplit - 1) / a.nsplit + KT - 1) / KT * KT;
  lo += per * split;
  const int64_t end = min(lo + per, hi);
  const int64_t w0 = r0 + 32 * w;  // this wave's first row
  const bool wave_live = w0 <= last;
  const int64_t pos_lo = sr.shift + min(w0, last) / a.G;
  const int64_t pos_hi = sr.shift + min(w0 + 31, last) / a.G;
  const int r = (int)min(w0 + n, last);
  const int tok = r / a.G, head = h * a.G + r % a.G;
  const int64_t pos = sr.shift + tok;
  const int64_t orow = ((sr.first + tok) * a.H + head) * a.nsplit + split;

  // q' in fp16, its largest value in [2^10, 2^11); the sign of the scale goes with it
  f16x8 q[KS];
  float qm;
  {
    const bf16_t* src = a.Q + (sr.first + tok) * a.ldq + head * HD;
    const float sign = a.scale2 == 0.f ? 0.f : a.scale2 < 0.f ? -1.f : 1.f;
    float top = 0.f;
    auto load = [&](int i, float (&v)[8]) __attribute__((always_inline)) {
      const int ch = i * 16 + hf * 8;
      const u32x4 x = *(const u32x4*)(src + ch);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[2 * j] = bf16lo(x[j]) * sign;
        v[2 * j + 1] = bf16hi(x[j]) * sign;
      }
      if (a.kdhi) {
        const float* d = a.kdhi + a.k_first + h * HD + ch;
        const f32x4 d0 = *(const f32x4*)d, d1 = *(const f32x4*)(d + 4);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          v[j] *= d0[j];
          v[4 + j] *= d1[j];
        }
      }
    };
#pragma unroll
    for (int i = 0; i < KS; ++i) {
      float v[8];
      load(i, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) top = fmaxf(top, __builtin_fabsf(v[j]));
    }
    top = fmaxf(top, __shfl_xor(top, 32));
    const int e = (top > 0.f ? min(ilogbf(top), 127) : 0) - 10;
#pragma unroll
    for (int i = 0; i < KS; ++i) {
      float v[8];
      load(i, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) q[i][j] = (_Float16)ldexpf(v[slot_code<CB>(j)], -e);
    }
    qm = sign == 0.f ? 1.f : fmaxf(ldexpf(__builtin_fabsf(a.scale2), e + U), 1.17549435e-38f);
  }

  f32x16 o[NCT];
#pragma unroll
  for (int i = 0; i < NCT; ++i)
#pragma unroll
    for (int j = 0; j < 16; ++j) o[i][j] = 0.f;
  float mrun = -kInf, sum = 0.f;
  int YK = -200, YV = -200;
  unsigned nan_groups = 0;

  // what this thread decodes of a tile: 16 channels of a key of K, 8 of two keys of V
  constexpr int KP = HD / 16, VP = HD / 8;
  const int kkey = tid / KP, kch = tid % KP * 16;
  const int vkey = tid / VP * 2, vch = tid % VP * 8;
  const int kpos = (kkey & ~31) + ((kkey >> 4) & 1) * 16 + ((kkey >> 2) & 1) * 8 + ((kkey >> 3) & 1) * 4 + (kkey & 3);
  struct Raw {
    unsigned k[CB / 2], v[2][CB / 4];
    float ks, km, vs[2], vm[2];
    bool kin, vin[2];
  };
  struct Pages {
    int k, v[2];
  };
  const int32_t* table = a.pages + seq * a.max_pages;
  const int64_t pmask = (int64_t(1) << a.pshift) - 1;
  const int64_t kc = a.k_first + h * HD + kch, vc = a.v_first + h * HD + vch;
  auto page_of = [&](int64_t key) __attribute__((always_inline)) { return key < end ? table[key >> a.pshift] : -1; };
  auto pages_of = [&](int64_t k0) __attribute__((always_inline)) {
    return Pages{page_of(k0 + kkey), {page_of(k0 + vkey), page_of(k0 + vkey + 1)}};
  };
  auto row_of = [&](int page, int64_t key, bool& in) __attribute__((always_inline)) {
    const int64_t at = ((int64_t)page << a.pshift) + (key & pmask);
    in = page >= 0 && at < a.n_slots;
    return in ? at : 0;  // (row 0 is there to be read)
  };
  auto fetch = [&](Raw& x, const Pages& p, int64_t k0) __attribute__((always_inline)) {
    {
      const int64_t row = row_of(p.k, k0 + kkey, x.kin);
      const uint8_t* c = a.kc + row * a.row_bytes + kc * CB / 8;
      if constexpr (CB == 8) {
        const u32x4 v = *(const u32x4*)c;
        x.k[0] = v.x; x.k[1] = v.y; x.k[2] = v.z; x.k[3] = v.w;
      } else {
        const u32x2 v = *(const u32x2*)c;
        x.k[0] = v.x; x.k[1] = v.y;
      }
      x.ks = a.ks[row * a.groups + (kc >> a.gshift)];
      x.km = a.km[row * a.groups + (kc >> a.gshift)];
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int64_t row = row_of(p.v[j], k0 + vkey + j, x.vin[j]);
      const uint8_t* c = a.vc + row * a.row_bytes + vc * CB / 8;
      if constexpr (CB == 8) {
        const u32x2 v = *(const u32x2*)c;
        x.v[j][0] = v.x; x.v[j][1] = v.y;
      } else {
        x.v[j][0] = *(const unsigned*)c;
      }
      x.vs[j] = a.vs[row * a.groups + (vc >> a.gshift)];
      x.vm[j] = a.vm[row * a.groups + (vc >> a.gshift)];
    }
  };
  auto nan = [](float s, float m) { return s != s || m != m; };

  // Decodes it into buffer b with YK and YV as they are; flags: 1 where they are too
  // small (what is then written is not used), 2 where mark() is needed.
  auto decode = [&](Raw& x, int b, int64_t k0, int slot) __attribute__((always_inline)) {
    int f = 0;
    {
      if (!x.kin) x.ks = x.km = 0.f;
      const float s = ldexpf(x.ks, -YK), m = ldexpf(x.km, -YK - U);
      if (s > kSMax || __builtin_fabsf(m) > 30000.f) f |= 1;
      const unsigned s1 = both(s, s), s16 = both(s * 0.0625f, s * 0.0625f), mm = both(m, m);
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const f16x8 c = CB == 8 ? codes8<CB, F8>(x.k[CB == 8 ? 2 * u : 0], x.k[CB == 8 ? 2 * u + 1 : 0])
                                : codes8<CB, F8>(x.k[u], 0u);
        u32x4 v = __builtin_bit_cast(u32x4, c);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = fma2(v[i], !F8 && slot_shift<CB>(2 * i) ? s16 : s1, mm);
        *(u32x4*)&sm_k[b][kpos * HD + (((kch >> 3) + u) ^ (kpos & 7)) * 8] = v;
      }
    }
    float s[2], m[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const bool bad = nan(x.vs[j], x.vm[j]);
      const bool none = !x.vin[j] || bad;
      if (x.vin[j] ? bad : k0 + vkey + j < end) f |= 2;
      s[j] = none ? 0.f : ldexpf(x.vs[j], -YV);
      m[j] = none ? 0.f : ldexpf(x.vm[j], -YV - U);
      if (s[j] > kSMax || __builtin_fabsf(m[j]) > 30000.f) f |= 1;
    }
    const unsigned s1 = both(s[0], s[1]), s16 = both(s[0] * 0.0625f, s[1] * 0.0625f), mm = both(m[0], m[1]);
    unsigned p[2][4];
#pragma unroll
    for (int i = 0; i < 2; ++i) key_pairs<CB, F8>(x.v[0], x.v[1], i, p[i]);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int ch = vch + i;
      const int sw = KT >= 64 ? (ch ^ (ch >> 3)) & 7 : ((ch >> 2) ^ (ch >> 3)) & 3;
      *(unsigned*)&sm_v[b][ch * KT + (((vkey >> 3) ^ sw) << 3) + (vkey & 7)] =
          fma2(p[i / 4][i % 4], !F8 && CB == 4 && (i & 1) ? s16 : s1, mm);
    }
    if (f) atomicOr(&sm_flag[slot], f);
  };

  // which keys of buffer b are in no page, and which groups of V are NaN
  auto mark = [&](const Raw& x, int b) __attribute__((always_inline)) {
    if (tid < KT) sm_bad[b][tid] = 0;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int g = (int)((vc >> a.gshift) - ((a.v_first + h * HD) >> a.gshift));
      const unsigned bits = !x.vin[j] ? kOut : nan(x.vs[j], x.vm[j]) ? 1u << g : 0u;
      if (bits) atomicOr(&sm_bad[b][vkey + j], bits);
    }
    __syncthreads();
  };

  // YK and YV for the tile that x is a part of, and O in the new units
  auto raise = [&](const Raw& x) __attribute__((always_inline)) {
    if (tid < 2) sm_y[tid] = -1000;
    __syncthreads();
    auto exponent = [&](float s, float m) __attribute__((always_inline)) {
      int e = -1000;
      if (s > 0.f) e = ilogbf(s);
      if (m != 0.f && m == m) e = max(e, ilogbf(m) - U);
      return e;
    };
    atomicMax(&sm_y[0], exponent(x.ks, x.km));
    int e = -1000;
#pragma unroll
    for (int j = 0; j < 2; ++j)
      if (x.vin[j] && !nan(x.vs[j], x.vm[j])) e = max(e, exponent(x.vs[j], x.vm[j]));
    atomicMax(&sm_y[1], e);
    __syncthreads();
    YK = max(YK, sm_y[0] + 1 - kSBits);
    const int y = max(YV, sm_y[1] + 1 - kSBits);
    const float f = ldexpf(1.f, YV - y);
#pragma unroll
    for (int i = 0; i < NCT; ++i) o[i] *= f;
    YV = y;
  };

  auto compute = [&](int b, int64_t k0, bool marked) __attribute__((always_inline)) {
    f32x16 s[NKT];
#pragma unroll
    for (int t = 0; t < NKT; ++t) {
#pragma unroll
      for (int j = 0; j < 16; ++j) s[t][j] = 0.f;
#pragma unroll
      for (int i = 0; i < KS; ++i) {
        const f16x8 k = *(const f16x8*)&sm_k[b][(t * 32 + n) * HD + ((2 * i + hf) ^ (n & 7)) * 8];
        s[t] = __builtin_amdgcn_mfma_f32_32x32x16_f16(k, q[i], s[t], 0, 0, 0);
      }
    }
    // value j of block t is that of key k0 + key_of(t, j)
    auto key_of = [&](int t, int j) __attribute__((always_inline)) { return t * 32 + (j >> 3) * 16 + hf * 8 + (j & 7); };
    if (marked || k0 + KT - 1 > pos_lo || k0 + KT > end || (a.window > 0 && k0 <= pos_hi - a.window)) {
      const int top = (int)min(min(pos, end - 1) - k0, (int64_t)KT);
      const int bottom = a.window > 0 ? (int)max(min(pos - a.window - k0, (int64_t)KT), (int64_t)-1) : -1;
#pragma unroll
      for (int t = 0; t < NKT; ++t)
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const int key = key_of(t, j);
          bool seen = key <= top && key > bottom;
          if (marked && seen) {
            const unsigned bad = sm_bad[b][key];
            if (bad & kOut) seen = false;
            else nan_groups |= bad;
          }
          if (!seen) s[t][j] = -kInf;
        }
    }
    float mx = -kInf;
#pragma unroll
    for (int t = 0; t < NKT; ++t)
#pragma unroll
      for (int j = 0; j < 16; ++j) mx = fmaxf(mx, s[t][j]);
    mx = fmaxf(mx, __shfl_xor(mx, 32));
    const float f = ldexpf(qm, YK), top = mx * f;
    if (__ballot(top > mrun + kLazy)) {
      const float mnew = fmaxf(mrun, top);
      const float g = mrun == -kInf ? 0.f : __builtin_amdgcn_exp2f(mrun - mnew);
#pragma unroll
      for (int i = 0; i < NCT; ++i) o[i] *= g;
      sum *= g;
      mrun = mnew;
    }
    const float base = mrun == -kInf ? 0.f : mrun;
    f16x8 p[PS];
#pragma unroll
    for (int i = 0; i < PS; ++i) {
      u32x4 v;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int at = (i & 1) * 8 + 2 * j;
        v[j] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_pkrtz(
            __builtin_amdgcn_exp2f(fmaf(s[i >> 1][at], f, -base)),
            __builtin_amdgcn_exp2f(fmaf(s[i >> 1][at + 1], f, -base))));
        sum = __builtin_amdgcn_fdot2(h2(v[j]), f16x2{(_Float16)1.f, (_Float16)1.f}, sum, false);
      }
      p[i] = __builtin_bit_cast(f16x8, v);
    }
#pragma unroll
    for (int t = 0; t < NCT; ++t) {
      const int ch = t * 32 + n;
      const int sw = KT >= 64 ? (ch ^ (ch >> 3)) & 7 : ((ch >> 2) ^ (ch >> 3)) & 3;
#pragma unroll
      for (int i = 0; i < PS; ++i) {
        const f16x8 v = *(const f16x8*)&sm_v[b][ch * KT + (((2 * i + hf) ^ sw) << 3)];
        o[t] = __builtin_amdgcn_mfma_f32_32x32x16_f16(v, p[i], o[t], 0, 0, 0);
      }
    }
  };

  if (lo < end) {  // uniform over the workgroup
    if (tid < 3) sm_flag[tid] = 0;
    Raw x;
    fetch(x, pages_of(lo), lo);
    Pages next = pages_of(lo + KT);
    __syncthreads();
    // tile t is decoded into buffer t % 2 with flags t % 3, which are cleared a tile
    // before: whoever reads them has done so two barriers ago
    int t = 0;
    auto settle = [&](int64_t k0) __attribute__((always_inline)) {
      if (tid == 0) sm_flag[(t + 1) % 3] = 0;
      decode(x, t & 1, k0, t % 3);
      __syncthreads();
      const int f = sm_flag[t % 3];
      if (f & 1) {
        raise(x);
        decode(x, t & 1, k0, t % 3);
        __syncthreads();
      }
      if (f & 2) mark(x, t & 1);
      return (f & 2) != 0;
    };
    bool marked = settle(lo);
    for (int64_t k0 = lo;; k0 += KT) {
      const bool more = k0 + KT < end;
      if (more) {
        fetch(x, next, k0 + KT);
        next = pages_of(k0 + 2 * KT);
      }
      if (wave_live && k0 <= pos_hi && (a.window <= 0 || k0 + KT - 1 > pos_lo - a.window))
        compute(t & 1, k0, marked);
      if (!more) break;
      ++t;
      marked = settle(k0 + KT);
    }
  }

  sum += __shfl_xor(sum, 32);
  nan_groups |= __shfl_xor(nan_groups, 32);
  if (w0 + n > last) return;
  const bool any = sum > 0.f || sum != sum;
  const float inv = any ? 1.f / sum : 0.f;
  if (a.nsplit > 1) {
    if (hf == 0) {
      a.ml[2 * orow] = mrun;
      a.ml[2 * orow + 1] = sum;
    }
    if (!any) return;
  }
#pragma unroll
  for (int t = 0; t < NCT; ++t)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int ch = t * 32 + i * 8 + hf * 4;
      const int64_t at = a.v_first + h * HD;
      const bool bad = (nan_groups >> (((at + ch) >> a.gshift) - (at >> a.gshift))) & 1;
      f32x4 x;
#pragma unroll
      for (int j = 0; j < 4; ++j) x[j] = bad ? __builtin_nanf("") : ldexpf(o[t][4 * i + j] * inv, YV + U);
      if (a.vdhi) x *= *(const f32x4*)(a.vdhi + at + ch);
      if (a.nsplit > 1)
        *(f32x4*)(a.part + orow * HD + ch) = x;
      else
        *(u32x2*)(a.out + ((sr.first + tok) * a.H + head) * HD + ch) =
            u32x2{pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3])};
    }
}

}  // namespace

hipError_t launch_attn_tile(const AttnArgs& a, int head_dim, int cb, int qf, const Launch& L) {
  const dim3 grid((unsigned)(a.tiles * a.nsplit * a.KV)), blk(512);
#define TTQ_AT(HDV)                                                                        \
  if (head_dim == HDV) {                                                                   \
    if (qf == QF_FP8) return ext_launch(k_attn_tile<HDV, 8, true>, grid, blk, 0, L, a);    \
    if (cb == 8) return ext_launch(k_attn_tile<HDV, 8, false>, grid, blk, 0, L, a);        \
    return ext_launch(k_attn_tile<HDV, 4, false>, grid, blk, 0, L, a);                     \
  }
  TTQ_AT(64)
  TTQ_AT(128)
  TTQ_AT(256)
#undef TTQ_AT
  return hipErrorInvalidValue;
}

}  // namespace ttq
