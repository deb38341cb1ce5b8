// A cache of rows that is quantized as it is written and read back (the K and
// V rows of a decoder: "Test-time quantization: quantising on the fly with no
// calibration dataset", lo0 blog, names KV-cache scales derived on the fly as
// the same logic applied to the cache).
//
// A cache row holds all C channels of a token (every head of K and V) and is
// laid out as ttq_quantize lays out a weight row: CB-bit containers, a scale and
// an offset per group of GS channels.  With D^{1/2} given (e.g. of the
// prompt's queries) the codes are those of u = x D^{1/2} and the row reads
// back as u_hat D^{-1/2}.
//
// Both kernels are one pass over their data and bound by memory: the write by
// the rows it reads, the read by the rows it writes (a bf16 row of 4-bit codes
// in groups of 128 is 2 C bytes out for 0.56 C in).  8 sequences of up to 4096
// rows of 8192 channels read back: 111 us, 4.4 TB/s; 2047 float32 rows of as many
// channels written in 2 bits: 18 us, 3.9 TB/s.
#include "cache_row.h"

namespace ttq {

namespace {

// One wave quantizes 512 channels of one row, 8 a lane (cache_row.h).
template <int GS, int QF>
__global__ __launch_bounds__(256) void k_cache_write(CacheWriteArgs a) {
  const int l = threadIdx.x & 63;
  const int64_t wid = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int64_t nchunk = (a.C + 511) / 512;
  const int64_t row = wid / nchunk;
  if (row >= a.T) return;  // uniform over the wave
  const int64_t slot = a.slots[row];  // (looked at once x is on its way)
  const int64_t c0 = (wid % nchunk) * 512 + l * 8;
  const bool live = c0 < a.C;  // C is a multiple of GS: whole groups

  float u[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) u[j] = 0.f;
  if (live) {
    if (a.x_f32) {
      const float* x = static_cast<const float*>(a.X) + row * a.ldx + c0;
      const f32x4 x0 = *(const f32x4*)x, x1 = *(const f32x4*)(x + 4);
      u[0] = x0.x; u[1] = x0.y; u[2] = x0.z; u[3] = x0.w;
      u[4] = x1.x; u[5] = x1.y; u[6] = x1.z; u[7] = x1.w;
    } else {
      const u32x4 x = *(const u32x4*)(static_cast<const bf16_t*>(a.X) + row * a.ldx + c0);
      u[0] = bf16lo(x.x); u[1] = bf16hi(x.x); u[2] = bf16lo(x.y); u[3] = bf16hi(x.y);
      u[4] = bf16lo(x.z); u[5] = bf16hi(x.z); u[6] = bf16lo(x.w); u[7] = bf16hi(x.w);
    }
    if (a.dh) {
      const f32x4 h0 = *(const f32x4*)(a.dh + c0), h1 = *(const f32x4*)(a.dh + c0 + 4);
      u[0] *= h0.x; u[1] *= h0.y; u[2] *= h0.z; u[3] *= h0.w;
      u[4] *= h1.x; u[5] *= h1.y; u[6] *= h1.z; u[7] *= h1.w;
    }
  }
  if (slot < 0 || slot >= a.n_slots) return;  // uniform
  quantize8<GS, QF>(u, live, slot, c0, a.C, a.row_bytes, a.Nf, a.rN, a.cb, a.codes, a.s, a.m);
}

// One wave reads 512 channels of CR consecutive rows of one sequence, 8 a
// lane.  Rows at or past the sequence's length, and rows whose page lies
// outside the cache, are left as they were.
//
// NT: the result is written past the last-level cache.  Where it is far larger
// than that cache, keeping it out gives the codes room (8 sequences of up to
// 4096 rows of 8192 channels, 4-bit -> bf16: 125 -> 111 us, 4.4 TB/s, where a
// plain copy reaches 4.8); where it fits, whoever reads it next finds it there
// (2047 rows of 8192 float32: 18 us written through the cache, 30 past it).
template <int CB, bool F8, bool OF32, int CR, bool NT>
__global__ __launch_bounds__(256) void k_cache_read(CacheReadArgs a) {
  auto store = [](auto v, auto* at) {
    if constexpr (NT) __builtin_nontemporal_store(v, at);
    else *at = v;
  };
  const int l = threadIdx.x & 63;
  const int64_t nchunk = (a.C + 511) / 512;
  const int64_t wid = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int64_t t0 = wid / nchunk * CR;
  const int64_t seq = blockIdx.y;
  const int64_t len = min((int64_t)a.lens[seq], a.T);
  if (t0 >= len) return;  // uniform over the wave
  const int64_t c0 = (wid % nchunk) * 512 + l * 8;
  if (c0 >= a.C) return;
  const int64_t G = a.C >> a.gshift, g = c0 >> a.gshift;

  unsigned w[CR][2];
  float s[CR], m[CR];
  bool ok[CR];
#pragma unroll
  for (int i = 0; i < CR; ++i) {
    const int64_t t = t0 + i;
    const int64_t pi = t >> a.pshift;
    ok[i] = t < len && pi < a.max_pages;
    const int64_t page = ok[i] ? a.pages[seq * a.max_pages + pi] : -1;
    const int64_t row = (page << a.pshift) + (t & ((1 << a.pshift) - 1));
    ok[i] = ok[i] && page >= 0 && row < a.n_slots;
    w[i][0] = w[i][1] = 0u;
    s[i] = m[i] = 0.f;
    if (ok[i]) {
      const uint8_t* src = a.codes + row * a.row_bytes + c0 * CB / 8;
      if (CB == 8) {
        const u32x2 v = *(const u32x2*)src;
        w[i][0] = v.x;
        w[i][1] = v.y;
      } else if (CB == 4) {
        w[i][0] = *(const unsigned*)src;
      } else if (CB == 2) {
        w[i][0] = *(const uint16_t*)src;
      } else {
        w[i][0] = *src;
      }
      s[i] = a.s[row * G + g];
      m[i] = a.m[row * G + g];
    }
  }
  float h[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) h[j] = 1.f;
  if (a.dhi) {
    const f32x4 h0 = *(const f32x4*)(a.dhi + c0), h1 = *(const f32x4*)(a.dhi + c0 + 4);
    h[0] = h0.x; h[1] = h0.y; h[2] = h0.z; h[3] = h0.w;
    h[4] = h1.x; h[5] = h1.y; h[6] = h1.z; h[7] = h1.w;
  }
#pragma unroll
  for (int i = 0; i < CR; ++i) {
    if (!ok[i]) continue;
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float q;
      if constexpr (F8) q = e4m3_byte(w[i][j / 4], j % 4);
      else if (CB == 8) q = (float)((w[i][j / 4] >> (8 * (j % 4))) & 0xffu);
      else q = (float)((w[i][0] >> (j * CB)) & ((1u << CB) - 1u));
      v[j] = fmaf(s[i], q, m[i]) * h[j];
    }
    const int64_t o = (seq * a.T + t0 + i) * a.C + c0;
    if constexpr (OF32) {
      float* out = static_cast<float*>(a.out) + o;
      store(f32x4{v[0], v[1], v[2], v[3]}, (f32x4*)out);
      store(f32x4{v[4], v[5], v[6], v[7]}, (f32x4*)(out + 4));
    } else {
      store(u32x4{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]),
                  pack_bf16(v[6], v[7])},
            (u32x4*)(static_cast<bf16_t*>(a.out) + o));
    }
  }
}

}  // namespace

hipError_t launch_cache_write(const CacheWriteArgs& a, int group, const Launch& L) {
  const int64_t waves = a.T * ((a.C + 511) / 512);
  if (waves == 0) return hipSuccess;
  const dim3 grid((unsigned)((waves + 3) / 4)), blk(256);
#define TTQ_CW_QF(GSV)                                                                      \
  case GSV:                                                                                 \
    switch (a.qf) {                                                                         \
      case QF_ASYM: return ext_launch(k_cache_write<GSV, QF_ASYM>, grid, blk, 0, L, a);     \
      case QF_SYM: return ext_launch(k_cache_write<GSV, QF_SYM>, grid, blk, 0, L, a);       \
      case QF_INTZP: return ext_launch(k_cache_write<GSV, QF_INTZP>, grid, blk, 0, L, a);   \
      case QF_FP8: return ext_launch(k_cache_write<GSV, QF_FP8>, grid, blk, 0, L, a);       \
      default: return hipErrorInvalidValue;                                                 \
    }
  switch (group) {
    TTQ_CW_QF(32)
    TTQ_CW_QF(64)
    TTQ_CW_QF(128)
    TTQ_CW_QF(256)
    default: return hipErrorInvalidValue;
  }
#undef TTQ_CW_QF
}

hipError_t launch_cache_read(const CacheReadArgs& a, int cb, const Launch& L) {
  const int64_t chunks = (a.C + 511) / 512;
  if (a.T == 0 || a.n_seq == 0) return hipSuccess;
  // more than the last-level cache holds (256 MiB), by the room for the rows;
  // there a wave's four rows in flight also pay (133 us with two), while short
  // reads want the most waves (33 rows of 1024: 3.5 us with four, 2.7 with one)
  const bool nt = a.n_seq * a.T * a.C > (int64_t(256) << 20) / (a.out_f32 ? 4 : 2);
  auto go = [&](auto kernel, int rows) {
    return ext_launch(kernel, dim3((unsigned)(((a.T + rows - 1) / rows * chunks + 3) / 4),
                                   (unsigned)a.n_seq), dim3(256), 0, L, a);
  };
#define TTQ_CR(CBV, F8)                                                                       \
  if (a.out_f32)                                                                              \
    return nt ? go(k_cache_read<CBV, F8, true, 4, true>, 4) : go(k_cache_read<CBV, F8, true, 1, false>, 1); \
  return nt ? go(k_cache_read<CBV, F8, false, 4, true>, 4) : go(k_cache_read<CBV, F8, false, 1, false>, 1);
  if (a.qf == QF_FP8) {
    if (cb != 8) return hipErrorInvalidValue;
    TTQ_CR(8, true)
  }
  switch (cb) {
    case 1: TTQ_CR(1, false)
    case 2: TTQ_CR(2, false)
    case 4: TTQ_CR(4, false)
    case 8: TTQ_CR(8, false)
    default: return hipErrorInvalidValue;
  }
#undef TTQ_CR
}

}  // namespace ttq
