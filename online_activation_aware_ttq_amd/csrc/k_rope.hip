// Norms of the query and key heads of a step's rows and their rotation by
// position, with the K and V rows quantized into the cache in the same pass:
// what the projection leaves is read once, and K and V are never written in
// between.
//
// For a head x of HD channels, pairs (a, b) of channels and position t,
//   y = (x r) w,  r = 1 / sqrt(mean(x^2) + eps)
//   (a, b) -> (a c - b s, b c + a s),  c, s = cos, sin(t f_i).
// r and the angles are float64 (float32 loses the angles of far positions: at a
// position of 10^6 half a unit of the first angle is 0.03), rounded once to
// float32; products and sums are float32, each rounded, none fused, because the
// codes that follow are decided by exact comparisons.  Queries are rounded once
// more, to bf16.
//
// One wave takes 512 channels of a row at a time, 8 a lane: 512 is a whole number
// of heads (a head is HD / 8 adjacent lanes) and of groups, and a lane has the
// same channels of a head in each of its chunks, so it needs its 8 (interleaved:
// 4) angles once; a chunk is asked for while the one before is worked on (42 -> 38 us).
//
// 4096 rows of 32 / 8 heads of 128 to 4 bits: 38 us, 2.3 TB/s of the 89 MB that it has to
// read and write (a copy reaches 4.8); waves wait for memory 45 % of their time, with one
// chunk of 16 bytes a lane on its way, and issue vector instructions 23 % of it.  One row:
// 6 us, most of it the launch, the angles in float64 and two loads after one another.
#include <algorithm>

#include "cache_row.h"

namespace ttq {

namespace {

// Cosine and sine of an angle of any size, in float64: x less its nearest multiple
// n of pi / 2 (pi / 2 as a sum of two doubles; n below 2^52, the first product in
// fma is exact, so the error is that of the result), then the power series of both
// on [-pi/4, pi/4] up to x^17 and x^16, whose next terms are below 2^-57.
__device__ __forceinline__ void sincos64(double x, double& s, double& c) {
  const double n = __builtin_rint(x * 0.63661977236758134308);
  double r = __builtin_fma(-n, 1.57079632679489655800, x);
  r = __builtin_fma(-n, 6.12323399573676603587e-17, r);
  const double z = r * r;
  double p = 1.0 / 355687428096000.0;
  p = __builtin_fma(p, z, -1.0 / 1307674368000.0);
  p = __builtin_fma(p, z, 1.0 / 6227020800.0);
  p = __builtin_fma(p, z, -1.0 / 39916800.0);
  p = __builtin_fma(p, z, 1.0 / 362880.0);
  p = __builtin_fma(p, z, -1.0 / 5040.0);
  p = __builtin_fma(p, z, 1.0 / 120.0);
  p = __builtin_fma(p, z, -1.0 / 6.0);
  const double sn = __builtin_fma(p * z, r, r);
  double q = 1.0 / 20922789888000.0;
  q = __builtin_fma(q, z, -1.0 / 87178291200.0);
  q = __builtin_fma(q, z, 1.0 / 479001600.0);
  q = __builtin_fma(q, z, -1.0 / 3628800.0);
  q = __builtin_fma(q, z, 1.0 / 40320.0);
  q = __builtin_fma(q, z, -1.0 / 720.0);
  q = __builtin_fma(q, z, 1.0 / 24.0);
  q = __builtin_fma(q, z, -0.5);
  const double cs = __builtin_fma(q, z, 1.0);
  const long long k = (long long)n;
  const double a = (k & 1) ? cs : sn, b = (k & 1) ? sn : cs;
  s = (k & 2) ? -a : a;
  c = ((k + 1) & 2) ? -b : b;
}

// 8 values of a row, bf16 (the first 16 bytes) or float32
struct Raw {
  u32x4 x, y;
};
__device__ __forceinline__ void load8(const void* X, int64_t at, int f32, Raw& r) {
  if (f32) {
    const u32x4* p = (const u32x4*)(static_cast<const float*>(X) + at);
    r.x = p[0];
    r.y = p[1];
  } else {
    r.x = *(const u32x4*)(static_cast<const bf16_t*>(X) + at);
  }
}
__device__ __forceinline__ void values8(const Raw& r, int f32, float (&u)[8]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (f32) {
      u[j] = __uint_as_float(r.x[j]);
      u[4 + j] = __uint_as_float(r.y[j]);
    } else {
      u[2 * j] = bf16lo(r.x[j]);
      u[2 * j + 1] = bf16hi(r.x[j]);
    }
  }
}

template <int GS, int QF>
__global__ __launch_bounds__(256) void k_cache_rope(RopeArgs a) {
  const int l = threadIdx.x & 63;
  const int64_t wid = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int64_t row = wid / a.parts;
  if (row >= a.T) return;  // uniform over the wave
  const int part = (int)(wid % a.parts);
  const int lph = a.head_dim / 8;          // lanes of a head
  const int ch = (l & (lph - 1)) * 8;      // this lane's channels of a head
  const int half = a.rot_dim / 2;
  const bool inter = a.inter != 0;
  const int nq = (a.q_width + 511) / 512, nk = (a.kv_width + 511) / 512;
  const int64_t slot = a.slots[row];

  // a chunk's channels of this lane, asked for a chunk ahead
  auto column = [&](int chunk) {
    return (chunk < nq ? chunk : chunk >= nq + nk ? chunk - nq - nk : chunk - nq) * 512 + l * 8;
  };
  auto fetch = [&](int chunk) {
    Raw r{};
    const int cl = column(chunk);
    if (chunk < nq) {
      if (cl < a.q_width) load8(a.Q, row * a.ldq + cl, a.x_f32, r);
    } else if (cl < a.kv_width && chunk < nq + 2 * nk) {
      if (chunk >= nq + nk) load8(a.V, row * a.ldv + cl, a.x_f32, r);
      else load8(a.K, row * a.ldk + cl, a.x_f32, r);
    }
    return r;
  };
  Raw next = fetch(part);

  // angles: of this lane's 4 pairs (interleaved), or of its 8 channels, whose
  // other halves are rot_dim / 16 lanes on or back
  float co[8], si[8];
  const bool rotated = ch < a.rot_dim;
  const bool upper = !inter && ch >= half;
  const int other = inter || !rotated ? l : upper ? l - half / 8 : l + half / 8;
  if (a.rot_dim && part < nq + nk) {
    const double t = a.positions[row];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      co[j] = 1.f;
      si[j] = 0.f;
      if (!rotated || (inter && j >= 4)) continue;
      double s, c;
      sincos64(t * (double)a.inv_freq[inter ? ch / 2 + j : upper ? ch - half + j : ch + j], s, c);
      co[j] = (float)c;
      si[j] = (float)s;
    }
  }

  for (int chunk = part; chunk < nq + 2 * nk; chunk += a.parts) {
    const bool is_q = chunk < nq, is_v = chunk >= nq + nk;
    const int cl = column(chunk);
    const bool live = cl < (is_q ? a.q_width : a.kv_width);
    float u[8];
    values8(next, a.x_f32, u);
    next = fetch(chunk + a.parts);
    const float* w = is_q ? a.wq : a.wk;
    if (!is_v && w) {
      double ss = 0.0;
#pragma unroll
      for (int j = 0; j < 8; ++j) ss = __builtin_fma((double)u[j], (double)u[j], ss);
      for (int off = 1; off < lph; off <<= 1) ss += __shfl_xor(ss, off);
      const float r = (float)(1.0 / __builtin_sqrt(ss * a.inv_hd + a.eps));
      const f32x4 w0 = *(const f32x4*)(w + ch), w1 = *(const f32x4*)(w + ch + 4);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        u[j] = u[j] * r * w0[j];
        u[j + 4] = u[j + 4] * r * w1[j];
      }
    }
    if (!is_v && a.rot_dim) {
      if (inter) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float x = u[2 * j], y = u[2 * j + 1];
          if (rotated) {
            u[2 * j] = x * co[j] - y * si[j];
            u[2 * j + 1] = y * co[j] + x * si[j];
          }
        }
      } else {
        float y[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = __shfl(u[j], other);
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (rotated) u[j] = upper ? u[j] * co[j] + y[j] * si[j] : u[j] * co[j] - y[j] * si[j];
      }
    }
    if (is_q) {
      if (live)
        *(u32x4*)(a.Q_out + row * a.q_width + cl) =
            u32x4{pack_bf16(u[0], u[1]), pack_bf16(u[2], u[3]), pack_bf16(u[4], u[5]),
                  pack_bf16(u[6], u[7])};
      continue;
    }
    const int64_t c0 = (is_v ? a.v_first : a.k_first) + cl;
    const float* dh = is_v ? a.v_dh : a.k_dh;
    if (live && dh) {
      const f32x4 h0 = *(const f32x4*)(dh + c0), h1 = *(const f32x4*)(dh + c0 + 4);
      u[0] *= h0.x; u[1] *= h0.y; u[2] *= h0.z; u[3] *= h0.w;
      u[4] *= h1.x; u[5] *= h1.y; u[6] *= h1.z; u[7] *= h1.w;
    }
    if (slot < 0 || slot >= a.n_slots) continue;  // uniform
    quantize8<GS, QF>(u, live, slot, c0, a.C, a.row_bytes, a.Nf, a.rN, a.cb,
                      is_v ? a.v_codes : a.k_codes, is_v ? a.v_s : a.k_s,
                      is_v ? a.v_m : a.k_m);
  }
}

}  // namespace

hipError_t launch_cache_rope(RopeArgs a, int group, const Launch& L) {
  const int chunks = (a.q_width + 511) / 512 + 2 * ((a.kv_width + 511) / 512);
  // a wave's chunks share its angles: as few waves a row as still fill the chip (4096
  // rows of 32 / 8 heads of 128: twice as many waves take 2 us longer, four times 6)
  a.parts = (int)std::min<int64_t>(chunks, std::max<int64_t>(1, (4096 + a.T - 1) / a.T));
  const int64_t waves = a.T * a.parts;
  const dim3 grid((unsigned)((waves + 3) / 4)), blk(256);
#define TTQ_RP_QF(GSV)                                                                      \
  case GSV:                                                                                 \
    switch (a.qf) {                                                                         \
      case QF_ASYM: return ext_launch(k_cache_rope<GSV, QF_ASYM>, grid, blk, 0, L, a);      \
      case QF_SYM: return ext_launch(k_cache_rope<GSV, QF_SYM>, grid, blk, 0, L, a);        \
      case QF_INTZP: return ext_launch(k_cache_rope<GSV, QF_INTZP>, grid, blk, 0, L, a);    \
      case QF_FP8: return ext_launch(k_cache_rope<GSV, QF_FP8>, grid, blk, 0, L, a);        \
      default: return hipErrorInvalidValue;                                                 \
    }
  switch (group) {
    TTQ_RP_QF(32)
    TTQ_RP_QF(64)
    TTQ_RP_QF(128)
    TTQ_RP_QF(256)
    default: return hipErrorInvalidValue;
  }
#undef TTQ_RP_QF
}

}  // namespace ttq
