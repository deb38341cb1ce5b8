// Attention over a cache of quantized rows where many query rows share their keys
// (prompts and chunks of them): tiles of keys, decoded once for 256 rows.
//
// A workgroup takes 256 query rows of one K/V head (a token's G heads, then the next
// token's) and its keys, KT = 8192 / HD at a time, decoded once for all of them as
// fp16(s (c - mid) + (m + mid s)) into LDS rows of K and of V.  Each of its eight waves has 32 rows:
//   S^T = K q'^T   (32 keys x 32 rows an instruction block).  Key 16s + 8h + 4a + b
//                  of a block is row 16s + 8a + 4h + b, so that the lane of a row (h
//                  = lane / 32) ends with the 8 adjacent keys 16s + 8h ..  of it
//   O^T += V^T P^T that it has to give here: nothing passes between lanes but the
//                  maximum.  V is transposed as it is read (16 lanes, 4 keys).
// The sums of p are those of the fp16 values that weight V (v_dot2).
//
// A SIMD has two waves (256 registers each), and a wave's tile is 32 matrix
// instructions of 32 cycles and about 300 vector ones, 32 of them exponentials.  Left
// to themselves both waves do the same at the same time.  So half of the waves are
// half a step behind: while they do their products, the others do the softmax.  The
// decoding of the next tile is spread between the products, whose operands are read
// four ahead of them; the order is fixed by hand, for the compiler's waits for each
// operand before its product (a tile of 64 keys and 128 channels: 3.6 us with waves
// that decode, multiply and weigh all together, 2.3 so; an order left to the compiler
// 5.8).  With all that a compute unit's tile is 5000 cycles where the matrix
// instructions are 2048: a products' phase takes 2200 and the other's 1850 and the
// two have to wait for each other twice a tile.  LDS is read for 1360 cycles of it and
// has 500 of conflicts.  64 rows a wave would halve its reads, for twice the registers.
//
// Besides, a workgroup of one tile takes 21 us: its rows, pages and codes are a chain
// of loads, and a compute unit holds one workgroup.  4 prompts of up to 2047 tokens, 32 / 8 heads
// of 128, 4 bits: 121 us a call, 518 TFLOP/s of the visible keys.
//
// fp16's range is kept by powers of two: K and V are decoded as 2^-YK and 2^-YV of what
// they are, YK and YV a group's (for all keys of the block), which put the median of a
// few keys that all rows see at 2 to 4; q' is times 2^YK, and as in k_attention.hip.  A
// key whose groups are all 2^-8 to 4000 in these units (or 0) keeps 11 bits, or 2^-16 of
// its group's largest value.  Keys of another size, 2^9 and more from that, are left out
// of the tiles, and what they give the rows that see them is added from their
// codes in float32, one after another: so no row depends on the size of a key that it
// does not see, and a seen one costs the others no bits.  That is slow, about 12 us a key
// of a workgroup, most of it waiting for its codes (4 prompts of 2048 tokens, 32 / 8 heads of
// 128: 242 us, with one such token in 1024 297, with one in 64 1080).
// The maximum of a row follows only steps of 2^8 (p and the sums may be as much
// larger), so O is seldom scaled; p is 2^7 of what it is, so that fp16 holds the many
// small ones of a long context, to 2^-32 of the largest.
#include <algorithm>

#include "attn.h"
#include "block_order.h"

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

// Of 16 lanes that read 4 values each, 4 lanes a row, lane i is given column i of the
// four rows
typedef __attribute__((ext_vector_type(4))) _Float16 f16x4;
typedef __attribute__((ext_vector_type(4))) short i16x4;
__device__ __forceinline__ f16x4 read_columns(const _Float16* p) {
  return __builtin_bit_cast(f16x4, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
      (__attribute__((address_space(3))) i16x4*)p));
}

// A value in a register of its own, so that a load can go to the one it was in: without
// it the compiler copies what a step loads at that step's end, and waits for it there
template <typename T>
__device__ __forceinline__ void copy_reg(T& to, T from) {
  asm("v_mov_b32 %0, %1" : "=&v"(to) : "v"(from));
}

// LDS is as all waves left it; global loads stay in flight
__device__ __forceinline__ void step_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_sched_barrier(0);
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_sched_barrier(0);
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// Sums of x over lanes 0 .. l
__device__ __forceinline__ int lane_scan(int x) {
  x += __builtin_amdgcn_update_dpp(0, x, 0x111, 0xf, 0xf, true);   // row_shr 1, 2, 4, 8
  x += __builtin_amdgcn_update_dpp(0, x, 0x112, 0xf, 0xf, true);
  x += __builtin_amdgcn_update_dpp(0, x, 0x114, 0xf, 0xf, true);
  x += __builtin_amdgcn_update_dpp(0, x, 0x118, 0xf, 0xf, true);
  x += __builtin_amdgcn_update_dpp(0, x, 0x142, 0xa, 0xf, false);  // row_bcast 15, 31
  x += __builtin_amdgcn_update_dpp(0, x, 0x143, 0xc, 0xf, false);
  return x;
}

// The lanes of a wave, each with a sequence (block_order.h)
struct LaneWave {
  LaneSeq own;
  template <class F>
  __device__ __forceinline__ int total(F f) const {
    return __builtin_amdgcn_readlane(lane_scan(f(own)), 63);
  }
  template <class F>
  __device__ __forceinline__ int owner(F f, int i, int& at) const {
    const int n = f(own), scan = lane_scan(n);
    const int lane = __builtin_ctzll(__ballot(scan > i));
    at = i - __builtin_amdgcn_readlane(scan - n, lane);
    return lane;
  }
  template <class F>
  __device__ __forceinline__ int of(int lane, F f) const {
    return __builtin_amdgcn_readlane(f(own), lane);
  }
};

// find_block with the blocks in another order, those of the most keys first (to within
// 256 keys): the last workgroups to begin are then short, where prompts of 2047 and
// 900 tokens in the order of the batch leave a fifth of the time to a few.  For up to
// 64 sequences, one a lane; more have enough blocks for any order.
__device__ __forceinline__ bool find_long_block(const AttnArgs& a, int64_t b, int64_t& seq, SeqRows& s,
                                                int64_t& r0) {
  const int l = threadIdx.x & 63;
  int64_t first = 0;
  LaneWave w{};
  if (l < a.n_seq) {
    first = min(max((int64_t)a.offsets[l], (int64_t)0), a.T);
    const int64_t tokens = max(min(max((int64_t)a.offsets[l + 1], (int64_t)0), a.T) - first, (int64_t)0);
    w.own.len = max(a.lens[l], 0);
    w.own.rows = tokens * a.G;
    w.own.shift = w.own.len - tokens;
  }
  int from = 0;
  if (!long_block(w, (int)b, a.max_len, a.G, from, r0)) return false;
  auto of = [&](int64_t v) __attribute__((always_inline)) {
    const unsigned lo = __builtin_amdgcn_readlane((int)v, from), hi = __builtin_amdgcn_readlane((int)(v >> 32), from);
    return (int64_t)((uint64_t)hi << 32 | lo);
  };
  seq = from;
  s.first = of(first);
  s.rows = (int)of(w.own.rows);
  s.shift = of(w.own.shift);
  s.len = min(min(of(w.own.len), a.max_len), a.max_pages << a.pshift);
  return true;
}

template <int HD, int CB, bool F8>
__global__ __launch_bounds__(512, 2) void k_attn_tile(AttnArgs a) {
  constexpr int KT = 8192 / HD;      // keys of a tile
  constexpr int NKT = KT / 32;       // blocks of 32 keys
  constexpr int NCT = HD / 32;       // blocks of 32 channels
  constexpr int KS = HD / 16;        // steps of 16 channels
  constexpr int PS = KT / 16;        // steps of 16 keys
  constexpr int KP = HD / 16;        // threads that decode a key
  constexpr float kInf = __builtin_inff();
  constexpr float kLazy = 8.f, kLift = 7.f;  // p of the largest score: 2^kLift to 2^(kLift + kLazy)
  // sizes of a group in a tile's units; and codes there are (c - mid) / 64 (E4M3: / 256),
  // so that a group's scale is about as large as its values
  constexpr float kMost = 4000.f, kLeast = 0x1p-8f;
  constexpr int kCode = F8 ? 8 : 6;
  constexpr int kNoUnit = 1000;  // (of a key that is not there, or 0; if all are, -1)
  // LDS rows are of 16-byte pieces, K's in the order piece ^ key % 8.  Of V, 16 lanes
  // read 32 bytes of 4 keys, the next 16 the 32 bytes beside them: in eight parts of the
  // banks, and the first four in four of half of the banks.
  auto v_flip = [](int key) { return (key & 3) << 1 | (HD == 64 ? 0 : (key & 1) << 3); };
  constexpr unsigned kOut = 1u << 31;  // the key is in no page of the cache, or left out
  __shared__ __align__(16) _Float16 sm_k[2][KT * HD];
  __shared__ __align__(16) _Float16 sm_v[2][KT * HD];
  __shared__ unsigned sm_bad[3][KT];  // of a key: groups of V that are NaN; kOut
  __shared__ int sm_ctl[3];           // a key of the tile is in sm_bad
  __shared__ int sm_y[2][HD / 32];    // YK, YV of 32 channels
  __shared__ unsigned sm_far[33];     // tiles (mod 1024) that have left out keys, a bit each; any

  const int tid = threadIdx.x, l = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int n = l & 31, hf = l >> 5;
  const unsigned group = attn_group();
  const int h = (int)(group % a.KV);
  const unsigned bs = group / a.KV, nsplit = (unsigned)a.nsplit;
  const int split = (int)(bs % nsplit);
  const int64_t block = bs / nsplit;
  if (block >= a.tiles) return;
  int64_t seq, r0;
  SeqRows sr;
  if (!(a.offsets && a.n_seq <= 64 ? find_long_block(a, block, seq, sr, r0)
                                   : find_block<256>(a, a.tiles - 1 - block, seq, sr, r0)))
    return;  // uniform over the workgroup

  seq = uniform64(seq);
  r0 = uniform64(r0);
  sr.first = uniform64(sr.first);
  sr.shift = uniform64(sr.shift);
  sr.len = uniform64(sr.len);
  sr.rows = __builtin_amdgcn_readfirstlane(sr.rows);

  // keys of the workgroup, and of this wave; key numbers are from lo on
  // (32-bit divisions: all rows of a call are fewer than 2^31)
  const unsigned first = (unsigned)r0, last = (unsigned)sr.rows - 1, G = (unsigned)a.G;
  const int64_t wg_lo = sr.shift + first / G, wg_hi = sr.shift + min(first + 255, last) / G;
  int64_t lo = a.window > 0 ? max(wg_lo - a.window + 1, (int64_t)0) / KT * KT : 0;
  const int64_t hi = min(sr.len, wg_hi + 1);
  const int64_t tiles = max(hi - lo + KT - 1, (int64_t)0) / KT;  // (< 2^31)
  const int64_t per = (int64_t)(((unsigned)tiles + nsplit - 1) / nsplit) * KT;
  lo += per * split;
  auto rel = [&](int64_t key) { return (int)min(max(key - lo, (int64_t)INT32_MIN), (int64_t)INT32_MAX); };
  const int end = rel(min(lo + per, hi));
  const unsigned w0 = first + 32 * w;  // this wave's first row
  const int64_t pos_lo = sr.shift + min(w0, last) / G;
  const int64_t pos_hi = sr.shift + min(w0 + 31, last) / G;
  // the keys that all of its rows see
  const int full_hi = min(rel(pos_lo), end - 1);
  const int full_lo = a.window > 0 ? rel(pos_hi - a.window + 1) : 0;
  unsigned r = min(w0 + n, last);
  const int64_t pos = sr.shift + r / G;
  // this row's, neither far below 0: a tile's first key is taken from them
  const int top_key = max(min(rel(pos), end - 1), -1);
  const int low_key = a.window > 0 ? max(rel(pos - a.window + 1), 0) : 0;
  const bf16_t* src = hf * 8 + a.Q + (sr.first + r / G) * a.ldq + (h * G + r % G) * HD;

  u32x4 qraw[KS];
  f32x16 o[NCT];
#pragma unroll
  for (int i = 0; i < NCT; ++i)
#pragma unroll
    for (int j = 0; j < 16; ++j) o[i][j] = 0.f;
  float mrun = -kInf, sum = 0.f;
  unsigned nan_groups = 0;

  // what this thread decodes of a tile: 16 channels of a key of K, and of V
  const int kkey = tid / KP, kch = tid % KP * 16;
  const int kpos = (kkey & ~31) + ((kkey >> 4) & 1) * 16 + ((kkey >> 2) & 1) * 8 + ((kkey >> 3) & 1) * 4 + (kkey & 3);
  const int32_t* table = a.pages + seq * a.max_pages;
  const int64_t pmask = (int64_t(1) << a.pshift) - 1;
  const int64_t kc = a.k_first + h * HD + kch, vc = a.v_first + h * HD + kch;
  const int64_t kg = kc >> a.gshift, vg = vc >> a.gshift;
  const unsigned nan_bit = 1u << (int)(vg - ((a.v_first + h * HD) >> a.gshift));
  struct Codes {
    unsigned k[CB / 2], v[CB / 2];
  };
  struct Scales {
    float ks, km, vs, vm;
  };
  auto page_at = [&](int t) __attribute__((always_inline)) {
    return table[(lo + min(t * KT + kkey, end - 1)) >> a.pshift];
  };
  auto row_at = [&](int t, int page) __attribute__((always_inline)) {
    const int key = t * KT + kkey;
    const int64_t at = ((int64_t)page << a.pshift) + ((lo + key) & pmask);
    return (page >= 0) & (at < a.n_slots) & (key < end) ? (int)at : -1;
  };
  auto row_times = [](int row, int64_t by) { return (uint64_t)(unsigned)max(row, 0) * (unsigned)by; };
  // (a key in no page reads row 0, which is there to be read, and counts nothing)
  auto codes_of = [&](int rk, int rv) __attribute__((always_inline)) {
    Codes x;
    const uint8_t* ck = a.kc + row_times(rk, a.row_bytes) + kc * CB / 8;
    const uint8_t* cv = a.vc + row_times(rv, a.row_bytes) + vc * CB / 8;
    if constexpr (CB == 8) {
      const u32x4 k = *(const u32x4*)ck, v = *(const u32x4*)cv;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x.k[i] = k[i];
        x.v[i] = v[i];
      }
    } else {
      const u32x2 k = *(const u32x2*)ck, v = *(const u32x2*)cv;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        x.k[i] = k[i];
        x.v[i] = v[i];
      }
    }
    return x;
  };
  auto scales_of = [&](int rk, int rv) __attribute__((always_inline)) {
    const uint64_t k = row_times(rk, a.groups) + kg, v = row_times(rv, a.groups) + vg;
    return Scales{a.ks[k], a.km[k], a.vs[v], a.vm[v]};
  };
  auto nan = [](float s, float m) { return s != s || m != m; };
  // the largest value that a group may hold (NaN or infinite if s or m is)
  auto size_of = [&](float s, float m) __attribute__((always_inline)) {
    return F8 ? fmaf(m, 0.f, __builtin_fabsf(s) * 448.f)
              : __builtin_elementwise_maximum(__builtin_fabsf(s) * (float)a.mid,
                                              __builtin_fabsf(fmaf(s, (float)a.mid, m)));
  };
  auto unit_of = [&](float s, float m) __attribute__((always_inline)) {
    const float x = size_of(s, m);
    return x > 0.f && x <= 3.402823466e38f ? min(max(__builtin_amdgcn_frexp_expf(x) - 2, -100), 100) : kNoUnit;
  };
  // Is a group's size one of a tile's, 2^y kLeast to 2^y kMost: as bits of floats
  auto fits = [&](float s, float m, int y) __attribute__((always_inline)) {
    const unsigned least = __float_as_uint(kLeast), most = __float_as_uint(kMost);
    return __float_as_uint(size_of(s, m)) - (least + ((unsigned)y << 23)) <= most - least;
  };

  const int late = w >> 2;  // 0: the waves that are ahead, 1: half a step behind
  Codes x;           // of pair d
  Scales xs, next;   // of pairs d and d + 1
  int r1, r2, r3;    // rows of this thread's key in tiles d + 1, d + 2, d + 3
  int page;          // and its page in tile d + 4
  int YK = -1, YV = -1;  // of this thread's group
  bool bad_keys = false;  // tile d has keys of sm_bad
  int ctl;
  uint64_t far_k = 0;  // lanes whose key is left out for its K, before its V is there

  // Is a group left out for its size; and of which keys is one (the KP threads of a key
  // are lanes beside each other)
  auto far = [&](float s, float m, int y) __attribute__((always_inline)) {
    return !fits(s, m, y) && size_of(s, m) > 0.f && !nan(s, m);
  };
  auto of_key = [&](uint64_t lanes) __attribute__((always_inline)) {
    return (lanes & (((uint64_t(1) << KP) - 1) << (l & -KP))) != 0;
  };

  // The scales xs of pair d, K's of row rk and V's of row rv.  Rare: keys in no page,
  // NaN, and keys of another size than the tile's.
  auto check = [&](int d, int rk, int rv) __attribute__((always_inline)) {
    const bool usual = fits(xs.ks, xs.km, YK) & fits(xs.vs, xs.vm, YV) & ((rk | rv) >= 0);
    if (__builtin_expect((__ballot(!usual) | far_k) == 0, 1)) return;
    finite_or_nan(xs.ks, xs.km);
    finite_or_nan(xs.vs, xs.vm);
    const bool bad = nan(xs.vs, xs.vm);
    const bool k_far = far(xs.ks, xs.km, YK), v_far = far(xs.vs, xs.vm, YV);
    const int slot = (d + 3) % 3;
    const bool left = (of_key(far_k) | of_key(__ballot(v_far))) & (rv >= 0);
    if (d >= 0 && d * KT + kkey < end && (left || bad || rv < 0)) {
      atomicOr(&sm_bad[slot][kkey], (bad && rv >= 0 ? nan_bit : 0u) | (left || rv < 0 ? kOut : 0u));
      sm_ctl[slot] = 1;
      if (left) {
        atomicOr(&sm_far[d >> 5 & 31], 1u << (d & 31));
        sm_far[32] = 1;
      }
    }
    if (rk < 0) xs.ks = xs.km = 0.f;
    if (rv < 0 || bad || v_far) xs.vs = xs.vm = 0.f;
    far_k = __ballot(k_far);
  };
  // Pair d into LDS, and on with what later ones need, in kPieces of code.
  // (half of the threads begin with the other 8 channels, for the other banks)
  const bool v_odd = tid >> 2 & 1, k_odd = HD > 64 && v_odd;
  // (a code in the low bits of 16 counts 1 / 64, a nibble above another 1 / 4)
  const unsigned mid = (unsigned)a.mid * 0x00010001u + k16, mid16 = ((unsigned)a.mid * 0x00010001u << 4) + k16;
  unsigned k16v = k16;
  if constexpr (CB == 4) asm("" : "+v"(k16v));  // (in a register: and and or in one instruction)
  constexpr int kPieces = 10;
  struct Factors {
    unsigned s1, s16, m;
  } fk, fv;
  auto factors = [&](float s, float m, int y) __attribute__((always_inline)) {
    // the offset of the middle of the codes, which is small where that of the first is
    // half the range and would lose so many bits more
    const float x = ldexpf(s, kCode - y), b = F8 ? 0.f : ldexpf(fmaf(s, (float)a.mid, m), -y);
    return Factors{both(x, x), both(x * 0.0625f, x * 0.0625f), both(b, b)};
  };
  auto decode = [&](const unsigned (&code)[CB / 2], int u, const Factors& x, _Float16* dst, int flip, bool odd) __attribute__((always_inline)) {
    unsigned w[2];
#pragma unroll
    for (int i = 0; i < CB / 4; ++i) {
      const unsigned c0 = code[u * CB / 4 + i], c1 = code[(1 - u) * CB / 4 + i];
      w[i] = odd ? c1 : c0;
    }
    if (CB == 4) w[1] = 0u;
    // (E4M3 has NaN, and a row that is not this cache's may hold it)
    if (F8 && x.s1 == 0u) w[0] = w[1] = 0u;
    u32x4 v = codes8_normal<CB, F8>(w[0], w[1], k16v);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const bool by16 = !F8 && slot_shift<CB>(2 * i);
      if (!F8) v[i] = u2(h2(v[i]) - h2(by16 ? mid16 : mid));  // exact, as is a code
      v[i] = fma2(v[i], by16 ? x.s16 : x.s1, x.m);
    }
    *(u32x4*)&dst[(((kch >> 3) + (odd ? 1 - u : u)) ^ flip) * 8] = v;
  };
  auto stage = [&](int d, int piece) __attribute__((always_inline)) {
    if (piece == 0) {
      bad_keys = __builtin_amdgcn_readfirstlane(ctl) != 0;
      fk = factors(xs.ks, xs.km, YK);
    }
    if (piece == 1) decode(x.k, 0, fk, &sm_k[(d + 1) & 1][kpos * HD], kpos & 7, k_odd);
    if (piece == 2) decode(x.k, 1, fk, &sm_k[(d + 1) & 1][kpos * HD], kpos & 7, k_odd);
    if (piece == 3) fv = factors(xs.vs, xs.vm, YV);
    if (piece == 4) decode(x.v, 0, fv, &sm_v[d & 1][kkey * HD], v_flip(kkey), v_odd);
    if (piece == 5) decode(x.v, 1, fv, &sm_v[d & 1][kkey * HD], v_flip(kkey), v_odd);
    if (piece == 6) x = codes_of(r2, r1);
    if (piece == 7) {
      copy_reg(xs.ks, next.ks);
      copy_reg(xs.km, next.km);
      copy_reg(xs.vs, next.vs);
      copy_reg(xs.vm, next.vm);
      check(d + 1, r2, r1);
    }
    if (piece == 8) {
      next = scales_of(r3, r2);
      int pg;
      copy_reg(pg, page);
      r1 = r2;
      r2 = r3;
      r3 = row_at(d + 4, pg);
    }
    if (piece == 9) page = page_at(d + 5);
  };

  // the first keys, and the rows of Q meanwhile
  if (end > 0) {
    const int p0 = page_at(0), p1 = page_at(1), p2 = page_at(2);
    page = page_at(3);
#pragma unroll
    for (int i = 0; i < KS; ++i) qraw[i] = *(const u32x4*)(src + i * 16);
    if (w == 0) {
      // The units, by 64 / KP keys over the range that all rows see: of each group the
      // key in the middle of their sizes
      const int64_t to = min(max(wg_lo, (int64_t)0), sr.len - 1);
      const int64_t from = a.window > 0 ? min(max(wg_hi - a.window + 1, (int64_t)0), to) : 0;
      const int64_t key = to - (to - from) * kkey / (64 / KP);
      const int64_t at = ((int64_t)table[key >> a.pshift] << a.pshift) + (key & pmask);
      const int row = at >= 0 && at < a.n_slots ? (int)at : -1;
      const Scales unit = scales_of(row, row);
      int e[2] = {row >= 0 ? unit_of(unit.ks, unit.km) : kNoUnit, row >= 0 ? unit_of(unit.vs, unit.vm) : kNoUnit};
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        int below = 0, valid = 0;
#pragma unroll
        for (int j = 0; j < 64 / KP; ++j) {
          const int x = __shfl(e[i], j * KP + l % KP);
          below += x < e[i] || (x == e[i] && j < kkey);
          valid += x != kNoUnit;
        }
        if (below == (valid > 0 ? (valid - 1) / 2 : 0)) sm_y[i][kch / 32] = e[i] == kNoUnit ? -1 : e[i];
      }
    }
    r1 = row_at(0, p0);
    r2 = row_at(1, p1);
    r3 = row_at(2, p2);
    x = codes_of(r1, -1);
    xs = scales_of(r1, -1);
    next = scales_of(r2, r1);
  }

  // q' 2^YK in fp16, its largest value in [2^10, 2^11); the sign of the scale goes with
  // it.  Eight values at a time first, times a power of two of their own, while YK is on
  // its way.
  f16x8 q[KS];
  int qe[KS];
  float qm = 1.f;
  auto convert_q = [&]() __attribute__((always_inline)) {
    const unsigned flip = a.scale2 < 0.f ? 0x80008000u : 0u, keep = a.scale2 == 0.f ? 0u : ~0u;
#pragma unroll
    for (int i = 0; i < KS; ++i) qraw[i] = (qraw[i] ^ flip) & keep;
    auto value = [&](int i, int j) __attribute__((always_inline)) {
      return j & 1 ? bf16hi(qraw[i][j >> 1]) : bf16lo(qraw[i][j >> 1]);
    };
    auto convert = [&](auto times) __attribute__((always_inline)) {
#pragma unroll
      for (int i = 0; i < KS; ++i) {
        float top = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) top = fmaxf(top, __builtin_fabsf(times(value(i, j), i, j)));
        const int e = top > 3.402823466e38f ? 129 : __builtin_amdgcn_frexp_expf(top);
        qe[i] = top > 0.f ? e - 11 : -1000;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int c = slot_code<CB>(j);
          q[i][j] = (_Float16)ldexpf(times(value(i, c), i, c), 11 - e);
        }
      }
      // (scores of -inf alone would be a row without keys)
      bool inf = false;
#pragma unroll
      for (int i = 0; i < KS; ++i) inf |= qe[i] == 129 - 11;
      if (inf) q[0][0] = (_Float16)__builtin_nanf("");
    };
    if (a.kdhi) {
      const float* d = a.kdhi + a.k_first + h * HD + hf * 8;
      convert([&](float v, int i, int j) __attribute__((always_inline)) { return v * d[i * 16 + j]; });
    } else {
      convert([](float v, int, int) __attribute__((always_inline)) { return v; });
    }
  };
  auto join_q = [&]() __attribute__((always_inline)) {
    int e = -1000;
#pragma unroll
    for (int i = 0; i < KS; ++i) {
      qe[i] += sm_y[0][i / 2];
      e = max(e, qe[i]);
    }
    e = max(e, __shfl_xor(e, 32));
#pragma unroll
    for (int i = 0; i < KS; ++i) {
      const float f = ldexpf(1.f, max(qe[i] - e, -40));
      const unsigned f2 = both(f, f);
      u32x4 v = __builtin_bit_cast(u32x4, q[i]);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = u2(h2(v[j]) * h2(f2));
      q[i] = __builtin_bit_cast(f16x8, v);
    }
    if (a.scale2 != 0.f && e > -500)
      qm = fminf(fmaxf(ldexpf(__builtin_fabsf(a.scale2), e), 1.17549435e-38f), 3.402823466e38f);
  };

  f32x16 s[NKT];
  f16x8 p[PS];
#pragma unroll
  for (int i = 0; i < PS; ++i) p[i] = f16x8{};
  // value j of block t of s is that of key k0 + key_of(t, j)
  auto key_of = [&](int t, int j) __attribute__((always_inline)) { return t * 32 + (j >> 3) * 16 + hf * 8 + (j & 7); };
  // The products of p with the V of tile t - 1, then, but for the last, those of K of
  // tile t with q', and pair t staged between them; operands are read LEAD products
  // ahead.  The order is written out, since the compiler's puts each read before its
  // product and the staging after all.
  auto products = [&](int t, auto score) __attribute__((always_inline)) {
    constexpr int NW = NCT * PS, N = NW + (score ? NKT * KS : 0);
    constexpr int LEAD = 4, NA = HD == 64 ? 2 : 4;
    const _Float16 *vrow[NA], *krow[4];
    // 16 lanes read 4 keys of 16 channels, and each is given a channel of the 4
    const int key = hf * 8 + ((l & 15) >> 2), ch = (l & 16) + (l & 3) * 4;
#pragma unroll
    for (int i = 0; i < NA; ++i)
      vrow[i] = &sm_v[(t + 1) & 1][key * HD + ((i * 4 + (ch >> 3)) ^ v_flip(key)) * 8 + (ch & 4)];
#pragma unroll
    for (int i = 0; i < 4; ++i) krow[i] = &sm_k[t & 1][n * HD + ((2 * i + hf) ^ (n & 7)) * 8];
    auto operand = [&](int at) __attribute__((always_inline)) {
      if (at < NW) {
        const int c = at % NCT, i = at / NCT;
        const _Float16* from = vrow[c % NA] + c / NA * NA * 32 + i * 16 * HD;
        return __builtin_shufflevector(read_columns(from), read_columns(from + 4 * HD), 0, 1, 2, 3, 4, 5, 6, 7);
      }
      const int b = (at - NW) % NKT, i = (at - NW) / NKT;
      return *(const f16x8*)&krow[i & 3][b * 32 * HD + (i >> 2) * 64];
    };
    if (score) ctl = sm_ctl[t % 3];
    f16x8 f[LEAD];
#pragma unroll
    for (int i = 0; i < LEAD; ++i) f[i] = operand(i);
#pragma unroll
    for (int at = 0; at < N; ++at) {
      __builtin_amdgcn_sched_barrier(0);
      if (at < NW) {
        f32x16& x = o[at % NCT];
        x = __builtin_amdgcn_mfma_f32_32x32x16_f16(f[at % LEAD], p[at / NCT], x, 0, 0, 0);
      } else {
        const int i = (at - NW) / NKT;
        f32x16& x = s[(at - NW) % NKT];
        x = __builtin_amdgcn_mfma_f32_32x32x16_f16(f[at % LEAD], q[i], i ? x : f32x16{}, 0, 0, 0);
      }
      if (at + LEAD < N) f[at % LEAD] = operand(at + LEAD);
      if (score && at >= 4 && at % 2 == 0 && at / 2 - 2 < kPieces) stage(t, at / 2 - 2);
    }
  };
  auto softmax = [&](int t, float f, bool marked) __attribute__((always_inline)) {
    const int k0 = t * KT;
    if (__builtin_expect(k0 + KT - 1 > full_hi || k0 < full_lo, 0)) {
      const int top = min(top_key - k0, KT) - 8 * hf, bottom = max(low_key - k0, 0) - 8 * hf;
#pragma unroll
      for (int i = 0; i < NKT; ++i)
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const int key = key_of(i, j) - 8 * hf;  // a constant
          if ((key > top) | (key < bottom)) s[i][j] = -kInf;
        }
    }
    if (__builtin_expect(marked, 0)) {
      const int top = min(top_key - k0, KT), bottom = max(low_key - k0, 0);
#pragma unroll
      for (int i = 0; i < NKT; ++i)
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const int key = key_of(i, j);
          const unsigned bad = (key > top) | (key < bottom) ? 0u : sm_bad[t % 3][key];
          if (bad & kOut) s[i][j] = -kInf;
          nan_groups |= bad;
        }
    }
    float mx = -kInf;
#pragma unroll
    for (int i = 0; i < NKT; ++i)
#pragma unroll
      for (int j = 0; j < 16; ++j) mx = fmaxf(mx, s[i][j]);
    const unsigned ux = __float_as_uint(mx);
    const auto halves = __builtin_amdgcn_permlane32_swap(ux, ux, false, false);
    mx = __builtin_elementwise_maximum(__uint_as_float(halves[0]), __uint_as_float(halves[1]));
    const float top = mx * f;
    if (__ballot(top > mrun + kLazy)) {
      const float mnew = top > mrun + kLazy ? top : mrun;  // (by the row's own keys alone)
      const float g = mrun == -kInf ? 0.f : __builtin_amdgcn_exp2f(mrun - mnew);
#pragma unroll
      for (int i = 0; i < NCT; ++i) o[i] *= g;
      sum *= g;
      mrun = mnew;
    }
    const float low = mrun == -kInf ? 0.f : mrun;
    float base = low - kLift;
    const bool far_row = __builtin_fabsf(low) > kFarScore;
    if (__ballot(far_row)) {  // (k_attention.hip)
#pragma unroll
      for (int i = 0; i < 16 * NKT; ++i) s[i / 16][i % 16] = far_row ? s[i / 16][i % 16] * f - low : s[i / 16][i % 16];
      f = far_row ? 1.f : f;
      base = far_row ? -kLift : base;
    }
#pragma unroll
    for (int i = 0; i < PS; ++i) {
      u32x4 v;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int at = (i & 1) * 8 + 2 * j;
        v[j] = both(__builtin_amdgcn_exp2f(fmaf(s[i >> 1][at], f, -base)),
                    __builtin_amdgcn_exp2f(fmaf(s[i >> 1][at + 1], f, -base)));
        sum = __builtin_amdgcn_fdot2(h2(v[j]), f16x2{(_Float16)1.f, (_Float16)1.f}, sum, false);
      }
      p[i] = __builtin_bit_cast(f16x8, v);
    }
  };
  // The keys that were left out, each as the one tile of its own: all 32 rows of a wave
  // at once, a half of the channels a lane, from its codes.
  auto add_far = [&](int nt) __attribute__((always_inline)) {
    // 8 channels of row `row` from channel ch on, in units of 2^y, those that f names
    auto values = [&](const uint8_t* codes, const float* scales, const float* mins, int64_t row, int64_t ch, int y,
                      auto f, auto& v) __attribute__((always_inline)) {
      const int64_t g = row * a.groups + (ch >> a.gshift);
      float sc = scales[g], m = mins[g];
      finite_or_nan(sc, m);
      const unsigned* from = (const unsigned*)(codes + row * a.row_bytes + ch * CB / 8);
      const unsigned w0 = from[0], w1 = CB == 8 ? from[1] : 0u;
#pragma unroll
      for (int j = 0; j < (int)(sizeof(v) / sizeof(float)); ++j) {
        const int at = f(j);
        const unsigned c = CB == 8 ? (at & 4 ? w1 : w0) >> (at & 3) * 8 & 255u : w0 >> at * 4 & 15u;
        v[j] = ldexpf(F8 ? sc * __builtin_amdgcn_cvt_f32_fp8((int)c, 0) : fmaf(sc, (float)c, m), -y);
      }
      return sc == sc;
    };
    const int64_t k_at = a.k_first + h * HD, v_at = a.v_first + h * HD;
#pragma unroll 1
    for (int t = 0; t < nt; ++t) {
      if ((__builtin_amdgcn_readfirstlane(sm_far[t >> 5 & 31]) >> (t & 31) & 1) == 0) continue;
      const int mine = row_at(t, page_at(t));
      Scales sc = scales_of(mine, mine);
      finite_or_nan(sc.ks, sc.km);
      finite_or_nan(sc.vs, sc.vm);
      const bool left = of_key(__ballot(mine >= 0 && (far(sc.ks, sc.km, YK) || far(sc.vs, sc.vm, YV))));
      __syncthreads();
      if (kch == 0) sm_bad[0][kkey] = left;
      __syncthreads();
#pragma unroll 1
      for (int i = 0; i < KT; ++i) {
        const int key = t * KT + i;
        if (__builtin_amdgcn_readfirstlane(sm_bad[0][i]) == 0) continue;
        const int64_t row = ((int64_t)table[(lo + key) >> a.pshift] << a.pshift) + ((lo + key) & pmask);
        float x = 0.f;
#pragma unroll
        for (int i = 0; i < KS; ++i) {
          float v[8];
          values(a.kc, a.ks, a.km, row, k_at + i * 16 + hf * 8, sm_y[0][i / 2], [](int j) { return slot_code<CB>(j); }, v);
#pragma unroll
          for (int j = 0; j < 8; ++j) x = fmaf((float)q[i][j], v[j], x);
        }
        x = (x + __shfl_xor(x, 32)) * qm;
        const bool seen = key <= top_key && key >= low_key;
        if (!seen) x = -kInf;
        const float mnew = x > mrun + kLazy ? x : mrun;
        const float g = mrun == -kInf ? 0.f : __builtin_amdgcn_exp2f(mrun - mnew);
        const float p = seen ? __builtin_amdgcn_exp2f(x - (mnew == -kInf ? 0.f : mnew) + kLift) : 0.f;
        if (mnew != mrun) {
#pragma unroll
          for (int i = 0; i < NCT; ++i) o[i] *= g;
          sum *= g;
          mrun = mnew;
        }
        if (hf == 0) sum += p;
#pragma unroll
        for (int i = 0; i < HD / 8; ++i) {
          float v[4];
          const bool good = values(a.vc, a.vs, a.vm, row, v_at + i * 8, sm_y[1][i / 4],
                                   [&](int j) { return CB == 4 ? slot_code<CB>(j) + 2 * hf : j + 4 * hf; }, v);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int at = i % 4 * 4 + j;
            if (good && p != 0.f) o[i / 4][at] = fmaf(p, v[j], o[i / 4][at]);
          }
        }
      }
    }
  };

  if (end > 0) {  // uniform over the workgroup
    const int nt = (end + KT - 1) / KT;
    if (tid < 3) sm_ctl[tid] = 0;
    if (tid < 33) sm_far[tid] = 0;
    convert_q();
    for (int i = tid; i < 3 * KT; i += 512) (&sm_bad[0][0])[i] = 0;
    __syncthreads();
    YK = sm_y[0][kch / 32];
    YV = sm_y[1][kch / 32];
    join_q();
    check(-1, r1, -1);
    __syncthreads();
    ctl = sm_ctl[2];
#pragma unroll
    for (int i = 0; i < kPieces; ++i) stage(-1, i);
    __syncthreads();
    // A step of a wave is the products, a barrier, the softmax of tile t, a barrier;
    // the late waves do the one while the others do the other.
    if (late) step_barrier();
    for (int t = 0; t < nt; ++t) {
      __builtin_amdgcn_s_setprio(1);
      products(t, std::true_type{});  // (V of tile -1: zeros)
      __builtin_amdgcn_s_setprio(0);
      if (late && tid - 256 < KT) {   // of pair t - 1, whose slot pair t + 2 takes
        sm_bad[(t + 2) % 3][tid - 256] = 0;
        if (tid == 256) sm_ctl[(t + 2) % 3] = 0;
      }
      step_barrier();
      softmax(t, qm, bad_keys);
      step_barrier();
    }
    products(nt, std::false_type{});
    if (!late) step_barrier();
    if (__builtin_expect(sm_far[32] != 0, 0)) add_far(nt);
  }

  sum += __shfl_xor(sum, 32);
  nan_groups |= __shfl_xor(nan_groups, 32);
  if (w0 + n > last) return;
  asm("" : "+v"(r));  // (not kept in other forms through the loop)
  const int64_t row = (sr.first + r / G) * a.H + h * G + r % G, orow = row * a.nsplit + split;
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
  for (int t = 0; t < NCT; ++t) {
    const int64_t at = a.v_first + h * HD;
    const int y = any ? sm_y[1][t] : 0;
    f32x4 back[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) back[i] = f32x4{1.f, 1.f, 1.f, 1.f};
    if (a.vdhi) {
#pragma unroll
      for (int i = 0; i < 4; ++i) back[i] = *(const f32x4*)(a.vdhi + at + t * 32 + i * 8 + hf * 4);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int ch = t * 32 + i * 8 + hf * 4;
      const bool bad = (nan_groups >> (((at + ch) >> a.gshift) - (at >> a.gshift))) & 1;
      f32x4 x;
#pragma unroll
      for (int j = 0; j < 4; ++j) x[j] = ldexpf(o[t][4 * i + j] * inv, y);
      if constexpr (CB == 4) {  // from slots to codes (slot_code)
        const float y0 = __shfl_xor(hf ? x[0] : x[1], 32), y1 = __shfl_xor(hf ? x[2] : x[3], 32);
        x = hf ? f32x4{y0, y1, x[1], x[3]} : f32x4{x[0], x[2], y0, y1};
      }
      if (bad) x = f32x4{1.f, 1.f, 1.f, 1.f} * __builtin_nanf("");
      x *= back[i];
      if (a.nsplit > 1)
        *(f32x4*)(a.part + orow * HD + ch) = x;
      else
        *(u32x2*)(a.out + row * HD + ch) =
            u32x2{pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3])};
    }
  }
}

}  // namespace

hipError_t launch_attn_tile(const AttnArgs& a, int head_dim, int cb, int qf, const Launch& L) {
  const dim3 grid = attn_grid(a.tiles * a.nsplit * a.KV), blk(512);
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
