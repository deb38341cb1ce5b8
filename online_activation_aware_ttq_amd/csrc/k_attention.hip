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
// fp16 holds q' (times a power of two, its largest value in [2^10, 2^11)), p (times
// 2^kLift) and V's scales (divided by 2^Y): 11 bits each, an eighth of what the bf16 result
// is rounded by; V's offsets are two fp16 values each, which also make up for what a
// scale's 11 bits leave out, in the middle of its codes.  Y is a group's, from the median of
// the first keys that all rows of the block see; a key with a group 2^7 larger or 2^8 smaller
// than that has no V in the products, and its p v is added in float32: so no row depends on
// the size of a key that it does not see, and a seen one costs the others no bits.
//
// It is bound by memory where there is enough of it to ask for: codes and scales go
// to LDS without registers, two or three steps ahead, and all steps of all blocks are
// divided evenly over two workgroups a compute unit.  4 bits, 32 / 8 heads of 128: 64
// requests of up to 8192 keys 100 us (4.6 TB/s), one of 131071 keys in groups of 64 52 us
// (3.2 TB/s; groups of 128: 41), 8 requests 36 us (3.0 TB/s).  11 us of each are the chain
// before the first codes (lengths and their sums, pages, codes) and the join's 4 to 8.
// Groups of 32 are bound by the products per group and their scales (8 requests of 32 heads:
// 79 us where groups of 128 take 35).  A key that is added by itself takes a wave about
// 1.5 us (16 requests of 8192 keys, 32 / 8 heads: 40 us, 53 with one such key in 64).
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

// NB bytes at p, aligned to the smaller of NB and 16
template <int NB>
struct Words {
  unsigned w[NB >= 4 ? NB / 4 : 1];
};
template <int NB>
__device__ __forceinline__ void read_words(Words<NB>& d, const uint8_t* p) {
  if constexpr (NB >= 16) {
    static_assert(NB == 16);
    const u32x4 v = *(const u32x4*)p;
    d.w[0] = v.x; d.w[1] = v.y; d.w[2] = v.z; d.w[3] = v.w;
  } else if constexpr (NB == 8) {
    const u32x2 v = *(const u32x2*)p;
    d.w[0] = v.x; d.w[1] = v.y;
  } else if constexpr (NB == 4) {
    d.w[0] = *(const unsigned*)p;
  } else {
    d.w[0] = *(const uint16_t*)p;
  }
}

template <int N>
__device__ __forceinline__ void wait_vm() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | 0x0F70);
}

// 16 or 4 bytes a lane from each lane's address into LDS, lane after lane
__device__ __forceinline__ void load_lds16(const void* p, void* lds) {
  __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)p,
                                   (__attribute__((address_space(3))) void*)lds, 16, 0, 0);
}
__device__ __forceinline__ void load_lds4(const void* p, void* lds) {
  __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)p,
                                   (__attribute__((address_space(3))) void*)lds, 4, 0, 0);
}

// the maximum over lanes l % 16, l % 16 + 16, .. (NaN, if any is)
__device__ __forceinline__ float max_rows(float x) {
  unsigned u = __float_as_uint(x);
  const auto a = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  x = __builtin_elementwise_maximum(__uint_as_float(a[0]), __uint_as_float(a[1]));
  u = __float_as_uint(x);
  const auto b = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  return __builtin_elementwise_maximum(__uint_as_float(b[0]), __uint_as_float(b[1]));
}

__device__ __forceinline__ unsigned mul_pair(unsigned a, unsigned b) {
  return __builtin_bit_cast(unsigned, __builtin_bit_cast(f16x2, a) * __builtin_bit_cast(f16x2, b));
}
__device__ __forceinline__ unsigned fma_pair(unsigned a, unsigned b, unsigned c) {
  return __builtin_bit_cast(unsigned, __builtin_elementwise_fma(__builtin_bit_cast(f16x2, a), __builtin_bit_cast(f16x2, b),
                                                                __builtin_bit_cast(f16x2, c)));
}

// A block of 16 query rows and the keys that any of them sees
struct Item {
  int64_t seq, r0, lo, hi, pos_lo, pos_hi;
  SeqRows sr;
};
// its steps (a block without keys has one, which writes its rows; 0: no rows)
__device__ __forceinline__ int64_t find_item(const AttnArgs& a, int64_t b, int step, Item& x) {
  if (!find_block<16>(a, b, x.seq, x.sr, x.r0)) return 0;
  x.pos_lo = x.sr.shift + (int)x.r0 / a.G;
  x.pos_hi = x.sr.shift + (int)min(x.r0 + 15, (int64_t)x.sr.rows - 1) / a.G;
  x.lo = a.window > 0 ? max(x.pos_lo - a.window + 1, (int64_t)0) & ~int64_t(31) : 0;
  x.hi = min(x.sr.len, x.pos_hi + 1);
  return max((x.hi - x.lo + step - 1) / step, (int64_t)1);
}
// HD channels a head; GSE = min(group, HD) of them a group; CB-bit codes
template <int HD, int GSE, int CB, bool F8>
struct SplitShape {
  static constexpr int NG = HD / GSE;           // groups of a head
  static constexpr int HB = HD * CB / 8;        // bytes of a head
  static constexpr int NW = HB == 256 ? 2 : 4;  // waves
  static constexpr int NB = HB <= 64 && NG == 1 ? 2 : 1;  // 32 keys of a wave's step
  static constexpr int KS = 32 * NB;            // its keys
  static constexpr int NS = NB * HB <= 64 ? 3 : 2;  // buffers
  static constexpr int CODES = KS * NW * HB;    // bytes of K's (or V's) codes of a step
  static constexpr int SCALES = 4 * KS * NW * NG;  // of one of its four arrays of scales
  static constexpr int STEP = 2 * CODES + 4 * SCALES;
  static constexpr int NPAGE = 1024;            // entries of the page table at hand
  static constexpr int LDS = NS * STEP + 4 * NPAGE;
};

// LH: log2 of the K/V heads of a workgroup, or -1 where it is not known here
template <int HD, int GSE, int CB, bool F8, int LH>
__global__ __launch_bounds__(64 * (HD * CB == 2048 ? 2 : 4), HD * CB == 2048 ? 1 : 2) void k_attn_split(AttnArgs a) {
  using Sh = SplitShape<HD, GSE, CB, F8>;
  constexpr int NG = Sh::NG, HB = Sh::HB, NS = Sh::NS, NW = Sh::NW, NB = Sh::NB, KS = Sh::KS;
  constexpr int KB = GSE * CB / 32;      // bytes of a lane's quarter of a group of K
  constexpr int KP = KB > 16 ? KB / 16 : 1, KW = KB > 16 ? 16 : KB;  // in pieces
  constexpr int NC = HD / 16;            // channels of V of a lane
  constexpr int VB = NC * CB / 8;
  constexpr int U = kUnit<F8>;           // of K's codes
  constexpr float kInf = __builtin_inff();
  constexpr bool kP = NG == 1;           // V's scales go into p, not into V
  // V's codes in products: as stored (E4M3, or 2^24 of what they are); integers that are
  // multiplied by their scales first, as c / 64, so that products are normal fp16 numbers
  constexpr int UV = F8 ? 0 : kP ? 24 : 6;
  // p of a row's largest score is 2^kLift to 2^(kLift + kLazy)
  constexpr float kLazy = 4.f, kLift = 9.f;
  // A group's size, the larger of its scale and 2^(1 - bits) of its values' middle, in
  // units of 2^Y: what products take (with p, or with a code, below 2^16; and normal fp16
  // numbers to 2^-11 of a step, or 2^-20 of the largest p), and 2^kFirst to twice that
  // for the size that Y is from
  constexpr float kMost = kP ? 7.5f : F8 ? 128.f : 4000.f, kLeast = kP ? 0x1p-13f : F8 ? 0x1p-12f : 0x1p-8f;
  constexpr int kFirst = kP ? -5 : F8 ? -2 : 2;
  constexpr int MU = F8 ? 0 : kP ? 26 : 0;  // V's offsets: 2^MU of O's unit
  __shared__ __align__(16) float sm_k[NW][2][NG][KS];
  __shared__ __align__(16) _Float16 sm_s[NW][NG][KS], sm_m[NW][F8 ? 1 : 2 * NG][KS];
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  int* sm_page = (int*)(smem + NS * Sh::STEP);

  const int tid = threadIdx.x, l = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int n = l & 15, c = l >> 4;
  const float rmid = 1.f / (float)a.mid;  // (a power of two)
  unsigned k16v = k16;
  if constexpr (!kP && CB == 4) asm("" : "+v"(k16v));  // (in a register: and and or in one instruction)
  // A workgroup takes HW neighbouring K/V heads; wave w head w % HW and KS of a step's
  // KS * NW / HW keys.  The steps of all blocks, one block after another, are divided
  // evenly over the workgroups of a head group (a.parts of them), so a range may end
  // in one block and go on in the next; or (a.parts = 0) each takes a block.
  const int lh = LH < 0 ? a.hw_shift : LH, HW = 1 << lh, lg = (NW == 4 ? 2 : 1) - lh;
  const int hgroups = a.KV >> lh, step = KS << lg;
  // Workgroup b runs on die b % 8: the head groups of a part go to one die, whose L2
  // then reads the lines that their scales share once (a part's scales of four heads
  // are 16 bytes of a line).
  const int64_t count = a.parts > 0 ? a.parts : a.tiles, even = (count & ~int64_t(7)) * hgroups;
  const unsigned group = attn_group();
  const int64_t in_die = group / 8, rest = group - even;
  const int64_t part = group < even ? in_die / hgroups * 8 + group % 8 : (count & ~int64_t(7)) + rest / hgroups;
  const int h0 = (int)(group < even ? in_die % hgroups : rest % hgroups) << lh;
  const int hh = w & (HW - 1), sub = w >> lh, h = h0 + hh;
  int64_t block, left, skip;  // the first block, the steps to do, those of it to leave out
  if (a.parts > 0) {
    __shared__ int64_t sm_sum[NW], sm_skip;
    __shared__ int sm_first;
    int64_t* pre = (int64_t*)smem;  // where the steps of each block begin
    const int each = (int)((a.tiles + 64 * NW - 1) / (64 * NW)), b0 = tid * each;
    int64_t mine = 0;
    for (int i = b0; i < min((int64_t)(b0 + each), a.tiles); ++i) {
      Item x;
      mine += pre[i + 1] = find_item(a, i, step, x);
    }
    int64_t run = mine;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const int64_t o = __shfl_up((long long)run, off);
      if (l >= off) run += o;
    }
    if (l == 63) sm_sum[w] = run;
    __syncthreads();
    int64_t total = 0;
    run -= mine;
#pragma unroll
    for (int i = 0; i < NW; ++i) {
      run += i < w ? sm_sum[i] : 0;
      total += sm_sum[i];
    }
    total = uniform64(total);
    const int64_t per = (total + a.parts - 1) / a.parts, begin = part * per;
    if (tid == 0 && group == 0) a.pre[0] = 0;
    for (int i = b0; i < min((int64_t)(b0 + each), a.tiles); ++i) {
      const int64_t next = run + pre[i + 1];
      if (run <= begin && begin < next) {
        sm_first = i;
        sm_skip = begin - run;
      }
      if (group == 0) a.pre[i + 1] = next;
      run = next;
    }
    __syncthreads();
    if (begin >= total) return;  // uniform over the workgroup
    block = __builtin_amdgcn_readfirstlane(sm_first);
    skip = uniform64(sm_skip);
    left = min(per, total - begin);
  } else {
    block = part;
    skip = 0;
    left = int64_t(1) << 40;
    if (block >= a.tiles) return;
  }

  for (; left > 0 && block < a.tiles; ++block) {
  Item it;
  const int64_t steps = find_item(a, block, step, it);
  if (steps == 0) {
    if (a.parts == 0) return;  // (uniform; the next block has its own workgroup)
    continue;
  }
  const int64_t todo = min(steps - skip, left);
  const bool all = todo == steps && lg == 0;  // the block's keys are all this wave's
  const int64_t lo = it.lo + skip * step, hi = it.hi;
  const int64_t end = min(lo + todo * step, hi);
  left = a.parts > 0 ? left - todo : 0;
  skip = 0;
  const SeqRows& sr = it.sr;
  const int64_t seq = it.seq, r0 = it.r0, pos_lo = it.pos_lo, pos_hi = it.pos_hi;
  // this lane's row
  const int r = (int)min(r0 + n, (int64_t)sr.rows - 1);
  const int tok = r / a.G, head = h * a.G + r % a.G;
  const int64_t pos = sr.shift + tok;

  // q' of this lane's channels, by group and step, and its sums: the values are asked
  // for here and used once the first codes are
  f16x8 q[HD / 32];
  float qs[NG], qm;
  u32x4 xq[HD / 32];
  f32x4 dq[HD / 16];
  auto q_channel = [&](int i) __attribute__((always_inline)) { return i / (GSE / 32) * GSE + c * (GSE / 4) + i % (GSE / 32) * 8; };
  {
    const bf16_t* src = a.Q + (sr.first + tok) * a.ldq + head * HD;
#pragma unroll
    for (int i = 0; i < HD / 32; ++i) xq[i] = *(const u32x4*)(src + q_channel(i));
#pragma unroll
    for (int i = 0; i < HD / 16; ++i) dq[i] = f32x4{1.f, 1.f, 1.f, 1.f};
    if (a.kdhi) {
      const float* d = a.kdhi + a.k_first + h * HD;
#pragma unroll
      for (int i = 0; i < HD / 16; ++i) dq[i] = *(const f32x4*)(d + q_channel(i / 2) + i % 2 * 4);
    }
  }
  auto make_q = [&]() __attribute__((always_inline)) {
    const float sign = a.scale2 == 0.f ? 0.f : a.scale2 < 0.f ? -1.f : 1.f;
    float qf[HD / 4], top = 0.f;
#pragma unroll
    for (int i = 0; i < HD / 4; ++i) {
      const unsigned x = xq[i / 8][i % 8 / 2];
      qf[i] = (i % 2 ? bf16hi(x) : bf16lo(x)) * sign * dq[i / 4][i % 4];
      top = fmaxf(top, __builtin_fabsf(qf[i]));
    }
    top = max_rows(top);
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
    // (scores of -inf alone would be a row without keys)
    if (!(top <= 3.402823466e38f)) q[0][0] = (_Float16)__builtin_nanf("");
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      qs[g] += __shfl_xor(qs[g], 16);
      qs[g] += __shfl_xor(qs[g], 32);
      qs[g] = ldexpf(qs[g], -U);
    }
    // (to what float32 holds: q of 2^100 and more have scores that nothing is near)
    qm = sign == 0.f ? 1.f : fminf(fmaxf(ldexpf(__builtin_fabsf(a.scale2), e + U), 1.17549435e-38f), 3.402823466e38f);
  };

  f32x4 o[NC], om = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < NC; ++i) o[i] = om;
  float mrun = -kInf;
  int Y[NG];
  bool no_unit = true;
  unsigned nan_groups = 0;

  // LDS of a step: rows of HW heads' codes, K's then V's, key r of 32 in place (r & 7)
  // * 4 + r / 8, its 16-byte pieces p in slots p ^ fold(r): the reads below find all
  // banks; then the scales and offsets of K and V, as they lie in the cache.
  const int RB = HB << lh, pieces = RB / 16, lrb = __builtin_ctz((unsigned)RB);
  auto fold = [&](int r) __attribute__((always_inline)) { return ((r & 3) | (((r >> 3) >> lg) << 2)) & (pieces - 1); };
  const int32_t* table = a.pages + seq * a.max_pages;
  const int pmask = (1 << a.pshift) - 1, max_page = (a.n_slots - 1) >> a.pshift;
  int64_t e0 = 0;  // the first key of the first page at hand
  // page of a key (-1 behind the last one), and its cache row; where it has none,
  // row 0, which is there to be read
  auto page_of = [&](int64_t key) __attribute__((always_inline)) {
    const int page = sm_page[min((unsigned)(int)(key - e0) >> a.pshift, (unsigned)Sh::NPAGE - 1)];
    return key < end ? page : -1;
  };
  auto row_of = [&](int64_t key, int page, bool& in) __attribute__((always_inline)) {
    const unsigned row = ((unsigned)page << a.pshift) + ((int)(key - e0) & pmask);
    in = (unsigned)page <= (unsigned)max_page && row < (unsigned)a.n_slots;
    return in ? row : 0u;
  };
  const uint8_t* kbase = a.kc + (a.k_first + h0 * HD) * CB / 8;
  const uint8_t* vbase = a.vc + (a.v_first + h0 * HD) * CB / 8;
  // this wave's part of a step: 1 KiB of codes an instruction, and 4 / NW of the
  // arrays of scales, 64 values an instruction or, where a key's values are whole 16
  // bytes (a.wide), four times as many: a load of 4 bytes a lane takes the address
  // units as long (64 requests: groups of 64 142 us so, 133 with 16 bytes; of 32 297 and
  // 263; context 131071, groups of 64: 55 either way)
  constexpr int NQ = KS * HB / 1024, NI = KS * NW * NG / 64, NA = 4 / NW;
  constexpr int PER = 2 * NQ + NA * NI, NIW = (NI + 3) / 4, PERW = 2 * NQ + NA * NIW;
  const int lsg = lh + __builtin_ctz((unsigned)NG);  // log2 of a key's scales
  const bool wide = NI % 4 == 0 && a.wide;
  const int lw = wide ? 2 : 0, hg = (l << lw) & ((1 << lsg) - 1);
  const float* sbase[NA];
#pragma unroll
  for (int j = 0; j < NA; ++j) {
    const int x = w * NA + j;
    const int64_t first = x < 2 ? a.k_first : a.v_first;
    sbase[j] = (x == 0 ? a.ks : x == 1 ? a.km : x == 2 ? a.vs : a.vm) +
               ((first + (h0 + hg / NG) * HD) >> a.gshift) + hg % NG;
  }
  auto issue = [&](int64_t k0, int buf) __attribute__((always_inline)) {
    uint8_t* to = smem + buf * Sh::STEP;
    int pq[NQ], ps[NI];
    auto code_key = [&](int i, int& piece) __attribute__((always_inline)) {
      const int at = (w * NQ + i) * 1024 + l * 16, p = at >> lrb;
      const int r = ((p & 31) >> 2) | ((p & 3) << 3);
      piece = ((at >> 4) & (pieces - 1)) ^ fold(r);
      return k0 + (p & ~31) + r;
    };
    auto scale_key = [&](int i) __attribute__((always_inline)) { return k0 + (((i * 64 + l) << lw) >> lsg); };
    int piece;
#pragma unroll
    for (int i = 0; i < NQ; ++i) pq[i] = page_of(code_key(i, piece));
#pragma unroll
    for (int i = 0; i < NIW; ++i) ps[i] = page_of(scale_key(i));
    bool in;
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
      const int64_t key = code_key(i, piece);
      const uint64_t off = (uint64_t)row_of(key, pq[i], in) * (unsigned)a.row_bytes + piece * 16;
      load_lds16(kbase + off, to + (w * NQ + i) * 1024);
      load_lds16(vbase + off, to + Sh::CODES + (w * NQ + i) * 1024);
    }
    uint8_t* sto = to + 2 * Sh::CODES + w * NA * Sh::SCALES;
    if (wide) {
#pragma unroll
      for (int i = 0; i < NIW; ++i) {
        const uint64_t off = (uint64_t)row_of(scale_key(i), ps[i], in) * (unsigned)a.groups;
#pragma unroll
        for (int j = 0; j < NA; ++j) load_lds16(sbase[j] + off, sto + j * Sh::SCALES + i * 1024);
      }
    } else {
#pragma unroll
      for (int i = NIW; i < NI; ++i) ps[i] = page_of(scale_key(i));
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const uint64_t off = (uint64_t)row_of(scale_key(i), ps[i], in) * (unsigned)a.groups;
#pragma unroll
        for (int j = 0; j < NA; ++j) load_lds4(sbase[j] + off, sto + j * Sh::SCALES + i * 256);
      }
    }
  };
  // where this lane's operands lie in a step
  const int kat = ((sub * KS + (n & 3) * 4 + (n >> 2)) << lrb), kf = fold((n >> 2) * 8 + (n & 3));
  const int vat = ((sub * KS + c) << lrb), vf = fold(c * 8);
  const int kl = l & (KS - 1), sat = ((sub * KS + kl) << lsg) + hh * NG;

  auto rescale = [&](float f) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < NC; ++i) o[i] *= f;
    om *= f;
  };
  // (NaN or infinite if s or m is)
  auto size_of = [&](float s, float m) __attribute__((always_inline)) {
    return F8 ? fmaf(m, 0.f, __builtin_fabsf(s))
              : __builtin_elementwise_maximum(__builtin_fabsf(s), __builtin_fabsf(fmaf(m, rmid, s)));
  };
  // 2^y kLeast to 2^y kMost: as bits of floats
  auto fits = [&](float s, float m, int y) __attribute__((always_inline)) {
    const unsigned least = __float_as_uint(kLeast), most = __float_as_uint(kMost);
    return __float_as_uint(size_of(s, m)) - (least + ((unsigned)y << 23)) <= most - least;
  };

  // The pages of as many keys as the table takes, and the first steps of them
  const int64_t epoch = ((int64_t)(Sh::NPAGE - 1) << a.pshift) / step * step;
  auto open = [&](int64_t from) __attribute__((always_inline)) {
    const int64_t to = min(from + epoch, end);
    __syncthreads();  // the pages and buffers before have been read
    e0 = from >> a.pshift << a.pshift;
    for (int i = tid; i <= (int)((to - 1 - e0) >> a.pshift); i += 64 * NW) sm_page[i] = table[(e0 >> a.pshift) + i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NS - 1; ++i)
      if (from + i * step < to) issue(from + i * step, i);
  };
  if (lo < end) {
    open(lo);
    make_q();
  }
  for (int64_t from = lo; from < end; from += epoch) {
  const int64_t to = min(from + epoch, end);
  if (from > lo) open(from);
  int buf = 0;
  for (int64_t k1 = from; k1 < to; k1 += step, buf = buf + 1 == NS ? 0 : buf + 1) {
    // this step's part of each wave is there, then all of it; the buffer that is
    // filled next has been read
    if (NS == 2 || k1 + step >= to) wait_vm<0>();
    else if (wide) wait_vm<PERW>();
    else wait_vm<PER>();
    lds_barrier();
    if (k1 + (NS - 1) * step < to) issue(k1 + (NS - 1) * step, buf == 0 ? NS - 1 : buf - 1);
    const uint8_t* codes = smem + buf * Sh::STEP;
    const int64_t k0 = k1 + sub * KS;
    // scales and offsets of key kl, to where the lanes that need them find them
    bool now, usual = true, bad = false;
    (void)row_of(k0 + kl, page_of(k0 + kl), now);
    float vs[NG], vm[NG];
    {
      const float* p = (const float*)(codes + 2 * Sh::CODES) + sat;
      float ks[NG], km[NG];
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        ks[g] = p[g];
        if (!F8) km[g] = p[Sh::SCALES / 4 + g];
        vs[g] = p[2 * (Sh::SCALES / 4) + g];
        vm[g] = p[3 * (Sh::SCALES / 4) + g];
      }
      wave_sync();
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        if (F8) km[g] = 0.f;
        finite_or_nan(ks[g], km[g]);
        sm_k[w][0][g][kl] = now ? ks[g] : 0.f;
        if (!F8) sm_k[w][1][g][kl] = now ? km[g] : 0.f;
      }
    }
    const uint64_t seen = __ballot(now);
    if (__builtin_expect(no_unit, 0)) {
      // The first keys there are: of each group the median of their sizes, of keys that
      // all rows see if there are some
      const int64_t key = k0 + kl;
      const uint64_t common = __ballot(now && key <= pos_lo && (a.window == 0 || key > pos_hi - a.window));
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        const float x = size_of(vs[g], vm[g]);
        const uint64_t sized = __ballot(now && x > 0.f && x <= 3.402823466e38f);
        const uint64_t of = sized & common ? sized & common : sized;
        const int e = __builtin_amdgcn_frexp_expf(x) - 1;
        int y = -256;
#pragma unroll
        for (int bit = 256; bit > 0; bit >>= 1) {
          if (2 * __builtin_popcountll(__ballot(e >= y + bit) & of) > __builtin_popcountll(of)) y += bit;
        }
        Y[g] = of ? min(max(y - kFirst, -100), 100) : -kFirst;
        no_unit &= of == 0;
      }
    }
#pragma unroll
    for (int g = 0; g < NG; ++g) usual &= fits(vs[g], vm[g], Y[g]);
    // keys whose V is not in the products
    uint64_t far = 0;
    if (__ballot(!usual)) {
      bool other = false;
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        finite_or_nan(vs[g], vm[g]);
        if (!now) vs[g] = vm[g] = 0.f;
        bad |= vs[g] != vs[g];
        other |= size_of(vs[g], vm[g]) > 0.f && !fits(vs[g], vm[g], Y[g]);
      }
      far = __ballot(other);
      if (KS == 32) far &= 0xffffffffu;
#pragma unroll
      for (int g = 0; g < NG; ++g)
        if (other && vs[g] == vs[g]) vs[g] = vm[g] = 0.f;
    }
    const bool any_bad = __ballot(bad) != 0;
    uint64_t bad_keys[NG];
    if (any_bad) {
#pragma unroll
      for (int g = 0; g < NG; ++g) bad_keys[g] = __ballot(vs[g] != vs[g]);
    }
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      // V's scale in 11 bits; what it is off is made up for in the middle of the codes
      // by the offset, which is a sum of two fp16 values
      const bool x = vs[g] != vs[g];
      const float sv = x ? 0.f : ldexpf(vs[g], -Y[g]);
      const _Float16 s16 = (_Float16)sv;
      sm_s[w][g][kl] = s16;
      if constexpr (!F8) {
        const float mv = x ? 0.f : fmaf(sv - (float)s16, ldexpf((float)a.mid, MU - UV), ldexpf(vm[g], MU - UV - Y[g]));
        const _Float16 m16 = (_Float16)mv;
        sm_m[w][g][kl] = m16;
        sm_m[w][NG + g][kl] = (_Float16)(mv - (float)m16);
      }
    }
    wave_sync();

    float t[NB][8];
#pragma unroll
    for (int g = 0; g < NG; ++g) {
#pragma unroll
      for (int u = 0; u < NB; ++u) {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          f32x4 acc = {0.f, 0.f, 0.f, 0.f};
          unsigned kx[KB / 4];
#pragma unroll
          for (int i = 0; i < KP; ++i) {
            const int off = hh * HB + g * (GSE * CB / 8) + c * KB + i * 16;
            Words<KW> x;
            read_words<KW>(x, codes + kat + (32 * u + 16 * half << lrb) + (((off >> 4) ^ kf) << 4) + (off & 15));
#pragma unroll
            for (int j = 0; j < KW / 4; ++j) kx[4 * i + j] = x.w[j];
          }
#pragma unroll
          for (int s = 0; s < GSE / 32; ++s) {
            const f16x8 k = CB == 8 ? codes8<CB, F8>(kx[CB == 8 ? 2 * s : 0], kx[CB == 8 ? 2 * s + 1 : 0])
                                    : codes8<CB, F8>(kx[s], 0u);
            acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(k, q[g * (GSE / 32) + s], acc, 0, 0, 0);
          }
          const f32x4 s4 = *(const f32x4*)&sm_k[w][0][g][u * 32 + c * 8 + half * 4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            t[u][half * 4 + i] = g == 0 ? s4[i] * acc[i] : fmaf(s4[i], acc[i], t[u][half * 4 + i]);
          if constexpr (!F8) {
            const f32x4 m4 = *(const f32x4*)&sm_k[w][1][g][u * 32 + c * 8 + half * 4];
#pragma unroll
            for (int i = 0; i < 4; ++i) t[u][half * 4 + i] = fmaf(m4[i], qs[g], t[u][half * 4 + i]);
          }
        }
      }
    }
    // where not all rows see all keys: bit j of mask, this lane's row sees its key j
    unsigned mask[NB];
#pragma unroll
    for (int u = 0; u < NB; ++u) mask[u] = 0xffu;
    if (seen != ~uint64_t(0) || k0 + KS - 1 > pos_lo || (a.window > 0 && k0 <= pos_hi - a.window)) {
      const int top = (int)max(min(pos - k0, (int64_t)64), (int64_t)-1);
      const int bottom = a.window > 0 ? (int)max(min(pos - a.window - k0, (int64_t)64), (int64_t)-1) : -1;
#pragma unroll
      for (int u = 0; u < NB; ++u) {
        mask[u] = (unsigned)(seen >> (u * 32 + c * 8)) & 0xffu;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int key = u * 32 + c * 8 + i;
          if (key > top || key <= bottom) mask[u] &= ~(1u << i);
          if (!((mask[u] >> i) & 1)) t[u][i] = -kInf;
        }
      }
    }
    auto mx2 = [](float x, float y) { return __builtin_elementwise_maximum(x, y); };
    float mx = t[0][0];
#pragma unroll
    for (int i = 1; i < 8 * NB; ++i) mx = mx2(mx, t[i / 8][i % 8]);
    mx = max_rows(mx) * qm;
    if (__ballot(mx > mrun + kLazy)) {
      const float mnew = mx > mrun + kLazy ? mx : mrun;  // (by the row's own keys alone)
      rescale(mrun == -kInf ? 0.f : __builtin_amdgcn_exp2f(mrun - mnew));
      mrun = mnew;
    }
    // t qm - mrun, rounded once; where mrun is so far from 0 that its own rounding would
    // be a power of two in p, the product is rounded as it was for mrun
    const float low = mrun == -kInf ? 0.f : mrun;
    float base = kLift - low, factor = qm;
    const bool far_row = __builtin_fabsf(low) > kFarScore;
    if (__ballot(far_row)) {
#pragma unroll
      for (int i = 0; i < 8 * NB; ++i) t[i / 8][i % 8] = far_row ? t[i / 8][i % 8] * qm - low : t[i / 8][i % 8];
      base = far_row ? kLift : base;
      factor = far_row ? 1.f : qm;
    }
    if (any_bad) {  // a scale of V that is NaN: its group, in the rows that see it
#pragma unroll
      for (int g = 0; g < NG; ++g)
#pragma unroll
        for (int u = 0; u < NB; ++u)
          if (mask[u] & (unsigned)(bad_keys[g] >> (u * 32 + c * 8)) & 0xffu) nan_groups |= 1u << g;
    }
#pragma unroll
    for (int u = 0; u < NB; ++u) {
      f16x8 p;
#pragma unroll
      for (int i = 0; i < 8; ++i) p[i] = (_Float16)__builtin_amdgcn_exp2f(fmaf(t[u][i], factor, base));
      // V's operands, their scales (of this lane's channels: one group) in p or in V
      const u32x4 sv = *(const u32x4*)&sm_s[w][n * NC / GSE][u * 32 + c * 8];
      Words<VB> vw[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int off = hh * HB + n * VB;
        read_words<VB>(vw[j], codes + Sh::CODES + vat + (32 * u + 4 * j << lrb) +
                                  (((off >> 4) ^ vf ^ (j & 3 & (pieces - 1))) << 4) + (off & 15));
      }
      if (F8 && seen != ~uint64_t(0)) {
        // (E4M3 has NaN, and the row read for a key that is not there may hold it)
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
          for (int i = 0; i < (VB >= 4 ? VB / 4 : 1); ++i)
            if (!((seen >> (u * 32 + c * 8 + j)) & 1)) vw[j].w[i] = 0u;
      }
      // p v of keys that are not in the products, from their codes
      for (unsigned keys = (unsigned)(far >> (u * 32)); keys; keys &= keys - 1) {
        const int j = __builtin_ctz(keys);
        float pj = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) pj = i == (j & 7) ? (float)p[i] : pj;
        pj = __shfl(pj, n + (j >> 3) * 16);
        const float* sj = (const float*)(codes + 2 * Sh::CODES + 2 * Sh::SCALES) + ((sub * KS + u * 32 + j) << lsg) + hh * NG;
        const uint8_t* from = codes + Sh::CODES + ((sub * KS + u * 32 + (j & 7) * 4 + (j >> 3)) << lrb);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int ch = (c * 4 + i) * NC, off = hh * HB + ch * CB / 8, g = ch / GSE;
          float sc = sj[g], m = sj[Sh::SCALES / 4 + g];
          finite_or_nan(sc, m);
          int y = Y[0];
#pragma unroll
          for (int k = 1; k < NG; ++k) y = g == k ? Y[k] : y;
          Words<VB> x;
          read_words<VB>(x, from + (((off >> 4) ^ fold(j)) << 4) + (off & 15));
#pragma unroll
          for (int k = 0; k < NC; ++k) {
            const unsigned code = x.w[k * CB / 32] >> (k * CB % 32) & ((1u << CB) - 1);
            const float v = F8 ? sc * __builtin_amdgcn_cvt_f32_fp8((int)code, 0) : fmaf(sc, (float)code, m);
            const float add = ldexpf(v, (CB == 4 && (k & 1) ? 4 : 0) - y - UV);
            if (pj != 0.f && sc == sc) o[k][i] = fmaf(pj, add, o[k][i]);
          }
        }
      }
      f16x8 ps = p;
      if constexpr (kP) ps = p * __builtin_bit_cast(f16x8, sv);
      // s (16 + c / 64) - 16 s, rounded once (E4M3: s c)
      constexpr bool kNormal = !kP && !F8;
      u32x4 s16 = {0u, 0u, 0u, 0u};
      if constexpr (kNormal) {
#pragma unroll
        for (int j = 0; j < 4; ++j) s16[j] = mul_pair(sv[j], 0xcc00cc00u);
      }
      auto times_scale = [&](unsigned v, int j) __attribute__((always_inline)) {
        return kNormal ? fma_pair(v, sv[j], s16[j]) : mul_pair(v, sv[j]);
      };
#pragma unroll
      for (int i = 0; i < NC / 4; ++i) {
        unsigned vp[4][4];
#pragma unroll
        for (int j = 0; j < 4; ++j) key_pairs<CB, F8>(vw[2 * j].w, vw[2 * j + 1].w, i, kNormal ? k16v : 0u, vp[j]);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const u32x4 v = kP ? u32x4{vp[0][k], vp[1][k], vp[2][k], vp[3][k]}
                             : u32x4{times_scale(vp[0][k], 0), times_scale(vp[1][k], 1),
                                     times_scale(vp[2][k], 2), times_scale(vp[3][k], 3)};
          o[4 * i + k] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, v), ps, o[4 * i + k], 0, 0, 0);
        }
      }
      // rows 0 .. NG - 1 of this product: V's offsets; 15: ones
      u32x4 mv = {0x3c003c00u, 0x3c003c00u, 0x3c003c00u, 0x3c003c00u};
      if (n < 15) mv = u32x4{0u, 0u, 0u, 0u};
      if (!F8 && n < NG) mv = *(const u32x4*)&sm_m[w][n][u * 32 + c * 8];
      om = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, mv), p, om, 0, 0, 0);
      if constexpr (!F8) {
        u32x4 ml = {0u, 0u, 0u, 0u};
        if (n < NG) ml = *(const u32x4*)&sm_m[w][NG + n][u * 32 + c * 8];
        om = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, ml), p, om, 0, 0, 0);
      }
    }
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
  if (r0 + n >= sr.rows) continue;  // (no shuffles below)
  // a block that several waves share: row n of slot (part + block, sub), which no
  // other has, since a workgroup goes from block to block and from part to part
  const int64_t slot = ((a.parts > 0 ? part : 0) + block << lg) + sub;
  const int64_t orow = ((int64_t)h * a.slots + slot) * a.slot_rows + n;
  const bool any = sum > 0.f || sum != sum;
  if (!all) {
    if (c == 0) {
      a.ml[2 * orow] = mrun;
      a.ml[2 * orow + 1] = sum;
    }
    if (!any) continue;
  }
  f32x4 dv[NC];
#pragma unroll
  for (int i = 0; i < NC; ++i) dv[i] = f32x4{1.f, 1.f, 1.f, 1.f};
  if (a.vdhi) {
    const float* d = a.vdhi + a.v_first + h * HD + c * (HD / 4);
#pragma unroll
    for (int i = 0; i < NC; ++i) dv[i] = *(const f32x4*)(d + 4 * i);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float x[NC];
    const int ch = c * (HD / 4) + i * NC;
    float f = 0.f;
    int y = 0;
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      f = ch / GSE == g ? off[g] : f;
      y = any && ch / GSE == g ? Y[g] : y;
    }
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      const float v = o[j][i] * (CB == 4 && (j & 1) ? 0.0625f : 1.f);
      x[j] = ldexpf((v + ldexpf(f, -MU)) * inv, y + UV) * dv[(i * NC + j) / 4][j % 4];
    }
    if (!all) {
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
}

// One workgroup joins the parts of a row: out = sum_s w_s l_s o_s / sum_s w_s l_s,
// w_s = exp(m_s - max m), o_s the mean of part s.  The weights first, all at once, and
// divided by their sum (o_s may be as large as float32 goes); then HD / 4 lanes a part,
// NT / (HD / 4) parts side by side.
template <int HD, int NT>
__global__ __launch_bounds__(NT) void k_attn_join(AttnArgs a) {
  constexpr int LN = HD / 4, SB = NT / LN;
  __shared__ float sm_w[kAttnMaxParts], sm_red[2][NT / 64];
  __shared__ __align__(16) float sm[SB][HD];
  const int tid = threadIdx.x, l = tid & 63, w = tid >> 6;
  const int64_t row = attn_group(), t = row / a.H;
  if (t >= a.T) return;
  if (a.offsets && (t >= a.offsets[a.n_seq] || t < a.offsets[0])) return;  // uniform
  // its parts: rows base + s stride
  int64_t base = row * a.nsplit, stride = 1;
  int count = a.nsplit;
  if (a.slots > 0) {
    const int h = (int)(row % a.H) / a.G, g = (int)(row % a.H) % a.G;
    int64_t tile, n;
    if (a.offsets) {
      int64_t lo = 0, hi = a.n_seq;
      while (hi - lo > 1) {
        const int64_t mid = (lo + hi) >> 1;
        if (a.offsets[mid] <= t) lo = mid;
        else hi = mid;
      }
      const int64_t first = max(a.offsets[lo], 0), r = (t - first) * a.G + g;
      tile = first * a.G / 16 + lo + r / 16;
      n = r % 16;
    } else {
      tile = t * ((a.G + 15) / 16) + g / 16;
      n = g % 16;
    }
    if (tile >= a.tiles) return;
    int64_t from = 0, to = 0;
    if (a.parts > 0) {
      const int64_t per = (a.pre[a.tiles] + a.parts - 1) / a.parts;
      if (a.pre[tile + 1] == a.pre[tile]) return;
      from = a.pre[tile] / per;
      to = (a.pre[tile + 1] - 1) / per;
    }
    if (from == to && a.lg == 0) return;  // one wave had all of it and wrote it
    base = ((int64_t)h * a.slots + ((from + tile) << a.lg)) * a.slot_rows + n;
    stride = a.slot_rows;
    count = (int)((to - from + 1) << a.lg);
  }
  const float* ml = a.ml + base * 2;
  float mx = -__builtin_inff();
  for (int s = tid; s < count; s += NT) mx = fmaxf(mx, ml[2 * s * stride]);
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) mx = fmaxf(mx, __shfl_xor(mx, off));
  if (l == 0) sm_red[0][w] = mx;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < NT / 64; ++i) mx = fmaxf(mx, sm_red[0][i]);
  float total = 0.f;
  for (int s = tid; s < count; s += NT) {
    // (a part without keys has no sum and has written no row)
    const float sum = ml[2 * s * stride + 1];
    const float f = sum > 0.f || sum != sum ? __builtin_amdgcn_exp2f(ml[2 * s * stride] - mx) * sum : 0.f;
    sm_w[s] = f;
    total += f;
  }
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) total += __shfl_xor(total, off);
  if (l == 0) sm_red[1][w] = total;
  __syncthreads();
  total = 0.f;
#pragma unroll
  for (int i = 0; i < NT / 64; ++i) total += sm_red[1][i];
  const float inv = total == 0.f ? 0.f : 1.f / total;
  const int c = tid % LN * 4, s0 = tid / LN;
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
  const float* p = a.part + base * HD + c;
#pragma unroll 4
  for (int s = s0; s < count; s += SB) {
    const float g = sm_w[s] * inv;
    if (g == 0.f) continue;
    const f32x4 v = *(const f32x4*)(p + s * stride * HD);
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
    *(unsigned*)(a.out + row * HD + 2 * tid) = pack_bf16(x[0], x[1]);
  }
}

// The same where all rows have the same few parts beside each other (kMerge at most): 4
// channels a thread.  Weights are divided by a power of two that keeps their sum below 1
// until it is known.
constexpr int kMerge = 16;
template <int HD>
__global__ __launch_bounds__(256) void k_attn_merge(AttnArgs a) {
  constexpr int LN = HD / 4;
  const int64_t row = (int64_t)blockIdx.x * (256 / LN) + threadIdx.x / LN, t = row / a.H;
  const int c = threadIdx.x % LN * 4;
  if (row >= a.T * a.H) return;
  if (a.offsets && (t >= a.offsets[a.n_seq] || t < a.offsets[0])) return;
  const float* ml = a.ml + row * a.nsplit * 2;
  const float* p = a.part + row * a.nsplit * HD + c;
  float mx = -__builtin_inff(), most = 0.f;
  for (int s = 0; s < a.nsplit; ++s) {
    mx = fmaxf(mx, ml[2 * s]);
    most = fmaxf(most, ml[2 * s + 1]);
  }
  const float unit = ldexpf(1.f, -4 - __builtin_amdgcn_frexp_expf(most));
  float total = 0.f;
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int s = 0; s < a.nsplit; ++s) {
    const float sum = ml[2 * s + 1];
    const float f = sum > 0.f || sum != sum ? __builtin_amdgcn_exp2f(ml[2 * s] - mx) * (sum * unit) : 0.f;
    if (f == 0.f) continue;  // (a part without keys has written no row)
    total += f;
    const f32x4 v = *(const f32x4*)(p + s * HD);
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[j] = fmaf(f, v[j], acc[j]);
  }
  const float inv = total == 0.f ? 0.f : 1.f / total;
  *(u32x2*)(a.out + row * HD + c) = u32x2{pack_bf16(acc[0] * inv, acc[1] * inv), pack_bf16(acc[2] * inv, acc[3] * inv)};
}

template <int HD, int GSE, int CB, bool F8, int LH>
hipError_t go_split(const AttnArgs& a, const Launch& L) {
  using Sh = SplitShape<HD, GSE, CB, F8>;
  static hipError_t attr = hipFuncSetAttribute(
      reinterpret_cast<const void*>(k_attn_split<HD, GSE, CB, F8, LH>),
      hipFuncAttributeMaxDynamicSharedMemorySize, Sh::LDS);
  if (attr != hipSuccess) return attr;
  const int64_t groups = (a.parts > 0 ? a.parts : a.tiles) * (a.KV >> a.hw_shift);
  return ext_launch(k_attn_split<HD, GSE, CB, F8, LH>, attn_grid(groups), dim3(64 * Sh::NW),
                    Sh::LDS, L, a);
}

template <int HD, int GSE, int CB, bool F8>
hipError_t go_split(const AttnArgs& a, const Launch& L) {
  // (as many heads as waves: offsets in LDS are constants)
  constexpr int LW = SplitShape<HD, GSE, CB, F8>::NW == 4 ? 2 : 1;
  return a.hw_shift == LW ? go_split<HD, GSE, CB, F8, LW>(a, L) : go_split<HD, GSE, CB, F8, -1>(a, L);
}

}  // namespace

hipError_t launch_attn_split(const AttnArgs& a, int head_dim, int cb, int qf, int group,
                             const Launch& L) {
  const int gse = std::min(group, head_dim);
#define TTQ_AS(HDV, GSV)                                              \
  if (head_dim == HDV && gse == GSV) {                                \
    if (qf == QF_FP8) return go_split<HDV, GSV, 8, true>(a, L);       \
    if (cb == 8) return go_split<HDV, GSV, 8, false>(a, L);           \
    return go_split<HDV, GSV, 4, false>(a, L);                        \
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
  const int64_t rows = a.T * a.H;
  const dim3 grid = attn_grid(rows);
  const bool merge = a.slots == 0 && a.nsplit <= kMerge;
  // many parts of a row: more of them side by side
  const bool wide = a.parts > 64 * a.tiles;
#define TTQ_AJ(HDV)                                                                        \
  if (head_dim == HDV) {                                                                   \
    if (merge)                                                                             \
      return ext_launch(k_attn_merge<HDV>, dim3((unsigned)((rows * HDV + 1023) / 1024)),   \
                        dim3(256), 0, L, a);                                               \
    return wide ? ext_launch(k_attn_join<HDV, 1024>, grid, dim3(1024), 0, L, a)            \
                : ext_launch(k_attn_join<HDV, 256>, grid, dim3(256), 0, L, a);             \
  }
  TTQ_AJ(64)
  TTQ_AJ(128)
  TTQ_AJ(256)
#undef TTQ_AJ
  return hipErrorInvalidValue;
}

}  // namespace ttq
