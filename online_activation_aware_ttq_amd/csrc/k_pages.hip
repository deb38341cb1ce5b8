// Page tables and slot maps of a step, from its request lengths: which pages the
// sequences give back and take, and the position and cache row of each of the
// step's rows.
//
// With L_i rows held, a_i added and p rows a page, sequence i needs
//   need_i = ceil((L_i + a_i) / p) - ceil(L_i / p)
// pages; page k of the call is that of the sequence whose range of the running
// sum of need holds k, and comes from place top - 1 - k of the stack.  Row t
// belongs to the sequence whose range of the running sum of a holds it.  So
// everything but two running sums is independent: one workgroup takes the
// sequences a chunk at a time (a chunk is as many as it has threads) and keeps the
// sums between chunks; pages and rows are dealt to its threads by the index k or
// t and find their sequence by bisection in LDS.
//
// It is bound by latency, a chain of dependent loads, two running sums and the
// barriers between them: 8 sequences 5.4 us.  100 prompts of 65536 rows together take 10.9:
// one chunk too, but a thread deals out several pages, one after another, each a bisection
// and two accesses that wait for each other; and 4.3 for the second launch that deals more
// than 4096 rows to the whole chip.
#include <algorithm>

#include "ttq_internal.h"

namespace ttq {

namespace {

// inclusive running sum over the workgroup's threads; `total`: of all of them
template <int NT>
__device__ __forceinline__ int64_t block_sum(int64_t v, int64_t& total, int64_t* part) {
  const int l = threadIdx.x & 63, w = threadIdx.x >> 6;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int64_t o = __shfl_up((long long)v, off);
    if (l >= off) v += o;
  }
  if constexpr (NT == 64) {
    total = __shfl((long long)v, 63);
    return v;
  }
  __syncthreads();  // (part may still be read)
  if (l == 63) part[w] = v;
  __syncthreads();
  int64_t before = 0;
  total = 0;
#pragma unroll
  for (int i = 0; i < NT / 64; ++i) {
    before += i < w ? part[i] : 0;
    total += part[i];
  }
  return v + before;
}

// the last of n (a power of two) ascending values that is at most v; the first is
template <int N>
__device__ __forceinline__ int find(const int* at, int v) {
  int j = 0;
#pragma unroll
  for (int step = N / 2; step > 0; step >>= 1)
    if (at[j + step] <= v) j += step;
  return j;
}

constexpr int kNone = 0x7fffffff;

__device__ __forceinline__ int clip(int64_t v) { return (int)min(v, (int64_t)kNone); }

template <int NT>
__global__ __launch_bounds__(NT) void k_extend(ExtendArgs a) {
  __shared__ int64_t part[NT / 64];
  __shared__ int s_start[NT], s_len[NT], s_held[NT];
  __shared__ bool s_refused[NT];
  __shared__ int s_taken;
  const int tid = threadIdx.x;
  const int64_t pmask = (int64_t(1) << a.pshift) - 1;
  const int64_t c0 = min((int64_t)max(*a.free_count, 0), a.n_pages);
  auto length = [](int n) { return n < 0 ? -1 - n : n; };
  auto held_of = [&](int n) __attribute__((always_inline)) { return min((n + pmask) >> a.pshift, a.max_pages); };

  // the pages of sequences that have ended, onto the stack
  int64_t released = 0;
  for (int64_t base = 0; base < a.n_seq; base += NT) {
    const int64_t i = base + tid;
    const bool live = i < a.n_seq;
    const bool ended = live && a.added[i] < 0;
    if (!__syncthreads_or(ended)) continue;  // (also: s_start has been read)
    const int64_t gone = ended ? held_of(length(a.lens[i])) : 0;
    int64_t total;
    const int64_t sum = block_sum<NT>(gone, total, part);
    s_start[tid] = live ? clip(sum - gone) : kNone;
    __syncthreads();
    const int n = (int)min(total, a.n_pages - min(c0 + released, a.n_pages));
    for (int k = tid; k < n; k += NT) {
      const int j = find<NT>(s_start, k);
      a.free_pages[c0 + released + k] = a.pages[(base + j) * a.max_pages + k - s_start[j]];
    }
    released += total;
  }
  const int64_t top = min(c0 + released, a.n_pages);
  if (tid == 0) {
    a.offsets[0] = 0;
    s_taken = 0;
  }
  __syncthreads();

  int64_t rows0 = 0, need0 = 0;
  for (int64_t base = 0; base < a.n_seq; base += NT) {
    const int64_t i = base + tid;
    const bool live = i < a.n_seq;
    const int add = live ? a.added[i] : 0;
    const int64_t len = live ? length(a.lens[i]) : 0;
    const int64_t adds = max(add, 0);
    int64_t rows, need_total;
    const int64_t row_end = rows0 + block_sum<NT>(adds, rows, part);
    const int64_t want = (len + adds + pmask) >> a.pshift, held = held_of((int)len);
    const bool too = want > a.max_pages || row_end > a.T || len + adds > kNone;
    const int64_t need = add < 0 || too ? 0 : want - held;
    const int64_t got = need0 + block_sum<NT>(need, need_total, part);
    const bool refused = adds > 0 && (too || (need > 0 && got > top));
    if (live) {
      a.lens_out[i] = add < 0 ? 0 : refused ? (int)(-1 - len) : (int)(len + adds);
      a.offsets[i + 1] = (int)min(row_end, a.T);
      if (need > 0 && !refused) atomicMax(&s_taken, (int)got);
    }
    s_len[tid] = (int)len;
    s_held[tid] = (int)held;
    s_refused[tid] = refused;
    s_start[tid] = live ? clip(got - need) : kNone;
    __syncthreads();
    for (int64_t k = need0 + tid; k < min(need0 + need_total, top); k += NT) {
      const int j = find<NT>(s_start, (int)k);
      if (!s_refused[j])
        a.pages[(base + j) * a.max_pages + s_held[j] + (k - s_start[j])] = a.free_pages[top - 1 - k];
    }
    if (a.rows_here) {
      __syncthreads();  // the pages are there, s_start has been read
      s_start[tid] = live ? clip(row_end - adds) : kNone;
      __syncthreads();
      for (int64_t t = rows0 + tid; t < min(rows0 + rows, a.T); t += NT) {
        const int j = find<NT>(s_start, (int)t);
        const int64_t pos = s_len[j] + (t - s_start[j]);
        int64_t slot = -1;
        if (!s_refused[j])
          slot = ((int64_t)a.pages[(base + j) * a.max_pages + (pos >> a.pshift)] << a.pshift) + (pos & pmask);
        a.positions[t] = (int)pos;
        a.slots[t] = slot;
      }
    }
    rows0 += rows;
    need0 += need_total;
    __syncthreads();  // before the next chunk's writes
  }
  if (a.rows_here)
    for (int64_t t = rows0 + tid; t < a.T; t += NT) {
      a.positions[t] = 0;
      a.slots[t] = -1;
    }
  if (tid == 0) *a.free_count_out = (int)(top - s_taken);
}

// The rows of large steps, dealt to many workgroups once the lengths, offsets and
// pages are there: a sequence of n rows had lens_out - n before, one that was
// refused has -1 - lens_out.
__global__ __launch_bounds__(256) void k_extend_rows(ExtendArgs a) {
  const int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (t >= a.T) return;
  int64_t slot = -1;
  int pos = 0;
  if (t < a.offsets[a.n_seq]) {
    int64_t lo = 0, hi = a.n_seq;  // offsets[lo] <= t < offsets[hi]
    while (hi - lo > 1) {
      const int64_t mid = (lo + hi) >> 1;
      if (a.offsets[mid] <= t) lo = mid;
      else hi = mid;
    }
    const int after = a.lens_out[lo];
    const int first = a.offsets[lo];
    if (after < 0) {
      pos = (int)(-1 - (int64_t)after + (t - first));
    } else {
      pos = (int)(after - (a.offsets[lo + 1] - t));
      slot = ((int64_t)a.pages[lo * a.max_pages + (pos >> a.pshift)] << a.pshift) +
             (pos & ((1 << a.pshift) - 1));
    }
  }
  a.positions[t] = pos;
  a.slots[t] = slot;
}

// rows that the workgroup of k_extend takes itself, without a second launch
constexpr int64_t kRowsHere = 4096;

}  // namespace

bool extend_rows_apart(const ExtendArgs& a) { return a.T > kRowsHere; }

hipError_t launch_extend(const ExtendArgs& a, const Launch& L) {
  const int64_t n = std::max(a.n_seq, std::min(a.T, kRowsHere) / 4);
  if (n <= 64) return ext_launch(k_extend<64>, dim3(1), dim3(64), 0, L, a);
  if (n <= 256) return ext_launch(k_extend<256>, dim3(1), dim3(256), 0, L, a);
  return ext_launch(k_extend<1024>, dim3(1), dim3(1024), 0, L, a);
}

hipError_t launch_extend_rows(const ExtendArgs& a, const Launch& L) {
  return ext_launch(k_extend_rows, dim3((unsigned)((a.T + 255) / 256)), dim3(256), 0, L, a);
}

}  // namespace ttq
