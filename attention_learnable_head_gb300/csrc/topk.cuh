// The n-th largest of a row of values by one CTA.  Values are mapped to unsigned
// integers of the same order first (a NaN counts as the largest; 0xFFFFFFFF is free).  A
// histogram of their range, as it is, says which bin the n-th is in; a bin of few values is
// ranked value by value, one of many has a histogram of its own.  Floats as integers are
// about their logarithms, so that attention weights spread over the bins and few additions
// meet in one.  Bounded by the latency of passes that depend on each other: with 32 counts of
// the values above a candidate, one for each bit, in its place an eviction of 32 rows of
// 16384 weights took 42.5 us, not 26, and a selection of 8 rows of 8192 pages 44, not 31.
#pragma once
#include <cstdint>

namespace attn_sink {

__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t u = __float_as_uint(x == 0.0f ? 0.0f : x);   // -0 equals 0
  if (x != x) return 0xFFFFFFFEu;
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float unordered(uint32_t u) {
  return __uint_as_float(u & 0x80000000u ? u & 0x7FFFFFFFu : ~u);
}
__device__ __forceinline__ unsigned long long ordered(double x) {
  const unsigned long long u = __double_as_longlong(x == 0.0 ? 0.0 : x);
  if (x != x) return ~0ull;
  return u >> 63 ? ~u : u | 1ull << 63;
}

// Sum over the CTA; s: one int per warp, used in turn by the parity of *turn.
template <int kThreads>
__device__ __forceinline__ int block_sum(int x, int (*s)[kThreads / 32], int* turn) {
  constexpr int kWarps = kThreads / 32;
  static_assert(kWarps <= 32, "a lane per warp");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  x = __reduce_add_sync(0xffffffffu, x);
  int* at = s[*turn];
  *turn ^= 1;
  if (lane == 0) at[warp] = x;
  __syncthreads();
  return __reduce_add_sync(0xffffffffu, lane < kWarps ? at[lane] : 0);
}

// Exclusive scan over the CTA of one value a thread, in the order of the threads; *all
// receives the sum.  As block_sum, s in turn.
template <int kThreads>
__device__ __forceinline__ int block_scan(int x, int (*s)[kThreads / 32], int* turn, int* all) {
  constexpr int kWarps = kThreads / 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int inc = x;
  #pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, inc, d);
    if (lane >= d) inc += y;
  }
  int* at = s[*turn];
  *turn ^= 1;
  if (lane == 31) at[warp] = inc;
  __syncthreads();
  int sum = lane < kWarps ? at[lane] : 0;
  #pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, sum, d);
    if (lane >= d) sum += y;
  }
  *all = __shfl_sync(0xffffffffu, sum, 31);
  const int before = __shfl_sync(0xffffffffu, sum, max(warp - 1, 0));
  return (warp > 0 ? before : 0) + inc - x;
}

// What block_nth keeps in shared memory.
constexpr int kNthEach = 2;              // bins a thread
template <int kThreads>
struct NthShared {
  int sum[2][kThreads / 32];
  unsigned bins[kNthEach * kThreads];
  uint32_t list[kThreads];
  uint32_t low[kThreads / 32], high[kThreads / 32], value;
  int count, bin, before, same;
};

// What block_nth says of the value of a rank.
struct Nth {
  uint32_t value;
  int above, same;                         // how many are larger, and equal
};

// The value T of rank n from the top, 1 <= n <= count: count(v > T) < n <= count(v >= T),
// over the values that `each` passes to its argument, shared out over the threads.  low
// and high: the smallest and the largest of this thread's (0xFFFFFFFF and 0 of none).
// What `each` reads need not be visible to other threads yet.  *turn as in block_sum.
template <int kThreads, typename Each>
__device__ __forceinline__ Nth block_nth(int n, uint32_t low, uint32_t high, Each each,
                                         NthShared<kThreads>* s, int* turn) {
  constexpr int kNthBins = kNthEach * kThreads;
  constexpr int kBits = kThreads == 256 ? 9 : kThreads == 512 ? 10 : 11;
  constexpr int kWarps = kThreads / 32;
  static_assert(1 << kBits == kNthBins, "a power of two");
  const int tid = threadIdx.x, lane = tid & 31;
  low = __reduce_min_sync(0xffffffffu, low);
  high = __reduce_max_sync(0xffffffffu, high);
  if (lane == 0) {
    s->low[tid >> 5] = low;
    s->high[tid >> 5] = high;
  }
  #pragma unroll
  for (int i = 0; i < kNthEach; ++i) s->bins[tid + i * kThreads] = 0;
  if (tid == 0) s->count = 0;
  __syncthreads();
  low = __reduce_min_sync(0xffffffffu, lane < kWarps ? s->low[lane] : 0xFFFFFFFFu);
  high = __reduce_max_sync(0xffffffffu, lane < kWarps ? s->high[lane] : 0u);
  uint32_t base = low, span = high - low;
  int left = n;                            // rank within the range
  while (true) {
    const int shift = max(0, 32 - __clz(span) - kBits);        // span >> shift < kNthBins
    each([&](uint32_t v) {
      if (v - base <= span) atomicAdd(&s->bins[(v - base) >> shift], 1u);
    });
    __syncthreads();
    // the bin in which the rank lies, from the top
    int mine[kNthEach], sum = 0;
    #pragma unroll
    for (int i = 0; i < kNthEach; ++i) {
      mine[i] = (int)s->bins[kNthBins - 1 - (tid * kNthEach + i)];
      sum += mine[i];
    }
    int all;
    int upto = block_scan<kThreads>(sum, s->sum, turn, &all);
    #pragma unroll
    for (int i = 0; i < kNthEach; ++i) {
      if (upto < left && left <= upto + mine[i]) {
        s->bin = kNthBins - 1 - (tid * kNthEach + i);
        s->before = upto;
      }
      upto += mine[i];
    }
    __syncthreads();
    const uint32_t bin = (uint32_t)s->bin;
    const int many = (int)s->bins[bin];
    left -= s->before;
    base += bin << shift;
    span = shift > 0 ? min(span - (bin << shift), (1u << shift) - 1u) : 0u;
    if (shift == 0) return Nth{base, n - left, many};       // one value
    if (many <= kThreads) {
      each([&](uint32_t v) {
        if (v - base <= span) s->list[atomicAdd(&s->count, 1)] = v;   // in any order
      });
      __syncthreads();
      if (tid < many) {
        const uint32_t v = s->list[tid];
        int more = 0, same = 0;
        for (int i = 0; i < many; ++i) {
          more += s->list[i] > v;
          same += s->list[i] == v;
        }
        if (more < left && left <= more + same) {           // equal ones say the same
          s->value = v;
          s->before = more;
          s->same = same;
        }
      }
      __syncthreads();
      return Nth{s->value, n - left + s->before, s->same};
    }
    __syncthreads();                       // the bins have been read
    #pragma unroll
    for (int i = 0; i < kNthEach; ++i) s->bins[tid + i * kThreads] = 0;
    __syncthreads();
  }
}

// The same for 64-bit values, from the top bit by bit: count(v >= the result) >= n, and
// n exactly where *whole, else count(v > the result) < n.
template <int kThreads, typename Each>
__device__ __forceinline__ unsigned long long block_nth64(int n, Each each,
                                                          int (*s)[kThreads / 32], int* turn,
                                                          bool* whole) {
  unsigned long long bound = 0;
  *whole = false;
  for (unsigned long long bit = 1ull << 63; bit != 0; bit >>= 1) {
    const unsigned long long at = bound | bit;
    int c = 0;
    each([&](unsigned long long v) { c += v >= at; });
    c = block_sum<kThreads>(c, s, turn);
    if (c >= n) bound = at;
    if (c == n) {
      *whole = true;
      break;
    }
  }
  return bound;
}

}  // namespace attn_sink
