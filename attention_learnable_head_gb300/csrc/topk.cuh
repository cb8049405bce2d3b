// The n-th largest of a row of values by one CTA: its bits are found from the top, each
// by counting the values at or above a candidate.  Values are mapped to unsigned
// integers of the same order first; a NaN counts as the largest.
#pragma once
#include <cstdint>

namespace attn_sink {

__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t u = __float_as_uint(x == 0.0f ? 0.0f : x);   // -0 equals 0
  if (x != x) return 0xFFFFFFFFu;
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

// The value T with count(v > T) < n <= count(v >= T), 1 <= n <= count of all, over the
// values that `each` passes to its argument, v by v, shared out over the threads;
// they are ones that ordered() gave, T the smallest bound found: where a candidate
// has exactly n values at or above it the search ends, as no lower bit can matter.
// *exact: then count(v >= T) = n.
template <int kThreads, typename U, typename Each>
__device__ __forceinline__ U block_nth_largest(int n, Each each, int (*s)[kThreads / 32],
                                               int* turn, bool* exact) {
  U bound = 0;
  *exact = false;
  for (U bit = (U)1 << (8 * sizeof(U) - 1); bit != 0; bit >>= 1) {
    const U at = bound | bit;
    int c = 0;
    each([&](U v) { c += v >= at; });
    c = block_sum<kThreads>(c, s, turn);
    if (c >= n) bound = at;
    if (c == n) {
      *exact = true;
      break;
    }
  }
  return bound;
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

}  // namespace attn_sink
