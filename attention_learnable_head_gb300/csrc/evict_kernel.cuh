// Eviction from a paged cache by accumulated attention weight, sm_103a.
//
// One CTA for each (sequence, kv head) finds the weight of the last key that stays
// (topk.cuh), its row of weights in shared memory, and lists what moves: the n-th kept key
// at or behind the budget goes to the n-th hole below it.  Only as many rows move as there
// are holes, and no row is both read and written, so that they can be copied in any order,
// 8 lanes a move: by the same CTA where there are enough of them to fill the GPU, by a second
// kernel where there are few.  One more CTA of the first kernel scans the sequences for the
// pages that become free.
//
// 4 sequences x 8 heads, 8947 to 16384 keys to 2048: 22 us, of which 15 are the chain of one
// CTA a row (load, rank, list) on 33 of 152 SMs and the rest the moves; 64 sequences x 8 heads
// of 2183 to 4351 keys, 11 of them past 4096: 12 us, that chain alone.  Their bytes would take
// 5 and 3.  All 64 of 4351 keys: 26 us, 512 rows in two rounds (64 registers leave two CTAs of
// 512 threads an SM).
#pragma once
#include <climits>
#include <cuda_bf16.h>
#include "sm103_ptx.cuh"
#include "topk.cuh"

namespace attn_sink {

constexpr int kEvictStage = 49152;      // weights that a CTA keeps in shared memory
constexpr int kMoveThreads = 256;

struct EvictParams {
  uint4* k_cache;                 // [num_pages][page_size][H_kv][8 chunks of 16 bytes]
  uint4* v_cache;
  const int* block_table;         // [B][max_pages]
  const int* seq_lens;            // [B]
  const float* mass;              // [B][H_kv][max_keys]
  float* mass_out;
  int* new_lens;                  // [B]
  int* freed;                     // [max_freed]
  int* num_freed;                 // [1]
  int* counts;                    // [B][H_kv] moves
  int* to;                        // [B][H_kv][max_moves] holes, in order
  int* from;                      // [B][H_kv][max_moves] keys that move there, from the last
  int* err;
  int batch, heads_kv, page_size, num_pages, max_pages, max_keys;
  int budget, keep_first, keep_last, max_freed, max_moves, stage;
  int here;                       // one kernel: the CTA of a row moves it
  int lists;                      // the moves are listed in shared memory, behind the weights
};

constexpr uint32_t kNoRow = 0xFFFFFFFFu;
constexpr uint32_t kStays = 0xFFFFFFFFu;   // in the place of a weight: no competition

__device__ __forceinline__ int evict_len(const EvictParams& p, int b, bool* bad) {
  const int len = __ldg(p.seq_lens + b), cap = min(p.max_pages * p.page_size, p.max_keys);
  *bad |= len < 0 || len > cap;
  return max(0, min(len, cap));
}

// The moves first, first + step, .. of sequence b and kv head h, by 8 lanes each; `from` is
// listed from the last.
__device__ __forceinline__ void evict_move(const EvictParams& p, int b, int h, const int* to,
                                           const int* from, int moves, int first, int step) {
  const int c = threadIdx.x & 7;
  const int* table = p.block_table + (size_t)b * p.max_pages;
  auto cache_row = [&](int j) {
    const int pg = j / p.page_size, e = __ldg(table + pg);
    return (unsigned)e < (unsigned)p.num_pages
               ? (uint32_t)e * (uint32_t)p.page_size + (uint32_t)(j - pg * p.page_size)
               : kNoRow;
  };
  constexpr int kAtOnce = 4;               // chains of four loads
  for (int i = first; i < moves; i += kAtOnce * step) {
    uint32_t src[kAtOnce], dst[kAtOnce];
    #pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      const int m = i + u * step;
      src[u] = dst[u] = kNoRow;
      if (m < moves) {
        src[u] = cache_row(from[moves - 1 - m]);
        dst[u] = cache_row(to[m]);
        if (src[u] == kNoRow || dst[u] == kNoRow) {
          atomicCAS(p.err, 0, DEVERR_DECODE_INPUT);
          src[u] = kNoRow;
        }
      }
    }
    uint4 k[kAtOnce], v[kAtOnce];
    #pragma unroll
    for (int u = 0; u < kAtOnce; ++u)
      if (src[u] != kNoRow) {
        const size_t at = ((size_t)src[u] * p.heads_kv + h) * 8 + c;
        k[u] = __ldcg(p.k_cache + at);
        v[u] = __ldcg(p.v_cache + at);
      }
    #pragma unroll
    for (int u = 0; u < kAtOnce; ++u)
      if (src[u] != kNoRow) {
        const size_t at = ((size_t)dst[u] * p.heads_kv + h) * 8 + c;
        p.k_cache[at] = k[u];
        p.v_cache[at] = v[u];
      }
  }
}

// The pages that become free, and the new lengths.  Entries outside the cache are no pages:
// where a round has any, it is listed again without them.  A function of its own: inlined, it
// made the rows' CTAs slower (4 sequences of up to 16384 keys to 2048 22.4 us, 21.8 so).
template <int kThreads>
__device__ __noinline__ void evict_pages(const EvictParams& p, int (*s_sum)[kThreads / 32],
                                            int* s_from, int* s_first) {
  const int tid = threadIdx.x;
  int turn = 0, done = 0;
  bool bad = false;
  for (int b0 = 0; b0 < p.batch; b0 += kThreads) {
    const int b = b0 + tid;
    int count = 0, from = 0;
    if (b < p.batch) {
      const int len = evict_len(p, b, &bad), fewer = min(len, p.budget);
      p.new_lens[b] = fewer;
      from = (fewer + p.page_size - 1) / p.page_size;
      count = (len + p.page_size - 1) / p.page_size - from;
    }
    int all;
    const int before = block_scan<kThreads>(count, s_sum, &turn, &all);
    __syncthreads();                      // the last round's have been used
    s_from[tid] = from;
    s_first[tid] = before;
    __syncthreads();
    // entry by entry over the CTA; whose it is by bisection (few pages of many sequences, or
    // many of few: 10000 of two took 24 us with a warp a sequence)
    auto entry = [&](int x) {
      int i = 0;                          // the last sequence that starts at or before x
      #pragma unroll
      for (int d = kThreads / 2; d > 0; d >>= 1)
        if (s_first[i + d] <= x) i += d;
      return __ldg(p.block_table + (size_t)(b0 + i) * p.max_pages + s_from[i] + x - s_first[i]);
    };
    bool none = false;
    for (int x = tid; x < all; x += kThreads) {
      const int e = entry(x);
      none |= (unsigned)e >= (unsigned)p.num_pages;
      if (x < p.max_freed - done) p.freed[done + x] = e;
    }
    if (!__syncthreads_or(none)) {
      done += all;
      continue;
    }
    bad = true;
    for (int x0 = 0; x0 < all; x0 += kThreads) {
      const int e = x0 + tid < all ? entry(x0 + tid) : -1;
      const bool page = (unsigned)e < (unsigned)p.num_pages;
      int pages;
      const int at = done + block_scan<kThreads>(page, s_sum, &turn, &pages);
      if (page && at < p.max_freed) p.freed[at] = e;
      done += pages;
    }
  }
  if (bad) atomicCAS(p.err, 0, DEVERR_DECODE_INPUT);
  if (tid == 0) *p.num_freed = done;
  if (p.here)                             // no page behind the freed ones
    for (int i = done + tid; i < p.max_freed; i += kThreads) p.freed[i] = -1;
}

template <int kThreads>
__global__ void __launch_bounds__(kThreads, 1024 / kThreads)
attn_sink_evict_kernel(const __grid_constant__ EvictParams p) {
  extern __shared__ uint32_t s_mass[];                      // [stage]
  __shared__ NthShared<kThreads> s_nth;
  __shared__ uint32_t s_kept[kThreads], s_tie[kThreads];    // bitmaps of 32 kThreads keys
  __shared__ int s_holes;
  grid_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31;
  if (blockIdx.x == gridDim.x - 1) {
    evict_pages<kThreads>(p, s_nth.sum, reinterpret_cast<int*>(s_kept),
                          reinterpret_cast<int*>(s_tie));
    return;
  }
  const int b = (int)(blockIdx.x / (unsigned)p.heads_kv);
  const size_t row = blockIdx.x;
  const float* mass = p.mass + row * p.max_keys;
  float* mass_out = p.mass_out + row * p.max_keys;
  bool bad = false;
  const int len = evict_len(p, b, &bad), fewer = min(len, p.budget);
  // what stays where it is, and nothing behind; the holes are filled at the end
  if (len <= p.budget) {
    for (int j = tid; j < p.max_keys; j += kThreads) mass_out[j] = j < fewer ? __ldg(mass + j) : 0.0f;
    if (tid == 0) p.counts[row] = 0;
    return;
  }
  const bool staged = len <= p.stage;
  const int lo = p.keep_first, hi = len - p.keep_last;      // the keys that compete
  const int need = p.budget - p.keep_first - p.keep_last;   // < hi - lo
  uint32_t least = 0xFFFFFFFFu, largest = 0;
  for (int j0 = tid; j0 < p.max_keys; j0 += 8 * kThreads) {
    float m[8];                            // on their way together
    #pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int j = j0 + u * kThreads;
      m[u] = j < len ? __ldg(mass + j) : 0.0f;
    }
    #pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int j = j0 + u * kThreads;
      if (j < p.max_keys) mass_out[j] = j < fewer ? m[u] : 0.0f;
      if (j >= len) continue;
      const bool competes = j >= lo && j < hi;
      const uint32_t v = competes ? ordered(m[u]) : kStays;
      if (staged) s_mass[j] = v;
      if (competes) {
        least = min(least, v);
        largest = max(largest, v);
      }
    }
  }
  auto at = [&](int j) {
    return staged ? s_mass[j] : j >= lo && j < hi ? ordered(__ldg(mass + j)) : kStays;
  };
  int turn = 0, ties = 0;                                   // some of the equal ones stay
  uint32_t bound = 0, cut = kStays;                         // from `cut` on all stay
  if (need > 0) {
    // a thread reads what it stored itself: j = tid modulo kThreads
    const Nth nth = block_nth<kThreads>(
        need, least, largest, [&](auto&& take) {
          for (int j0 = tid; j0 < hi; j0 += 4 * kThreads) {
            uint32_t v[4];
            #pragma unroll
            for (int u = 0; u < 4; ++u) v[u] = j0 + u * kThreads < hi ? at(j0 + u * kThreads) : kStays;
            #pragma unroll
            for (int u = 0; u < 4; ++u)
              if (v[u] != kStays) take(v[u]);
          }
        }, &s_nth, &turn);
    bound = nth.value;
    if (need - nth.above < nth.same) ties = need - nth.above;
    cut = ties > 0 ? bound + 1 : bound;
  }
  // Bitmaps of 32 kThreads keys at a time, a word a thread.  With s kept keys in front of j,
  // a hole at j is number j - s, and a kept key at j >= budget is number budget - 1 - s
  // from the last.
  int* const lists = reinterpret_cast<int*>(s_mass + p.stage);
  int* const to = p.lists ? lists : p.to + row * p.max_moves;
  int* const come = p.lists ? lists + p.max_moves : p.from + row * p.max_moves;
  int stay = 0, holes = 0;
  for (int base = 0; base < len; base += 32 * kThreads) {
    __syncthreads();                                        // the last round's words are read
    const int words = min(kThreads, (len - base + 31) / 32);
    if (tid >= words) s_kept[tid] = s_tie[tid] = 0;
    for (int w = tid >> 5; w < words; w += kThreads / 32) {
      const int j = base + 32 * w + lane;
      const uint32_t v = j < len ? at(j) : 0;               // 0: no value
      const uint32_t k = __ballot_sync(0xffffffffu, v >= cut);
      if (lane == 0) s_kept[w] = k;
      if (ties > 0) {                                       // the same for the whole CTA
        const uint32_t e = __ballot_sync(0xffffffffu, v == bound);
        if (lane == 0) s_tie[w] = e;
      }
    }
    __syncthreads();
    uint32_t kept = s_kept[tid];
    int all;
    if (ties > 0) {                                         // the same for the whole CTA
      uint32_t equal = s_tie[tid];
      const int before = block_scan<kThreads>(__popc(equal), s_nth.sum, &turn, &all);
      for (int k = min(__popc(equal), ties - before); k > 0; --k) {
        kept |= equal & (0u - equal);
        equal &= equal - 1;
      }
      ties = max(0, ties - all);
    }
    const int j0 = base + 32 * tid;
    const int first = stay + block_scan<kThreads>(__popc(kept), s_nth.sum, &turn, &all);
    stay += all;
    // bits of the word below the budget
    const uint32_t below = fewer - j0 >= 32 ? 0xFFFFFFFFu : fewer <= j0 ? 0u : (1u << (fewer - j0)) - 1u;
    uint32_t hole = ~kept & below, mover = kept & ~below;
    int place = j0 - first;
    if (j0 < fewer) {
      while (hole != 0) {
        to[place++] = j0 + __ffs(hole) - 1;
        hole &= hole - 1;
      }
    }
    // kept keys of this word below the budget come first
    place = fewer - 1 - first - __popc(kept & below);
    while (mover != 0) {
      come[place--] = j0 + __ffs(mover) - 1;
      mover &= mover - 1;
    }
    // holes up to the budget: what is left of it when its kept keys are counted
    if (j0 < fewer && fewer <= j0 + 32) s_holes = fewer - first - __popc(kept & below);
  }
  __syncthreads();                                          // the moves are listed
  holes = fewer > 0 ? s_holes : 0;
  for (int i = tid; i < holes; i += kThreads)
    mass_out[to[i]] = __ldg(mass + come[holes - 1 - i]);
  if (p.here)
    evict_move(p, b, (int)(row - (size_t)b * p.heads_kv), to, come, holes, tid >> 3, kThreads / 8);
  else if (tid == 0)
    p.counts[row] = holes;
}

__global__ void __launch_bounds__(kMoveThreads)
attn_sink_evict_move_kernel(const __grid_constant__ EvictParams p) {
  grid_dependency_wait();
  const size_t rows = (size_t)p.batch * p.heads_kv;
  for (size_t row = blockIdx.y; row < rows; row += gridDim.y) {
    const int b = (int)(row / (unsigned)p.heads_kv);
    evict_move(p, b, (int)(row - (size_t)b * p.heads_kv), p.to + row * p.max_moves,
               p.from + row * p.max_moves, __ldcg(p.counts + row),
               blockIdx.x * (kMoveThreads / 8) + (threadIdx.x >> 3),
               gridDim.x * (kMoveThreads / 8));
  }
  // no page behind the freed ones
  const unsigned tid = (blockIdx.y * gridDim.x + blockIdx.x) * kMoveThreads + threadIdx.x;
  const unsigned threads = gridDim.x * gridDim.y * kMoveThreads;
  for (size_t i = (size_t)max(__ldcg(p.num_freed), 0) + tid; i < (size_t)p.max_freed; i += threads)
    p.freed[i] = -1;
}

}  // namespace attn_sink
