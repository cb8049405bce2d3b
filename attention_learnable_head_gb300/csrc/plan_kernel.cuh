// Plan of a serving step over the paged cache: new pages for the sequences'
// block tables, and a cache row and a position for every new token, from the
// request lengths alone.
//
// have_b = ceil(cached_b / P), need_b = ceil((cached_b + new_b) / P) - have_b;
// with base_b the exclusive sum of need, sequence b takes free[base_b ..
// base_b + need_b) in order.  Token i of b sits at position p = cached_b + i in
// row table[b, p / P] * P + p % P; where p / P >= have_b the entry is taken
// from the free list itself, so no CTA waits for a table entry that another
// writes, and the whole plan is one launch.
//
// CTA (x, y) handles the 256 sequences of group x: it sums the lengths of the
// groups before it (reads that stay in L2; of many sequences, where that would grow
// with their square, a kernel of one CTA before it does), scans its own group in
// shared memory, and writes every gridDim.y-th block of the group's tokens and new
// pages, found by bisection of the scanned offsets, so ragged lengths spread
// evenly.  What bounds it is latency: a plan moves 12 bytes a token and 8 a
// new page.  A decode step of 128 sequences takes 3.1 us, 1024 prompts of 64 to 128
// tokens 5.9 us on the device.
#pragma once
#include <climits>
#include "sm103_ptx.cuh"

namespace attn_sink {

constexpr int kPlanThreads = 256;
constexpr int kPlanSeqs = kPlanThreads;    // sequences of a group, one per thread
constexpr int DEVERR_PLAN = 0x1000;

struct PlanParams {
  const int* cached;
  const int* fresh;       // new tokens per sequence
  const int* free_pages;
  int* table;             // [B][max_pages]
  long long* slots;       // [max_tokens]
  int* positions;
  int* cu;                // [B + 1]
  int* lens;              // [B]
  int* needed;            // [1]
  int* err;
  int batch, page_size, num_pages, max_pages, num_free, max_tokens;
  int summed;             // the sums before each group are in cu and lens
};

struct PlanSeq {
  int cached, fresh, have, need;
};

__device__ __forceinline__ PlanSeq plan_seq(const PlanParams& p, int b, bool* bad) {
  PlanSeq s{0, 0, 0, 0};
  if (b >= p.batch) return s;
  const int cap = p.max_pages * p.page_size;             // <= 2^30, checked by the host
  const int c = __ldg(p.cached + b), n = __ldg(p.fresh + b);
  s.cached = min(max(c, 0), cap);
  s.fresh = min(max(n, 0), cap - s.cached);
  if (s.cached != c || s.fresh != n) *bad = true;
  const unsigned ps = (unsigned)p.page_size;
  s.have = (int)(((unsigned)s.cached + ps - 1) / ps);
  s.need = (int)(((unsigned)(s.cached + s.fresh) + ps - 1) / ps) - s.have;
  return s;
}

// Number of leading entries of the exclusive offsets first[0 .. kPlanSeqs) that
// are <= t, minus one: the sequence of the group that t falls into.
__device__ __forceinline__ int plan_find(const long long* first, long long t) {
  int lo = 0;
  #pragma unroll
  for (int step = kPlanSeqs / 2; step > 0; step >>= 1)
    if (first[lo + step] <= t) lo += step;
  return lo;
}

// Tokens and pages of the sequences before each group, left in the group's first
// entries of cu and lens, which the plan overwrites (its one CTA per group reads them
// first).  As unsigned 32-bit numbers: no max_tokens or num_free reaches the largest.
// A warp sums a group, 32 of them at a time.
constexpr int kPlanSumThreads = 1024;
__global__ void __launch_bounds__(kPlanSumThreads, 1)
attn_sink_plan_sum_kernel(const PlanParams p) {
  __shared__ long long s_tok[32], s_page[32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  bool dummy = false;
  long long tok0 = 0, pag0 = 0;            // before this round; kept by the first warp
  for (int b0 = 0; b0 < p.batch; b0 += 32 * kPlanSeqs) {
    long long tok = 0, pag = 0;
    #pragma unroll
    for (int i = 0; i < kPlanSeqs; i += 32) {
      const PlanSeq s = plan_seq(p, b0 + warp * kPlanSeqs + i + lane, &dummy);
      tok += s.fresh;
      pag += s.need;
    }
    #pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
      tok += __shfl_xor_sync(0xffffffffu, tok, d);
      pag += __shfl_xor_sync(0xffffffffu, pag, d);
    }
    if (lane == 0) {
      s_tok[warp] = tok;
      s_page[warp] = pag;
    }
    __syncthreads();
    if (warp == 0) {
      long long t = s_tok[lane], g = s_page[lane];
      const long long my_t = t, my_g = g;
      #pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const long long a = __shfl_up_sync(0xffffffffu, t, d), c = __shfl_up_sync(0xffffffffu, g, d);
        if (lane >= d) {
          t += a;
          g += c;
        }
      }
      const int b = b0 + lane * kPlanSeqs;
      if (b < p.batch) {
        p.cu[b] = (int)(unsigned)min(tok0 + t - my_t, (long long)UINT_MAX);
        p.lens[b] = (int)(unsigned)min(pag0 + g - my_g, (long long)UINT_MAX);
      }
      tok0 += __shfl_sync(0xffffffffu, t, 31);
      pag0 += __shfl_sync(0xffffffffu, g, 31);
    }
    __syncthreads();
  }
}

__global__ void __launch_bounds__(kPlanThreads)
attn_sink_plan_kernel(const PlanParams p) {
  constexpr int kWarps = kPlanThreads / 32;
  __shared__ long long s_tok[kPlanSeqs], s_page[kPlanSeqs];   // exclusive, within the group
  __shared__ int s_cached[kPlanSeqs], s_have[kPlanSeqs];
  __shared__ long long s_sum[2][kWarps];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int b0 = blockIdx.x * kPlanSeqs;
  bool bad = false, dummy = false;

  // tokens and pages of the sequences before this group (64-bit: lengths are
  // data; their sums are clamped only where they are stored)
  long long tok = 0, pag = 0;
  if (p.summed) {
    tok = (unsigned)p.cu[b0];
    pag = (unsigned)p.lens[b0];
    __syncthreads();                       // before they are overwritten
  } else if (b0 > 0) {
    for (int b = tid; b < b0; b += kPlanThreads) {
      const PlanSeq s = plan_seq(p, b, &dummy);
      tok += s.fresh;
      pag += s.need;
    }
    #pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
      tok += __shfl_xor_sync(0xffffffffu, tok, d);
      pag += __shfl_xor_sync(0xffffffffu, pag, d);
    }
    if (lane == 0) {
      s_sum[0][warp] = tok;
      s_sum[1][warp] = pag;
    }
    __syncthreads();
    tok = pag = 0;
    #pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      tok += s_sum[0][w];
      pag += s_sum[1][w];
    }
    __syncthreads();
  }
  const long long tok0 = tok, pag0 = pag;

  // exclusive scan of the group
  const int b = b0 + tid;
  const PlanSeq me = plan_seq(p, b, &bad);
  long long it = me.fresh, ip = me.need;
  #pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long a = __shfl_up_sync(0xffffffffu, it, d), c = __shfl_up_sync(0xffffffffu, ip, d);
    if (lane >= d) {
      it += a;
      ip += c;
    }
  }
  if (lane == 31) {
    s_sum[0][warp] = it;
    s_sum[1][warp] = ip;
  }
  __syncthreads();
  long long before_t = 0, before_p = 0, all_t = 0, all_p = 0;
  #pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) {
      before_t += s_sum[0][w];
      before_p += s_sum[1][w];
    }
    all_t += s_sum[0][w];
    all_p += s_sum[1][w];
  }
  const long long my_tok = before_t + it - me.fresh, my_page = before_p + ip - me.need;
  s_tok[tid] = my_tok;
  s_page[tid] = my_page;
  s_cached[tid] = me.cached;
  s_have[tid] = me.have;
  const bool last = b0 + kPlanSeqs >= p.batch;             // the group of the last sequence
  if (blockIdx.y == 0) {
    if (b < p.batch) {
      p.cu[b] = (int)min(tok0 + my_tok, (long long)p.max_tokens);
      p.lens[b] = me.cached + me.fresh;
    }
    if (last && tid == 0) {
      p.cu[p.batch] = (int)min(tok0 + all_t, (long long)p.max_tokens);
      *p.needed = (int)min(pag0 + all_p, (long long)INT_MAX);
      if (tok0 + all_t > p.max_tokens || pag0 + all_p > p.num_free) bad = true;
    }
  }
  __syncthreads();

  const long long step = (long long)gridDim.y * kPlanThreads;
  const long long first = (long long)blockIdx.y * kPlanThreads + tid;
  const unsigned ps = (unsigned)p.page_size;
  auto free_page = [&](long long i) -> int {               // entry i of the free list, or -1
    if (i >= p.num_free) return -1;
    const int pg = __ldg(p.free_pages + i);
    if (pg >= 0 && pg < p.num_pages) return pg;
    bad = true;
    return -1;
  };
  // new block-table entries of the group
  for (long long k = first; k < all_p; k += step) {
    const int s = plan_find(s_page, k);
    p.table[(size_t)(b0 + s) * p.max_pages + s_have[s] + (int)(k - s_page[s])] =
        free_page(pag0 + k);
  }
  // rows and positions of the group's tokens
  const long long n_tok = min(all_t, (long long)p.max_tokens - tok0);
  for (long long k = first; k < n_tok; k += step) {
    const int s = plan_find(s_tok, k);
    const unsigned pos = (unsigned)s_cached[s] + (unsigned)(k - s_tok[s]);
    const unsigned col = pos / ps;
    int pg;
    if ((int)col < s_have[s]) {
      pg = p.table[(size_t)(b0 + s) * p.max_pages + col];   // a page of the cached keys
      if (pg < 0 || pg >= p.num_pages) {
        bad = true;
        pg = -1;
      }
    } else {
      pg = free_page(pag0 + s_page[s] + (int)col - s_have[s]);
    }
    p.slots[tok0 + k] = pg < 0 ? -1ll : (long long)pg * p.page_size + (pos - col * ps);
    p.positions[tok0 + k] = (int)pos;
  }
  // entries behind the last token
  if (last) {
    for (long long t = tok0 + all_t + first; t < p.max_tokens; t += step) {
      p.slots[t] = -1;
      p.positions[t] = 0;
    }
  }
  if (bad) atomicCAS(p.err, 0, DEVERR_PLAN);
}

}  // namespace attn_sink
