// Bounds of the keys of a page, and the pages whose bounds promise a decode step's
// largest scores, sm_103a.
//
// For any key k of a page with elementwise bounds lo <= k <= hi,
//   q.k <= sum_d max(q_d, 0) hi_d + min(q_d, 0) lo_d,
// a dot product of 128 numbers: (min(q, 0), max(q, 0)) with the page's 256 bytes (lo,
// hi).  A page of 16 keys is so judged by 1/16 of what its keys and values weigh.
//
// Bounds: eight lanes of 16 bytes read a head's key, a warp four heads of a page, key
// by key, all of a page's loads on their way at once up to 16.  Bounded by the keys' bytes: 16
// prompts of 500 to 2047 new keys, 29 MB, 7.4 us with the launch; one page each of 128
// sequences 4.1 us.
//
// Scores: pages are the 16 rows, the group's heads the 8 columns of warp-level
// products m16n8k16 (a tcgen05 product has 64 rows of one operand at least, and its
// operands would go through shared memory: this is bound by the bounds' bytes).  As a
// dot product does not care for the order of its terms, the k index is permuted so
// that a lane's fragments are whole 16-byte chunks of a page's bounds: chunk 4 u + t of
// the 16 for lane t of four.  64 sequences x 8 heads x 1024 pages: 101 MB in 21 us.
//
// Selection: one CTA for each (sequence, kv head) finds the score of the last page it
// takes (topk.cuh).  The scores come from fp32 sums, so every page within
// twice their error of that one is computed again with the sums' rounding carried on, where
// any are left out (a fraction of a page a row, on average).  What is selected goes through
// a bitmap to ascending order.  Bounded by the latency of these passes: 128 pages for 64 x 8 rows
// of 1024 10 us, 256 for 8 rows of 8192 12 us.
#pragma once
#include <climits>
#include <cuda_bf16.h>
#include "sm103_ptx.cuh"
#include "topk.cuh"

namespace attn_sink {

// ----------------------------------------------------------------------------- bounds
constexpr int kBoundsThreads = 256;

struct BoundsParams {
  const __nv_bfloat16* k_cache;   // [num_pages][page_size][H_kv][64]
  const int* block_table;         // [B][max_pages]
  const int* cached;              // [B]
  const int* seq_lens;            // [B]
  __nv_bfloat16* bounds;          // [num_pages][H_kv][2][64]
  int* err;
  int batch, heads_kv, page_size, num_pages, max_pages;
};

__global__ void __launch_bounds__(kBoundsThreads)
attn_sink_page_bounds_kernel(const __grid_constant__ BoundsParams p) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int quads = (p.heads_kv + 3) / 4;
  const int cap = p.max_pages * p.page_size;
  const unsigned warps = gridDim.x * (kBoundsThreads / 32);
  for (int b = blockIdx.y; b < p.batch; b += gridDim.y) {
    const int l0 = __ldg(p.seq_lens + b), c0 = __ldg(p.cached + b);
    const int len = max(0, min(l0, cap)), from = max(0, min(c0, len));
    if ((len != l0 || c0 < 0) && threadIdx.x == 0) atomicCAS(p.err, 0, DEVERR_DECODE_INPUT);
    if (from >= len) continue;
    const int col0 = from / p.page_size, cols = (len - 1) / p.page_size + 1 - col0;
    const unsigned long long units = (unsigned long long)cols * (unsigned)quads;
    for (unsigned long long u = blockIdx.x * (kBoundsThreads / 32) + warp; u < units; u += warps) {
      const int at = (int)(u / (unsigned)quads);
      const int h = 4 * (int)(u - (unsigned long long)at * (unsigned)quads) + (lane >> 3);
      const int col = col0 + at;
      const int page = __ldg(p.block_table + (size_t)b * p.max_pages + col);
      if ((unsigned)page >= (unsigned)p.num_pages) {
        if (lane == 0) atomicCAS(p.err, 0, DEVERR_DECODE_INPUT);
        continue;
      }
      if (h >= p.heads_kv) continue;
      const int keys = min(p.page_size, len - col * p.page_size);
      const size_t step = (size_t)p.heads_kv * 8;           // 16-byte chunks from key to key
      const uint4* src = reinterpret_cast<const uint4*>(p.k_cache) +
                         (size_t)page * p.page_size * step + h * 8 + (lane & 7);
      __nv_bfloat162 lo[4], hi[4];
      const uint4 v0 = __ldg(src);
      const uint32_t w0[4] = {v0.x, v0.y, v0.z, v0.w};
      #pragma unroll
      for (int e = 0; e < 4; ++e) lo[e] = hi[e] = *reinterpret_cast<const __nv_bfloat162*>(&w0[e]);
      // 16 keys at a time; one behind the last stands for it
      for (int j = 0; j < keys; j += 16) {
        uint4 v[16];
        #pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = __ldg(src + min(j + i, keys - 1) * step);
        #pragma unroll
        for (int i = 0; i < 16; ++i) {
          const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
          #pragma unroll
          for (int e = 0; e < 4; ++e) {
            const __nv_bfloat162 x = *reinterpret_cast<const __nv_bfloat162*>(&w[e]);
            lo[e] = __hmin2_nan(lo[e], x);
            hi[e] = __hmax2_nan(hi[e], x);
          }
        }
      }
      uint4* dst = reinterpret_cast<uint4*>(p.bounds) + ((size_t)page * p.heads_kv + h) * 16 +
                   (lane & 7);
      dst[0] = *reinterpret_cast<const uint4*>(lo);
      dst[8] = *reinterpret_cast<const uint4*>(hi);
    }
  }
}

// ----------------------------------------------------------------------------- scores
constexpr int kScoreThreads = 256;
constexpr int kScoreStages = 2;         // groups of 16 pages on their way to a warp
constexpr int kScoreSmem = kScoreThreads / 32 * kScoreStages * 16 * 256;

struct SelectParams {
  const __nv_bfloat16* q;         // [B][H_q][64]
  const __nv_bfloat16* bounds;    // [num_pages][H_kv][2][64]
  const int* block_table;         // [B][max_pages]
  const int* seq_lens;            // [B]
  float* scores;                  // [B][H_kv][max_pages]; -inf: no page in the cache
  unsigned* peak;                 // [B][H_kv][tiles] largest |bound| of 16 pages, bf16 bits
  unsigned long long* exact;      // [B][H_kv][max_pages] ordered() of 64-bit scores, some
  int* selected;                  // [B][H_kv][count]
  int* err;
  int batch, heads_q, heads_kv, group, page_size, num_pages, max_pages, tiles;
  int count, keep_first, keep_last;
};

__device__ __forceinline__ int select_len(const SelectParams& p, int b, bool* bad) {
  const int len = __ldg(p.seq_lens + b), cap = p.max_pages * p.page_size;
  *bad = len < 0 || len > cap;
  return max(0, min(len, cap));
}

__global__ void __launch_bounds__(kScoreThreads, 3)
attn_sink_page_scores_kernel(const __grid_constant__ SelectParams p) {
  grid_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const unsigned id = blockIdx.x * (kScoreThreads / 32) + warp;
  const unsigned step = gridDim.x * (kScoreThreads / 32) / (unsigned)p.heads_kv;
  const unsigned first = id / (unsigned)p.heads_kv;
  const int h = (int)(id - first * (unsigned)p.heads_kv);
  const int b = blockIdx.y;
  bool bad;
  const int len = select_len(p, b, &bad);
  if (bad && id == 0 && lane == 0) atomicCAS(p.err, 0, DEVERR_DECODE_INPUT);
  const int have = (len + p.page_size - 1) / p.page_size;
  if (have <= p.count || first >= step) return;             // all are selected
  // B: head g, the dimensions of this lane's chunks; 0 for the columns behind the group
  uint32_t qb[16];
  #pragma unroll
  for (int u = 0; u < 2; ++u) {
    uint4 v = make_uint4(0, 0, 0, 0);
    if (g < p.group)
      v = __ldg(reinterpret_cast<const uint4*>(p.q) +
                ((size_t)b * p.heads_q + h * p.group + g) * 8 + 4 * u + t);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    #pragma unroll
    for (int e = 0; e < 4; ++e) {
      const __nv_bfloat162 x = *reinterpret_cast<const __nv_bfloat162*>(&w[e]);
      const __nv_bfloat162 zero = __floats2bfloat162_rn(0.0f, 0.0f);
      const __nv_bfloat162 lo = __hmin2_nan(x, zero), hi = __hmax2_nan(x, zero);
      qb[4 * u + e] = *reinterpret_cast<const uint32_t*>(&lo);
      qb[8 + 4 * u + e] = *reinterpret_cast<const uint32_t*>(&hi);
    }
  }
  const size_t row = (size_t)b * p.heads_kv + h;
  const int* table = p.block_table + (size_t)b * p.max_pages;
  extern __shared__ __align__(256) uint8_t score_smem[];
  const uint32_t ring = smem_u32(score_smem) + (uint32_t)warp * (kScoreStages * 16 * 256);
  // 16-byte chunk c of page r: every other page has the halves of its 128 bytes exchanged,
  // so that 8 lanes that read 4 chunks of 2 pages touch each bank once
  auto place = [](int r, int c) { return (uint32_t)r * 256u + (uint32_t)((c ^ ((r & 1) << 2)) << 4); };
  const unsigned tiles = (unsigned)(have + 15) / 16;
  auto entry = [&](unsigned tile) {                         // of page 16 tile + lane % 16
    const int c = 16 * (int)tile + (lane & 15);
    int e = -1;
    if (tile < tiles && c < have) {
      e = __ldg(table + c);
      if ((unsigned)e >= (unsigned)p.num_pages) {
        atomicCAS(p.err, 0, DEVERR_DECODE_INPUT);
        e = -1;
      }
    }
    return e;
  };
  auto issue = [&](int mine, int st) {
    #pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int r = 2 * u + (lane >> 4);
      const int e = __shfl_sync(0xffffffffu, mine, r);      // -1: nothing is read, 0 written
      cp_async_16_zfill(ring + st * (16 * 256) + place(r, lane & 15),
                        e >= 0 ? p.bounds + ((size_t)e * p.heads_kv + h) * 128 + 8 * (lane & 15) : p.q,
                        e >= 0 ? 16 : 0);
    }
  };
  int mine[kScoreStages];
  #pragma unroll
  for (int st = 0; st < kScoreStages; ++st) mine[st] = entry(first + st * step);
  #pragma unroll
  for (int st = 0; st < kScoreStages; ++st) {
    if (first + st * step < tiles) issue(mine[st], st);
    cp_async_commit();
  }
  int next = entry(first + kScoreStages * step);
  for (unsigned base = first; base < tiles; base += kScoreStages * step) {
    #pragma unroll
    for (int st = 0; st < kScoreStages; ++st) {
      const unsigned tile = base + st * step, ahead = tile + kScoreStages * step;
      if (tile >= tiles) continue;                          // the same for the whole warp
      cp_async_wait<kScoreStages - 1>();
      __syncwarp();
      uint32_t v[2][4][4];
      #pragma unroll
      for (int r = 0; r < 2; ++r)
        #pragma unroll
        for (int u = 0; u < 4; ++u)
          ld_shared_v4(ring + st * (16 * 256) + place(8 * r + g, 4 * u + t), v[r][u]);
      const bool in0 = __shfl_sync(0xffffffffu, mine[st], g) >= 0;
      const bool in1 = __shfl_sync(0xffffffffu, mine[st], g + 8) >= 0;
      __syncwarp();                                         // every lane has read the stage
      mine[st] = next;
      if (ahead < tiles) issue(next, st);
      cp_async_commit();
      next = entry(ahead + step);
      float c[4] = {0.0f, 0.0f, 0.0f, 0.0f};
      uint32_t peak = 0;
      #pragma unroll
      for (int u = 0; u < 4; ++u) {
        mma_16816_bf16(c, v[0][u][0], v[1][u][0], v[0][u][1], v[1][u][1], qb[4 * u], qb[4 * u + 1]);
        mma_16816_bf16(c, v[0][u][2], v[1][u][2], v[0][u][3], v[1][u][3], qb[4 * u + 2],
                       qb[4 * u + 3]);
        #pragma unroll
        for (int r = 0; r < 2; ++r)
          #pragma unroll
          for (int e = 0; e < 4; ++e) peak = __vmaxu2(peak, v[r][u][e] & 0x7fff7fffu);
      }
      // the largest head's score (a NaN among them counts: the row's peak says so too)
      #pragma unroll
      for (int r = 0; r < 2; ++r) {
        float m = 2 * t < p.group ? c[2 * r] : -INFINITY;
        if (2 * t + 1 < p.group) m = fmaxf(m, c[2 * r + 1]);
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
        const int at = 16 * (int)tile + g + 8 * r;
        if (t == 0 && at < have) p.scores[row * p.max_pages + at] = (r ? in1 : in0) ? m : -INFINITY;
      }
      peak = __reduce_max_sync(0xffffffffu, max(peak & 0xffffu, peak >> 16));
      if (lane == 0) p.peak[row * p.tiles + tile] = peak;
    }
  }
}

// ----------------------------------------------------------------------------- selection
constexpr int kSelectStage = 12288;     // scores that a CTA keeps in shared memory
constexpr int kSelectBand = 256;        // pages at the border that it ranks there

// The 64-bit score of a page, by a whole warp: lanes 4 i .. 4 i + 3 have head i, 16
// dimensions each.  Products of two bf16 are exact in fp32 where they do not leave its
// range (kWide: they may; then all is done in fp64, of which the GPU has little), and the
// rounding of each sum is carried on in a second one: 48 bits and more.
template <bool kWide>
__device__ __forceinline__ unsigned long long page_score_exact(const SelectParams& p, int b, int h,
                                                               int col) {
  const int lane = threadIdx.x & 31, i = lane >> 2, t = lane & 3;
  const int page = __ldg(p.block_table + (size_t)b * p.max_pages + col);
  if ((unsigned)page >= (unsigned)p.num_pages) return ordered(-(double)INFINITY);
  const uint4* src =
      reinterpret_cast<const uint4*>(p.bounds) + ((size_t)page * p.heads_kv + h) * 16 + 2 * t;
  const uint4* query = reinterpret_cast<const uint4*>(p.q) +
                       ((size_t)b * p.heads_q + h * p.group + (i < p.group ? i : 0)) * 8 + 2 * t;
  double wide = 0.0;
  float s[2] = {0.0f, 0.0f}, low[2] = {0.0f, 0.0f};
  #pragma unroll
  for (int u = 0; u < 2; ++u) {
    const uint4 q4 = __ldg(query + u), lo4 = __ldg(src + u), hi4 = __ldg(src + 8 + u);
    const uint32_t q[4] = {q4.x, q4.y, q4.z, q4.w};
    const uint32_t lo[4] = {lo4.x, lo4.y, lo4.z, lo4.w}, hi[4] = {hi4.x, hi4.y, hi4.z, hi4.w};
    #pragma unroll
    for (int e = 0; e < 4; ++e)
      #pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float x = k ? bf16_hi(q[e]) : bf16_lo(q[e]);
        const float y[2] = {k ? bf16_hi(hi[e]) : bf16_lo(hi[e]), k ? bf16_hi(lo[e]) : bf16_lo(lo[e])};
        const float z[2] = {x < 0.0f ? 0.0f : x, x > 0.0f ? 0.0f : x};    // NaN: both
        #pragma unroll
        for (int d = 0; d < 2; ++d) {
          if constexpr (kWide) {
            wide = fma((double)z[d], (double)y[d], wide);
          } else {
            // two-sum: next + (what its rounding lost) = s + the product
            const float v = __fmul_rn(z[d], y[d]);
            const float next = __fadd_rn(s[d], v), part = __fsub_rn(next, s[d]);
            low[d] = __fadd_rn(low[d], __fadd_rn(__fsub_rn(s[d], __fsub_rn(next, part)),
                                                 __fsub_rn(v, part)));
            s[d] = next;
          }
        }
      }
  }
  double all = kWide ? wide : ((double)s[0] + (double)s[1]) + ((double)low[0] + (double)low[1]);
  all += __shfl_xor_sync(0xffffffffu, all, 1);
  all += __shfl_xor_sync(0xffffffffu, all, 2);
  unsigned long long best = i < p.group ? ordered(all) : 0;
  #pragma unroll
  for (int d = 4; d < 32; d <<= 1) {
    const unsigned long long o = __shfl_xor_sync(0xffffffffu, best, d);
    best = o > best ? o : best;
  }
  return best;
}

template <int kThreads>
__global__ void __launch_bounds__(kThreads, 1024 / kThreads)
attn_sink_select_kernel(const __grid_constant__ SelectParams p) {
  extern __shared__ uint32_t s_score[];                     // [min(max_pages, kSelectStage)]
  __shared__ NthShared<kThreads> s_nth;
  __shared__ uint32_t s_sure[kThreads], s_tie[kThreads];    // bitmaps of 32 kThreads pages
  __shared__ unsigned long long s_key[kSelectBand];
  __shared__ int s_at[kSelectBand];
  __shared__ uint8_t s_take[kSelectBand];
  __shared__ int s_many, s_side;   // pages at the border, and above it
  __shared__ unsigned s_peak[kThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31;
  const int b = (int)(blockIdx.x / (unsigned)p.heads_kv);
  const int h = (int)(blockIdx.x - (unsigned)b * (unsigned)p.heads_kv);
  const size_t row = blockIdx.x;
  int* out = p.selected + row * p.count;
  bool bad;
  const int have = (select_len(p, b, &bad) + p.page_size - 1) / p.page_size;
  if (have <= p.count) {
    for (int i = tid; i < p.count; i += kThreads) out[i] = i < have ? i : -1;
    grid_dependency_wait();               // not to end before the kernel in front does
    return;
  }
  for (int i = tid; i < p.keep_first; i += kThreads) out[i] = i;
  for (int i = tid; i < p.keep_last; i += kThreads)
    out[p.count - p.keep_last + i] = have - p.keep_last + i;
  const int n = have - p.keep_first - p.keep_last;          // pages between them
  const int need = p.count - p.keep_first - p.keep_last;    // < n
  if (need == 0) {
    grid_dependency_wait();
    return;
  }
  // the largest sum of |q| of a head, lanes 4 i .. 4 i + 3 have head i (a NaN is the
  // largest as an integer, too)
  float norm = 0.0f;
  if ((lane >> 2) < p.group) {
    const uint4* query = reinterpret_cast<const uint4*>(p.q) +
                         ((size_t)b * p.heads_q + h * p.group + (lane >> 2)) * 8 + 2 * (lane & 3);
    #pragma unroll
    for (int u = 0; u < 2; ++u) {
      const uint4 v = __ldg(query + u);
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
      #pragma unroll
      for (int e = 0; e < 4; ++e) norm += fabsf(bf16_lo(w[e])) + fabsf(bf16_hi(w[e]));
    }
  }
  norm += __shfl_xor_sync(0xffffffffu, norm, 1);
  norm += __shfl_xor_sync(0xffffffffu, norm, 2);
  norm = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(norm) & 0x7fffffffu));
  if (tid == 0) {
    s_many = s_side = 0;
  }
  grid_dependency_wait();                                   // the scores
  const float* scores = p.scores + row * p.max_pages + p.keep_first;
  const bool staged = n <= kSelectStage;
  uint32_t least = 0xFFFFFFFFu, largest = 0;
  for (int i0 = tid; i0 < n; i0 += 8 * kThreads) {
    float x[8];                                             // on their way together
    #pragma unroll
    for (int u = 0; u < 8; ++u)
      x[u] = i0 + u * kThreads < n ? __ldcg(scores + i0 + u * kThreads) : 0.0f;
    #pragma unroll
    for (int u = 0; u < 8; ++u) {
      if (i0 + u * kThreads >= n) break;
      const uint32_t v = ordered(x[u]);
      least = min(least, v);
      largest = max(largest, v);
      if (staged) s_score[i0 + u * kThreads] = v;
    }
  }
  unsigned peak = 0;
  for (int i = tid; i < (have + 15) / 16; i += kThreads)
    peak = max(peak, __ldcg(p.peak + row * p.tiles + i));
  peak = __reduce_max_sync(0xffffffffu, peak);
  if (lane == 0) s_peak[tid >> 5] = peak;
  auto at = [&](int i) { return staged ? s_score[i] : ordered(__ldcg(scores + i)); };
  int turn = 0;
  const uint32_t low = block_nth<kThreads>(
      need, least, largest, [&](auto&& take) {
        for (int i0 = tid; i0 < n; i0 += 4 * kThreads) {
          uint32_t v[4];
          #pragma unroll
          for (int u = 0; u < 4; ++u) v[u] = i0 + u * kThreads < n ? at(i0 + u * kThreads) : 0u;
          #pragma unroll
          for (int u = 0; u < 4; ++u)
            if (i0 + u * kThreads < n) take(v[u]);
        }
      }, &s_nth, &turn).value;             // the smallest score that is taken
  // No score is further off than the rounding of its sums: 8 products of 16 terms and the sum
  // so far, each of the 17 cut below 2^-23 of what the terms' sizes add up to at most, 8 * 17 *
  // 2^-23 = 1.0625 * 2^-16; and 2^-119 where small terms are lost, nothing of 2^-90.
  peak = __reduce_max_sync(0xffffffffu, lane < kThreads / 32 ? s_peak[lane] : 0u);
  const float top = __uint_as_float(peak << 16), most = norm * top;
  // Infinities, NaN, and scores so small that fp32 loses some of their products: all of them
  // in fp64.  (None of that where there are only zeros.)
  const bool wide =
      !(most < 1e37f) || (most < 0x1p-90f && norm != 0.0f && top != 0.0f);
  const float off = most * 0x1.2p-15f;                      // more than twice that: both sides
  const float last = unordered(low);
  uint32_t from = low, upto = low;                      // the border, both ends inside
  if (wide) {
    from = 0;
    upto = 0xFFFFFFFFu;
  } else if (off > 0.0f) {
    from = ordered(__fsub_rd(last, off));
    upto = ordered(__fadd_ru(last, off));
  }
  int sure = 0;
  for (int i0 = tid; i0 < n; i0 += 4 * kThreads) {
    uint32_t v[4];
    #pragma unroll
    for (int u = 0; u < 4; ++u) v[u] = i0 + u * kThreads < n ? at(i0 + u * kThreads) : 0u;
    #pragma unroll
    for (int u = 0; u < 4; ++u) {
      sure += v[u] > upto;
      if (v[u] < from || v[u] > upto || i0 + u * kThreads >= n) continue;
      const int x = atomicAdd(&s_many, 1);                  // their order does not matter
      if (x < kSelectBand) s_at[x] = i0 + u * kThreads;
    }
  }
  sure = __reduce_add_sync(0xffffffffu, sure);
  if (lane == 0 && sure != 0) atomicAdd(&s_side, sure);     // whole numbers: any order
  __syncthreads();
  const int left = need - s_side, border = s_many;          // of the border, left <= border
  // which of the border: all, by their ranks in shared memory, or by a 64-bit bound
  const bool every = left == border;
  const bool again = !every && (off > 0.0f || wide);
  const bool ranked = again && border <= kSelectBand;
  const unsigned long long* exact = p.exact + row * p.max_pages;
  unsigned long long bound64 = 0;
  if (again) {
    auto score = [&](int i) {
      return wide ? page_score_exact<true>(p, b, h, p.keep_first + i)
                  : page_score_exact<false>(p, b, h, p.keep_first + i);
    };
    if (ranked) {
      for (int x = tid >> 5; x < border; x += kThreads / 32) {
        const unsigned long long key = score(s_at[x]);
        if (lane == 0) s_key[x] = key;
      }
    } else {
      for (int i0 = tid - lane; i0 < n; i0 += kThreads) {
        const uint32_t v = i0 + lane < n ? at(i0 + lane) : 0;
        unsigned todo = __ballot_sync(0xffffffffu, i0 + lane < n && v >= from && v <= upto);
        for (; todo != 0; todo &= todo - 1) {
          const int i = i0 + __ffs(todo) - 1;
          const unsigned long long key = score(i);
          if (lane == 0) p.exact[row * p.max_pages + i] = key;
        }
      }
    }
    __syncthreads();
    if (ranked) {
      if (tid < border) {
        int before = 0;
        for (int y = 0; y < border; ++y)
          before += s_key[y] > s_key[tid] || (s_key[y] == s_key[tid] && s_at[y] < s_at[tid]);
        s_take[tid] = before < left;
      }
      __syncthreads();
    } else {
      bool whole;
      bound64 = block_nth64<kThreads>(
          left, [&](auto&& take) {
            for (int i = tid; i < n; i += kThreads) {
              const uint32_t v = at(i);
              if (v >= from && v <= upto) take(exact[i]);
            }
          }, s_nth.sum, &turn, &whole);
      if (whole && bound64 > 0) --bound64;                  // all at or above it: none is a tie
    }
  }
  int ties = !again ? left : 0;                             // equals that are taken
  if (again && !ranked) {
    int above = 0;
    for (int i = tid; i < n; i += kThreads) {
      const uint32_t v = at(i);
      above += v >= from && v <= upto && exact[i] > bound64;
    }
    ties = left - block_sum<kThreads>(above, s_nth.sum, &turn);
  }
  if (every) ties = 0;
  int done = p.keep_first;
  for (int base = 0; base < n; base += 32 * kThreads) {
    __syncthreads();                                        // the last round's words are read
    const int words = min(kThreads, (n - base + 31) / 32);
    if (tid >= words) s_sure[tid] = s_tie[tid] = 0;
    for (int w = tid >> 5; w < words; w += kThreads / 32) {
      const int i = base + 32 * w + lane;
      const uint32_t v = i < n ? at(i) : 0;                 // 0: no score
      bool take = v > upto || (every && v >= from && i < n), tie = false;
      if (!every && i < n && v >= from && v <= upto) {      // few: of whom some may be taken
        if (!again) {
          tie = true;                                       // the first ones of equals
        } else if (ranked) {
          int x = 0;
          while (s_at[x] != i) ++x;
          take = s_take[x] != 0;
        } else {
          take = exact[i] > bound64;
          tie = exact[i] == bound64;
        }
      }
      const uint32_t s = __ballot_sync(0xffffffffu, take), e = __ballot_sync(0xffffffffu, tie);
      if (lane == 0) {
        s_sure[w] = s;
        s_tie[w] = e;
      }
    }
    __syncthreads();
    uint32_t word = s_sure[tid];
    int all;
    if (ties > 0) {                                         // the same for the whole CTA
      uint32_t equal = s_tie[tid];
      const int before = block_scan<kThreads>(__popc(equal), s_nth.sum, &turn, &all);
      for (int k = min(__popc(equal), ties - before); k > 0; --k) {
        word |= equal & (0u - equal);
        equal &= equal - 1;
      }
      ties = max(0, ties - all);
    }
    int place = done + block_scan<kThreads>(__popc(word), s_nth.sum, &turn, &all);
    done += all;
    while (word != 0) {
      out[place++] = p.keep_first + base + 32 * tid + __ffs(word) - 1;
      word &= word - 1;
    }
  }
}

}  // namespace attn_sink
