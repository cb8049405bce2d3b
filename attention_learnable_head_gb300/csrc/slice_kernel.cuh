// A decode step over some of a sequence's cached keys, sm_103a: the pages selected for
// each kv head (attn_sink_decode_pages), or the keys behind a prefix that a group of
// sequences shares (attn_sink_decode_shared, whose prefix shared_kernel.cuh computes).
//
// CTA (slice, kv head, sequence) attends the G query heads of the kv head to one slice of
// the keys; slices and prefix are joined with the sink by attn_sink_join_kernel below, a
// single slice by its own CTA.
//
// Every warp has a pipeline of its own: blocks of 32 keys of K and V, every fourth block of
// the slice, in a ring of kSliceStages stages that only this warp waits for; nothing but
// the end synchronises the CTA.  (With blocks of 64 keys shared by the four warps, as in
// attn_sink_decode_kernel, the two barriers a block made the slowest warp's chain bound
// it: 64 sequences x 2048 selected keys 65 us at 4 to 5 CTAs an SM, at any depth.)  Where
// the page size is a power of two from 8 on, the first lanes of a warp copy a page or 32
// keys of one each by TMA; other page sizes are copied 16 bytes a lane with cp.async.
// List entries are read two blocks, table entries one block in front of the copies.
//
// The products are warp-level m16n8k16 (a tcgen05 product has 64 rows of keys or queries
// at least).  The G <= 8 query heads fill half of the 16 rows: S = Q K^T uses the others
// for nothing, O = P V for the lower halves of the probabilities: P = hi + lo in two bf16
// (17 bits), rows 0-7 and 8-15, so that bf16 values enter as they are.
//
// Bounded by the keys' and values' bytes: 64 sequences x 8 heads x 2048 selected keys 56 us
// (269 MB, 4.9 TB/s: rows of 128 bytes, each head of pages of its own), 192 sequences x 512 to
// 1024 own keys 57 us (5.3 TB/s).  One sequence of 4096 selected keys: 6 us, the chain
// of the two kernels.
#pragma once
#include <climits>
#include <cuda_bf16.h>
#include "fwd_kernel.cuh"

namespace attn_sink {

constexpr int kSliceThreads = 128;
constexpr int kSliceWarps = kSliceThreads / 32;
constexpr int kSliceKeys = 32;           // of a warp's block
constexpr int kSliceStages = 2;
constexpr int kSliceCtas = 3;            // per SM
constexpr int kSliceStageBytes = 2 * kSliceKeys * 128;
constexpr int kSliceSmem = 1024 + kSliceWarps * kSliceStages * kSliceStageBytes;
constexpr int kSliceMax = 64;            // slices of a sequence
constexpr int kSharedMinSeqs = 2;        // smaller groups and shorter prefixes are read by each
constexpr int kSharedMinKeys = 64;       //   sequence for itself
constexpr int kNoKey = INT_MIN;          // no entry of the list, or no key of the slice

// The prefix of a sequence: its tile's partial results.
struct alignas(16) SharedRef {
  int first, parts;               // of [partial][kv head][128 rows]; 0 parts: no prefix
  int place, pad;                 // the sequence's place in the tile
};

struct SliceParams {
  CUtensorMap tm_k;               // k_cache as [num_pages * page_size][H_kv][64], box
  CUtensorMap tm_v;               //   64 x 1 x min(page_size, 32), 128B swizzle (TMA path)
  const __nv_bfloat16* q;         // [B][H_q][64]
  const __nv_bfloat16* k_cache;   // [num_pages][page_size][H_kv][64]
  const __nv_bfloat16* v_cache;
  const int* block_table;         // [B][max_pages]
  const int* seq_lens;            // [B]
  const int* selected;            // pages: [B][H_kv][count] columns of the block table
  const int* cu_groups;           // shared: [num_groups + 1] first sequences
  const int* prefix_lens;         //   [num_groups]
  const SharedRef* refs;          //   [B]
  const float* prefix_o;          //   [partial][H_kv][128 rows][64] sums
  const float2* prefix_ml;        //   [partial][H_kv][128 rows]: maximum (log2 units), sum
  const float* sink;              // [H_q]
  float* slice_o;                 // [B][H_q][splits][64] sums
  float2* slice_ml;               // [B][H_q][splits]: maximum (log2 units), sum
  __nv_bfloat16* out;             // [B][H_q][64]
  float* lse;                     // [H_q][B] (natural log)
  int* err;
  int batch, heads_q, heads_kv;
  int page_size, num_pages, max_pages, count, num_groups;
  int splits;
  int whole;                      // a single slice, joined where it is computed
  int log2_page;                  // TMA path: log2(page_size)
  float scale_log2;               // softmax_scale * log2(e)
#ifdef ATTN_SINK_TEST_HOOKS
  int skip_k_tile;
#endif
};

// Page sizes that are copied by TMA: whole 128-byte swizzle atoms of 8 keys, and blocks
// that are whole pages or parts of one.
__host__ __device__ constexpr bool slice_tma_page(int page_size) {
  return page_size >= 8 && (page_size & (page_size - 1)) == 0;
}

__device__ __forceinline__ int slice_seq_len(const int* seq_lens, int b, int cap) {
  return max(0, min(__ldg(seq_lens + b), cap));
}

// The group of sequence b among [cu[p], cu[p + 1]), p < groups: p (groups: none), and its
// bounds; by a whole warp, of which every lane gets the answer.
struct SharedGroup {
  int at, first, end;
};
__device__ __forceinline__ SharedGroup shared_find(const int* cu, int groups, int b) {
  const int lane = threadIdx.x & 31;
  int lo = 0, span = groups + 1;             // the last p with cu[p] <= b is in [lo, lo + span)
  while (true) {
    const int step = (span + 30) / 31;       // 31 places, and one behind
    const int at = min(lo + lane * step, groups);
    const int v = __ldg(cu + at);
    const int i = max(0, 31 - __clz(__ballot_sync(0xffffffffu, lane * step < span && v <= b)));
    if (step == 1) {
      const int first = __shfl_sync(0xffffffffu, v, i), end = __shfl_sync(0xffffffffu, v, i + 1);
      return SharedGroup{lo + i, first, lo + i < groups ? end : first};
    }
    lo += i * step;
    span = min(step, span - i * step);
  }
}

// Keys that the group of sequence b reads together (see attn_sink_shared_plan_kernel);
// by a whole CTA, of which every thread gets the answer.
__device__ __forceinline__ int shared_prefix(const SliceParams& p, int b, int cap) {
  __shared__ int s_min[kSliceWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const SharedGroup group = shared_find(p.cu_groups, p.num_groups, b);
  const int c0 = max(0, group.first), c1 = min(p.batch, group.end);
  const int keys = group.at < p.num_groups ? __ldg(p.prefix_lens + group.at) : 0;
  int least = INT_MAX;
  for (int i = c0 + (int)threadIdx.x; i < c1; i += kSliceThreads)
    least = min(least, slice_seq_len(p.seq_lens, i, cap));
  least = __reduce_min_sync(0xffffffffu, least);
  if (lane == 0) s_min[warp] = least;
  __syncthreads();
  #pragma unroll
  for (int w = 0; w < kSliceWarps; ++w) least = min(least, s_min[w]);
  const int shared = min(keys, least);
  return c0 <= b && b < c1 && c1 - c0 >= kSharedMinSeqs && shared >= kSharedMinKeys ? shared : 0;
}

// G = query heads per kv head (1, 2, 4 or 8).
template <int G, bool kTma, bool kShared>
__global__ void __launch_bounds__(kSliceThreads, kSliceCtas)
attn_sink_slice_kernel(const __grid_constant__ SliceParams p) {
  extern __shared__ uint8_t slice_smem[];
  __shared__ __align__(8) uint64_t full[kSliceWarps][kSliceStages];   // TMA path: copies landed
  __shared__ uint32_t s_seen[kSliceWarps][kSliceStages];              // keys of the block to use
  __shared__ float s_m[kSliceWarps][8], s_l[kSliceWarps][8];
  grid_launch_dependents();
  const int split = blockIdx.x, g = blockIdx.y, b = blockIdx.z;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int gr = lane >> 2;          // fragment row = query head of the group
  const int t4 = lane & 3;           // fragment column pair
  // the warps' rings, and their O rows at the end
  uint8_t* const base = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(slice_smem) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* const ring = base + warp * (kSliceStages * kSliceStageBytes);
  float (*s_o)[8][64] = reinterpret_cast<float (*)[8][64]>(base);
  static_assert(sizeof(float) * kSliceWarps * 8 * 64 <= kSliceSmem - 1024, "O rows in the rings");

  const int l0 = __ldg(p.seq_lens + b), cap = p.max_pages * p.page_size;
  const int len = max(0, min(l0, cap));
  if (len != l0 && tid == 0) atomicCAS(p.err, 0, DEVERR_DECODE_INPUT);
  const int have = (len + p.page_size - 1) / p.page_size;   // pages of the sequence
  // keys [lo, end): of the sequence, or of the list of pages one after the other
  const int lo = kShared ? shared_prefix(p, b, cap) : 0;
  const int end = kShared ? len : min(p.count, have) * p.page_size;
  const int* listed = kShared ? nullptr : p.selected + ((size_t)b * p.heads_kv + g) * p.count;
  const int* table = p.block_table + (size_t)b * p.max_pages;
  const int lo_blk = lo & ~(kSliceKeys - 1);
  const int per = ((end - lo_blk + p.splits - 1) / p.splits + kSliceKeys - 1) & ~(kSliceKeys - 1);
  const int k0 = lo_blk + split * per;                      // this slice
  const int k1 = min(end, k0 + per);
  const int blocks = k1 > k0 ? (k1 - k0 + kSliceKeys - 1) / kSliceKeys : 0;
  const int n = blocks > warp ? (blocks - warp + kSliceWarps - 1) / kSliceWarps : 0;   // this warp's

  // The kernel in front computes the prefix at the same time.  This one has ended only
  // when that one has: where no CTA waits for the prefix, one waits here.
  auto leave = [&] {
    if (kShared && split == 0 && g == 0 && b == 0) grid_dependency_wait();
  };
  if (blocks == 0 && !p.whole) {                            // an empty slice
    if (tid < G)
      p.slice_ml[((size_t)b * p.heads_q + g * G + tid) * p.splits + split] =
          make_float2(-INFINITY, 0.0f);
    leave();
    return;
  }

  // Q as the A operand (rows >= G are zero): a0 = dims 16 kk + 2 t4 .. + 1, a2 = the same
  // + 8, of head row gr; a1 = a3 = 0 (rows 8..15)
  uint32_t qa0[4], qa2[4];
  #pragma unroll
  for (int kk = 0; kk < 4; ++kk) {
    qa0[kk] = 0u;
    qa2[kk] = 0u;
    if (gr < G) {
      const uint32_t* qp = reinterpret_cast<const uint32_t*>(
          p.q + ((size_t)b * p.heads_q + g * G + gr) * 64 + 16 * kk + 2 * t4);
      qa0[kk] = __ldg(qp);
      qa2[kk] = __ldg(qp + 4);
    }
  }

  // What a lane copies of a block: a box of 1 << log2_box keys by TMA (the first lanes), or a key
  // of which the warp's lanes copy 16 bytes each.
  const int log2_box = kTma ? min(p.log2_page, 5) : 0;
  const int box = 1 << log2_box;
  const bool mine = !kTma || lane < (kSliceKeys >> log2_box);
  auto at = [&](int i) { return k0 + (warp + kSliceWarps * i) * kSliceKeys + (lane << log2_box); };
  auto page_of = [&](int j) { return kTma ? j >> p.log2_page : j / p.page_size; };
  struct Copy {
    int entry, seen;                 // of the block table; how many of the keys are there
  };
  auto list = [&](int i) {           // the column of the block table; kNoKey: none
    const int j = at(i);
    if (!mine || i >= n || j >= k1 || j + box <= lo) return kNoKey;
    return kShared ? page_of(j) : __ldg(listed + page_of(j));
  };
  auto entry = [&](int i, int col) {
    if (col < 0) return Copy{kNoKey, 0};
    if (col >= have) return Copy{-1, 0};                    // behind the sequence: recorded
    const int j = at(i);
    const int first = kShared ? j : col * p.page_size + (j - page_of(j) * p.page_size);
    const int seen = min(max(len - first, 0), box);
    if (seen == 0) return Copy{kNoKey, 0};
    return Copy{max(-1, __ldg(table + col)), seen};
  };
  auto issue = [&](int i, int st, const Copy& e) {          // by the whole warp
    const int j = at(i);
    const bool ok = (unsigned)e.entry < (unsigned)p.num_pages;
    if (!ok && e.entry != kNoKey) atomicCAS(p.err, 0, DEVERR_DECODE_INPUT);
    uint32_t seen = ok ? (e.seen >= 32 ? 0xFFFFFFFFu : (1u << e.seen) - 1u) << (lane << log2_box) : 0u;
    if (kTma && !mine) seen = 0u;
    seen = __reduce_or_sync(0xffffffffu, seen);
    const int first = k0 + (warp + kSliceWarps * i) * kSliceKeys;
    if (first < lo) seen &= ~0u << (lo - first);            // less than a block
    if (first + kSliceKeys > k1) seen &= ~0u >> (first + kSliceKeys - k1);
    if (lane == 0) s_seen[warp][st] = seen;
    uint8_t* const dst = ring + st * kSliceStageBytes;
    const int off = j - page_of(j) * p.page_size;
    if (kTma) {
      const bool send = TEST_HOOK_FWD_ISSUE_K(i);
      if (lane == 0 && send) mbar_arrive_expect_tx(&full[warp][st], kSliceStageBytes);
      __syncwarp();
      if (mine && send) {
        const int row = ok ? e.entry * p.page_size + off : p.num_pages * p.page_size;   // zeros
        tma_load_3d(&p.tm_k, &full[warp][st], dst + (lane << log2_box) * 128, 0, g, row);
        tma_load_3d(&p.tm_v, &full[warp][st], dst + kSliceKeys * 128 + (lane << log2_box) * 128, 0, g,
                    row);
      }
    } else {
      const uint32_t row = ok ? ((uint32_t)e.entry * (uint32_t)p.page_size + (uint32_t)off) *
                                        (uint32_t)p.heads_kv + (uint32_t)g
                              : 0xFFFFFFFFu;
      #pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int r = 4 * u + (lane >> 3), c = lane & 7;
        const uint32_t x = __shfl_sync(0xffffffffu, row, r);
        const bool in = x != 0xFFFFFFFFu;                   // else nothing is read, 0 written
        const uint32_t to = smem_u32(dst) + sw128_offset((uint32_t)r, (uint32_t)c);
        cp_async_16_zfill(to, in ? p.k_cache + (size_t)x * 64 + 8 * c : p.q, in ? 16 : 0);
        cp_async_16_zfill(to + kSliceKeys * 128, in ? p.v_cache + (size_t)x * 64 + 8 * c : p.q,
                          in ? 16 : 0);
      }
    }
  };
  if (kTma) {
    if (lane == 0) {
      #pragma unroll
      for (int st = 0; st < kSliceStages; ++st) mbar_init(&full[warp][st], 1);
      fence_mbarrier_init();
    }
    __syncwarp();
  }
  Copy next;
  int col_next;
  int issued = min(n, kSliceStages);   // of this warp's blocks
  {
    int col[kSliceStages + 2];
    Copy c[kSliceStages + 1];
    #pragma unroll
    for (int i = 0; i < kSliceStages + 2; ++i) col[i] = list(i);
    #pragma unroll
    for (int i = 0; i < kSliceStages + 1; ++i) c[i] = entry(i, col[i]);
    #pragma unroll
    for (int i = 0; i < kSliceStages; ++i) {
      if (i < n) issue(i, i, c[i]);
      if (!kTma) cp_async_commit();
    }
    next = c[kSliceStages];
    col_next = col[kSliceStages + 1];
  }

  float m_r = -INFINITY;   // running max of head row gr (log2 units)
  float l_r = 0.0f;        // this thread's share of the row sum
  float oacc[8][4];        // O: n-tile nd = dims 8 nd ..; c0, c1: row gr with P hi, c2, c3: with P lo
  #pragma unroll
  for (int nd = 0; nd < 8; ++nd)
    #pragma unroll
    for (int e = 0; e < 4; ++e) oacc[nd][e] = 0.0f;
  const int mi = lane >> 3, ri = lane & 7;   // ldmatrix: matrix and row this lane addresses
  bool ok = true;
  for (int i = 0; i < n; ++i) {
    const int st = i % kSliceStages;
    if (kTma) {
      ok = mbar_wait_warp(&full[warp][st], (i / kSliceStages) & 1, nullptr);
      if (!ok) break;
    } else {
      cp_async_wait<kSliceStages - 1>();
    }
    __syncwarp();
    const uint32_t kt = smem_u32(ring + st * kSliceStageBytes), vt = kt + kSliceKeys * 128;
    const uint32_t seen = s_seen[warp][st];
    if (seen != 0xFFFFFFFFu) {
      // value rows that are not seen may hold anything, and 0 * inf is not 0
      for (int x = lane; x < kSliceKeys * 8; x += 32)
        if (!(seen >> (x >> 3) & 1u)) st_shared_v4(vt + (uint32_t)x * 16u, 0, 0, 0, 0);
      if (kTma) fence_proxy_async_smem();   // the stage's next copy comes through the async proxy
      __syncwarp();
    }
    // S = Q K^T, n-tiles of 8 keys; matrices of the x4 load: (keys +0, dims 16 kk), (keys +0,
    // dims +8), (keys +8, ...), (keys +8, +8)
    float sc[4][4];
    #pragma unroll
    for (int nt = 0; nt < 4; ++nt)
      #pragma unroll
      for (int e = 0; e < 4; ++e) sc[nt][e] = 0.0f;
    #pragma unroll
    for (int kk = 0; kk < 4; ++kk)
      #pragma unroll
      for (int half = 0; half < 2; ++half) {
        uint32_t b00, b01, b10, b11;
        ldmatrix_x4(kt + sw128_offset(16 * half + (mi >> 1) * 8 + ri, 2 * kk + (mi & 1)), b00, b01,
                    b10, b11);
        mma_16816_bf16(sc[2 * half], qa0[kk], 0u, qa2[kk], 0u, b00, b01);
        mma_16816_bf16(sc[2 * half + 1], qa0[kk], 0u, qa2[kk], 0u, b10, b11);
      }
    // online softmax of row gr over keys 8 nt + 2 t4 + e (log2 units)
    float x[4][2];
    float mx = -INFINITY;
    #pragma unroll
    for (int nt = 0; nt < 4; ++nt)
      #pragma unroll
      for (int e = 0; e < 2; ++e) x[nt][e] = sc[nt][e] * p.scale_log2;
    if (seen != 0xFFFFFFFFu) {
      #pragma unroll
      for (int nt = 0; nt < 4; ++nt)
        #pragma unroll
        for (int e = 0; e < 2; ++e)
          if (!(seen >> (8 * nt + 2 * t4 + e) & 1u)) x[nt][e] = -INFINITY;
    }
    #pragma unroll
    for (int nt = 0; nt < 4; ++nt) mx = fmax3(mx, x[nt][0], x[nt][1]);
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
    const float mn = fmaxf(m_r, mx);
    const float mb = (mn == -INFINITY) ? 0.0f : mn;
    if (__any_sync(0xffffffffu, mn != m_r)) {
      const float alpha = ex2_approx(m_r - mb);             // 0 while m is -inf
      l_r *= alpha;
      #pragma unroll
      for (int nd = 0; nd < 8; ++nd)
        #pragma unroll
        for (int e = 0; e < 4; ++e) oacc[nd][e] *= alpha;
      m_r = mn;
    }
    // P = hi + lo as the A operand: rows 0-7 hi, rows 8-15 lo; a0, a1 = keys 2 t4 .. + 1 of
    // 16, a2, a3 = keys 8 + 2 t4 .. + 1
    uint32_t hi[4], lo2[4];
    #pragma unroll
    for (int nt = 0; nt < 4; ++nt) {
      const float p0 = ex2_approx(x[nt][0] - mb), p1 = ex2_approx(x[nt][1] - mb);
      l_r += p0 + p1;
      hi[nt] = pack_bf16x2(p0, p1);
      lo2[nt] = pack_bf16x2(p0 - bf16_lo(hi[nt]), p1 - bf16_hi(hi[nt]));
    }
    // O += P V; transposed x4 load matrices: (keys +0, dims 16 u), (keys +8, dims 16 u), (keys
    // +0, dims +8), (keys +8, dims +8)
    #pragma unroll
    for (int half = 0; half < 2; ++half)
      #pragma unroll
      for (int u = 0; u < 4; ++u) {
        uint32_t v0, v1, v2, v3;
        ldmatrix_x4_trans(vt + sw128_offset(16 * half + (mi & 1) * 8 + ri, 2 * u + (mi >> 1)), v0,
                          v1, v2, v3);
        mma_16816_bf16(oacc[2 * u], hi[2 * half], lo2[2 * half], hi[2 * half + 1],
                       lo2[2 * half + 1], v0, v1);
        mma_16816_bf16(oacc[2 * u + 1], hi[2 * half], lo2[2 * half], hi[2 * half + 1],
                       lo2[2 * half + 1], v2, v3);
      }
    __syncwarp();                    // every lane is done with the stage before it is refilled
    if (i + kSliceStages < n) {
      issue(i + kSliceStages, st, next);
      issued = i + kSliceStages + 1;
      next = entry(i + kSliceStages + 1, col_next);
      col_next = list(i + kSliceStages + 2);
    }
    if (!kTma) cp_async_commit();
  }
  if (!kTma) cp_async_wait<0>();
  if (!__syncthreads_and(ok)) {
    // a copy that did not land within the wait limit: report it, give the copies in flight
    // time to land before the CTA releases its shared memory, and write nothing
    if (lane == 0 && !ok) {
      atomicCAS(p.err, 0, DEVERR_TIMEOUT_FWD + 0x18);
      for (int i = max(0, issued - kSliceStages); i < issued; ++i)
        mbar_wait(&full[warp][i % kSliceStages], (i / kSliceStages) & 1, nullptr);
    }
    __syncthreads();
    leave();
    return;
  }

  // the row sum over the 4 lanes of row gr, then the 4 warps' states joined
  l_r += __shfl_xor_sync(0xffffffffu, l_r, 1);
  l_r += __shfl_xor_sync(0xffffffffu, l_r, 2);
  if (t4 == 0) {
    s_m[warp][gr] = m_r;
    s_l[warp][gr] = l_r;
  }
  // hi is above zero where P is, lo of any sign: an infinite value is infinite in hi's sum,
  // and may be NaN or the other infinity in lo's
  auto both = [](float hi, float lo) { return isinf(hi) ? hi : hi + lo; };
  #pragma unroll
  for (int nd = 0; nd < 8; ++nd)
    *reinterpret_cast<float2*>(&s_o[warp][gr][8 * nd + 2 * t4]) =
        make_float2(both(oacc[nd][0], oacc[nd][2]), both(oacc[nd][1], oacc[nd][3]));
  __syncthreads();
  // thread t: head t / 16, dims 4 (t % 16) .. + 4
  const int h = tid >> 4;
  const int d0 = 4 * (tid & 15);
  const bool whole = p.whole != 0;
  if (kShared && whole) grid_dependency_wait();             // the prefix
  if (h < G) {
    float mm = -INFINITY;
    #pragma unroll
    for (int w = 0; w < kSliceWarps; ++w) mm = fmaxf(mm, s_m[w][h]);
    const int hq = g * G + h;
    const size_t row = (size_t)b * p.heads_q + hq;
    const float s2 = whole ? __ldg(p.sink + hq) * kLog2e : -INFINITY;
    // the parts of the prefix: a tile's rows apart
    int parts = 0;
    const float2* ml = nullptr;
    const float* po = nullptr;
    const size_t pstep = (size_t)p.heads_kv * kBlockM;
    if (kShared && whole && lo > 0) {
      const int4 r = __ldcg(reinterpret_cast<const int4*>(p.refs + b));   // a SharedRef
      const size_t to = ((size_t)r.x * p.heads_kv + g) * kBlockM + r.z * G + h;
      parts = r.y;
      ml = p.prefix_ml + to;
      po = p.prefix_o + to * 64 + d0;
      #pragma unroll 8
      for (int i = 0; i < parts; ++i) mm = fmaxf(mm, __ldcg(ml + i * pstep).x);
    }
    const float mf = fmaxf(mm, s2);
    const float mb = mf == -INFINITY ? 0.0f : mf;
    float z = 0.0f, acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    #pragma unroll
    for (int w = 0; w < kSliceWarps; ++w) {
      const float wt = ex2_approx(s_m[w][h] - mb);          // NaN sums reach the result
      z = fmaf(wt, s_l[w][h], z);
      const float4 o = *reinterpret_cast<const float4*>(&s_o[w][h][d0]);
      acc[0] = fmaf(wt, o.x, acc[0]);
      acc[1] = fmaf(wt, o.y, acc[1]);
      acc[2] = fmaf(wt, o.z, acc[2]);
      acc[3] = fmaf(wt, o.w, acc[3]);
    }
    if (kShared && whole) {
      #pragma unroll 4
      for (int i = 0; i < parts; ++i) {
        const float2 x = __ldcg(ml + i * pstep);
        const float4 o = __ldcg(reinterpret_cast<const float4*>(po + i * pstep * 64));
        const float wt = ex2_approx(x.x - mb);
        if (wt != 0.0f) {                                   // an empty part has stored no sums
          z = fmaf(wt, x.y, z);
          acc[0] = fmaf(wt, o.x, acc[0]);
          acc[1] = fmaf(wt, o.y, acc[1]);
          acc[2] = fmaf(wt, o.z, acc[2]);
          acc[3] = fmaf(wt, o.w, acc[3]);
        }
      }
    }
    if (whole) {
      z += s2 == mb ? 1.0f : ex2_approx(s2 - mb);           // 1 where both are inf
      const float inv = z != 0.0f ? 1.0f / z : 0.0f;
      *reinterpret_cast<uint2*>(p.out + row * 64 + d0) = make_uint2(
          pack_bf16x2(acc[0] * inv, acc[1] * inv), pack_bf16x2(acc[2] * inv, acc[3] * inv));
      if (d0 == 0)
        p.lse[(size_t)hq * p.batch + b] = z != 0.0f ? (mb + __log2f(z)) * kLn2 : -INFINITY;
    } else {
      const size_t to = row * p.splits + split;
      *reinterpret_cast<float4*>(p.slice_o + to * 64 + d0) =
          make_float4(acc[0], acc[1], acc[2], acc[3]);
      if (d0 == 0) p.slice_ml[to] = make_float2(mf, z);
    }
  }
  leave();
}

// ----------------------------------------------------------------------------- join
// Joins the slices, the parts of a shared prefix and the sink, in a fixed order:
//   M = max(m_c, sink), Z = sum l_c 2^(m_c - M) + 2^(sink - M), O = sum 2^(m_c - M) o_c / Z.
// A warp takes a row (sequence, query head): 16 lanes of 4 dimensions for the even
// slices, 16 for the odd ones.  It costs the chain of its loads, so the sums of 16 slices
// go out together, before their weights are known.  A kernel of its own, launched
// while the slices are computed: counting the slices and letting the last CTA of a row
// join them takes a memory fence in every CTA and the counters' clearing in front.
constexpr int kJoinThreads = 128;
constexpr int kJoinParts = 128;       // slices (up to 64) and prefix parts (up to 64)

template <bool kShared>
__global__ void __launch_bounds__(kJoinThreads)
attn_sink_join_kernel(const __grid_constant__ SliceParams p) {
  const int lane = threadIdx.x & 31, odd = lane >> 4, d = 4 * (lane & 15);
  const unsigned row = blockIdx.x * (kJoinThreads / 32) + (threadIdx.x >> 5);
  const unsigned b = row / (unsigned)p.heads_q;
  const int hq = (int)(row - b * (unsigned)p.heads_q);
  const bool in = b < (unsigned)p.batch;
  const float s2 = in ? __ldg(p.sink + hq) * kLog2e : 0.0f;
  grid_dependency_wait();
  if (!in) return;
  // part c: slice c, then the prefix's parts, whose rows lie a tile's rows apart
  int parts = p.splits;
  const float2* ml = p.slice_ml + (size_t)row * p.splits;
  const float* o = p.slice_o + (size_t)row * p.splits * 64 + d;
  const float2* pml = nullptr;
  const float* po = nullptr;
  const size_t pstep = (size_t)p.heads_kv * kBlockM;
  if constexpr (kShared) {
    const int4 r = __ldcg(reinterpret_cast<const int4*>(p.refs + b));     // a SharedRef
    const int group = p.heads_q / p.heads_kv, g = hq / group;
    const size_t at = ((size_t)r.x * p.heads_kv + g) * kBlockM + r.z * group + (hq - g * group);
    parts += r.y;
    pml = p.prefix_ml + at - (size_t)p.splits * pstep;
    po = p.prefix_o + at * 64 + d - (size_t)p.splits * pstep * 64;
  }
  auto load = [&](int c) {
    const float* src = kShared && c >= p.splits ? po + (size_t)c * pstep * 64 : o + (size_t)c * 64;
    return c < parts ? __ldcg(reinterpret_cast<const float4*>(src))
                     : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  };
  constexpr int kEach = (kShared ? kJoinParts : kJoinParts / 2) / 32;
  float2 x[kEach];                         // of parts lane, lane + 32, ..
  #pragma unroll
  for (int u = 0; u < kEach; ++u) {
    const int c = lane + 32 * u;
    const float2* src = kShared && c >= p.splits ? pml + (size_t)c * pstep : ml + c;
    x[u] = c < parts ? __ldcg(src) : make_float2(-INFINITY, 0.0f);
  }
  float4 v[8];
  #pragma unroll
  for (int u = 0; u < 8; ++u) v[u] = load(2 * u + odd);
  float m = s2;
  #pragma unroll
  for (int u = 0; u < kEach; ++u) m = fmaxf(m, x[u].x);
  #pragma unroll
  for (int k = 16; k > 0; k >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, k));
  const float mb = m == -INFINITY ? 0.0f : m;
  float w[kEach], z = 0.0f;
  #pragma unroll
  for (int u = 0; u < kEach; ++u) {
    w[u] = ex2_approx(x[u].x - mb);        // 0: an empty part
    z = fmaf(x[u].y, w[u], z);
  }
  #pragma unroll
  for (int k = 16; k > 0; k >>= 1) z += __shfl_xor_sync(0xffffffffu, z, k);
  z += s2 == mb ? 1.0f : ex2_approx(s2 - mb);               // 1 where both are inf
  float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  for (int c = 0; c < parts; c += 16) {
    float mine = w[0];
    #pragma unroll
    for (int u = 1; u < kEach; ++u) mine = c >= 32 * u ? w[u] : mine;
    #pragma unroll
    for (int u = 0; u < 8; ++u) {
      const float wk = __shfl_sync(0xffffffffu, mine, (c + 2 * u + odd) & 31);
      if (wk != 0.0f) {                    // an empty part has stored no sums
        acc.x = fmaf(v[u].x, wk, acc.x);
        acc.y = fmaf(v[u].y, wk, acc.y);
        acc.z = fmaf(v[u].z, wk, acc.z);
        acc.w = fmaf(v[u].w, wk, acc.w);
      }
    }
    if (c + 16 < parts)
      #pragma unroll
      for (int u = 0; u < 8; ++u) v[u] = load(c + 16 + 2 * u + odd);
  }
  acc.x += __shfl_xor_sync(0xffffffffu, acc.x, 16);
  acc.y += __shfl_xor_sync(0xffffffffu, acc.y, 16);
  acc.z += __shfl_xor_sync(0xffffffffu, acc.z, 16);
  acc.w += __shfl_xor_sync(0xffffffffu, acc.w, 16);
  const float inv = z != 0.0f ? 1.0f / z : 0.0f;            // NaN for a NaN score
  if (odd == 0)
    *reinterpret_cast<uint2*>(p.out + (size_t)row * 64 + d) = make_uint2(
        pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
  if (lane == 0)
    p.lse[(size_t)hq * p.batch + b] = z != 0.0f ? (mb + __log2f(z)) * kLn2 : -INFINITY;
}

}  // namespace attn_sink
