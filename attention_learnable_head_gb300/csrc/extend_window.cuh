// Windowed attention of several new tokens over a paged cache, on the band kernel
// (fwd_band_kernel.cuh): one product covers a tile's whole window there, and its
// persistent CTAs overlap tiles, where the general kernel of extend_kernel.cuh
// spends 17000 cycles on the two 128-key blocks of a window of 128.
//
// The band kernel reads packed keys and values, so the keys that a sequence's new
// tokens see (n + W - 1 of them at most) are first gathered from their pages:
// K as it is, V as fp16 (as the forward does with v).  Regions of zero rows lie
// between the sequences, so that the band kernel's boxes, which reach beyond a
// sequence's keys, find zeros there and nothing of another sequence.  A schedule
// kernel of one CTA lays out the regions and lists every tile as a sequence of
// its own for the band kernel: its queries and the keys that they see, bottom-right
// aligned.  Where a block-table entry is outside the cache the gather says so, and the
// band kernel masks the keys of such entries.
#pragma once
#include "extend_kernel.cuh"
#include "fwd_band_kernel.cuh"

namespace attn_sink {

constexpr int kGatherThreads = 256;
constexpr int kGatherPad = kBandMaxCols;   // zero rows before, between and behind the sequences

struct GatherRegion {
  int base, first, rows, pad;              // first gathered row; its key; keys; zero rows behind
};

struct GatherParams {
  ExtParams e;                             // lengths, tables, cache, window
  int4* spans;                             // [max_tiles], see FwdBandParams
  GatherRegion* regions;                   // [B]
  __nv_bfloat16* k;                        // [rows][H_kv][64]
  uint16_t* v;                             // the same, fp16
  int* any_lost;                           // is there a key without a page?
  int max_tiles;
  long long rows;                          // of k and v
};

__global__ void __launch_bounds__(kExtSchedThreads, 1)
attn_sink_gather_plan_kernel(const __grid_constant__ GatherParams g) {
  __shared__ int s_scan[kExtSchedThreads / 32];
  grid_launch_dependents();
  const ExtParams& p = g.e;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  bool bad = false;
  if (tid == 0) *g.any_lost = 0;
  int row0 = kGatherPad, tile0 = 0;        // of the sequences before this round
  for (int b0 = 0; b0 < p.batch; b0 += kExtSchedThreads) {
    const int b = b0 + 32 * lane + warp;   // neighbours go to different warps
    ExtSeq s{0, 0, 0};
    int tiles = 0, first = 0, rows = 0;
    if (b < p.batch) {
      s = ext_seq(p, b, &bad);
      tiles = (s.n + p.tokens - 1) / p.tokens;
      if (tiles > 0) {
        first = ext_tile(p, s, 0).lo;
        rows = max(0, s.len - first);
      }
    }
    int all_r, all_t;
    const int base = row0 + ext_scan(tiles > 0 ? rows + kGatherPad : 0, s_scan, &all_r);
    const int tile = tile0 + ext_scan(tiles, s_scan, &all_t);
    row0 += all_r;
    tile0 += all_t;
    if (b < p.batch)
      g.regions[b] = GatherRegion{base, first, rows, tiles > 0 ? kGatherPad : 0};
    for (unsigned todo = __ballot_sync(0xffffffffu, tiles > 0); todo; todo &= todo - 1) {
      const int l = __ffs(todo) - 1;
      ExtSeq x;
      x.q0 = __shfl_sync(0xffffffffu, s.q0, l);
      x.n = __shfl_sync(0xffffffffu, s.n, l);
      x.len = __shfl_sync(0xffffffffu, s.len, l);
      const int nt = __shfl_sync(0xffffffffu, tiles, l), at = __shfl_sync(0xffffffffu, tile, l);
      const int shift = __shfl_sync(0xffffffffu, base - first, l);
      const int seq = b0 + 32 * l + warp;
      for (int t = lane; t < nt; t += 32) {
        const ExtTile e = ext_tile(p, x, t);
        const int n = min(p.tokens, x.n - t * p.tokens);       // < 128
        const int lo = min(e.lo, e.hi);    // no key: an empty span; kBandMaxCols keys at most
        // more tiles than fit are only listed by a cu_seqlens that descends
        if ((unsigned)(at + t) < (unsigned)g.max_tiles)
          g.spans[at + t] =
              make_int4(x.q0 + t * p.tokens, lo + shift, (e.hi - lo) << 8 | n, seq);
      }
    }
  }
  if (bad) atomicCAS(p.err, 0, DEVERR_DECODE_INPUT);
  for (int t = max(tile0, 0) + tid; t < g.max_tiles; t += kExtSchedThreads)
    g.spans[t] = make_int4(0, 0, 0, 0);
}

// A thread copies 16 bytes of K and of V of a row.  Bound by the latency of the table
// entries and rows behind them: 8 sequences of 513 + 127 keys, 8 heads, 6.5 us.
__global__ void __launch_bounds__(kGatherThreads)
attn_sink_gather_kernel(const __grid_constant__ GatherParams g) {
  grid_dependency_wait();
  grid_launch_dependents();
  const ExtParams& p = g.e;
  const int per = p.heads_kv * 8;          // chunks of a row
  bool over = false, lost = false;
  auto put = [&](long long row, int c, uint4 k, uint4 v) {
    // a cu_seqlens that descends (recorded) may want more rows than there are
    if ((unsigned long long)row >= (unsigned long long)g.rows) return;
    const size_t at = ((size_t)row * per + c) * 8;
    *reinterpret_cast<uint4*>(g.k + at) = k;
    *reinterpret_cast<uint4*>(g.v + at) = v;
  };
  const uint4 zero = make_uint4(0, 0, 0, 0);
  if (blockIdx.y == 0)                     // before the first sequence
    for (int u = blockIdx.x * kGatherThreads + threadIdx.x; u < kGatherPad * per;
         u += gridDim.x * kGatherThreads)
      put(u / per, u % per, zero, zero);
  for (int b = blockIdx.y; b < p.batch; b += gridDim.y) {
    const int4 r = *reinterpret_cast<const int4*>(g.regions + b);
    if (r.w == 0) continue;
    const int* table = p.block_table + (size_t)b * p.max_pages;
    const long long units = ((long long)r.z + r.w) * per;
    for (long long u = blockIdx.x * kGatherThreads + threadIdx.x; u < units;
         u += (long long)gridDim.x * kGatherThreads) {
      const int i = (int)(u / per), c = (int)(u - (long long)i * per);
      uint4 k = zero, v = zero;
      if (i < r.z) {
        const int j = r.y + i, pg = j / p.page_size;
        const int e = __ldg(table + pg);
        if (e >= 0 && e < p.num_pages) {
          const size_t src = (((size_t)e * p.page_size + (j - pg * p.page_size)) * per + c) * 8;
          k = *reinterpret_cast<const uint4*>(p.k_cache + src);
          v = *reinterpret_cast<const uint4*>(p.v_cache + src);
          v.x = bf16x2_to_f16x2(v.x, &over);
          v.y = bf16x2_to_f16x2(v.y, &over);
          v.z = bf16x2_to_f16x2(v.z, &over);
          v.w = bf16x2_to_f16x2(v.w, &over);
        } else {
          lost = true;
        }
      }
      put((long long)r.x + i, c, k, v);
    }
  }
  if (lost) {
    *g.any_lost = 1;
    atomicCAS(p.err, 0, DEVERR_DECODE_INPUT);
  }
  if (over) atomicCAS(p.err, 0, DEVERR_FP16_RANGE);
}

}  // namespace attn_sink
