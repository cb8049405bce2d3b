// The prefix of groups of sequences in a decode step, sm_103a: the keys that a
// group's sequences share are read once for all of them.
//
// A tile is T = floor(128 / G) consecutive sequences of a group times the G query
// heads of one kv head: their new tokens' rows lie next to each other in q, so the
// tile is a tile of attn_sink_extend_kernel whose tokens all see the whole prefix,
// and that kernel computes it, with P as two bf16 (ext_split: with one, as for a prompt's
// tokens, outputs were off by 0.0023 of their norm, of which 0.0017 is their own rounding; the
// second costs 18 us of the larger call below, 0.4 of the smaller): it leaves each part's
// maximum, sum and unnormalised output in the workspace.  The keys behind the prefix are
// each sequence's own; attn_sink_slice_kernel reads them, at the same time, and a last
// kernel joins everything with the sink (slice_kernel.cuh).
//
// This schedule kernel of one CTA lists the tiles' parts.  Their keys are cut so that
// rounds of CTAs times what the longest takes is least, over chunks of kSharedTries sizes
// from an even share of all blocks on (three prompts of 4608 to 8192 keys, 192 samples, 64
// heads on 8, P as one bf16: 38 us, 556 TFLOP/s, bound by the chain of a tile's softmax; cut by
// the even share itself, 1.2 rounds, 52 us).  With 512 to 1024 own keys each the call takes
// 118 us: own keys and prefix share the SMs, whose registers hold two CTAs of the one or three
// of the other.  8 sequences of 200 own keys behind 1024: 13.5 us, three dependent kernels.
// Groups of one sequence and short prefixes have none (kSharedMinSeqs, kSharedMinKeys): their
// sequences read all keys themselves.
#pragma once
#include "extend_kernel.cuh"
#include "slice_kernel.cuh"

namespace attn_sink {

constexpr int kSharedWarps = 32;
constexpr int kSharedTries = 32;
constexpr int kSharedListed = 1024;      // groups up to which sizes are tried
constexpr int kSharedMinBlocks = 1;      // key blocks of a part

struct SharedPlan {
  ExtParams e;                             // batch, heads, cache, items, slots
  const int* cu_groups;                    // [num_groups + 1]
  const int* prefix_lens;                  // [num_groups]
  SharedRef* refs;                         // [B]
  int num_groups;
};

__global__ void __launch_bounds__(32 * kSharedWarps, 1)
attn_sink_shared_plan_kernel(const __grid_constant__ SharedPlan p) {
  __shared__ int s_scan[32];
  __shared__ unsigned long long s_work, s_best;
  __shared__ int s_tiles[kSharedListed], s_blocks[kSharedListed];
  __shared__ int s_first[kSharedListed], s_end[kSharedListed], s_keys[kSharedListed];
  grid_launch_dependents();
  const ExtParams& e = p.e;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cap = e.max_pages * e.page_size;
  if (tid == 0) {
    s_work = 0;
    s_best = ~0ull;
  }
  // a sequence that no group has keeps this
  for (int b = tid; b < e.batch; b += 32 * kSharedWarps) p.refs[b] = SharedRef{0, 0, 0, 0};
  __syncthreads();
  bool bad = false;
  // The keys that group i reads together, and its sequences [c0, c1); by a whole warp.
  auto group = [&](int i, int* c0, int* c1) {
    const int a0 = __ldg(p.cu_groups + i), a1 = __ldg(p.cu_groups + i + 1);
    const int keys = __ldg(p.prefix_lens + i);
    *c0 = max(0, a0);
    *c1 = min(e.batch, a1);
    bad |= a0 < 0 || a1 > e.batch || a1 < a0 || keys < 0 || (i == 0 && a0 != 0) ||
           (i == p.num_groups - 1 && a1 != e.batch);
    int least = INT_MAX;
    for (int b = *c0 + lane; b < *c1; b += 32) {
      const int len = __ldg(e.seq_lens + b);
      bad |= len < 0 || len > cap;
      least = min(least, max(0, min(len, cap)));
    }
    least = __reduce_min_sync(0xffffffffu, least);
    const int shared = min(keys, least);
    return *c1 - *c0 >= kSharedMinSeqs && shared >= kSharedMinKeys ? shared : 0;
  };
  // all tiles' blocks of keys: what a slot's share is
  unsigned long long work = 0;
  for (int i = warp; i < p.num_groups; i += kSharedWarps) {
    int c0, c1;
    const int keys = group(i, &c0, &c1);
    const int tiles = keys > 0 ? (c1 - c0 + e.tokens - 1) / e.tokens : 0;
    const int blocks = (keys + kBlockN - 1) / kBlockN;
    work += (unsigned long long)tiles * (unsigned)blocks;
    if (lane == 0 && i < kSharedListed) {
      s_tiles[i] = tiles;
      s_blocks[i] = blocks;
      s_first[i] = c0;
      s_end[i] = c1;
      s_keys[i] = keys;
    }
  }
  if (lane == 0 && work > 0) atomicAdd(&s_work, work);      // whole numbers: any order
  if (bad) atomicCAS(e.err, 0, DEVERR_DECODE_INPUT);
  __syncthreads();
  const unsigned long long all = s_work * (unsigned)e.heads_kv;
  const unsigned long long share = (all + (unsigned)e.slots - 1) / (unsigned)e.slots;
  int chunk = (int)min(max(share, (unsigned long long)kSharedMinBlocks), 1ull << 20);
  if (p.num_groups <= kSharedListed) {
    // warp i tries the share times (16 + i) / 16
    const int c = max(chunk, (int)min((share * (16 + warp) + 15) / 16, 1ull << 20));
    unsigned ctas = 0;
    int longest = 0;
    for (int i = lane; i < p.num_groups; i += 32)
      if (s_tiles[i] > 0) {
        const int parts = ext_parts(s_blocks[i], c);
        ctas += (unsigned)s_tiles[i] * (unsigned)parts;
        longest = max(longest, (s_blocks[i] + parts - 1) / parts);
      }
    ctas = __reduce_add_sync(0xffffffffu, ctas) * (unsigned)e.heads_kv;   // a launch grid
    longest = __reduce_max_sync(0xffffffffu, longest);
    const unsigned long long rounds = (ctas + (unsigned)e.slots - 1) / (unsigned)e.slots;
    if (lane == 0)
      atomicMin(&s_best, rounds * (unsigned)(longest + kExtOver) << 21 | (unsigned)c);
    __syncthreads();
    chunk = (int)(s_best & ((1u << 21) - 1));
  }
  // the items of 32 groups at a time, one group a warp
  int listed = 0;
  bool over = false;                       // more than the workspace holds: no valid cu_groups
  for (int i0 = 0; i0 < p.num_groups; i0 += kSharedWarps) {
    const int i = i0 + warp;
    int c0 = 0, c1 = 0, keys = 0;
    if (i < p.num_groups && p.num_groups > kSharedListed) {
      keys = group(i, &c0, &c1);
    } else if (i < p.num_groups) {
      c0 = s_first[i];
      c1 = s_end[i];
      keys = s_keys[i];
    }
    const int blocks = (keys + kBlockN - 1) / kBlockN;
    const int tiles = keys > 0 ? (c1 - c0 + e.tokens - 1) / e.tokens : 0;
    const int parts = keys > 0 ? ext_parts(blocks, chunk) : 0;
    __syncthreads();                       // the last round's counts have been read
    if (lane == 0) s_scan[warp] = tiles * parts;
    __syncthreads();
    const int mine = s_scan[lane];
    int upto = mine;
    #pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, upto, d);
      if (lane >= d) upto += y;
    }
    const int first = listed + __shfl_sync(0xffffffffu, upto - mine, warp);
    listed += __shfl_sync(0xffffffffu, upto, 31);           // 32 groups: below 2^31
    over = listed > e.n_items;             // never where cu_groups ascends: recorded
    if (over) break;
    for (int x = lane; x < tiles * parts; x += 32) {
      const int tile = x / parts, part = x - tile * parts;
      const int per = (blocks + parts - 1) / parts, skip = min(blocks, part * per);
      ExtItem it;
      it.num = min(per, blocks - skip);
      it.blk0 = skip;
      it.seq = c0;                         // whose block-table row the keys are read through
      it.row0 = c0 + tile * e.tokens;
      it.lo = 0;
      it.hi = keys;
      it.mlo = 0;
      it.mhi = keys / kBlockN - skip;      // the last block may hold keys behind the prefix
      it.rows = min(e.tokens, c1 - it.row0) * e.group;
      it.at0 = 1 << 30;                    // every row sees them all
      it.split = part << 16 | max(parts, 2);   // one part, too, leaves its sums
      it.first = first + tile * parts;
      const uint4* src = reinterpret_cast<const uint4*>(&it);
      uint4* dst = reinterpret_cast<uint4*>(e.items + first + x);
      dst[0] = src[0];
      dst[1] = src[1];
      dst[2] = src[2];
    }
    for (int b = c0 + lane; b < c1; b += 32)
      p.refs[b] = keys > 0 ? SharedRef{first + (b - c0) / e.tokens * parts, parts,
                                       (b - c0) % e.tokens, 0}
                           : SharedRef{0, 0, 0, 0};
  }
  if (over) {                              // the same for every thread
    __syncthreads();
    for (int b = tid; b < e.batch; b += 32 * kSharedWarps) p.refs[b] = SharedRef{0, 0, 0, 0};
  }
  for (int x = (over ? 0 : listed) + tid; x < e.n_items; x += 32 * kSharedWarps)
    e.items[x].num = -1;
}

}  // namespace attn_sink
