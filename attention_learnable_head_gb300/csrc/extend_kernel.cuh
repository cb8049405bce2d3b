// Attention with a per-head sink of several new tokens per sequence over a
// paged key/value cache, sm_103a (tcgen05 + TMA): chunks of prompts on cached
// prefixes, drafted tokens, long conversations.
//
// Rows.  A tile is T = floor(128 / G) consecutive tokens of a sequence times
// the G query heads of one kv head (row = token * G + head, the order [tokens]
// [heads][64] stores them, so one TMA box loads Q): 128 rows of the matrix
// product that all read the same keys, where a tile of one head would fill
// only as many rows as there are new tokens.
//
// Keys.  Blocks of 128 keys, copied page by page through the block table into
// 128-byte-swizzled shared memory.  Where the page size is a multiple of 8 one
// warp issues TMA boxes of as many keys as divide both the page and the block
// (a box without a needed key is read past the tensor, which fills zeros);
// other page sizes are copied 16 bytes a lane with cp.async.  (32 sequences of
// up to 8192 keys: 86 us in boxes of 64 keys, 90 of 16, 97 of 8, and 120 key by
// key, where the warp issues 64 copies a block.)
//
// Work items.  A schedule kernel of one CTA lists (sequence, tile, key range)
// in the workspace; the hardware hands them out, each to one CTA per kv head
// (which go through the same keys at the same time: each reads 128 bytes of a
// cache row that holds them all).  Tiles with more keys than an even share of
// the launch's work are split, so that a long cache with few new tokens fills
// the GPU; the parts leave fp32 sums in the workspace and a third kernel joins
// them and adds the sink.  The three are chained by programmatic dependent
// launch.  Where the table or the window leaves a tile too few keys for a cut to
// pay there is no join, and few CTAs of up to 128 sequences need no schedule either:
// each finds its tile (5 new tokens on 10 keys: 7.5 us, 14.4 with all three).
//
// The rest is the forward kernel's pipeline: S = Q K^T into TMEM, online
// softmax by two warpgroups (one per key half), P to TMEM, O += P V with P
// read from TMEM, lazy rescaling.  P is rounded to bf16, not fp16: the cache
// holds bf16 values, and an fp16 product would need every value tile converted
// by each CTA; one more rounding of 2^-8 next to that of the bf16 output.  The
// row sums add the fp32 probabilities.
//
// With full tiles a CTA's chain bounds it, 2400 clocks per 128 keys (S from TMEM 300,
// maximum and its exchange 550, 64 exponentials a thread and P 1300, waits 250), two
// CTAs an SM: 4 sequences of 8192 to 16384 keys with up to 1024 new tokens, 64 + 8
// heads, take 760 us, 835 TFLOP/s.  With few tokens the cache does: 32 sequences of
// 4096 to 8192 keys with up to 5 new tokens 91 us (393 MB, 58 us at the copy rate), 5
// of them each for the schedule and the join.
#pragma once
#include <climits>
#include "fwd_kernel.cuh"

namespace attn_sink {

constexpr int kExtThreads = 320;           // 8 softmax warps, copy warp, MMA warp
constexpr int kExtMaxGroup = 128;
constexpr int kExtMaxSplits = 64;          // parts of a tile
constexpr int kExtMinBlocks = 4;           // key blocks of a part
constexpr int kExtFindMax = 128;           // sequences of a single launch
constexpr int kExtTries = 24;              // candidates for the cut, up to 3 rounds of CTAs
constexpr int kExtOver = 5;                // what a CTA costs beside its blocks, in blocks
constexpr int kExtSchedThreads = 1024;
constexpr int kExtJoinThreads = 256;
constexpr int kExtJoinCtas = 4;            // resident CTAs per SM of the join

// One CTA's work for each kv head: a tile, or a range of its key blocks.
struct alignas(16) ExtItem {
  int num, blk0, seq, row0;                // blocks (-1: unused entry); first block; sequence;
  int lo, hi, mlo, mhi;                    // first row of q; keys the tile sees; blocks [mlo, mhi)
  int rows, at0, split, first;             // that need no mask; rows with a token; key position of
};                                         // the first token; part << 16 | parts; first partial
static_assert(sizeof(ExtItem) == 48, "three 16-byte loads");

// A tile whose parts are to be joined.
struct ExtTileRef {
  int first, parts, rows, row0;            // first partial result; rows with a token; row of q
};

struct ExtParams {
  CUtensorMap tm_q;        // [T][H_q][64] bf16, box 64 x G x tokens per tile
  CUtensorMap tm_out;
  CUtensorMap tm_k;        // cache as [rows][H_kv][64], box 64 x 1 x box
  CUtensorMap tm_v;
  const __nv_bfloat16* k_cache;
  const __nv_bfloat16* v_cache;
  const int* block_table;  // [B][max_pages]
  const int* seq_lens;     // [B]
  const int* cu_q;         // [B + 1]
  const float* sink;       // [H_q]
  __nv_bfloat16* out;      // [T][H_q][64]
  float* lse;              // [H_q][T]
  ExtItem* items;          // null: see ext_find
  float* o_part;           // [partial][kv head][128 rows][64]
  float2* ml_part;         // [partial][kv head][128 rows]: maximum (log2 units), sum
  ExtTileRef* tiles;       // tiles that are split, for the join
  int2* n_tiles;           // how many, and the rows of the largest
  int* err;
  int batch, total_q, heads_q, heads_kv, group, tokens;
  int page_size, num_pages, max_pages, window;
  int box;                 // keys of a TMA box (0: cp.async copies)
  int n_items, max_parts, max_tiles;   // sizes of items, partial results, tiles
  int slots;               // CTAs the GPU holds at once
  float scale_log2;
#ifdef ATTN_SINK_TEST_HOOKS
  int skip_k_tile;
#endif
};

// A sequence's span: rows [q0, q0 + n) of q, L cached keys (clamped to what
// the arrays hold).
struct ExtSeq {
  int q0, n, len;
};

__device__ __forceinline__ ExtSeq ext_seq(const ExtParams& p, int b, bool* bad) {
  const int c0 = __ldg(p.cu_q + b), c1 = __ldg(p.cu_q + b + 1), len = __ldg(p.seq_lens + b);
  ExtSeq s;
  s.q0 = min(max(c0, 0), p.total_q);
  s.n = max(0, min(c1, p.total_q) - s.q0);
  s.len = min(max(len, 0), p.max_pages * p.page_size);
  *bad |= s.q0 != c0 || s.q0 + s.n != c1 || s.len != len;
  return s;
}

// Keys [lo, hi) that tile `t` of the sequence sees, and their blocks.
struct ExtTile {
  int lo, hi, blocks;
};
__device__ __forceinline__ ExtTile ext_tile(const ExtParams& p, const ExtSeq& s, int t) {
  const int i0 = t * p.tokens, i1 = min(i0 + p.tokens, s.n) - 1;
  const int off = s.len - s.n;             // key position of token 0
  ExtTile x;
  x.hi = max(0, min(s.len, i1 + off + 1));
  x.lo = p.window > 0 ? max(0, i0 + off - p.window + 1) : 0;
  x.blocks = x.hi > x.lo ? (x.hi + kBlockN - 1) / kBlockN - x.lo / kBlockN : 0;
  return x;
}

// Part `part` of `np` of a tile; `first`: the tile's first partial result.
__device__ __forceinline__ ExtItem ext_item(const ExtParams& p, const ExtSeq& s, int seq, int tile,
                                            int part, int np, int first) {
  const ExtTile e = ext_tile(p, s, tile);
  const int i0 = tile * p.tokens, i1 = min(i0 + p.tokens, s.n) - 1, off = s.len - s.n;
  const int per = (e.blocks + np - 1) / np, skip = min(e.blocks, part * per);
  ExtItem it;
  it.num = min(per, e.blocks - skip);
  it.blk0 = e.lo / kBlockN + skip;
  it.seq = seq;
  it.row0 = s.q0 + i0;
  it.lo = e.lo;
  it.hi = e.hi;
  // blocks before mlo hold keys behind some token's window, blocks from mhi on
  // keys after some token
  const int lost = i1 + off - p.window;    // last key some token has lost
  it.mlo = p.window > 0 && lost >= 0 ? lost / kBlockN + 1 - it.blk0 : 0;
  it.mhi = max(0, min(s.len, i0 + off + 1)) / kBlockN - it.blk0;
  it.rows = (i1 - i0 + 1) * p.group;
  it.at0 = i0 + off;
  it.split = part << 16 | np;
  it.first = first;
  return it;
}

// Without a list (items null: up to kExtFindMax sequences, tiles that are not cut):
// item i is the i-th tile of the batch, found by every warp for itself.  A lane
// holds up to four neighbouring sequences.
__device__ __forceinline__ ExtItem ext_find(const ExtParams& p, int i, bool record) {
  const int lane = threadIdx.x & 31;
  const int each = (p.batch + 31) >> 5;
  static_assert(kExtFindMax == 4 * 32, "four sequences a lane");
  bool bad = false;
  ExtSeq s[4];
  // < 2^30 tiles each; sums stay there too: for a cu_seqlens that ascends they do by
  // themselves, others have been recorded
  int tiles = 0, before[4];
  #pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int b = lane * each + u;
    s[u] = ExtSeq{0, 0, 0};
    if (u < each && b < p.batch) s[u] = ext_seq(p, b, &bad);
  }
  #pragma unroll
  for (int u = 0; u < 4; ++u) {
    before[u] = tiles;
    tiles = min(tiles + (s[u].n + p.tokens - 1) / p.tokens, 1 << 30);
  }
  if (bad && record) atomicCAS(p.err, 0, DEVERR_DECODE_INPUT);
  int upto = tiles;
  #pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, upto, d);
    if (lane >= d) upto = (int)min((unsigned)upto + (unsigned)y, 1u << 30);
  }
  const unsigned after = __ballot_sync(0xffffffffu, upto > i);
  ExtItem it;
  it.num = -1;
  if (after == 0) return it;
  const int who = __ffs(after) - 1;
  const int j = i - __shfl_sync(0xffffffffu, upto - tiles, who);   // tile of that lane's
  int u = 0;
  #pragma unroll
  for (int v = 1; v < 4; ++v)
    if (__shfl_sync(0xffffffffu, before[v], who) <= j &&
        __shfl_sync(0xffffffffu, s[v].n, who) > 0)
      u = v;
  ExtSeq x{0, 0, 0};
  int tile = 0;
  #pragma unroll
  for (int v = 0; v < 4; ++v) {
    const int q0 = __shfl_sync(0xffffffffu, s[v].q0, who);
    const int n = __shfl_sync(0xffffffffu, s[v].n, who);
    const int len = __shfl_sync(0xffffffffu, s[v].len, who);
    const int at = __shfl_sync(0xffffffffu, before[v], who);
    if (v == u) {
      x = ExtSeq{q0, n, len};
      tile = j - at;
    }
  }
  if ((long long)tile * p.tokens >= x.n) return it;        // sums that were cut off
  return ext_item(p, x, who * each + u, tile, 0, 1, 0);
}

// Parts of a tile of `blocks` blocks, of at least c blocks each (rounded up).
__device__ __forceinline__ int ext_parts(int blocks, int c) {
  return min(kExtMaxSplits, max(1, (blocks + c - 1) / c));
}

// Exclusive scan of the block's values; *all receives their sum.
__device__ __forceinline__ int ext_scan(int x, int* s_warp, int* all) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int inc = x;
  #pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, inc, d);
    if (lane >= d) inc += y;
  }
  __syncthreads();                         // the last scan's sums have been read
  if (lane == 31) s_warp[warp] = inc;
  __syncthreads();
  // every warp scans the 32 warps' sums
  int sum = s_warp[lane];
  #pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, sum, d);
    if (lane >= d) sum += y;
  }
  *all = __shfl_sync(0xffffffffu, sum, 31);
  const int before = __shfl_sync(0xffffffffu, sum, max(warp - 1, 0));
  return (warp > 0 ? before : 0) + inc - x;
}

// Exclusive scans of three values a thread, in one pass; all[i] receives the sums.
__device__ __forceinline__ void ext_scan3(int (&x)[3], int (*s_warp)[32], int (&all)[3]) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int inc[3], sum[3];
  #pragma unroll
  for (int i = 0; i < 3; ++i) inc[i] = x[i];
  #pragma unroll
  for (int d = 1; d < 32; d <<= 1)
    #pragma unroll
    for (int i = 0; i < 3; ++i) {
      const int y = __shfl_up_sync(0xffffffffu, inc[i], d);
      if (lane >= d) inc[i] += y;
    }
  __syncthreads();                         // the last round's sums have been read
  if (lane == 31)
    #pragma unroll
    for (int i = 0; i < 3; ++i) s_warp[i][warp] = inc[i];
  __syncthreads();
  #pragma unroll
  for (int i = 0; i < 3; ++i) sum[i] = s_warp[i][lane];
  #pragma unroll
  for (int d = 1; d < 32; d <<= 1)
    #pragma unroll
    for (int i = 0; i < 3; ++i) {
      const int y = __shfl_up_sync(0xffffffffu, sum[i], d);
      if (lane >= d) sum[i] += y;
    }
  #pragma unroll
  for (int i = 0; i < 3; ++i) {
    all[i] = __shfl_sync(0xffffffffu, sum[i], 31);
    const int before = __shfl_sync(0xffffffffu, sum[i], max(warp - 1, 0));
    x[i] = (warp > 0 ? before : 0) + inc[i] - x[i];
  }
}

// Lists the work items.  With W the key blocks of all tiles (each taken as long
// as its sequence's last) times the kv heads, a tile is cut into ceil(blocks / c)
// parts.  Candidates for c spread W over 1/8, 2/8, .. 3 times the CTAs the GPU
// holds at once (slots); the first leaves whole what a slot's share would not
// cut.  Taken is the one with the least ceil(CTAs / slots) * (blocks of the
// longest part + kExtOver): rounds of CTAs, and what a CTA costs beside its
// blocks.  (With c = W / slots, W / (2 slots) or no cut alone, 32 sequences of
// 4096 to 8192 keys and 5 new tokens fill 2.2 rounds and take 104 us.)  That
// makes tiles + 3 slots / H_kv items at most.  A thread takes a sequence, later
// an item, whose sequence it finds by bisection of the scanned counts: 5 us in
// front of the tiles (7 with a warp per sequence and a scan for each count).
__global__ void __launch_bounds__(kExtSchedThreads, 1)
attn_sink_extend_plan_kernel(const __grid_constant__ ExtParams p) {
  __shared__ int s_scan[3][32];
  __shared__ unsigned long long s_work;
  __shared__ int s_tiles[kExtSchedThreads], s_blocks[kExtSchedThreads];
  __shared__ int s_item[kExtSchedThreads], s_part[kExtSchedThreads], s_split[kExtSchedThreads];
  __shared__ ExtSeq s_seq[kExtSchedThreads];
  __shared__ unsigned long long s_cost[kExtTries];
  __shared__ int s_chunk[kExtTries], s_rows;
  static_assert(kExtTries <= 32 && kExtSchedThreads == 1024, "a warp per candidate");
  grid_launch_dependents();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  bool bad = false;
  ExtSeq s{0, 0, 0};
  int tiles = 0, blocks = 0;               // of the sequence; of its last tile
  auto load = [&](int b) {
    s = ExtSeq{0, 0, 0};
    tiles = blocks = 0;
    if (b >= p.batch) return;
    s = ext_seq(p, b, &bad);
    tiles = (s.n + p.tokens - 1) / p.tokens;
    if (tiles > 0) blocks = ext_tile(p, s, tiles - 1).blocks;
  };
  if (tid == 0) {
    s_work = 0;
    s_rows = 0;
  }
  __syncthreads();
  unsigned long long w = 0;
  for (int b0 = 0; b0 < p.batch; b0 += kExtSchedThreads) {
    load(b0 + tid);
    w += (unsigned long long)tiles * (unsigned)blocks;
  }
  if (bad) atomicCAS(p.err, 0, DEVERR_DECODE_INPUT);
  if (__any_sync(0xffffffffu, w > 0)) {
    #pragma unroll
    for (int d = 16; d > 0; d >>= 1) w += __shfl_xor_sync(0xffffffffu, w, d);
    if (lane == 0) atomicAdd(&s_work, w);                  // whole numbers: any order
  }
  s_tiles[tid] = tiles;                    // of the last (mostly the only) round
  s_blocks[tid] = blocks;
  __syncthreads();
  int chunk = 1 << 24;                     // > any tile's blocks
  if (p.max_parts > 0) {
    // warp i tries candidate i; with several rounds of sequences they go through
    // shared memory again
    const unsigned long long per = s_work * (unsigned)p.heads_kv;
    const unsigned share = (unsigned)(warp + 1) * (unsigned)p.slots;
    const int c = 8 * per < (1ull << 31)   // the division of 64 bits takes 0.3 us
                      ? max((int)(((unsigned)(8 * per) + share - 1) / share), kExtMinBlocks)
                      : (int)min((8 * per + share - 1) / share, 1ull << 24);   // > any tile's
    unsigned long long ctas = 0;
    int longest = 0;
    for (int b0 = 0; b0 < p.batch; b0 += kExtSchedThreads) {
      if (p.batch > kExtSchedThreads) {
        load(b0 + tid);
        __syncthreads();                   // the last round's have been read
        s_tiles[tid] = tiles;
        s_blocks[tid] = blocks;
        __syncthreads();
      }
      if (warp >= kExtTries) continue;
      for (int i = lane; i < min(kExtSchedThreads, p.batch - b0); i += 32) {
        const int n = s_blocks[i];
        if (s_tiles[i] == 0) continue;
        const int k = ext_parts(n, c);
        ctas += (unsigned long long)s_tiles[i] * (unsigned)k;
        longest = max(longest, (n + k - 1) / k);
      }
    }
    if (warp < kExtTries) {
      #pragma unroll
      for (int d = 16; d > 0; d >>= 1) ctas += __shfl_xor_sync(0xffffffffu, ctas, d);
      longest = __reduce_max_sync(0xffffffffu, longest);
      if (lane == 0) {
        // the grid is below 2^31 CTAs, more of them are a cu_seqlens that does not ascend
        const unsigned all = (unsigned)min(ctas * (unsigned)p.heads_kv, 1ull << 31);
        s_cost[warp] = (unsigned long long)((all + (unsigned)p.slots - 1) / (unsigned)p.slots) *
                       (unsigned)(longest + kExtOver);
        s_chunk[warp] = c;
      }
    }
    __syncthreads();
    unsigned long long cost = lane < kExtTries ? s_cost[lane] : ~0ull;
    int best = lane;
    #pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
      const unsigned long long other = __shfl_xor_sync(0xffffffffu, cost, d);
      const int who = __shfl_xor_sync(0xffffffffu, best, d);
      if (other < cost || (other == cost && who < best)) {
        cost = other;
        best = who;
      }
    }
    chunk = s_chunk[best];
  }

  int done = 0, part0 = 0, split0 = 0;     // items listed; partial results, split tiles so far
  bool over = false;                       // more than the workspace holds: no valid cu_seqlens
  for (int b0 = 0; b0 < p.batch; b0 += kExtSchedThreads) {
    if (p.batch > kExtSchedThreads) load(b0 + tid);        // else still at hand
    const int parts = tiles > 0 ? ext_parts(blocks, chunk) : 0;
    int at[3] = {tiles * parts, parts > 1 ? tiles * parts : 0, parts > 1 ? tiles : 0}, all[3];
    const int rows = parts > 1 ? min(s.n, p.tokens) * p.group : 0;
    const int most = __reduce_max_sync(0xffffffffu, rows);
    if (lane == 0 && most > 0) atomicMax(&s_rows, most);
    ext_scan3(at, s_scan, all);            // and its barriers: the last round has been written
    s_item[tid] = at[0];
    s_part[tid] = part0 + at[1];
    s_split[tid] = split0 + at[2];
    s_tiles[tid] = tiles;
    s_blocks[tid] = parts;
    s_seq[tid] = s;
    __syncthreads();
    over = all[0] < 0 || all[0] > p.n_items - done || all[1] < 0 ||
           all[1] > p.max_parts - part0 || all[2] < 0 || all[2] > p.max_tiles - split0;
    if (over) break;
    for (int k = tid; k < all[0]; k += kExtSchedThreads) {
      int i = 0;                           // the last sequence that starts at or before k
      #pragma unroll
      for (int d = kExtSchedThreads / 2; d > 0; d >>= 1)
        if (s_item[i + d] <= k) i += d;
      const ExtSeq x = s_seq[i];
      const int np = max(s_blocks[i], 1), nt = s_tiles[i], j = k - s_item[i];
      const int up = j / np, tile = nt - 1 - up, part = j - up * np;   // the longest tiles first
      ExtItem it;
      it.num = -1;
      if ((unsigned)tile < (unsigned)nt) {                 // else sums that wrapped round
        it = ext_item(p, x, b0 + i, tile, part, np, s_part[i] + up * np);
        // for every cu_seqlens that ascends the bounds hold; one that does not has
        // been recorded
        if (np > 1 && (unsigned)it.first > (unsigned)(p.max_parts - np)) it.num = -1;
        if (np > 1 && part == 0 && (unsigned)(s_split[i] + up) < (unsigned)p.max_tiles)
          p.tiles[s_split[i] + up] =
              ExtTileRef{it.first, it.num < 0 ? 0 : np, it.num < 0 ? 0 : it.rows, it.row0};
      }
      const uint4* src = reinterpret_cast<const uint4*>(&it);
      uint4* dst = reinterpret_cast<uint4*>(p.items + done + k);
      dst[0] = src[0];
      dst[1] = src[1];
      dst[2] = src[2];
    }
    done += all[0];
    part0 += all[1];
    split0 += all[2];
  }
  // over: uniform, as the sums are
  for (int k = (over ? 0 : done) + tid; k < p.n_items; k += kExtSchedThreads) p.items[k].num = -1;
  if (tid == 0) *p.n_tiles = over ? make_int2(0, 0) : make_int2(split0, s_rows);
}

// The sink's term 2^(s - m) of a row sum, s <= m; 1 where both are inf.
__device__ __forceinline__ float ext_sink(float s, float m) {
  return s == m ? 1.0f : ex2_approx(s - m);
}

// The bits below bit n of a word.
__device__ __forceinline__ uint32_t ext_below(int n) {
  return n >= 32 ? 0xFFFFFFFFu : n <= 0 ? 0u : (1u << n) - 1u;
}

// Two bf16 each whose sums are p0 and p1 to 2^-14 of them: the upper 8 bits, and the rest of
// (1 + 2^-17) p.  Both are above zero where p is, so that an infinite value stays one (a rest
// of p itself may be zero, one of a rounded first negative: 0 * inf is not 0).
__device__ __forceinline__ void ext_split(float p0, float p1, uint32_t* first, uint32_t* second) {
  const uint32_t w0 = __float_as_uint(p0), w1 = __float_as_uint(p1);
  *first = __byte_perm(w0, w1, 0x7632);
  const uint64_t rest = ffma2(f2(p0, p1), f2(1.0f + 0x1p-17f, 1.0f + 0x1p-17f),
                              f2(__uint_as_float((w0 & 0xFFFF0000u) | 0x80000000u),
                                 __uint_as_float((w1 & 0xFFFF0000u) | 0x80000000u)));
  *second = pack_bf16x2(f2_lo(rest), f2_hi(rest));
}

// kTwo: P as the sum of two bf16 (ext_split), the second in the columns of the scores, which
// the threads have read: O += P_2 v comes first, then the next block's scores, then O += P_1 v.
// A CTA waits longer for its scores, which the tiles of shared prefixes take on
// (shared_kernel.cuh): one token a sequence is asked for as exactly as by attn_sink_decode.
template <bool kTma, bool kTwo = false>
__global__ void __maxnreg__(96)
attn_sink_extend_kernel(const __grid_constant__ ExtParams p) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t q_full, mma_drained;
  __shared__ __align__(8) uint64_t k_full[kFwdKStages], k_empty[kFwdKStages];
  __shared__ __align__(8) uint64_t v_full[kFwdVStages], v_empty[kFwdVStages];
  __shared__ __align__(8) uint64_t s_full, s_free, p_full, pv_done, low_done;
  __shared__ uint32_t tmem_base_sh;
  __shared__ volatile int abort_flag;
  __shared__ float s_mx[2][2][kBlockM];
  __shared__ float s_red_l[2][kBlockM];
  __shared__ int s_at[kBlockM];            // key position of a row's token
  __shared__ int s_lo, s_hi, s_bad;        // keys of the tile; some page is missing

  const int item = (int)(blockIdx.x / (unsigned)p.heads_kv);
  const int g = (int)(blockIdx.x - (unsigned)item * (unsigned)p.heads_kv);
  uint4 d0, d1, d2;                                       // an ExtItem
  if (p.items != nullptr) {
    const uint4* desc = reinterpret_cast<const uint4*>(p.items + item);
    grid_dependency_wait();
    grid_launch_dependents();
    d0 = __ldcg(desc);
    d1 = __ldcg(desc + 1);
    d2 = __ldcg(desc + 2);
  } else {
    const ExtItem it = ext_find(p, item, blockIdx.x == 0 && threadIdx.x < 32);
    const uint4* desc = reinterpret_cast<const uint4*>(&it);
    d0 = desc[0];
    d1 = desc[1];
    d2 = desc[2];
  }
  const int num = (int)d0.x, blk0 = (int)d0.y, row0 = (int)d0.w;
  if (num < 0) return;                                    // uniform per CTA
  const int lo = (int)d1.x, hi = (int)d1.y, mlo0 = (int)d1.z, mhi0 = (int)d1.w;
  const int rows = (int)d2.x;                             // rows that hold a token
  const int part = (int)(d2.z >> 16), parts = (int)(d2.z & 0xFFFFu), first = (int)d2.w;
  const int row_warps = (rows + 31) / 32;                 // the other rows' warps only wait
  const int tid = threadIdx.x;
  const int warp = tid >> 5, lane = tid & 31;
  const size_t pidx = (size_t)(first + part) * p.heads_kv + g;   // this CTA's partial result
  const int* table = p.block_table + (size_t)d0.z * p.max_pages;

  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* sQ = smem;
  uint8_t* sK = sQ + kTileBytes;
  uint8_t* sV = sK + kFwdKStages * kTileBytes;

  if (num > 0) {
    // The copy warp's first table entries, on their way while the CTA sets up.
    // Lanes 0-15 copy the K boxes of a block, lanes 16-31 know the V boxes; each
    // holds the table entry of its next box, loaded one block ahead.
    const int half = lane >> 4, ci = lane & 15;
    int ent = -1, in_page = 0;
    auto fetch = [&](int n) {
      const int j = (blk0 + n) * kBlockN + ci * p.box;
      ent = -1;
      if (ci * p.box < kBlockN && n < num && j < hi && j + p.box > lo) {
        const int pg = j / p.page_size;
        in_page = j - pg * p.page_size;
        ent = __ldg(table + pg);
      }
    };
    if (kTma && warp == kFwdTmaWarp) fetch(0);
    if (tid == 0) {
      abort_flag = 0;
      mbar_init(&q_full, 1);
      mbar_init(&mma_drained, 1);
      for (int s = 0; s < kFwdKStages; ++s) {
        mbar_init(&k_full[s], kTma ? 1 : 32);
        mbar_init(&k_empty[s], 1);
      }
      for (int s = 0; s < kFwdVStages; ++s) {
        mbar_init(&v_full[s], kTma ? 1 : 32);
        mbar_init(&v_empty[s], 1);
      }
      mbar_init(&s_full, 1);
      mbar_init(&s_free, 64 * row_warps);
      mbar_init(&p_full, 64 * row_warps);
      mbar_init(&pv_done, 1);
      if (kTwo) mbar_init(&low_done, 1);
      fence_mbarrier_init();
      s_lo = lo;
      s_hi = hi;
    }
    if (tid < kBlockM) s_at[tid] = (int)d2.y + tid / p.group;
    if (warp == kFwdMmaWarp) {
      tmem_alloc(&tmem_base_sh, kFwdTmemCols);
      tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_base_sh;

    if (warp == kFwdTmaWarp) {
      // -------------------------------------------------------------- copies
      const uint32_t q_bytes = (uint32_t)(p.tokens * p.group) * 128u;
      if (lane == 0) {
        tma_prefetch_desc(&p.tm_q);
        mbar_arrive_expect_tx(&q_full, q_bytes);
        tma_load_3d(&p.tm_q, &q_full, sQ, 0, g * p.group, row0);
      }
      __syncwarp();
      if (kTma) {
        const bool mine = ci < kBlockN / p.box;
        // cache row of the fetched box; past the tensor (zero fill) without a page
        auto row = [&]() {
          return (unsigned)ent < (unsigned)p.num_pages ? ent * p.page_size + in_page
                                                       : p.num_pages * p.page_size;
        };
        const uint64_t keep = l2_policy_evict_last();
        int nk = 0, nv = 0;
        unsigned long long t_last = global_timer_ns();
        bool ok = true;
        while (nk < num || nv < num) {
          // one lane's answer for the warp: the lanes issue together
          bool can_k = false, can_v = false;
          if (lane == 0) {
            can_k = nk < num && TEST_HOOK_FWD_ISSUE_K(nk) &&
                    (nk < kFwdKStages || mbar_test_wait(smem_u32(&k_empty[nk % kFwdKStages]),
                                                        ((nk / kFwdKStages) & 1) ^ 1));
            can_v = nv < nk + (can_k ? 1 : 0) && nv < num &&
                    (nv < kFwdVStages || mbar_test_wait(smem_u32(&v_empty[nv % kFwdVStages]),
                                                        ((nv / kFwdVStages) & 1) ^ 1));
            if (can_k) mbar_arrive_expect_tx(&k_full[nk % kFwdKStages], kTileBytes);
            if (can_v) mbar_arrive_expect_tx(&v_full[nv % kFwdVStages], kTileBytes);
          }
          __syncwarp();
          can_k = __shfl_sync(0xffffffffu, can_k, 0);
          can_v = __shfl_sync(0xffffffffu, can_v, 0);
          if (can_k) {
            if (half == 0) {
              const int st = nk % kFwdKStages;
              if (mine)
                tma_load_3d_hint(&p.tm_k, &k_full[st], sK + st * kTileBytes + ci * p.box * 128, 0,
                                 g, row(), keep);
              fetch(nk + 1);
            }
            ++nk;
          }
          if (can_v) {
            if (half == 1) {
              const int st = nv % kFwdVStages;
              if (mine)
                tma_load_3d_hint(&p.tm_v, &v_full[st], sV + st * kTileBytes + ci * p.box * 128, 0,
                                 g, row(), keep);
              fetch(nv + 1);
            }
            ++nv;
          }
          if (can_k || can_v) {
            t_last = global_timer_ns();
          } else {
            const bool stop = abort_flag || global_timer_ns() - t_last > kWaitLimitNs;
            if (__any_sync(0xffffffffu, stop)) {
              ok = false;
              break;
            }
            __nanosleep(32);
          }
        }
        if (!ok && lane == 0) {
          abort_flag = 1;
          atomicCAS(p.err, 0, DEVERR_TIMEOUT_FWD + 6);
          // let the copies in flight land before the CTA releases its SMEM
          mbar_wait(&q_full, 0, nullptr);
          for (int it = max(0, nk - kFwdKStages); it < nk; ++it)
            mbar_wait(&k_full[it % kFwdKStages], (it / kFwdKStages) & 1, nullptr);
          for (int it = max(0, nv - kFwdVStages); it < nv; ++it)
            mbar_wait(&v_full[it % kFwdVStages], (it / kFwdVStages) & 1, nullptr);
        }
        __syncwarp();
      } else {
        // Loads x = 0, 1, 2, ...: K(0), V(0), K(1), V(1), ...; load x is handed
        // over (landed, fenced for the async proxy, arrived on) once load x + 2
        // has been issued.
        auto hand_over = [&](int x) {
          fence_proxy_async_smem();
          const int n = x >> 1;
          mbar_arrive((x & 1) ? &v_full[n % kFwdVStages] : &k_full[n % kFwdKStages]);
        };
        // Lane l holds the cache rows (128-byte units) of keys l, l + 32, .. of a
        // block, and all lanes which keys have one; the table entries of the next
        // block are on their way meanwhile.
        uint32_t at[4], has[4];
        bool all = true;
        int pg_e[4], pg_at[4];
        auto entries = [&](int n) {
          #pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int j = (blk0 + n) * kBlockN + 32 * i + lane;
            pg_e[i] = -1;
            if (n < num && j >= lo && j < hi) {
              const int pg = j / p.page_size;
              pg_at[i] = j - pg * p.page_size;
              pg_e[i] = __ldg(table + pg);
            }
          }
        };
        entries(0);
        bool ok = true;
        int x = 0;
        for (; x < 2 * num; ++x) {
          const int n = x >> 1;
          const bool is_v = x & 1;
          if (!is_v && !TEST_HOOK_FWD_ISSUE_K(n)) {
            ok = false;
            break;
          }
          if (!is_v) {
            all = true;
            #pragma unroll
            for (int i = 0; i < 4; ++i) {
              const bool in = (unsigned)pg_e[i] < (unsigned)p.num_pages;
              at[i] = in ? ((uint32_t)pg_e[i] * (uint32_t)p.page_size + (uint32_t)pg_at[i]) *
                                   (uint32_t)p.heads_kv + (uint32_t)g
                         : 0;
              has[i] = __ballot_sync(0xffffffffu, in);
              all = all && has[i] == 0xffffffffu;
            }
            entries(n + 1);
          }
          if (is_v ? n >= kFwdVStages : n >= kFwdKStages) {
            uint64_t* e = is_v ? &v_empty[n % kFwdVStages] : &k_empty[n % kFwdKStages];
            const int par = is_v ? ((n / kFwdVStages) & 1) ^ 1 : ((n / kFwdKStages) & 1) ^ 1;
            if (!mbar_wait_warp(e, par, &abort_flag)) {
              ok = false;
              break;
            }
          }
          const uint32_t dst = smem_u32(is_v ? sV + (n % kFwdVStages) * kTileBytes
                                             : sK + (n % kFwdKStages) * kTileBytes);
          const int c = lane & 7;
          const __nv_bfloat16* cache = (is_v ? p.v_cache : p.k_cache) + 8 * c;
          if (all) {
            #pragma unroll
            for (int i = 0; i < 4; ++i)
              #pragma unroll
              for (int u = 0; u < 8; ++u) {
                const int r = 4 * u + (lane >> 3);
                const uint32_t row = __shfl_sync(0xffffffffu, at[i], r);
                cp_async_16_zfill(dst + sw128_offset((uint32_t)(32 * i + r), (uint32_t)c),
                                  cache + (size_t)row * 64, 16);
              }
          } else {
            #pragma unroll
            for (int i = 0; i < 4; ++i)
              #pragma unroll 2
              for (int u = 0; u < 8; ++u) {
                const int r = 4 * u + (lane >> 3);
                const uint32_t row = __shfl_sync(0xffffffffu, at[i], r);
                const bool in = has[i] >> r & 1u;           // else nothing is read, 0 written
                cp_async_16_zfill(dst + sw128_offset((uint32_t)(32 * i + r), (uint32_t)c),
                                  in ? (const void*)(cache + (size_t)row * 64)
                                     : (const void*)p.out,
                                  in ? 16u : 0u);
              }
          }
          cp_async_commit();
          if (x >= 2) {
            cp_async_wait<2>();
            hand_over(x - 2);
          }
        }
        cp_async_wait<0>();
        if (ok) {
          for (int y = max(0, x - 2); y < x; ++y) hand_over(y);
        } else if (lane == 0) {
          abort_flag = 1;
          atomicCAS(p.err, 0, DEVERR_TIMEOUT_FWD + 6);
          mbar_wait(&q_full, 0, nullptr);
        }
        __syncwarp();
      }
    } else if (warp == kFwdMmaWarp) {
      // -------------------------------------------------------------- MMA issuer
      // As in the forward kernel: S(n + 1) before PV(n).
      if (lane == 0) {
        const uint32_t idesc_s = make_idesc_bf16(kBlockM, kBlockN, false, false);
        const uint32_t idesc_o = make_idesc_bf16(kBlockM, kHeadDim, false, true);
        const uint64_t dQ = make_sdesc_sw128(smem_u32(sQ), 16, 1024);
        const uint64_t dK0 = make_sdesc_sw128(smem_u32(sK), 16, 1024);
        const uint64_t dV0 = make_sdesc_sw128(smem_u32(sV), 16384, 1024);   // MN-major
        constexpr uint32_t kTileU = kTileBytes >> 4;
        auto issue_s = [&](int n) -> bool {
          const int st = n % kFwdKStages;
          if (!mbar_wait(&k_full[st], (n / kFwdKStages) & 1, &abort_flag)) return false;
          tc_fence_after();
          #pragma unroll
          for (int k = 0; k < kHeadDim / 16; ++k)
            mma_ss(tmem + kFwdColS, dQ + 2 * k, dK0 + st * kTileU + 2 * k, idesc_s, k > 0);
          mma_commit(&s_full);
          mma_commit(&k_empty[st]);
          return true;
        };
        bool ok = mbar_wait(&q_full, 0, &abort_flag) && issue_s(0);
        for (int n = 0; ok && n < num; ++n) {
          if (!kTwo && n + 1 < num) {
            if (!mbar_wait(&s_free, n & 1, &abort_flag) || !issue_s(n + 1)) {
              ok = false;
              break;
            }
          }
          const int sv = n % kFwdVStages;
          if (!mbar_wait(&v_full[sv], (n / kFwdVStages) & 1, &abort_flag) ||
              !mbar_wait(&p_full, n & 1, &abort_flag)) {
            ok = false;
            break;
          }
          tc_fence_after();
          if constexpr (kTwo) {
            #pragma unroll
            for (int k = 0; k < kBlockN / 16; ++k)
              mma_ts(tmem + kFwdColO, tmem + kFwdColS + 64 * (k >> 2) + 8 * (k & 3),
                     dV0 + sv * kTileU + 128 * k, idesc_o, (n > 0 || k > 0));
            mma_commit(&low_done);
            if (n + 1 < num && (!mbar_wait(&low_done, n & 1, &abort_flag) || !issue_s(n + 1))) {
              ok = false;
              break;
            }
          }
          #pragma unroll
          for (int k = 0; k < kBlockN / 16; ++k)
            mma_ts(tmem + kFwdColO, tmem + kFwdColP + 8 * k, dV0 + sv * kTileU + 128 * k, idesc_o,
                   (kTwo || n > 0 || k > 0));
          mma_commit(&pv_done);
          mma_commit(&v_empty[sv]);
        }
        if (!ok) {
          abort_flag = 1;
          atomicCAS(p.err, 0, DEVERR_TIMEOUT_FWD + 7);
        }
        // every MMA issued above has finished before TMEM is released
        mma_commit(&mma_drained);
        mbar_wait(&mma_drained, 0, nullptr);
      }
    } else {
      // -------------------------------------------------------------- softmax warps
      // Key half c = warp / 4; thread = row = TMEM lane.  Warps whose rows hold no
      // token go straight to the end.
      const int c = warp >> 2;
      const int r = tid & 127;
      const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
      const uint32_t tS = tmem + kFwdColS + 64 * c + lane_base;
      const uint32_t tP = tmem + kFwdColP + 32 * c + lane_base;
      const uint32_t tO = tmem + kFwdColO + 32 * c + lane_base;
      const bool working = (warp & 3) < row_warps;
      // Does every page of these keys lie in the cache?  (Rarely not: then every
      // block is masked, and the entries of its keys are looked up one by one.)
      bool bad_page = false;
      {
        const int k0 = max(lo, blk0 * kBlockN), k1 = min(hi, (blk0 + num) * kBlockN);
        const int pg1 = (k1 - 1) / p.page_size;
        for (int pg = k0 / p.page_size + tid; pg <= pg1; pg += 2 * kBlockM) {
          const int e = __ldg(table + pg);
          bad_page |= e < 0 || e >= p.num_pages;
        }
      }
      bad_page = !named_barrier_and(1, 2 * kBlockM, !bad_page);
      s_bad = bad_page;                                     // by every thread, for itself
      if (bad_page && tid == 0) atomicCAS(p.err, 0, DEVERR_DECODE_INPUT);
      float m = -INFINITY, l = 0.0f;
      const float sl2 = p.scale_log2;
      const uint64_t sl2x2 = f2(sl2, sl2);
      // Blocks before mlo hold keys behind some token's window, blocks from mhi on
      // keys after some token; with a missing page every block is masked.
      int mlo = 0, mhi = 0;
      if (!bad_page) {
        mlo = mlo0;
        mhi = mhi0;
      }
      bool ok = true;
      for (int it = 0; working && it < num; ++it) {
        uint32_t a[64];
        bool got = mbar_wait_warp(&s_full, it & 1, &abort_flag);
        float mx_half = -INFINITY;
        if (got) {
          tc_fence_after();
          tmem_ld_x32(tS, a);
          tmem_ld_x32(tS + 32, a + 32);
          tmem_ld_wait();
          tc_fence_before();
          mbar_arrive(&s_free);
          if (it < mlo || it >= mhi) {
            const int j0 = (blk0 + it) * kBlockN + 64 * c;  // first key of this half
            const int at = s_at[r];
            const int jmax = min(s_hi - 1, at) - j0;        // inclusive, within the half
            const int jmin = (p.window > 0 ? at - p.window + 1 : 0) - j0;
            // bit e: key e of the half is not seen (two words tested bit by bit cost
            // half of what two comparisons an element do)
            uint32_t w0 = ~(ext_below(jmax + 1) & ~ext_below(jmin));
            uint32_t w1 = ~(ext_below(jmax - 31) & ~ext_below(jmin - 32));
            if (s_bad) {                                    // keys without a page
              #pragma unroll 1
              for (int e = 0; e < 64; ++e) {
                const int j = j0 + e;
                if (j < s_lo || j >= s_hi) continue;
                const int pe = __ldg(table + j / p.page_size);
                if (pe >= 0 && pe < p.num_pages) continue;
                if (e < 32) w0 |= 1u << e;
                else w1 |= 1u << (e - 32);
              }
            }
            #pragma unroll
            for (int e = 0; e < 32; ++e) {
              if (w0 & (1u << e)) a[e] = __float_as_uint(-INFINITY);
              if (w1 & (1u << e)) a[32 + e] = __float_as_uint(-INFINITY);
            }
          }
          // row max over the 64 columns: four independent 3-input max chains
          float q0 = __uint_as_float(a[0]), q1 = __uint_as_float(a[1]);
          float q2 = __uint_as_float(a[2]), q3 = __uint_as_float(a[3]);
          #pragma unroll
          for (int e = 4; e < 64; e += 8) {
            q0 = fmax3(q0, __uint_as_float(a[e]), __uint_as_float(a[e + 1]));
            q1 = fmax3(q1, __uint_as_float(a[e + 2]), __uint_as_float(a[e + 3]));
            q2 = fmax3(q2, __uint_as_float(a[e + 4]), __uint_as_float(a[e + 5]));
            q3 = fmax3(q3, __uint_as_float(a[e + 6]), __uint_as_float(a[e + 7]));
          }
          mx_half = fmaxf(fmax3(q0, q1, q2), q3);
          s_mx[it & 1][c][r] = mx_half;
        }
        if (!named_barrier_and(2 + (warp & 3), 64, got && ok)) {
          ok = false;
          abort_flag = 1;
          break;
        }
        // The first and the last block may hold value rows that no token sees, and
        // those may hold anything: 0 * inf is not 0.
        if (it == 0 || it == num - 1) {
          const int jb = (blk0 + it) * kBlockN;
          if (jb < s_lo || jb + kBlockN > s_hi) {
            const int sv = it % kFwdVStages;
            if (mbar_wait_warp(&v_full[sv], (it / kFwdVStages) & 1, &abort_flag)) {
              const uint32_t base = smem_u32(sV + sv * kTileBytes);
              // 16-byte chunks over the 64 * row_warps threads
              for (int ch = 32 * (2 * (warp & 3) + c) + lane; ch < kBlockN * 8;
                   ch += 64 * row_warps) {
                const int j = jb + (ch >> 3);
                if (j < s_lo || j >= s_hi) st_shared_v4(base + (uint32_t)ch * 16u, 0, 0, 0, 0);
              }
              fence_proxy_async_smem();
            } else {
              ok = false;
            }
          }
        }
        const float mx = fmaxf(mx_half, s_mx[it & 1][c ^ 1][r]) * sl2;
        // lazy rescale: the max only moves when it grows by more than the threshold
        float alpha = 1.0f;
        if (mx > m + kRescaleThreshold || (m == -INFINITY && mx > -INFINITY)) {
          alpha = ex2_approx(m - mx);
          m = mx;
        }
        const float m_use = (m == -INFINITY) ? 0.0f : m;
        const uint64_t negm2 = f2(-m_use, -m_use);
        uint64_t rs = f2(0.0f, 0.0f);
        uint32_t pk[16];
        uint32_t low[8];                                    // kTwo: what pk leaves of P
        auto exponentials = [&](int at, int n) {            // of columns at .. at + n - 1
          #pragma unroll
          for (int e = 0; e < n; e += 2) {
            const uint64_t x = ffma2(f2(__uint_as_float(a[at + e]), __uint_as_float(a[at + e + 1])),
                                     sl2x2, negm2);
            const float e0 = ex2_approx(f2_lo(x));
            const float e1 = ex2_approx(f2_hi(x));
            rs = fadd2(rs, f2(e0, e1));
            if constexpr (kTwo) ext_split(e0, e1, &pk[e >> 1], &low[(e >> 1) & 7]);
            else pk[e >> 1] = pack_bf16x2(e0, e1);
          }
        };
        // PV(it - 1) has read the P columns and updated O
        auto pv_read = [&] {
          if (it > 0 && !mbar_wait_warp(&pv_done, (it - 1) & 1, &abort_flag)) ok = false;
        };
        if (!kTwo) exponentials(0, 32);
        pv_read();
        if (ok) {
          tc_fence_after();
          if constexpr (kTwo) {
            #pragma unroll
            for (int u = 0; u < 4; ++u) {
              exponentials(16 * u, 16);
              tmem_st_x8(tP + 8 * u, pk);
              tmem_st_x8(tS + 8 * u, low);
            }
          } else {
            tmem_st_x16(tP, pk);
            exponentials(32, 32);
            tmem_st_x16(tP + 16, pk);
          }
          l = l * alpha + (f2_lo(rs) + f2_hi(rs));
          if (it > 0 && __any_sync(0xffffffffu, alpha != 1.0f)) {
            #pragma unroll
            for (int q = 0; q < 32; q += 16) {
              uint32_t o[16];
              tmem_ld_x16(tO + q, o);
              tmem_ld_wait();
              #pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
              tmem_st_x16(tO + q, o);
            }
          }
          tmem_st_wait();
          tc_fence_before();
          mbar_arrive(&p_full);
        } else {
          abort_flag = 1;
        }
      }
      bool fin = ok && mbar_wait_warp(&pv_done, (num - 1) & 1, &abort_flag);
      s_red_l[c][r] = l;
      fin = named_barrier_and(1, 2 * kBlockM, fin);
      if (!fin) {
        abort_flag = 1;
        atomicCAS(p.err, 0, DEVERR_TIMEOUT_FWD + 8);
      } else {
        tc_fence_after();
        const int tok = r / p.group;
        const int hq = g * p.group + (r - tok * p.group);
        const bool valid = r < rows;
        const float lt = s_red_l[0][r] + s_red_l[1][r];
        uint32_t o[32];
        tmem_ld_x32(tO, o);
        tmem_ld_wait();
        if (parts > 1) {
          // this part's sums, unnormalised and without the sink
          if (valid) {
            float4* dst = reinterpret_cast<float4*>(p.o_part + (pidx * kBlockM + r) * kHeadDim +
                                                    32 * c);
            #pragma unroll
            for (int u = 0; u < 8; ++u)
              dst[u] = make_float4(__uint_as_float(o[4 * u]), __uint_as_float(o[4 * u + 1]),
                                   __uint_as_float(o[4 * u + 2]), __uint_as_float(o[4 * u + 3]));
            if (c == 0) p.ml_part[pidx * kBlockM + r] = make_float2(m, lt);
          }
        } else {
          // with the sink: Z = l 2^m + 2^sink (log2 units, relative to the larger)
          const float s2 = valid ? __ldg(p.sink + hq) * kLog2e : -INFINITY;
          const float mf = fmaxf(m, s2);
          const float mb = (mf == -INFINITY) ? 0.0f : mf;
          const float wk = ex2_approx(m - mb);
          const float z = fmaf(lt, wk, ext_sink(s2, mb));
          const float scale = z != 0.0f ? wk / z : 0.0f;
          const bool whole = rows == p.tokens * p.group;    // same for every row
          const size_t row = (size_t)row0 + tok;
          if (whole || valid) {
            const size_t base = (row * p.heads_q + hq) * kHeadDim + 32 * c;
            #pragma unroll
            for (int u = 0; u < 4; ++u) {
              uint32_t hi2[4];
              #pragma unroll
              for (int e = 0; e < 4; ++e)
                hi2[e] = pack_bf16x2(__uint_as_float(o[8 * u + 2 * e]) * scale,
                                     __uint_as_float(o[8 * u + 2 * e + 1]) * scale);
              if (whole)
                st_shared_v4(smem_u32(sK) + sw128_offset((uint32_t)r, (uint32_t)(4 * c + u)),
                             hi2[0], hi2[1], hi2[2], hi2[3]);
              else
                reinterpret_cast<uint4*>(p.out + base)[u] =
                    make_uint4(hi2[0], hi2[1], hi2[2], hi2[3]);
            }
            if (c == 0 && valid)
              p.lse[(size_t)hq * p.total_q + row] =         // NaN for a NaN score
                  z != 0.0f ? (mb + __log2f(z)) * kLn2 : -INFINITY;
          }
          if (whole) {
            fence_proxy_async_smem();
            named_barrier_sync(1, 2 * kBlockM);
            if (warp == 0 && lane == 0) {
              tma_store_3d_hint(&p.tm_out, sK, 0, g * p.group, row0, l2_policy_evict_first());
              bulk_commit_group();
              bulk_wait_group_read0();
            }
          }
        }
      }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kFwdMmaWarp) {
      tc_fence_after();
      tmem_dealloc(tmem, kFwdTmemCols);
    }
  } else if (parts > 1) {
    for (int r = tid; r < rows; r += kExtThreads)
      p.ml_part[pidx * kBlockM + r] = make_float2(-INFINITY, 0.0f);
  } else {
    // no row of this tile sees a key: the sink alone
    for (int x = tid; x < rows * 8; x += kExtThreads) {
      const int r = x >> 3, tok = r / p.group;
      const int hq = g * p.group + (r - tok * p.group);
      const size_t row = (size_t)row0 + tok;
      reinterpret_cast<uint4*>(p.out + (row * p.heads_q + hq) * kHeadDim)[x & 7] =
          make_uint4(0, 0, 0, 0);
      if ((x & 7) == 0) p.lse[(size_t)hq * p.total_q + row] = __ldg(p.sink + hq);
    }
  }
}

// Joins the parts of the split tiles, in the order of their keys, with the sink:
// M = max(m_c, sink), Z = sum l_c 2^(m_c - M) + 2^(sink - M).  A warp takes a row
// (tile, kv head, row): 16 lanes of 4 dimensions for the even parts, 16 for the
// odd ones.  What it costs is the chain of its loads (count, tile, statistics and
// sums), so those of 16 parts go out together, before their weights are known.
// It adds 5 us to a call (two rows a warp, loads behind the weights: 6.5).  A
// kernel of its own: joined by the CTA that stored the last part, 38 parts of 128
// rows (1.2 MB through one SM) took 60 us.
__global__ void __launch_bounds__(kExtJoinThreads, kExtJoinCtas)
attn_sink_extend_join_kernel(const __grid_constant__ ExtParams p) {
  grid_dependency_wait();
  const int lane = threadIdx.x & 31, odd = lane >> 4, d = 4 * (lane & 15);
  const int2 n = __ldcg(p.n_tiles);
  const unsigned pairs = (unsigned)n.x * (unsigned)p.heads_kv;            // < 2^30
  if (pairs == 0) return;
  const unsigned warps = gridDim.x * (kExtJoinThreads / 32);
  const unsigned up = warps / pairs, on = warps - up * pairs;
  unsigned x = blockIdx.x * (kExtJoinThreads / 32) + (threadIdx.x >> 5);
  unsigned row_at = x / pairs;
  x -= row_at * pairs;
  const size_t step = (size_t)p.heads_kv * kBlockM;         // from part to part
  // rows in the outer order: the warps of a last round are those of rows that
  // few tiles have
  for (; (int)row_at < n.y; row_at += up, x += on) {
    if (x >= pairs) {
      x -= pairs;
      if ((int)++row_at >= n.y) break;
    }
    const int r = (int)row_at;
    const unsigned t = x / (unsigned)p.heads_kv;
    const int g = (int)(x - t * (unsigned)p.heads_kv);
    const int4 ref = __ldcg(reinterpret_cast<const int4*>(p.tiles + t));   // an ExtTileRef
    const int parts = ref.y;
    if (r >= ref.z) continue;
    const int tok = r / p.group;
    const int hq = g * p.group + (r - tok * p.group);
    const size_t pr = ((size_t)ref.x * p.heads_kv + g) * kBlockM + r;
    const float* o = p.o_part + (pr + odd * step) * kHeadDim + d;
    auto load = [&](int c) {                                // parts c + odd, c + odd + 2, ..
      return c + odd < parts ? __ldcs(reinterpret_cast<const float4*>(o + c * step * kHeadDim))
                             : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    };
    static_assert(kExtMaxSplits <= 64, "two parts a lane");
    const float s2 = __ldg(p.sink + hq) * kLog2e;
    float2 ml[2];                                           // of parts lane and lane + 32
    #pragma unroll
    for (int u = 0; u < 2; ++u)
      ml[u] = lane + 32 * u < parts ? __ldcg(p.ml_part + pr + (lane + 32 * u) * step)
                                    : make_float2(-INFINITY, 0.0f);
    float4 v[8];
    #pragma unroll
    for (int u = 0; u < 8; ++u) v[u] = load(2 * u);
    float mf = fmaxf(s2, fmaxf(ml[0].x, ml[1].x));
    #pragma unroll
    for (int k = 16; k > 0; k >>= 1) mf = fmaxf(mf, __shfl_xor_sync(0xffffffffu, mf, k));
    const float mb = (mf == -INFINITY) ? 0.0f : mf;
    const float w0 = ex2_approx(ml[0].x - mb), w1 = ex2_approx(ml[1].x - mb);   // 0: empty part
    float z = fmaf(ml[1].y, w1, ml[0].y * w0);
    #pragma unroll
    for (int k = 16; k > 0; k >>= 1) z += __shfl_xor_sync(0xffffffffu, z, k);
    z += ext_sink(s2, mb);
    float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int c = 0; c < parts; c += 16) {
      #pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int k = c + 2 * u + odd;
        const float wk = __shfl_sync(0xffffffffu, c < 32 ? w0 : w1, k & 31);
        if (wk != 0.0f) {                                   // an empty part stored no sums
          acc.x = fmaf(v[u].x, wk, acc.x);
          acc.y = fmaf(v[u].y, wk, acc.y);
          acc.z = fmaf(v[u].z, wk, acc.z);
          acc.w = fmaf(v[u].w, wk, acc.w);
        }
      }
      if (c + 16 < parts)
        #pragma unroll
        for (int u = 0; u < 8; ++u) v[u] = load(c + 16 + 2 * u);
    }
    acc.x += __shfl_xor_sync(0xffffffffu, acc.x, 16);
    acc.y += __shfl_xor_sync(0xffffffffu, acc.y, 16);
    acc.z += __shfl_xor_sync(0xffffffffu, acc.z, 16);
    acc.w += __shfl_xor_sync(0xffffffffu, acc.w, 16);
    const float inv = z != 0.0f ? 1.0f / z : 0.0f;          // NaN for a NaN score
    const size_t row = (size_t)ref.w + tok;
    if (odd == 0)
      *reinterpret_cast<uint2*>(p.out + (row * p.heads_q + hq) * kHeadDim + d) = make_uint2(
          pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
    if (lane == 0)
      p.lse[(size_t)hq * p.total_q + row] = z != 0.0f ? (mb + __log2f(z)) * kLn2 : -INFINITY;
  }
}

}  // namespace attn_sink
