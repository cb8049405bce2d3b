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
// other page sizes are copied 16 bytes a lane with cp.async.
//
// Work items.  A schedule kernel of one CTA lists (sequence, tile, key range)
// in the workspace.  Sequences whose keys exceed an even share of the launch's
// work are split over several CTAs per tile, so that a long cache with few new
// tokens fills the GPU; the CTA of a tile that finishes last joins the parts
// and adds the sink (counters that the schedule kernel zeroes).  The parts are
// joined in the order of their keys, whichever CTA does it.
//
// The rest is the forward kernel's pipeline: S = Q K^T into TMEM, online
// softmax by two warpgroups (one per key half), P to TMEM, O += P V with P
// read from TMEM, lazy rescaling.  P is rounded to bf16, not fp16: the cache
// holds bf16 values, and an fp16 product would need every value tile converted
// by each CTA; one more rounding of 2^-8 next to that of the bf16 output.  The
// row sums add the fp32 probabilities.
#pragma once
#include "fwd_kernel.cuh"

namespace attn_sink {

constexpr int kExtThreads = 320;           // 8 softmax warps, copy warp, MMA warp
constexpr int kExtMaxGroup = 128;
constexpr int kExtMaxSplits = 64;
constexpr int kExtSchedThreads = 1024;
constexpr uint32_t kExtNone = 0xFFFFFFFFu;

struct ExtItem {                           // one CTA's work for each kv head
  uint32_t seq;                            // kExtNone: unused entry
  uint32_t tile;
  uint32_t split;                          // part << 16 | parts of the tile
  uint32_t first;                          // index of the tile's first partial result
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
  ExtItem* items;
  float* o_part;           // [partial][kv head][128 rows][64]
  float2* ml_part;         // [partial][kv head][128 rows]: maximum (log2 units), sum
  int* done;               // [partial][kv head], counted at a tile's first partial
  int* err;
  int batch, total_q, heads_q, heads_kv, group, tokens;
  int page_size, num_pages, max_pages, window;
  int box;                 // keys of a TMA box (0: cp.async copies)
  int n_items, max_parts;  // sizes of items, and of the partial results
  int target;              // CTAs the work is spread over
  int min_blocks;          // key blocks a part has at least
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

// Keys [lo, hi) that tokens i0 .. i1 of the sequence see.
__device__ __forceinline__ void ext_keys(const ExtSeq& s, int i0, int i1, int window, int* lo,
                                         int* hi) {
  const int off = s.len - s.n;             // key position of token 0
  *hi = max(0, min(s.len, i1 + off + 1));
  *lo = window > 0 ? max(0, i0 + off - window + 1) : 0;
}

__device__ __forceinline__ int ext_blocks(int lo, int hi) {
  return hi > lo ? (hi + kBlockN - 1) / kBlockN - lo / kBlockN : 0;
}

// Lists the work items.  With W the key blocks of all tiles (each taken as long
// as its sequence's last) times the kv heads, a part has at least c = W / target
// blocks and a tile ceil(blocks / c) parts: tiles + target / H_kv items at most.
__global__ void __launch_bounds__(kExtSchedThreads, 1)
attn_sink_extend_plan_kernel(const __grid_constant__ ExtParams p) {
  constexpr int kWarps = kExtSchedThreads / 32;
  __shared__ long long s_red[kWarps];
  __shared__ int s_scan[2][kWarps];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  bool bad = false;
  auto tiles_of = [&](const ExtSeq& s) { return (s.n + p.tokens - 1) / p.tokens; };
  auto blocks_of = [&](const ExtSeq& s, int tiles) {     // of the last tile
    int lo, hi;
    ext_keys(s, (tiles - 1) * p.tokens, s.n - 1, p.window, &lo, &hi);
    return ext_blocks(lo, hi);
  };
  // total work
  long long w = 0;
  for (int b = tid; b < p.batch; b += kExtSchedThreads) {
    const ExtSeq s = ext_seq(p, b, &bad);
    const int tiles = tiles_of(s);
    if (tiles > 0) w += (long long)tiles * blocks_of(s, tiles);
  }
  if (bad) atomicCAS(p.err, 0, DEVERR_DECODE_INPUT);
  #pragma unroll
  for (int d = 16; d > 0; d >>= 1) w += __shfl_xor_sync(0xffffffffu, w, d);
  if (lane == 0) s_red[warp] = w;
  // the tiles' completion counters, and the table's entries behind the last item
  for (int i = tid; i < p.max_parts * p.heads_kv; i += kExtSchedThreads) p.done[i] = 0;
  __syncthreads();
  w = 0;
  #pragma unroll
  for (int i = 0; i < kWarps; ++i) w += s_red[i];
  const long long share = (w * p.heads_kv + p.target - 1) / p.target;
  const int chunk = (int)min(max((long long)p.min_blocks, share), 1ll << 24);   // > any tile's blocks

  int item0 = 0, part0 = 0;                // of the sequences before this round
  for (int b0 = 0; b0 < p.batch; b0 += kExtSchedThreads) {
    const int b = b0 + tid;
    ExtSeq s{0, 0, 0};
    int tiles = 0, parts = 0;
    if (b < p.batch) {
      s = ext_seq(p, b, &bad);
      tiles = tiles_of(s);
      if (tiles > 0)
        parts = min(kExtMaxSplits, max(1, (blocks_of(s, tiles) + chunk - 1) / chunk));
    }
    const int mine_i = tiles * parts, mine_p = parts > 1 ? tiles * parts : 0;
    int it = mine_i, ip = mine_p;          // inclusive scans
    #pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int a = __shfl_up_sync(0xffffffffu, it, d), c = __shfl_up_sync(0xffffffffu, ip, d);
      if (lane >= d) {
        it += a;
        ip += c;
      }
    }
    if (lane == 31) {
      s_scan[0][warp] = it;
      s_scan[1][warp] = ip;
    }
    __syncthreads();
    int bi = item0, bp = part0, all_i = 0, all_p = 0;
    #pragma unroll
    for (int i = 0; i < kWarps; ++i) {
      if (i < warp) {
        bi += s_scan[0][i];
        bp += s_scan[1][i];
      }
      all_i += s_scan[0][i];
      all_p += s_scan[1][i];
    }
    bi += it - mine_i;
    bp += ip - mine_p;
    // a warp writes its 32 sequences' items, 32 at a time
    for (int l = 0; l < 32; ++l) {
      const int n = __shfl_sync(0xffffffffu, mine_i, l);
      if (n == 0) continue;
      const int sp = __shfl_sync(0xffffffffu, parts, l), nt = __shfl_sync(0xffffffffu, tiles, l);
      const int wi = __shfl_sync(0xffffffffu, bi, l), wp = __shfl_sync(0xffffffffu, bp, l);
      for (int k = lane; k < n; k += 32) {
        const int tile = k / sp, part = k - tile * sp;
        ExtItem e;
        e.seq = (uint32_t)(b0 + 32 * warp + l);
        e.tile = (uint32_t)(nt - 1 - tile);            // the longest tiles first
        e.split = (uint32_t)part << 16 | (uint32_t)sp;
        e.first = (uint32_t)(wp + tile * sp);
        // both bounds hold for every cu_seqlens that ascends; one that does not
        // may list more, which is dropped (and was recorded)
        if (sp > 1 && wp + tile * sp + sp > p.max_parts) e.seq = kExtNone;
        if (wi + k < p.n_items) reinterpret_cast<uint4*>(p.items)[wi + k] = *reinterpret_cast<uint4*>(&e);
      }
    }
    item0 += all_i;
    part0 += all_p;
    __syncthreads();
  }
  for (int k = item0 + tid; k < p.n_items; k += kExtSchedThreads) p.items[k].seq = kExtNone;
}

template <bool kTma>
__global__ void __maxnreg__(96)
attn_sink_extend_kernel(const __grid_constant__ ExtParams p) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t q_full, mma_drained;
  __shared__ __align__(8) uint64_t k_full[kFwdKStages], k_empty[kFwdKStages];
  __shared__ __align__(8) uint64_t v_full[kFwdVStages], v_empty[kFwdVStages];
  __shared__ __align__(8) uint64_t s_full, s_free, p_full, pv_done;
  __shared__ uint32_t tmem_base_sh;
  __shared__ volatile int abort_flag;
  __shared__ float s_mx[2][2][kBlockM];
  __shared__ float s_red_l[2][kBlockM];
  __shared__ int s_last;

  const int item = (int)(blockIdx.x / (unsigned)p.heads_kv);
  const int g = (int)(blockIdx.x - (unsigned)item * (unsigned)p.heads_kv);
  const uint4 raw = __ldg(reinterpret_cast<const uint4*>(p.items) + item);
  if (raw.x == kExtNone) return;                          // uniform per CTA
  const int seq = (int)raw.x, tile = (int)raw.y;
  const int part = (int)(raw.z >> 16), parts = (int)(raw.z & 0xFFFFu);
  bool dummy = false;
  const ExtSeq sp = ext_seq(p, seq, &dummy);
  const int i0 = tile * p.tokens;
  const int i1 = min(i0 + p.tokens, sp.n) - 1;            // last token of the tile
  const int rows = (i1 - i0 + 1) * p.group;               // rows that hold a token
  const int off = sp.len - sp.n;
  const int tid = threadIdx.x;
  const int warp = tid >> 5, lane = tid & 31;
  // keys [lo, hi) of the tile, and of them the blocks [blk0, blk0 + num) of
  // this part
  int lo, hi;
  ext_keys(sp, i0, i1, p.window, &lo, &hi);
  int blk0 = lo / kBlockN, num = ext_blocks(lo, hi);
  if (parts > 1) {
    const int per = (num + parts - 1) / parts;
    const int skip = min(num, part * per);
    blk0 += skip;
    num = min(per, num - skip);
  }
  const size_t pidx = (size_t)(raw.w + part) * p.heads_kv + g;   // this CTA's partial result
  const int* table = p.block_table + (size_t)seq * p.max_pages;

  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* sQ = smem;
  uint8_t* sK = sQ + kTileBytes;
  uint8_t* sV = sK + kFwdKStages * kTileBytes;
  bool failed = false;

  if (num > 0) {
    // Does every page of these keys lie in the cache?  (Rarely not: then the
    // softmax looks its keys' entries up one by one.)
    bool bad_page = false;
    {
      const int k0 = max(lo, blk0 * kBlockN), k1 = min(hi, (blk0 + num) * kBlockN);
      const int pg1 = (k1 - 1) / p.page_size;
      for (int pg = k0 / p.page_size + tid; pg <= pg1; pg += kExtThreads) {
        const int e = __ldg(table + pg);
        bad_page |= e < 0 || e >= p.num_pages;
      }
    }
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
      mbar_init(&s_free, 2 * kBlockM);
      mbar_init(&p_full, 2 * kBlockM);
      mbar_init(&pv_done, 1);
      fence_mbarrier_init();
    }
    if (warp == kFwdMmaWarp) {
      tmem_alloc(&tmem_base_sh, kFwdTmemCols);
      tmem_relinquish();
    }
    tc_fence_before();
    bad_page = __syncthreads_or(bad_page);
    tc_fence_after();
    const uint32_t tmem = tmem_base_sh;
    if (bad_page && tid == 0) atomicCAS(p.err, 0, DEVERR_DECODE_INPUT);

    if (warp == kFwdTmaWarp) {
      // -------------------------------------------------------------- copies
      const uint32_t q_bytes = (uint32_t)(p.tokens * p.group) * 128u;
      if (lane == 0) {
        tma_prefetch_desc(&p.tm_q);
        mbar_arrive_expect_tx(&q_full, q_bytes);
        tma_load_3d(&p.tm_q, &q_full, sQ, 0, g * p.group, sp.q0 + i0);
      }
      __syncwarp();
      if (kTma) {
        // Lanes 0-15 copy the K boxes of a block, lanes 16-31 the V boxes; each
        // holds the page of its next box, read one block ahead.
        const int half = lane >> 4, ci = lane & 15;
        const int boxes = kBlockN / p.box;
        const bool mine = ci < boxes;
        const int oob = p.num_pages * p.page_size;          // first row past the cache
        auto row_of = [&](int n) -> int {                   // cache row of this lane's box
          const int j = (blk0 + n) * kBlockN + ci * p.box;
          if (!mine || n >= num || j >= hi || j + p.box <= lo) return oob;
          const int pg = j / p.page_size;
          const int e = __ldg(table + pg);
          return e >= 0 && e < p.num_pages ? e * p.page_size + (j - pg * p.page_size) : oob;
        };
        int row = row_of(0);
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
                tma_load_3d(&p.tm_k, &k_full[st], sK + st * kTileBytes + ci * p.box * 128, 0, g,
                            row);
              row = row_of(nk + 1);
            }
            ++nk;
          }
          if (can_v) {
            if (half == 1) {
              const int st = nv % kFwdVStages;
              if (mine)
                tma_load_3d(&p.tm_v, &v_full[st], sV + st * kTileBytes + ci * p.box * 128, 0, g,
                            row);
              row = row_of(nv + 1);
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
        bool ok = true;
        int x = 0;
        for (; x < 2 * num; ++x) {
          const int n = x >> 1;
          const bool is_v = x & 1;
          if (!is_v && !TEST_HOOK_FWD_ISSUE_K(n)) {
            ok = false;
            break;
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
          const __nv_bfloat16* cache = is_v ? p.v_cache : p.k_cache;
          const int jb = (blk0 + n) * kBlockN;
          const int c = lane & 7;
          #pragma unroll 4
          for (int u = 0; u < kBlockN / 4; ++u) {
            const int r = 4 * u + (lane >> 3);
            const int j = jb + r;
            const void* src = p.out;                        // any address: 0 bytes are read
            uint32_t bytes = 0;
            if (j >= lo && j < hi) {
              const int pg = j / p.page_size;
              const int e = __ldg(table + pg);
              if (e >= 0 && e < p.num_pages) {
                src = cache + ((size_t)e * p.page_size + (j - pg * p.page_size)) *
                                  ((size_t)p.heads_kv * 64) + g * 64 + 8 * c;
                bytes = 16;
              }
            }
            cp_async_16_zfill(dst + sw128_offset((uint32_t)r, (uint32_t)c), src, bytes);
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
          if (n + 1 < num) {
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
          #pragma unroll
          for (int k = 0; k < kBlockN / 16; ++k)
            mma_ts(tmem + kFwdColO, tmem + kFwdColP + 8 * k, dV0 + sv * kTileU + 128 * k, idesc_o,
                   (n > 0 || k > 0));
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
      // Key half c = warp / 4; thread = row = TMEM lane.
      const int c = warp >> 2;
      const int r = tid & 127;
      const int tok = r / p.group;
      const int hq = g * p.group + (r - tok * p.group);
      const int i = i0 + tok;
      const bool valid = r < rows;
      const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
      const uint32_t tS = tmem + kFwdColS + 64 * c + lane_base;
      const uint32_t tP = tmem + kFwdColP + 32 * c + lane_base;
      const uint32_t tO = tmem + kFwdColO + 32 * c + lane_base;
      // a warp without a row that holds a token only keeps the barriers going
      const bool idle = 32 * (warp & 3) >= rows;
      float m = -INFINITY, l = 0.0f;
      const float sl2 = p.scale_log2;
      const uint64_t sl2x2 = f2(sl2, sl2);
      const int jmax = min(sp.len - 1, i + off);            // inclusive
      const int jmin = p.window > 0 ? i + off - p.window + 1 : 0;
      bool ok = true;
      for (int it = 0; it < num; ++it) {
        uint32_t a[64];
        const int jb = (blk0 + it) * kBlockN;
        bool got = mbar_wait_warp(&s_full, it & 1, &abort_flag);
        float mx_half = -INFINITY;
        if (got) {
          tc_fence_after();
          if (!idle) {
            tmem_ld_x32(tS, a);
            tmem_ld_x32(tS + 32, a + 32);
            tmem_ld_wait();
          }
          tc_fence_before();
          mbar_arrive(&s_free);
          if (!idle) {
            const int j0 = jb + 64 * c;                     // first key of this half
            const bool need_mask = j0 + 64 > sp.len || j0 + 63 > i0 + off ||
                                   (p.window > 0 && j0 <= i1 + off - p.window);
            if (need_mask) {
              #pragma unroll
              for (int e = 0; e < 64; ++e) {
                const int j = j0 + e;
                if (j > jmax || j < jmin) a[e] = __float_as_uint(-INFINITY);
              }
            }
            if (bad_page) {
              uint32_t off_lo = 0, off_hi = 0;              // keys without a page
              #pragma unroll 1
              for (int e = 0; e < 64; ++e) {
                const int j = j0 + e;
                if (j < lo || j >= hi) continue;
                const int pe = __ldg(table + j / p.page_size);
                if (pe >= 0 && pe < p.num_pages) continue;
                if (e < 32) off_lo |= 1u << e;
                else off_hi |= 1u << (e - 32);
              }
              #pragma unroll
              for (int e = 0; e < 64; ++e)
                if (((e < 32 ? off_lo : off_hi) >> (e & 31)) & 1u)
                  a[e] = __float_as_uint(-INFINITY);
            }
            float q0 = __uint_as_float(a[0]), q1 = __uint_as_float(a[1]);
            float q2 = __uint_as_float(a[2]), q3 = __uint_as_float(a[3]);
            #pragma unroll
            for (int e = 4; e < 64; e += 8) {
              q0 = fmax3(q0, __uint_as_float(a[e]), __uint_as_float(a[e + 1]));
              q1 = fmax3(q1, __uint_as_float(a[e + 2]), __uint_as_float(a[e + 3]));
              q2 = fmax3(q2, __uint_as_float(a[e + 4]), __uint_as_float(a[e + 5]));
              q3 = fmax3(q3, __uint_as_float(a[e + 6]), __uint_as_float(a[e + 7]));
            }
            mx_half = valid ? fmaxf(fmax3(q0, q1, q2), q3) : -INFINITY;
            s_mx[it & 1][c][r] = mx_half;
          }
        }
        if (!named_barrier_and(2 + (warp & 3), 64, got && ok)) {
          ok = false;
          abort_flag = 1;
          break;
        }
        // A block at the edge of the keys: value rows that no token sees may hold
        // anything, and 0 * inf is not 0.
        if (jb < lo || jb + kBlockN > hi) {
          const int sv = it % kFwdVStages;
          if (mbar_wait_warp(&v_full[sv], (it / kFwdVStages) & 1, &abort_flag)) {
            const uint32_t base = smem_u32(sV + sv * kTileBytes);
            #pragma unroll
            for (int u = 0; u < 4; ++u) {
              const int chunk = u * 256 + tid;
              const int j = jb + (chunk >> 3);
              if (j < lo || j >= hi) st_shared_v4(base + (uint32_t)chunk * 16u, 0, 0, 0, 0);
            }
            fence_proxy_async_smem();
          } else {
            ok = false;
          }
        }
        float alpha = 1.0f;
        if (!idle) {
          const float mx = fmaxf(mx_half, s_mx[it & 1][c ^ 1][r]) * sl2;
          if (mx > m + kRescaleThreshold || (m == -INFINITY && mx > -INFINITY)) {
            alpha = ex2_approx(m - mx);
            m = mx;
          }
        }
        const float m_use = (m == -INFINITY) ? 0.0f : m;
        const uint64_t negm2 = f2(-m_use, -m_use);
        uint64_t rs = f2(0.0f, 0.0f);
        uint32_t pk[16];
        if (!idle) {
          #pragma unroll
          for (int e = 0; e < 32; e += 2) {
            const uint64_t x =
                ffma2(f2(__uint_as_float(a[e]), __uint_as_float(a[e + 1])), sl2x2, negm2);
            const float e0 = ex2_approx(f2_lo(x));
            const float e1 = ex2_approx(f2_hi(x));
            rs = fadd2(rs, f2(e0, e1));
            pk[e >> 1] = pack_bf16x2(e0, e1);
          }
        }
        // PV(it - 1) has read the P columns and updated O
        if (it > 0 && !mbar_wait_warp(&pv_done, (it - 1) & 1, &abort_flag)) ok = false;
        if (ok) {
          tc_fence_after();
          if (!idle) {
            tmem_st_x16(tP, pk);
            #pragma unroll
            for (int e = 0; e < 32; e += 2) {
              const uint64_t x =
                  ffma2(f2(__uint_as_float(a[32 + e]), __uint_as_float(a[33 + e])), sl2x2, negm2);
              const float e0 = ex2_approx(f2_lo(x));
              const float e1 = ex2_approx(f2_hi(x));
              rs = fadd2(rs, f2(e0, e1));
              pk[e >> 1] = pack_bf16x2(e0, e1);
            }
            tmem_st_x16(tP + 16, pk);
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
          }
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
          const float z = fmaf(lt, wk, ex2_approx(s2 - mb));
          const float scale = z > 0.0f ? wk / z : 0.0f;
          const bool whole = i0 + p.tokens <= sp.n;         // same for every row
          const size_t row = (size_t)sp.q0 + i;
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
              p.lse[(size_t)hq * p.total_q + row] =
                  z > 0.0f ? (mb + __log2f(z)) * kLn2 : -INFINITY;
          }
          if (whole) {
            fence_proxy_async_smem();
            named_barrier_sync(1, 2 * kBlockM);
            if (warp == 0 && lane == 0) {
              tma_store_3d_hint(&p.tm_out, sK, 0, g * p.group, sp.q0 + i0,
                                l2_policy_evict_first());
              bulk_commit_group();
              bulk_wait_group_read0();
            }
          }
        }
      }
    }
    tc_fence_before();
    __syncthreads();
    failed = abort_flag != 0;
    if (warp == kFwdMmaWarp) {
      tc_fence_after();
      tmem_dealloc(tmem, kFwdTmemCols);
    }
    if (failed) return;                                     // uniform: recorded, nothing joined
  } else if (parts > 1) {
    for (int r = tid; r < rows; r += kExtThreads)
      p.ml_part[pidx * kBlockM + r] = make_float2(-INFINITY, 0.0f);
  } else {
    // no row of this tile sees a key: the sink alone
    for (int x = tid; x < rows * 8; x += kExtThreads) {
      const int r = x >> 3, tok = r / p.group;
      const int hq = g * p.group + (r - tok * p.group);
      const size_t row = (size_t)sp.q0 + i0 + tok;
      reinterpret_cast<uint4*>(p.out + (row * p.heads_q + hq) * kHeadDim)[x & 7] =
          make_uint4(0, 0, 0, 0);
      if ((x & 7) == 0) p.lse[(size_t)hq * p.total_q + row] = __ldg(p.sink + hq);
    }
  }
  if (parts == 1) return;

  // ---- the last CTA of the tile joins the parts, in the order of their keys,
  // with the sink: M = max(m_c, sink), Z = sum l_c 2^(m_c - M) + 2^(sink - M).
  __threadfence();
  __syncthreads();
  if (tid == 0)
    s_last = atomicAdd(p.done + (size_t)raw.w * p.heads_kv + g, 1) == parts - 1;
  __syncthreads();
  if (!s_last) return;
  __threadfence();
  for (int x = tid; x < rows * 16; x += kExtThreads) {      // thread: a row, 4 dimensions
    const int r = x >> 4, d = 4 * (x & 15);
    const int tok = r / p.group;
    const int hq = g * p.group + (r - tok * p.group);
    const size_t row = (size_t)sp.q0 + i0 + tok;
    const size_t first = ((size_t)raw.w * p.heads_kv + g) * kBlockM + r;
    const size_t step = (size_t)p.heads_kv * kBlockM;
    const float s2 = __ldg(p.sink + hq) * kLog2e;
    float mf = s2;
    #pragma unroll 8
    for (int c = 0; c < parts; ++c) mf = fmaxf(mf, __ldcg(p.ml_part + first + c * step).x);
    const float mb = (mf == -INFINITY) ? 0.0f : mf;
    float z = ex2_approx(s2 - mb);
    float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    #pragma unroll 8
    for (int c = 0; c < parts; ++c) {
      const float2 ml = __ldcg(p.ml_part + first + c * step);
      const float4 o = __ldcg(
          reinterpret_cast<const float4*>(p.o_part + (first + c * step) * kHeadDim + d));
      if (ml.x == -INFINITY) continue;                      // no key: its sums were not written
      const float wt = ex2_approx(ml.x - mb);
      z = fmaf(ml.y, wt, z);
      acc.x = fmaf(o.x, wt, acc.x);
      acc.y = fmaf(o.y, wt, acc.y);
      acc.z = fmaf(o.z, wt, acc.z);
      acc.w = fmaf(o.w, wt, acc.w);
    }
    const float inv = z > 0.0f ? 1.0f / z : 0.0f;
    *reinterpret_cast<uint2*>(p.out + (row * p.heads_q + hq) * kHeadDim + d) =
        make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
    if (d == 0)
      p.lse[(size_t)hq * p.total_q + row] = z > 0.0f ? (mb + __log2f(z)) * kLn2 : -INFINITY;
  }
}

}  // namespace attn_sink
