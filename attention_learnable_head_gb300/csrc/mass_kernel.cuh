// The attention weight that each cached key gets from a step's new tokens, sm_103a.
//
//   mass[b, h, j] (+)= sum over tokens i that see j, heads of h's group, exp(S_ij - lse_i)
//
// With the lse at hand nothing has to be known of the other keys: a weight needs its
// score alone, and values are not read.  The keys are the rows of the product, the
// (token, head) rows of q its columns, so that a thread sums the weights of its own keys
// and nothing is exchanged before the end.
//
// Few rows of q a sequence (one new token): the keys' bytes bound it.  Every warp walks
// through keys of one head by itself, 32 at a time with the next 32 on their way, with
// all rows of q in registers, and multiplies with m16n8k16 (a tcgen05 product has 64 rows
// of keys at least, which would have to go through shared memory).  As a dot product does
// not care for the order of its terms, the k index is permuted so that a lane's
// fragments are whole 16-byte chunks (chunks t and 4 + t for lane t of four).  32 sequences
// of 4 to 8 k keys, 64 heads on 8: 220 MB in 43 us, 5.1 TB/s.
//
// Many rows (prompts): an exponential a score bounds it.  A CTA holds 256 keys in TMEM, as the
// A operands of two products (from shared memory they would be read again for every tile),
// and q passes by in tiles of 96 rows through a TMA ring.  The rows' lse is part of the
// product: 16 more terms, of which three are ones on the keys' side and -(lse - c) /
// softmax_scale in three bf16 (24 bits) on the rows', with c a constant of the tile, so that
// a thread, with two keys and 48 of the rows, has one fma and one exponential for each
// score and reads nothing but TMEM.  Eight warps of 48 rows wait less often than twelve of
// 32.  Tiles with masks (the last 256 keys' triangle, rows without a token, lse that are
// infinite; all tiles where G does not divide 96) have a loop of their own: with the masks in
// the same one all tiles paid for them.  4 sequences of 280 to 512 new tokens on 13.6 to 16.4 k
// keys, 64 heads on 8: 275 us, of which 168 are exponentials at the unit's rate; about 30 are the blocks'
// beginnings and 35 the hand-over of products to weights.
#pragma once
#include <cuda_bf16.h>
#include "fwd_kernel.cuh"

namespace attn_sink {

struct MassParams {
  CUtensorMap tm_q;               // [T][H_q][64] bf16, box 64 x G x tokens per tile
  const __nv_bfloat16* q;         // [T][H_q][64]
  const __nv_bfloat16* k_cache;   // [num_pages][page_size][H_kv][64]
  const int* block_table;         // [B][max_pages]
  const int* seq_lens;            // [B]
  const int* cu_q;                // [B + 1]
  const float* lse;               // [H_q][T]
  float* mass;                    // [B][H_kv][max_keys]
  int* err;
  int batch, total_q, heads_q, heads_kv, group, tokens;
  int page_size, num_pages, max_pages, max_keys, accumulate;
  float scale_log2, inv_scale;    // softmax_scale log2(e), 1 / softmax_scale
#ifdef ATTN_SINK_TEST_HOOKS
  int skip_k_tile;
#endif
};

// A sequence: its new tokens [q0, q0 + n) of q, its keys, and those with an entry.
struct MassSeq {
  int q0, n, len, keys;
};
__device__ __forceinline__ MassSeq mass_seq(const MassParams& p, int b, bool* bad) {
  const int c0 = __ldg(p.cu_q + b), c1 = __ldg(p.cu_q + b + 1), l0 = __ldg(p.seq_lens + b);
  MassSeq s;
  s.q0 = min(max(c0, 0), p.total_q);
  s.n = max(0, min(c1, p.total_q) - s.q0);
  s.len = max(0, min(l0, p.max_pages * p.page_size));
  s.keys = min(s.len, p.max_keys);
  *bad = s.q0 != c0 || s.q0 + s.n != c1 || s.len != l0 || s.keys != s.len;
  return s;
}

constexpr uint32_t kMassNoRow = 0xFFFFFFFFu;

// The row of key j in the cache, in units of a head's 128 bytes, from its page's entry e of
// the table; kMassNoRow (and recorded) without a page.
__device__ __forceinline__ uint32_t mass_row(const MassParams& p, int e, int h, int j) {
  if ((unsigned)e >= (unsigned)p.num_pages) {
    atomicCAS(p.err, 0, DEVERR_DECODE_INPUT);
    return kMassNoRow;
  }
  return ((uint32_t)e * (uint32_t)p.page_size + (uint32_t)(j % p.page_size)) *
             (uint32_t)p.heads_kv + (uint32_t)h;
}

// ----------------------------------------------------------------------------- few rows
constexpr int kMassFewThreads = 256;
constexpr int kMassFewStages = 3;        // groups of 32 keys on their way to a warp
constexpr int kMassFewSmem = kMassFewThreads / 32 * kMassFewStages * 32 * 128;

// 16-byte chunk c of row r of a warp's stage: the halves of every 128 bytes are exchanged
// in every other row, so that 8 lanes that read 4 chunks of 2 rows touch each bank once.
__device__ __forceinline__ uint32_t mass_few_at(int r, int c) {
  return (uint32_t)r * 128u + (uint32_t)((c ^ ((r & 1) << 2)) << 4);
}

// Sequences of up to 8 kTiles rows of q; those with more take them in turns.
template <int kTiles>
__global__ void __launch_bounds__(kMassFewThreads, 2)
attn_sink_key_mass_few_kernel(const __grid_constant__ MassParams p) {
  extern __shared__ __align__(128) uint8_t few_smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const unsigned id = blockIdx.x * (kMassFewThreads / 32) + warp;
  const unsigned step = gridDim.x * (kMassFewThreads / 32) / (unsigned)p.heads_kv;
  const unsigned first = id / (unsigned)p.heads_kv;
  const int h = (int)(id - first * (unsigned)p.heads_kv);
  const int b = blockIdx.y;
  bool bad;
  const MassSeq s = mass_seq(p, b, &bad);
  if (bad && id == 0 && lane == 0) atomicCAS(p.err, 0, DEVERR_DECODE_INPUT);
  if (first >= step) return;
  float* mass = p.mass + ((size_t)b * p.heads_kv + h) * p.max_keys;
  const int* table = p.block_table + (size_t)b * p.max_pages;
  if (!p.accumulate)
    for (long long j = (s.n > 0 ? s.keys : 0) + 32ll * first + lane; j < p.max_keys; j += 32ll * step)
      mass[j] = 0.0f;
  const long long rows = (long long)s.n * p.group;
  const int at0 = s.len - s.n;             // key position of token 0
  const uint32_t ring = smem_u32(few_smem) + (uint32_t)warp * (kMassFewStages * 32 * 128);
  for (long long r0 = 0; r0 < rows; r0 += 8 * kTiles) {
    // B: row g of every tile, the dimensions of this lane's chunks; lse and the last key
    // seen of the two rows 2 t, 2 t + 1 whose scores it gets (-1: none, no weight)
    uint32_t bq[kTiles][8];
    float z[kTiles][2];
    int at[kTiles][2];
    int least = INT_MAX;
    #pragma unroll
    for (int i = 0; i < kTiles; ++i) {
      #pragma unroll
      for (int u = 0; u < 2; ++u) {
        uint4 v = make_uint4(0, 0, 0, 0);
        const long long r = r0 + 8 * i + g;
        if (r < rows) {
          const int tok = (int)(r / p.group), hd = (int)(r - (long long)tok * p.group);
          v = __ldg(reinterpret_cast<const uint4*>(p.q) +
                    ((size_t)(s.q0 + tok) * p.heads_q + h * p.group + hd) * 8 + 4 * u + t);
        }
        bq[i][4 * u] = v.x;
        bq[i][4 * u + 1] = v.y;
        bq[i][4 * u + 2] = v.z;
        bq[i][4 * u + 3] = v.w;
        const long long c = r0 + 8 * i + 2 * t + u;
        z[i][u] = 0.0f;
        at[i][u] = -1;
        if (c < rows) {
          const int tok = (int)(c / p.group), hd = (int)(c - (long long)tok * p.group);
          const float x = __ldg(p.lse + (size_t)(h * p.group + hd) * p.total_q + s.q0 + tok);
          if (!isinf(x)) {
            z[i][u] = -x * kLog2e;
            at[i][u] = at0 + tok;
          }
        }
        least = min(least, at[i][u]);
      }
    }
    least = __reduce_min_sync(0xffffffffu, least);
    const bool add = p.accumulate || r0 > 0;
    // this lane's key of a group of 32, whose row the others get from it
    auto row_of = [&](unsigned grp) {
      const int j = 32 * (int)grp + lane;
      return j < s.keys ? mass_row(p, __ldg(table + j / p.page_size), h, j) : kMassNoRow;
    };
    auto issue = [&](uint32_t mine, int st) {
      #pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int r = 4 * u + (lane >> 3);
        const uint32_t row = __shfl_sync(0xffffffffu, mine, r);
        const bool in = row != kMassNoRow;                  // else nothing is read, 0 written
        cp_async_16_zfill(ring + st * (32 * 128) + mass_few_at(r, lane & 7),
                          in ? p.k_cache + (size_t)row * 64 + 8 * (lane & 7) : p.q, in ? 16 : 0);
      }
    };
    const unsigned groups = (unsigned)(s.keys + 31) / 32;
    auto use = [&](unsigned grp, uint32_t mine, const uint32_t (*a)[2][4], float old) {
      float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
      const int j0 = 32 * (int)grp;
      #pragma unroll
      for (int i = 0; i < kTiles; ++i) {
        #pragma unroll
        for (int m = 0; m < 2; ++m) {
          float c[4] = {0.0f, 0.0f, 0.0f, 0.0f};
          #pragma unroll
          for (int u = 0; u < 2; ++u) {
            mma_16816_bf16(c, a[2 * m][u][0], a[2 * m + 1][u][0], a[2 * m][u][1],
                           a[2 * m + 1][u][1], bq[i][4 * u], bq[i][4 * u + 1]);
            mma_16816_bf16(c, a[2 * m][u][2], a[2 * m + 1][u][2], a[2 * m][u][3],
                           a[2 * m + 1][u][3], bq[i][4 * u + 2], bq[i][4 * u + 3]);
          }
          #pragma unroll
          for (int r = 0; r < 2; ++r) {
            float w0 = ex2_approx(fmaf(c[2 * r], p.scale_log2, z[i][0]));
            float w1 = ex2_approx(fmaf(c[2 * r + 1], p.scale_log2, z[i][1]));
            if (j0 + 31 > least) {         // the same for the whole warp
              const int j = j0 + 16 * m + 8 * r + g;
              w0 = j <= at[i][0] ? w0 : 0.0f;
              w1 = j <= at[i][1] ? w1 : 0.0f;
            }
            sum[2 * m + r] += w0 + w1;
          }
        }
      }
      #pragma unroll
      for (int r = 0; r < 4; ++r) {
        sum[r] += __shfl_xor_sync(0xffffffffu, sum[r], 1);
        sum[r] += __shfl_xor_sync(0xffffffffu, sum[r], 2);
      }
      // lane t of four has key 8 t + g
      const float w = t == 0 ? sum[0] : t == 1 ? sum[1] : t == 2 ? sum[2] : sum[3];
      const bool has = __shfl_sync(0xffffffffu, mine, 8 * t + g) != kMassNoRow;
      const int j = j0 + 8 * t + g;
      if (j < s.keys) mass[j] = old + (has ? w : 0.0f);
    };
    auto before = [&](unsigned grp) {
      const int j = 32 * (int)grp + 8 * t + g;
      return add && j < s.keys ? mass[j] : 0.0f;
    };
    // the table one group ahead of the copies, those kMassFewStages ahead of their use
    uint32_t mine[kMassFewStages];
    float old[kMassFewStages];
    #pragma unroll
    for (int st = 0; st < kMassFewStages; ++st) {
      const unsigned grp = first + st * step;
      mine[st] = grp < groups ? row_of(grp) : kMassNoRow;
    }
    #pragma unroll
    for (int st = 0; st < kMassFewStages; ++st) {
      const unsigned grp = first + st * step;
      if (grp < groups) issue(mine[st], st);
      cp_async_commit();
      old[st] = grp < groups ? before(grp) : 0.0f;
    }
    uint32_t next = first + kMassFewStages * step < groups ? row_of(first + kMassFewStages * step)
                                                           : kMassNoRow;
    for (unsigned base = first; base < groups; base += kMassFewStages * step) {
      #pragma unroll
      for (int st = 0; st < kMassFewStages; ++st) {
        const unsigned now = base + st * step, ahead = now + kMassFewStages * step;
        if (now < groups) {                // the same for the whole warp
          cp_async_wait<kMassFewStages - 1>();
          __syncwarp();
          uint32_t a[4][2][4];
          #pragma unroll
          for (int r = 0; r < 4; ++r)
            #pragma unroll
            for (int u = 0; u < 2; ++u)
              ld_shared_v4(ring + st * (32 * 128) + mass_few_at(8 * r + g, 4 * u + t), a[r][u]);
          const uint32_t rows_now = mine[st];
          const float was = old[st];
          __syncwarp();                    // every lane has read the stage
          mine[st] = next;
          if (ahead < groups) {
            issue(next, st);
            old[st] = before(ahead);
          }
          cp_async_commit();
          next = ahead + step < groups ? row_of(ahead + step) : kMassNoRow;
          use(now, rows_now, a, was);
        }
      }
    }
    cp_async_wait<0>();
    __syncwarp();
  }
}

// ----------------------------------------------------------------------------- many rows
constexpr int kMassKeys = 256;           // of a CTA: two products of 128
constexpr int kMassRows = 96;            // of a tile of q
constexpr int kMassMaxGroup = kMassRows;
constexpr int kMassWarps = 8;            // of weights, a key of each half and 48 rows a thread
constexpr int kMassCols = kMassRows / 2;
constexpr int kMassCopyWarp = kMassWarps;
constexpr int kMassMmaWarp = kMassWarps + 1;
constexpr int kMassThreads = 32 * (kMassWarps + 2);
constexpr int kMassStages = 4;
// What the warps read of a tile i is free once the product of tile i + 1 is there, for which
// they have all read the scores of tile i: with a stage's next tile but one.
constexpr int kMassInfos = 2 * kMassStages;
constexpr uint32_t kMassTileBytes = kMassRows * 128;
constexpr uint32_t kMassLseBytes = kMassRows * 32;    // of a stage: 16 bf16 a row
constexpr uint32_t kMassOneBytes = kBlockM * 32;      // the keys' side
constexpr uint32_t kMassTmemCols = 256;  // keys: 2 x 32 columns of bf16 pairs, scores: 2 x 96
constexpr uint32_t kMassColS = 64;
constexpr int kMassSmemBytes =
    1024 + (int)((kMassTileBytes + kMassLseBytes) * kMassStages + kMassOneBytes);
// softmax_scale for which (lse - c) / softmax_scale is an ordinary number
constexpr float kMassLeastScale = 0x1p-10f, kMassMostScale = 0x1p10f;

// Byte offset of 16-byte chunk c (0, 1) of row r of the 16 more terms: core matrices of 8 rows
// x 16 bytes, the two of 8 rows next to each other.
__device__ __forceinline__ uint32_t mass_more_at(int r, int c) {
  return (uint32_t)(r >> 3) * 256u + (uint32_t)c * 128u + (uint32_t)(r & 7) * 16u;
}
// Its descriptor: no swizzle, 128 bytes from core matrix to core matrix along the terms, 256
// along the rows.
__device__ __forceinline__ uint64_t mass_more_desc(uint32_t saddr) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | (uint64_t)(128 >> 4) << 16 |
         (uint64_t)(256 >> 4) << 32 | (uint64_t)1 << 46;
}

// mbar_wait_warp for the inner loop, where it mostly need not wait: what follows a first
// try is a call.
__device__ __noinline__ bool mass_wait_more(uint64_t* bar, uint32_t parity,
                                            volatile int* abort_flag) {
  return mbar_wait_warp(bar, parity, abort_flag);
}
__device__ __forceinline__ bool mass_wait(uint64_t* bar, uint32_t parity,
                                          volatile int* abort_flag) {
  return __all_sync(0xffffffffu, mbar_try_wait(smem_u32(bar), parity)) ||
         mass_wait_more(bar, parity, abort_flag);
}

__global__ void __launch_bounds__(kMassThreads, 2)
attn_sink_key_mass_kernel(const __grid_constant__ MassParams p) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t q_full[kMassStages], q_empty[kMassStages];
  __shared__ __align__(8) uint64_t s_full[2], s_empty[2], mma_drained;
  // of a tile: last key the row sees (-1: none); -c log2(e); 0 where all 96 rows have a token
  // that sees every key
  __shared__ __align__(16) int s_at[kMassInfos][kMassRows];
  __shared__ float s_base[kMassInfos];
  __shared__ int s_mask[kMassInfos];
  __shared__ float s_part[kMassKeys];
  __shared__ uint8_t s_has[kMassKeys];
  __shared__ uint32_t tmem_base_sh;
  __shared__ volatile int abort_flag;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int h = blockIdx.y, b = blockIdx.z;
  const int j0 = blockIdx.x * kMassKeys;
  bool bad;
  const MassSeq s = mass_seq(p, b, &bad);
  if (bad && tid == 0 && blockIdx.x == 0 && h == 0) atomicCAS(p.err, 0, DEVERR_DECODE_INPUT);
  float* mass = p.mass + ((size_t)b * p.heads_kv + h) * p.max_keys;
  const int at0 = s.len - s.n;             // key position of token 0
  // tiles of q from the first token that sees a key of the block
  const int t0 = max(0, j0 - at0) / p.tokens * p.tokens;
  const int tiles = j0 < s.keys && s.n > t0 ? (s.n - t0 + p.tokens - 1) / p.tokens : 0;
  if (tiles == 0) {                        // the same for the whole CTA
    const int j = j0 + tid;
    if (!p.accumulate && tid < kMassKeys && j < p.max_keys) mass[j] = 0.0f;
    return;
  }
  uint8_t* sQ = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                           ~static_cast<uintptr_t>(1023));
  uint8_t* sLse = sQ + kMassStages * kMassTileBytes;
  uint8_t* sOne = sLse + kMassStages * kMassLseBytes;
  const int rows = p.tokens * p.group;     // of a tile; behind them zeros, with no weight
  // the page of the thread's key is looked up meanwhile
  const int entry = tid < kMassKeys && j0 + tid < s.keys
                        ? __ldg(p.block_table + (size_t)b * p.max_pages + (j0 + tid) / p.page_size)
                        : -1;
  if (tid == 0) {
    abort_flag = 0;
    for (int i = 0; i < kMassStages; ++i) {
      mbar_init(&q_full[i], 2);            // the copy, and the rows' lse
      mbar_init(&q_empty[i], 1);           // the product
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 2);            // the product, and what its thread has seen of the tile
      mbar_init(&s_empty[i], kMassWarps);
    }
    mbar_init(&mma_drained, 1);
    fence_mbarrier_init();
  }
  if (warp == kMassMmaWarp) {
    tmem_alloc(&tmem_base_sh, kMassTmemCols);
    tmem_relinquish();
  }
  // the rows of a tile that no copy writes; three ones for each key, and zeros
  for (int x = rows * 8 + tid; x < kMassRows * 8; x += kMassThreads)
    for (int i = 0; i < kMassStages; ++i)
      st_shared_v4(smem_u32(sQ + i * kMassTileBytes) + (uint32_t)x * 16u, 0, 0, 0, 0);
  for (int x = tid; x < kMassRows * kMassStages; x += kMassThreads)
    st_shared_v4(smem_u32(sLse + (x / kMassRows) * kMassLseBytes) + mass_more_at(x % kMassRows, 1), 0,
                 0, 0, 0);
  for (int x = tid; x < kBlockM; x += kMassThreads) {
    st_shared_v4(smem_u32(sOne) + mass_more_at(x, 0), 0x3F803F80u, 0x00003F80u, 0, 0);
    st_shared_v4(smem_u32(sOne) + mass_more_at(x, 1), 0, 0, 0, 0);
  }
  fence_proxy_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // a thread's key goes from its page into TMEM
  const int c = warp >> 2, r = tid & 127;
  uint32_t key[32];
  float old[2] = {0.0f, 0.0f};
  if (warp < 8) {
    const int j = j0 + tid;
    const uint32_t row = j < s.keys ? mass_row(p, entry, h, j) : kMassNoRow;
    const bool has = row != kMassNoRow;
    #pragma unroll
    for (int u = 0; u < 8; ++u) {
      const uint4 v = has ? __ldg(reinterpret_cast<const uint4*>(p.k_cache) + (size_t)row * 8 + u)
                          : make_uint4(0, 0, 0, 0);
      key[4 * u] = v.x;
      key[4 * u + 1] = v.y;
      key[4 * u + 2] = v.z;
      key[4 * u + 3] = v.w;
    }
    s_has[tid] = has;
    if (p.accumulate && c == 0) {          // keys r and r + 128
      #pragma unroll
      for (int k = 0; k < 2; ++k)
        if (j + 128 * k < s.keys) old[k] = mass[j + 128 * k];
    }
  }
  const uint32_t tmem = tmem_base_sh;
  const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
  if (warp < 8) {
    tmem_st_x32(tmem + 32 * c + lane_base, key);
    tmem_st_wait();
    tc_fence_before();
  }
  if (warp != kMassCopyWarp) {             // which need not wait for the keys
    named_barrier_sync(2, kMassThreads - 32);
    tc_fence_after();
  }

  if (warp == kMassCopyWarp) {
    // ---------------------------------------------------------------- q and its lse
    constexpr int kCols = kMassRows / 32;
    int tok[kCols], hd[kCols];             // of rows lane, lane + 32, ..
    #pragma unroll
    for (int u = 0; u < kCols; ++u) {
      tok[u] = (lane + 32 * u) / p.group;
      hd[u] = lane + 32 * u - tok[u] * p.group;
    }
    // the lse of the next kAhead tiles is on its way: a load takes as long as a tile
    constexpr int kAhead = 4;
    float z[kAhead][kCols];
    auto fetch = [&](int i, float* z) {
      #pragma unroll
      for (int u = 0; u < kCols; ++u) {
        const int x = t0 + i * p.tokens + tok[u];
        z[u] = tok[u] < p.tokens && x < s.n
                   ? __ldg(p.lse + (size_t)(h * p.group + hd[u]) * p.total_q + s.q0 + x)
                   : INFINITY;
      }
    };
    const int last = min(j0 + kMassKeys, s.keys) - 1;      // of the block
    const uint32_t bytes = (uint32_t)rows * 128u;
    if (lane == 0) tma_prefetch_desc(&p.tm_q);
    #pragma unroll
    for (int k = 0; k < kAhead; ++k) fetch(k, z[k]);
    int i = 0;
    auto tile = [&](float* z) {
      const int st = i % kMassStages;
      if (i >= kMassStages && !mbar_wait_warp(&q_empty[st], ((i / kMassStages) & 1) ^ 1, &abort_flag))
        return false;
      if (lane == 0 && TEST_HOOK_FWD_ISSUE_K(i)) {
        mbar_arrive_expect_tx(&q_full[st], bytes);
        tma_load_3d(&p.tm_q, &q_full[st], sQ + st * kMassTileBytes, 0, h * p.group,
                    s.q0 + t0 + i * p.tokens);
      }
      // c: of the rows' lse the one next to zero (0 if they are out of fp32's middle range).  A
      // score's sum then is off by the rounding of |lse - c| <= 2 |lse| of its own row: with the
      // first row's lse for c, weights next to a head switched off by a sink of 1e4, 1e6 and
      // 1e10 were off by 0.06, 4.7 and 100 %; so by 3e-7.
      uint32_t size = 0x7F800000u;
      #pragma unroll
      for (int u = 0; u < kCols; ++u) size = min(size, __float_as_uint(z[u]) & 0x7FFFFFFFu);
      size = __reduce_min_sync(0xffffffffu, size);
      bool above = false;
      #pragma unroll
      for (int u = 0; u < kCols; ++u) above = above || __float_as_uint(z[u]) == size;
      const float least = __uint_as_float(size);
      const float base = !(least < 1e30f) ? 0.0f : __any_sync(0xffffffffu, above) ? least : -least;
      bool clear = true;
      #pragma unroll
      for (int u = 0; u < kCols; ++u) {
        const int at = at0 + t0 + i * p.tokens + tok[u];
        const bool weight = !isinf(z[u]);
        float y = weight ? (base - z[u]) * p.inv_scale : -1e30f;
        if (fabsf(y) > 1e37f) y = copysignf(1e37f, y);      // its three parts stay finite
        const uint32_t hi = pack_bf16x2(y, 0.0f) & 0xFFFFu;
        const float y1 = y - bf16_lo(hi);
        const uint32_t mid = pack_bf16x2(y1, 0.0f) & 0xFFFFu;
        const uint32_t low = pack_bf16x2(y1 - bf16_lo(mid), 0.0f) & 0xFFFFu;
        st_shared_v4(smem_u32(sLse + st * kMassLseBytes) + mass_more_at(lane + 32 * u, 0),
                     hi | mid << 16, weight ? low : 0u, 0, 0);
        s_at[i % kMassInfos][lane + 32 * u] = weight ? at : -1;
        clear = clear && weight && at >= last;
      }
      clear = __all_sync(0xffffffffu, clear);
      if (lane == 0) {
        s_mask[i % kMassInfos] = !clear;
        s_base[i % kMassInfos] = -base * kLog2e;
      }
      fence_proxy_async_smem();            // the product reads the lse
      __syncwarp();
      if (lane == 0) mbar_arrive(&q_full[st]);
      fetch(i + kAhead, z);
      ++i;
      return true;
    };
    bool ok = true;
    while (ok && i < tiles)
      #pragma unroll
      for (int k = 0; k < kAhead; ++k)
        if (ok && i < tiles) ok = tile(z[k]);
    if (lane == 0) {
      if (!ok) {
        abort_flag = 1;
        atomicCAS(p.err, 0, DEVERR_TIMEOUT_FWD + 0x10);
      }
      // the copies in flight land before the CTA releases its shared memory, also where the
      // other warps have given up
      for (int k = max(0, i - kMassStages); k < i; ++k)
        mbar_wait(&q_full[k % kMassStages], (k / kMassStages) & 1, nullptr);
    }
    __syncwarp();
  } else if (warp == kMassMmaWarp) {
    // ---------------------------------------------------------------- products
    if (lane == 0) {
      const uint32_t idesc = make_idesc_bf16(kBlockM, kMassRows, false, false);
      const uint64_t dQ = make_sdesc_sw128(smem_u32(sQ), 16, 1024);
      const uint64_t dLse = mass_more_desc(smem_u32(sLse)), dOne = mass_more_desc(smem_u32(sOne));
      bool ok = true;
      for (int i = 0; ok && i < tiles; ++i) {
        const int st = i % kMassStages;
        ok = mbar_wait(&q_full[st], (i / kMassStages) & 1, &abort_flag);
        #pragma unroll
        for (int e = 0; e < 2; ++e) {
          ok = ok && (i < 1 || mbar_wait(&s_empty[e], (i & 1) ^ 1, &abort_flag));
          if (!ok) break;
          tc_fence_after();
          mbar_arrive(&s_full[e]);
          const uint32_t d = tmem + kMassColS + kMassRows * e;
          #pragma unroll
          for (int k = 0; k < kHeadDim / 16; ++k)
            mma_ts(d, tmem + 32 * e + 8 * k, dQ + st * (kMassTileBytes >> 4) + 2 * k, idesc, k > 0);
          mma_ss(d, dOne, dLse + st * (kMassLseBytes >> 4), idesc, 1);
          mma_commit(&s_full[e]);
        }
        if (ok) mma_commit(&q_empty[st]);
      }
      if (!ok) {
        abort_flag = 1;
        atomicCAS(p.err, 0, DEVERR_TIMEOUT_FWD + 0x11);
      }
      mma_commit(&mma_drained);            // before TMEM is released
      mbar_wait(&mma_drained, 0, nullptr);
    }
    __syncwarp();
  } else {
    // ---------------------------------------------------------------- weights
    // warpgroup c has rows 48 c .. 48 c + 47 of every tile; thread = TMEM lane = keys r and
    // r + 128
    const uint32_t tS = tmem + kMassColS + kMassCols * c + lane_base;
    const uint64_t scale = f2(p.scale_log2, p.scale_log2);
    uint64_t sum[2][2] = {{f2(0.0f, 0.0f), f2(0.0f, 0.0f)}, {f2(0.0f, 0.0f), f2(0.0f, 0.0f)}};
    float more[2] = {0.0f, 0.0f};          // of tiles with masks
    int end[kMassCols / 16];               // the token of a tile that every 16 rows end with
    #pragma unroll
    for (int u = 0; u < kMassCols / 16; ++u) end[u] = (kMassCols * c + 16 * u + 15) / p.group;
    bool ok = true;
    for (int i = 0; ok && i < tiles; ++i) {
      ok = mass_wait(&s_full[0], i & 1, &abort_flag);
      if (!ok) break;
      const int info = i % kMassInfos;
      const int mask = s_mask[info];       // the same for the whole CTA
      if (mask == 0) {
        const uint64_t off = f2(s_base[info], s_base[info]);
        #pragma unroll
        for (int e = 0; e < 2; ++e) {
          ok = ok && (e == 0 || mass_wait(&s_full[e], i & 1, &abort_flag));
          if (!ok) break;
          tc_fence_after();
          uint32_t x[kMassCols];
          tmem_ld_x32(tS + kMassRows * e, x);
          tmem_ld_x16(tS + kMassRows * e + 32, x + 32);
          tmem_ld_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&s_empty[e]);          // the next product may begin
          #pragma unroll
          for (int k = 0; k < kMassCols; k += 2) {
            const uint64_t v =
                ffma2(f2(__uint_as_float(x[k]), __uint_as_float(x[k + 1])), scale, off);
            sum[e][(k >> 1) & 1] =
                fadd2(sum[e][(k >> 1) & 1], f2(ex2_approx(f2_lo(v)), ex2_approx(f2_hi(v))));
          }
        }
      } else {
        const float off = s_base[info];
        const int x0 = t0 + i * p.tokens, at_i = at0 + x0;
        const int rows_i = min(p.tokens, s.n - x0) * p.group;
        #pragma unroll 1
        for (int e = 0; e < 2; ++e) {
          ok = ok && (e == 0 || mass_wait(&s_full[e], i & 1, &abort_flag));
          if (!ok) break;
          tc_fence_after();
          uint32_t x[kMassCols];
          tmem_ld_x32(tS + kMassRows * e, x);
          tmem_ld_x16(tS + kMassRows * e + 32, x + 32);
          tmem_ld_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&s_empty[e]);
          const int least = j0 + 128 * e + (r & ~31), j = least + lane;   // the warp's first key
          float w = 0.0f;
          #pragma unroll
          for (int u = 0; u < kMassCols / 16; ++u) {
            // none of the 16 rows has a token that sees one of the warp's keys
            if (kMassCols * c + 16 * u >= rows_i || at_i + end[u] < least) continue;
            const int2* at2 = reinterpret_cast<const int2*>(&s_at[info][kMassCols * c + 16 * u]);
            #pragma unroll
            for (int k = 16 * u; k < 16 * u + 16; k += 2) {
              const int2 at = at2[(k >> 1) - 8 * u];
              const float w0 = ex2_approx(fmaf(__uint_as_float(x[k]), p.scale_log2, off));
              const float w1 = ex2_approx(fmaf(__uint_as_float(x[k + 1]), p.scale_log2, off));
              w += (j <= at.x ? w0 : 0.0f) + (j <= at.y ? w1 : 0.0f);
            }
          }
          if (e == 0) more[0] += w;
          else more[1] += w;
        }
      }
    }
    float w[2];
    #pragma unroll
    for (int k = 0; k < 2; ++k) {
      const uint64_t both = fadd2(sum[k][0], sum[k][1]);
      w[k] = f2_lo(both) + f2_hi(both) + more[k];
      if (c > 0) s_part[128 * k + r] = w[k];
    }
    ok = named_barrier_and(1, 32 * kMassWarps, ok);
    if (!ok) {
      abort_flag = 1;
      atomicCAS(p.err, 0, DEVERR_TIMEOUT_FWD + 0x12);
    } else if (c == 0) {
      #pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int x = 128 * k + r, j = j0 + x;
        const float all = s_has[x] ? w[k] + s_part[x] : 0.0f;
        if (j < s.keys) mass[j] = old[k] + all;
        else if (!p.accumulate && j < p.max_keys) mass[j] = 0.0f;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMassMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, kMassTmemCols);
  }
}

}  // namespace attn_sink
