// The attention weight that each cached key gets from a step's new tokens, sm_103a.
//
//   mass[b, h, j] (+)= sum over tokens i that see j, heads of h's group, exp(S_ij - lse_i)
//
// With the lse at hand nothing has to be known of the other keys: a weight needs its
// score alone, and values are not read.  The keys are the rows of the product, the
// (token, head) rows of q its columns, so that a thread sums the weights of its own keys
// and nothing is exchanged before the end.  Warp-level products m16n8k16 hold 32 keys
// of a warp in registers for as long as q passes by; as a dot product does not care for
// the order of its terms, the k index is permuted so that a lane's fragments are whole
// 16-byte chunks (chunks t and 4 + t for lane t of four): keys go from their pages
// straight into registers, q comes from shared memory 16 bytes a lane.
//
// One new token a sequence: the keys' bytes bound it.  Prompts: an exponential a score.
#pragma once
#include <cuda_bf16.h>
#include "sm103_ptx.cuh"

namespace attn_sink {

constexpr int kMassThreads = 256;
constexpr int kMassKeys = 256;           // of a CTA at a time: 32 a warp
constexpr int kMassRows = 64;            // rows of q in shared memory at a time, two buffers

struct MassParams {
  const __nv_bfloat16* q;         // [T][H_q][64]
  const __nv_bfloat16* k_cache;   // [num_pages][page_size][H_kv][64]
  const int* block_table;         // [B][max_pages]
  const int* seq_lens;            // [B]
  const int* cu_q;                // [B + 1]
  const float* lse;               // [H_q][T]
  float* mass;                    // [B][H_kv][max_keys]
  int* err;
  int batch, total_q, heads_q, heads_kv, group;
  int page_size, num_pages, max_pages, max_keys, accumulate;
  float scale_log2;
};

// 16-byte chunk c of row r of q in shared memory: rows of 128 bytes, whose two halves
// are exchanged in every other row, so that 8 lanes that read 4 chunks of 2 rows
// touch every bank once.
__device__ __forceinline__ uint32_t mass_q_at(int r, int c) {
  return (uint32_t)r * 128u + (uint32_t)((c ^ ((r & 1) << 2)) << 4);
}

__global__ void __launch_bounds__(kMassThreads, 3)
attn_sink_key_mass_kernel(const __grid_constant__ MassParams p) {
  __shared__ __align__(128) uint8_t s_q[2][kMassRows * 128];
  __shared__ float s_lse[2][kMassRows];    // times log2(e)
  __shared__ int s_at[2][kMassRows];       // last key the row sees; -1: no weight at all
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t = lane & 3;
  const int h = blockIdx.y, b = blockIdx.z;
  const int c0 = __ldg(p.cu_q + b), c1 = __ldg(p.cu_q + b + 1), l0 = __ldg(p.seq_lens + b);
  const int q0 = min(max(c0, 0), p.total_q), n = max(0, min(c1, p.total_q) - q0);
  const int cap = p.max_pages * p.page_size;
  const int len = max(0, min(l0, cap)), keys = min(len, p.max_keys);
  if (tid == 0 && blockIdx.x == 0 && h == 0 &&
      (q0 != c0 || q0 + n != c1 || len != l0 || keys != len))
    atomicCAS(p.err, 0, DEVERR_DECODE_INPUT);
  const long long rows = (long long)n * p.group;
  const int at0 = len - n;                 // key position of token 0
  float* mass = p.mass + ((size_t)b * p.heads_kv + h) * p.max_keys;
  const int* table = p.block_table + (size_t)b * p.max_pages;
  // what of C there is to write
  const int end = p.accumulate ? (n > 0 ? keys : 0) : p.max_keys;
  for (int j0 = blockIdx.x * kMassKeys; j0 < end; j0 += gridDim.x * kMassKeys) {
    if (j0 >= keys || n == 0) {
      if (j0 + tid < end) mass[j0 + tid] = 0.0f;
      continue;
    }
    // A: this warp's 32 keys, two fragments of 16: rows g and g + 8 of each
    uint4 a[4][2];
    bool has[4];
    #pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int j = j0 + 32 * warp + 8 * r + g;
      has[r] = false;
      size_t row = 0;
      if (j < keys) {
        const int pg = j / p.page_size, e = __ldg(table + pg);
        has[r] = (unsigned)e < (unsigned)p.num_pages;
        row = ((size_t)e * p.page_size + (j - pg * p.page_size)) * p.heads_kv + h;
        if (!has[r] && t == 0) atomicCAS(p.err, 0, DEVERR_DECODE_INPUT);
      }
      const uint4* src = reinterpret_cast<const uint4*>(p.k_cache) + row * 8 + t;
      #pragma unroll
      for (int u = 0; u < 2; ++u) a[r][u] = has[r] ? __ldg(src + 4 * u) : make_uint4(0, 0, 0, 0);
    }
    // rows of q from the first token that sees a key of this block
    const long long first = (long long)max(0, j0 - at0) * p.group / kMassRows * kMassRows;
    const int last = min(j0 + kMassKeys, keys) - 1;        // last key of the block
    const int chunks = (int)((rows - first + kMassRows - 1) / kMassRows);
    auto load = [&](int chunk) {
      const long long r0 = first + (long long)chunk * kMassRows;
      const int buf = chunk & 1;
      #pragma unroll
      for (int x = tid; x < kMassRows * 8; x += kMassThreads) {
        const int r = x >> 3;
        const bool in = r0 + r < rows;
        const int tok = in ? (int)((r0 + r) / p.group) : 0;
        const int hd = in ? (int)(r0 + r - (long long)tok * p.group) : 0;
        cp_async_16_zfill(smem_u32(s_q[buf]) + mass_q_at(r, x & 7),
                          p.q + ((size_t)(q0 + tok) * p.heads_q + h * p.group + hd) * 64 +
                              8 * (x & 7),
                          in ? 16 : 0);
      }
      cp_async_commit();
      if (tid < kMassRows) {
        const bool in = r0 + tid < rows;
        float z = 0.0f;
        int at = -1;
        if (in) {
          const int tok = (int)((r0 + tid) / p.group);
          const int hd = (int)(r0 + tid - (long long)tok * p.group);
          z = __ldg(p.lse + (size_t)(h * p.group + hd) * p.total_q + q0 + tok);
          if (!isinf(z)) at = at0 + tok;
        }
        s_lse[buf][tid] = z * kLog2e;
        s_at[buf][tid] = at;
      }
    };
    float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    load(0);
    for (int chunk = 0; chunk < chunks; ++chunk) {
      const int buf = chunk & 1;
      if (chunk + 1 < chunks) {
        load(chunk + 1);
        cp_async_wait<1>();
      } else {
        cp_async_wait<0>();
      }
      __syncthreads();
      const long long left = rows - first - (long long)chunk * kMassRows;
      const int tiles = (int)((min((long long)kMassRows, left) + 7) / 8);
      const bool clear = __all_sync(0xffffffffu, min(s_at[buf][lane], s_at[buf][lane + 32]) >= last);
      const uint32_t base = smem_u32(s_q[buf]);
      for (int i = 0; i < tiles; ++i) {
        uint32_t bq[2][4];
        #pragma unroll
        for (int u = 0; u < 2; ++u)
          ld_shared_v4(base + mass_q_at(8 * i + g, 4 * u + t), bq[u]);
        const float2 z = *reinterpret_cast<const float2*>(&s_lse[buf][8 * i + 2 * t]);
        float c[2][4];
        #pragma unroll
        for (int s = 0; s < 2; ++s) {
          #pragma unroll
          for (int e = 0; e < 4; ++e) c[s][e] = 0.0f;
          #pragma unroll
          for (int u = 0; u < 2; ++u) {
            mma_16816_bf16(c[s], a[2 * s][u].x, a[2 * s + 1][u].x, a[2 * s][u].y,
                           a[2 * s + 1][u].y, bq[u][0], bq[u][1]);
            mma_16816_bf16(c[s], a[2 * s][u].z, a[2 * s + 1][u].z, a[2 * s][u].w,
                           a[2 * s + 1][u].w, bq[u][2], bq[u][3]);
          }
        }
        if (clear) {
          #pragma unroll
          for (int s = 0; s < 2; ++s)
            #pragma unroll
            for (int r = 0; r < 2; ++r)
              sum[2 * s + r] += ex2_approx(fmaf(c[s][2 * r], p.scale_log2, -z.x)) +
                                ex2_approx(fmaf(c[s][2 * r + 1], p.scale_log2, -z.y));
        } else {
          const int2 at = *reinterpret_cast<const int2*>(&s_at[buf][8 * i + 2 * t]);
          #pragma unroll
          for (int s = 0; s < 2; ++s)
            #pragma unroll
            for (int r = 0; r < 2; ++r) {
              const int j = j0 + 32 * warp + 16 * s + 8 * r + g;
              const float w0 = ex2_approx(fmaf(c[s][2 * r], p.scale_log2, -z.x));
              const float w1 = ex2_approx(fmaf(c[s][2 * r + 1], p.scale_log2, -z.y));
              sum[2 * s + r] += (j <= at.x ? w0 : 0.0f) + (j <= at.y ? w1 : 0.0f);
            }
        }
      }
      __syncthreads();                     // the buffer is filled again
    }
    #pragma unroll
    for (int r = 0; r < 4; ++r) {
      sum[r] += __shfl_xor_sync(0xffffffffu, sum[r], 1);
      sum[r] += __shfl_xor_sync(0xffffffffu, sum[r], 2);
      if (!has[r]) sum[r] = 0.0f;
    }
    // lane t of four writes key 8 t + g
    const float mine = t == 0 ? sum[0] : t == 1 ? sum[1] : t == 2 ? sum[2] : sum[3];
    const int j = j0 + 32 * warp + 8 * t + g;
    if (j < keys) mass[j] = p.accumulate ? mass[j] + mine : mine;
    else if (j < end) mass[j] = 0.0f;
  }
}

}  // namespace attn_sink
