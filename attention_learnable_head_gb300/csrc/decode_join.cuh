// Joins the slices of a decode step (decode_kernel.cuh, kDecPages and kDecShared), the
// parts of a shared prefix (shared_kernel.cuh) and the sink, in a fixed order:
//   M = max(m_c, sink), Z = sum l_c 2^(m_c - M) + 2^(sink - M), O = sum 2^(m_c - M) o_c / Z.
//
// A warp takes a row (sequence, query head): 16 lanes of 4 dimensions for the even
// slices, 16 for the odd ones.  It costs the chain of its loads, so the sums of 16 slices
// go out together, before their weights are known.  A kernel of its own, launched
// while the slices are computed: counting the slices and letting the last CTA of a row
// join them takes a memory fence in every CTA and the counters' clearing in front.
#pragma once
#include "decode_kernel.cuh"

namespace attn_sink {

constexpr int kDecJoinThreads = 128;
constexpr int kDecJoinParts = 128;       // slices (up to 64) and prefix parts (up to 64)

template <bool kShared>
__global__ void __launch_bounds__(kDecJoinThreads)
attn_sink_decode_join_kernel(const __grid_constant__ DecodeParams p) {
  const int lane = threadIdx.x & 31, odd = lane >> 4, d = 4 * (lane & 15);
  const unsigned row = blockIdx.x * (kDecJoinThreads / 32) + (threadIdx.x >> 5);
  const unsigned b = row / (unsigned)p.heads_q;
  const int hq = (int)(row - b * (unsigned)p.heads_q);
  const bool in = b < (unsigned)p.batch;
  const float s2 = in ? __ldg(p.sink + hq) * kLog2eDec : 0.0f;
  grid_dependency_wait();
  if (!in) return;
  // part c: slice c, then the prefix's parts, whose rows lie a tile's rows apart
  int parts = p.splits;
  const float2* ml = p.slice_ml + (size_t)row * p.splits;
  const float* o = p.slice_o + (size_t)row * p.splits * 64 + d;
  const float2* pml = nullptr;
  const float* po = nullptr;
  const size_t pstep = (size_t)p.heads_kv * kDecTileRows;
  if constexpr (kShared) {
    const int4 r = __ldcg(reinterpret_cast<const int4*>(p.refs + b));     // a SharedRef
    const int group = p.heads_q / p.heads_kv, g = hq / group;
    const size_t at = ((size_t)r.x * p.heads_kv + g) * kDecTileRows + r.z * group + (hq - g * group);
    parts += r.y;
    pml = p.prefix_ml + at - (size_t)p.splits * pstep;
    po = p.prefix_o + at * 64 + d - (size_t)p.splits * pstep * 64;
  }
  auto load = [&](int c) {
    const float* src = kShared && c >= p.splits ? po + (size_t)c * pstep * 64 : o + (size_t)c * 64;
    return c < parts ? __ldcg(reinterpret_cast<const float4*>(src))
                     : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  };
  constexpr int kEach = (kShared ? kDecJoinParts : kDecJoinParts / 2) / 32;
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
    p.lse[(size_t)hq * p.batch + b] = z != 0.0f ? (mb + __log2f(z)) * kLn2Dec : -INFINITY;
}

}  // namespace attn_sink
