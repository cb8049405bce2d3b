// RMS norm of every query and key head and rotary positions, in one pass over
// the packed projection, and its gradient.
//
//   u = x r w,  r = 1 / sqrt(mean(x^2) + eps)          (x: one head, 64 numbers)
//   y = a R(angle) u                                   (pairs of dimensions)
// Forward: with C[d] = a cos and S[d] = -+ a sin of dimension d's pair (C = 1,
// S = 0 where d is not rotated) and d' the other dimension of the pair,
//   y_d = r (x_d w_d C_d + x_d' w_d' S_d).
// Gradient, g = a R^T dy (the same with S negated), h = w g:
//   dw = sum over tokens and heads of g x r,
//   dx = r (h - x r^2 mean(h x)).
//
// Both are bound by memory: they read and write each number once.  Eight lanes
// hold a head (16 bytes each), so a warp takes four heads at a time; the
// mean square (and mean(h x)) are three shuffles, the other dimension of a
// pair comes from another lane by shuffle (halves) or lies in the lane's own
// eight (interleaved).  A warp computes the 32 angles of a token once, one per
// lane, and keeps C and S in shared memory for all heads of the token.  The
// angle is positions * inv_freq / 2 pi in fp64, reduced to one turn there, so
// that the fp32 sine and cosine of a position of a million are as exact as
// those of position one (an fp32 product would be off by 0.06 radians).
#pragma once
#include <cuda_bf16.h>
#include "sm103_ptx.cuh"

namespace attn_sink {

constexpr int kRopeThreads = 256;
constexpr int kRopeWarps = kRopeThreads / 32;

struct RopeParams {
  const __nv_bfloat16* q;      // [T] rows of q_stride elements
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  const int* positions;        // [axes][T]
  const float* inv_freq;       // [rotary / 2]
  const void* q_weight;        // [64] fp32 or bf16
  const void* k_weight;
  const long long* slots;      // [T] or null
  __nv_bfloat16* q_out;        // [T][H_q][64]
  __nv_bfloat16* k_out;        // [T][H_kv][64] or null
  __nv_bfloat16* v_out;
  __nv_bfloat16* k_cache;      // [rows][H_kv][64]
  __nv_bfloat16* v_cache;
  // gradient: dy from the attention, dx into the projection's gradient
  const void* dq;
  const void* dk;
  const void* dv;
  __nv_bfloat16* dq_in;
  __nv_bfloat16* dk_in;
  __nv_bfloat16* dv_in;
  float* dw_part;              // [CTAs][2][64]
  int* err;
  long long q_stride, k_stride, v_stride;
  long long dq_in_stride, dk_in_stride, dv_in_stride;
  long long cache_rows;
  int tokens, heads_q, heads_kv;
  int rotary;
  int parts;                   // warps that share the heads of a token
  int weight_bf16;
  float eps, amplitude;
  unsigned char pair_axis[32];
};

// The eight numbers a lane holds of a head.
struct Oct {
  float e[8];
};

__device__ __forceinline__ Oct oct_from_bf16(uint4 w) {
  Oct o;
  o.e[0] = bf16_lo(w.x); o.e[1] = bf16_hi(w.x);
  o.e[2] = bf16_lo(w.y); o.e[3] = bf16_hi(w.y);
  o.e[4] = bf16_lo(w.z); o.e[5] = bf16_hi(w.z);
  o.e[6] = bf16_lo(w.w); o.e[7] = bf16_hi(w.w);
  return o;
}
__device__ __forceinline__ uint4 oct_to_bf16(const Oct& o) {
  return make_uint4(pack_bf16x2(o.e[0], o.e[1]), pack_bf16x2(o.e[2], o.e[3]),
                    pack_bf16x2(o.e[4], o.e[5]), pack_bf16x2(o.e[6], o.e[7]));
}
__device__ __forceinline__ Oct oct_load(const float* s) {
  Oct o;
  const float4 a = reinterpret_cast<const float4*>(s)[0], b = reinterpret_cast<const float4*>(s)[1];
  o.e[0] = a.x; o.e[1] = a.y; o.e[2] = a.z; o.e[3] = a.w;
  o.e[4] = b.x; o.e[5] = b.y; o.e[6] = b.z; o.e[7] = b.w;
  return o;
}
__device__ __forceinline__ float sum8(float x) {       // over the eight lanes of a head
  x += __shfl_xor_sync(0xffffffffu, x, 1);
  x += __shfl_xor_sync(0xffffffffu, x, 2);
  x += __shfl_xor_sync(0xffffffffu, x, 4);
  return x;
}
__device__ __forceinline__ uint4 ld_stream(const void* p) {   // read once: not kept in L1
  uint4 r;
  asm volatile("ld.global.nc.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p));
  return r;
}

__device__ __forceinline__ float rope_weight(const void* w, int bf16, int d) {
  if (w == nullptr) return 1.0f;
  return bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(w)[d])
              : static_cast<const float*>(w)[d];
}

// The other dimension of d's pair (d itself where d is not rotated).
template <bool kInter>
__device__ __forceinline__ int rope_partner(int d, int rotary) {
  if (d >= rotary) return d;
  if (kInter) return d ^ 1;
  const int half = rotary >> 1;
  return d < half ? d + half : d - half;
}

// C and S of a token into sC, sS [64]: lane i computes pair i.
template <bool kInter>
__device__ __forceinline__ void rope_angles(const RopeParams& p, int t, int lane, double freq,
                                            float* sC, float* sS) {
  __syncwarp();                            // the last token's heads have read C and S
  const int pairs = p.rotary >> 1;
  if (lane < pairs) {
    const int pos = __ldg(p.positions + (size_t)p.pair_axis[lane] * p.tokens + t);
    double turns = (double)pos * freq;     // freq = inv_freq / 2 pi
    turns -= rint(turns);
    float s, c;
    sincospif(2.0f * (float)turns, &s, &c);
    s *= p.amplitude;
    c *= p.amplitude;
    const int d0 = kInter ? 2 * lane : lane;
    const int d1 = kInter ? d0 + 1 : lane + pairs;
    sC[d0] = c;
    sC[d1] = c;
    sS[d0] = -s;
    sS[d1] = s;
  }
  __syncwarp();
}

template <bool kInter>
__device__ __forceinline__ Oct oct_partner(const Oct& x, int src_lane) {
  Oct o;
  if (kInter) {
    #pragma unroll
    for (int e = 0; e < 8; ++e) o.e[e] = x.e[e ^ 1];
  } else {
    #pragma unroll
    for (int e = 0; e < 8; ++e) o.e[e] = __shfl_sync(0xffffffffu, x.e[e], src_lane);
  }
  return o;
}
template <bool kInter>
__device__ __forceinline__ Oct oct_partner_bf16(uint4 w, int src_lane) {
  if (kInter) return oct_partner<true>(oct_from_bf16(w), 0);
  uint4 o;
  o.x = __shfl_sync(0xffffffffu, w.x, src_lane);
  o.y = __shfl_sync(0xffffffffu, w.y, src_lane);
  o.z = __shfl_sync(0xffffffffu, w.z, src_lane);
  o.w = __shfl_sync(0xffffffffu, w.w, src_lane);
  return oct_from_bf16(o);
}

// Where lane `lane` of a warp sits: eight lanes a head, four heads a step.
struct RopeLane {
  int sub, j, src;      // head of the step, chunk of the head, lane of the pairs' other halves
  double freq;
};
template <bool kInter>
__device__ __forceinline__ RopeLane rope_lane(const RopeParams& p, int lane) {
  RopeLane r;
  r.sub = lane >> 3;
  r.j = lane & 7;
  r.src = (lane & 24) | (rope_partner<kInter>(8 * r.j, p.rotary) >> 3);
  r.freq = lane < (p.rotary >> 1)
               ? (double)__ldg(p.inv_freq + lane) * 0.15915494309189533577   // 1 / (2 pi)
               : 0.0;
  return r;
}

// Heads [h0, h1) of one tensor of a token that a part works on: whole steps of
// four heads, spread over the parts.
__device__ __forceinline__ void rope_share(int heads, int part, int parts, int* h0, int* h1) {
  const int steps = (heads + 3) >> 2;
  *h0 = 4 * (int)((long long)steps * part / parts);
  *h1 = min(heads, 4 * (int)((long long)steps * (part + 1) / parts));
}

template <bool kNorm, bool kInter>
__global__ void __launch_bounds__(kRopeThreads)
attn_sink_rope_kernel(const RopeParams p) {
  __shared__ __align__(16) float s_w[2][2][64];            // q, k: weight, the partner's weight
  __shared__ __align__(16) float s_cs[kRopeWarps][2][64];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (kNorm && tid < 128) {
    const int which = tid >> 6, d = tid & 63;
    const void* w = which ? p.k_weight : p.q_weight;
    s_w[which][0][d] = rope_weight(w, p.weight_bf16, d);
    s_w[which][1][d] = rope_weight(w, p.weight_bf16, rope_partner<kInter>(d, p.rotary));
  }
  float* sC = s_cs[warp][0];
  float* sS = s_cs[warp][1];
  for (int d = lane; d < 64; d += 32) {                    // the dimensions that pass
    sC[d] = 1.0f;
    sS[d] = 0.0f;
  }
  const RopeLane me = rope_lane<kInter>(p, lane);
  __syncthreads();
  const size_t kv_row = (size_t)p.heads_kv * 64;
  const long long items = (long long)p.tokens * p.parts;
  for (long long it = (long long)blockIdx.x * kRopeWarps + warp; it < items;
       it += (long long)gridDim.x * kRopeWarps) {
    const int t = (int)(it / p.parts), part = (int)(it - (long long)t * p.parts);
    rope_angles<kInter>(p, t, lane, me.freq, sC, sS);
    long long slot = -1;
    if (p.slots != nullptr) {
      slot = __ldg(p.slots + t);
      if (slot < -1 || slot >= p.cache_rows) {
        if (lane == 0) atomicCAS(p.err, 0, DEVERR_DECODE_INPUT);
        slot = -1;
      }
    }
    #pragma unroll
    for (int which = 0; which < 2; ++which) {              // q, then k
      const int heads = which ? p.heads_kv : p.heads_q;
      if (which && p.k_out == nullptr && slot < 0) break;
      Oct a = oct_load(sC + 8 * me.j), b = oct_load(sS + 8 * me.j);
      if (kNorm) {
        const Oct w = oct_load(&s_w[which][0][8 * me.j]), wp = oct_load(&s_w[which][1][8 * me.j]);
        #pragma unroll
        for (int e = 0; e < 8; ++e) {
          a.e[e] *= w.e[e];
          b.e[e] *= wp.e[e];
        }
      }
      const __nv_bfloat16* src = which ? p.k + (size_t)t * p.k_stride : p.q + (size_t)t * p.q_stride;
      int h0, h1;
      rope_share(heads, part, p.parts, &h0, &h1);
      #pragma unroll 4
      for (int h = h0; h < h1; h += 4) {
        const int hd = h + me.sub;
        const bool on = hd < h1;
        uint4 raw = make_uint4(0, 0, 0, 0);
        if (on) raw = ld_stream(src + (size_t)hd * 64 + 8 * me.j);
        const Oct x = oct_from_bf16(raw);
        const Oct xp = oct_partner_bf16<kInter>(raw, me.src);
        float inv = 1.0f;
        if (kNorm) {
          float ss = 0.0f;
          #pragma unroll
          for (int e = 0; e < 8; ++e) ss = fmaf(x.e[e], x.e[e], ss);
          inv = rsqrtf(sum8(ss) * (1.0f / 64.0f) + p.eps);
        }
        Oct y;
        #pragma unroll
        for (int e = 0; e < 8; ++e) {
          y.e[e] = fmaf(xp.e[e], b.e[e], x.e[e] * a.e[e]);
          if (kNorm) y.e[e] *= inv;
        }
        const uint4 o = oct_to_bf16(y);
        if (on) {
          const size_t off = (size_t)hd * 64 + 8 * me.j;
          if (which == 0) {
            *reinterpret_cast<uint4*>(p.q_out + (size_t)t * p.heads_q * 64 + off) = o;
          } else {
            if (p.k_out) *reinterpret_cast<uint4*>(p.k_out + (size_t)t * kv_row + off) = o;
            if (slot >= 0) *reinterpret_cast<uint4*>(p.k_cache + (size_t)slot * kv_row + off) = o;
          }
        }
      }
    }
    if (p.v_out != nullptr || slot >= 0) {
      int h0, h1;
      rope_share(p.heads_kv, part, p.parts, &h0, &h1);
      for (int h = h0; h < h1; h += 4) {
        const int hd = h + me.sub;
        if (hd >= h1) continue;
        const size_t off = (size_t)hd * 64 + 8 * me.j;
        const uint4 raw = ld_stream(p.v + (size_t)t * p.v_stride + off);
        if (p.v_out) *reinterpret_cast<uint4*>(p.v_out + (size_t)t * kv_row + off) = raw;
        if (slot >= 0) *reinterpret_cast<uint4*>(p.v_cache + (size_t)slot * kv_row + off) = raw;
      }
    }
  }
}

template <bool kFp32>
__device__ __forceinline__ Oct grad_load(const void* base, size_t off) {
  if (kFp32) {
    const float* f = static_cast<const float*>(base) + off;
    const uint4 a = ld_stream(f), b = ld_stream(f + 4);
    Oct o;
    o.e[0] = __uint_as_float(a.x); o.e[1] = __uint_as_float(a.y);
    o.e[2] = __uint_as_float(a.z); o.e[3] = __uint_as_float(a.w);
    o.e[4] = __uint_as_float(b.x); o.e[5] = __uint_as_float(b.y);
    o.e[6] = __uint_as_float(b.z); o.e[7] = __uint_as_float(b.w);
    return o;
  }
  return oct_from_bf16(ld_stream(static_cast<const __nv_bfloat16*>(base) + off));
}

template <bool kNorm, bool kInter, bool kFp32>
__global__ void __launch_bounds__(kRopeThreads)
attn_sink_rope_bwd_kernel(const RopeParams p) {
  __shared__ __align__(16) float s_w[2][64];
  __shared__ __align__(16) float s_cs[kRopeWarps][2][64];
  __shared__ __align__(16) float s_dw[kRopeWarps][2][64];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (kNorm && tid < 128)
    s_w[tid >> 6][tid & 63] =
        rope_weight(tid >> 6 ? p.k_weight : p.q_weight, p.weight_bf16, tid & 63);
  float* sC = s_cs[warp][0];
  float* sS = s_cs[warp][1];
  for (int d = lane; d < 64; d += 32) {
    sC[d] = 1.0f;
    sS[d] = 0.0f;
  }
  const RopeLane me = rope_lane<kInter>(p, lane);
  __syncthreads();
  float dw[2][8];
  #pragma unroll
  for (int e = 0; e < 8; ++e) dw[0][e] = dw[1][e] = 0.0f;
  const long long items = (long long)p.tokens * p.parts;
  for (long long it = (long long)blockIdx.x * kRopeWarps + warp; it < items;
       it += (long long)gridDim.x * kRopeWarps) {
    const int t = (int)(it / p.parts), part = (int)(it - (long long)t * p.parts);
    rope_angles<kInter>(p, t, lane, me.freq, sC, sS);
    #pragma unroll
    for (int which = 0; which < 2; ++which) {
      const int heads = which ? p.heads_kv : p.heads_q;
      const Oct c = oct_load(sC + 8 * me.j), s = oct_load(sS + 8 * me.j);
      Oct w;
      if (kNorm) w = oct_load(&s_w[which][8 * me.j]);
      const void* dy = which ? p.dk : p.dq;
      const __nv_bfloat16* src = which ? p.k + (size_t)t * p.k_stride : p.q + (size_t)t * p.q_stride;
      __nv_bfloat16* dst = which ? p.dk_in + (size_t)t * p.dk_in_stride
                                 : p.dq_in + (size_t)t * p.dq_in_stride;
      int h0, h1;
      rope_share(heads, part, p.parts, &h0, &h1);
      #pragma unroll 2
      for (int h = h0; h < h1; h += 4) {
        const int hd = h + me.sub;
        const bool on = hd < h1;
        Oct d, x;
        #pragma unroll
        for (int e = 0; e < 8; ++e) d.e[e] = x.e[e] = 0.0f;
        if (on) {
          d = grad_load<kFp32>(dy, ((size_t)t * heads + hd) * 64 + 8 * me.j);
          if (kNorm) x = oct_from_bf16(ld_stream(src + (size_t)hd * 64 + 8 * me.j));
        }
        const Oct dp = oct_partner<kInter>(d, me.src);
        Oct g;
        #pragma unroll
        for (int e = 0; e < 8; ++e) g.e[e] = fmaf(-dp.e[e], s.e[e], d.e[e] * c.e[e]);
        if (kNorm) {
          float ss = 0.0f, hx = 0.0f;
          #pragma unroll
          for (int e = 0; e < 8; ++e) {
            ss = fmaf(x.e[e], x.e[e], ss);
            hx = fmaf(g.e[e] * w.e[e], x.e[e], hx);
          }
          ss = sum8(ss);
          hx = sum8(hx);
          const float inv = rsqrtf(ss * (1.0f / 64.0f) + p.eps);
          const float back = hx * (1.0f / 64.0f) * inv * inv;
          #pragma unroll
          for (int e = 0; e < 8; ++e) {
            dw[which][e] = fmaf(g.e[e] * inv, x.e[e], dw[which][e]);
            g.e[e] = inv * fmaf(-x.e[e], back, g.e[e] * w.e[e]);
          }
        }
        if (on) *reinterpret_cast<uint4*>(dst + (size_t)hd * 64 + 8 * me.j) = oct_to_bf16(g);
      }
    }
    if (p.dv != nullptr) {
      int h0, h1;
      rope_share(p.heads_kv, part, p.parts, &h0, &h1);
      for (int h = h0; h < h1; h += 4) {
        const int hd = h + me.sub;
        if (hd >= h1) continue;
        const Oct d = grad_load<kFp32>(p.dv, ((size_t)t * p.heads_kv + hd) * 64 + 8 * me.j);
        *reinterpret_cast<uint4*>(p.dv_in + (size_t)t * p.dv_in_stride + (size_t)hd * 64 +
                                  8 * me.j) = oct_to_bf16(d);
      }
    }
  }
  if constexpr (kNorm) {
    // this CTA's weight gradients: the four heads of a step, then the warps, in order
    #pragma unroll
    for (int which = 0; which < 2; ++which) {
      #pragma unroll
      for (int e = 0; e < 8; ++e) {
        float x = dw[which][e];
        x += __shfl_xor_sync(0xffffffffu, x, 8);
        x += __shfl_xor_sync(0xffffffffu, x, 16);
        if (me.sub == 0) s_dw[warp][which][8 * me.j + e] = x;
      }
    }
    __syncthreads();
    if (tid < 128) {
      float x = 0.0f;
      #pragma unroll
      for (int w = 0; w < kRopeWarps; ++w) x += s_dw[w][tid >> 6][tid & 63];
      p.dw_part[(size_t)blockIdx.x * 128 + tid] = x;
    }
  }
}

// The CTAs' partial weight gradients in a fixed order: thread (g, d) sums every
// eighth CTA's, then the eight sums are added in order.
constexpr int kRopeSumThreads = 1024;
__global__ void __launch_bounds__(kRopeSumThreads)
attn_sink_rope_dw_kernel(const float* part, int ctas, float* dwq, float* dwk) {
  __shared__ float s[8][128];
  const int d = threadIdx.x & 127, g = threadIdx.x >> 7;
  float x = 0.0f;
  for (int c = g; c < ctas; c += 8) x += part[(size_t)c * 128 + d];
  s[g][d] = x;
  __syncthreads();
  if (g == 0) {
    #pragma unroll
    for (int i = 1; i < 8; ++i) x += s[i][d];
    (d < 64 ? dwq : dwk)[d & 63] = x;
  }
}

}  // namespace attn_sink
