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
// hold a head, each the eight numbers that turn together: four of the first and
// the same four of the second half of the pairs (interleaved: eight neighbours),
// so that no number of a pair has to come from another lane, and the mean square
// (and mean(h x)) are three shuffles.  Where fewer dimensions are rotated the
// lanes behind the pairs hold eight neighbours too.  A warp takes four heads at
// a time.  What keeps the memory busy is a ring of chunks of heads per warp in
// shared memory, filled by bulk copies several chunks ahead and across tokens:
// loads into registers (four steps ahead, then a wait) left 57 % of the time
// waiting, and 16-byte cp.async cost 20 instructions a step.  A warp computes the
// 32 angles of a token once, one per lane, and keeps C and S in shared memory for
// all heads of the token.  The angle is positions * inv_freq / 2 pi; with the
// factor's fraction of a turn as a 64-bit integer the product is the fraction that is
// left (whole turns drop out of the multiplication), so the fp32 sine and cosine of a
// position of a million are as exact as those of position one (an fp32 product would
// be off by 0.06 radians).  10 + 2 + 2 heads take 59.2 us with all 64 bits of it and
// 58.2 with the upper 32.
#pragma once
#include <cuda_bf16.h>
#include "sm103_ptx.cuh"

namespace attn_sink {

constexpr int kRopeThreads = 128;
constexpr int kRopeWarps = kRopeThreads / 32;
// Chosen by sweeping CTAs per SM, heads of a bulk copy and chunks of the ring on
// 65536 tokens of 64 + 8 + 8 heads: the forward takes 205 us (floor at the
// measured copy rate 198) with 5 x 8 x 2 or 3 x 16 x 3, and 214 to 254 with more
// or larger copies in flight, which set the reads against the writes; the
// gradient 296 us (floor 287) with 4 x 8 x 3 and 317 to 380 with smaller chunks
// or more CTAs.
constexpr int kRopeCtas = 5;       // resident CTAs per SM, forward
constexpr int kRopeChunk = 8;      // heads of a bulk copy
constexpr int kRopeDepth = 2;      // chunks in a warp's ring
constexpr int kRopeBwdCtas = 4;    // and of the gradient
constexpr int kRopeBwdChunk = 8;
constexpr int kRopeBwdDepth = 3;
// Where a warp's share of a token is this many heads of q, k and v together or less,
// a stage of the ring takes them all, with one wait for the three tensors (kWhole): a
// token of few heads is bound by instructions (750 for 5 + 1 + 1 heads with a wait for
// each tensor) and few tokens by the chain of waits.  Whole and by chunks: 65536
// tokens of 8 + 1 + 1 heads 58 and 69 us, of 10 + 2 + 2 59 and 79, of 16 + 2 + 2 61
// and 82, of 20 + 4 + 4 86 and 94, of 16 + 8 + 8 (not taken) 97 and 92; 64 tokens 4.4
// and 5.2.  The gradient, 12 + 2 + 2 heads 82 and 112, 8 + 1 + 1 73 and 95, with fp32
// gradients 75 and 97; its stages hold dy too and have to fit 48 KB with four warps.
constexpr int kRopeWhole = 28;
constexpr int kRopeBwdWhole = 17;      // of the gradient, dy in bf16
constexpr int kRopeBwdWholeFp32 = 11;
constexpr int kRopeWholeDepth = 2;

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
  int weight_bf16;
  float eps, amplitude;
  unsigned char pair_axis[32];
};

// The eight numbers a lane holds of a head, as packed fp32 pairs: numbers 0-3 lie
// at dimension d0, numbers 4-7 at d1.  The other number of number i's pair is
// number i ^ 4 (interleaved: i ^ 1).  In odd heads of a step d0 and d1 change
// places, so that the lanes of two heads read different banks of shared memory.
struct Oct {
  uint64_t e[4];
};

__device__ __forceinline__ uint64_t bf16x2_to_f2(uint32_t w) { return f2(bf16_lo(w), bf16_hi(w)); }
__device__ __forceinline__ uint32_t f2_to_bf16x2(uint64_t v) {
  return pack_bf16x2(f2_lo(v), f2_hi(v));
}
__device__ __forceinline__ Oct oct_from_bf16(uint2 a, uint2 b) {
  Oct o;
  o.e[0] = bf16x2_to_f2(a.x);
  o.e[1] = bf16x2_to_f2(a.y);
  o.e[2] = bf16x2_to_f2(b.x);
  o.e[3] = bf16x2_to_f2(b.y);
  return o;
}
// number i -> the other number of its pair
template <bool kInter>
__device__ __forceinline__ Oct oct_other(const Oct& x) {
  Oct o;
  if (kInter) {
    #pragma unroll
    for (int i = 0; i < 4; ++i) o.e[i] = f2(f2_hi(x.e[i]), f2_lo(x.e[i]));
  } else {
    o.e[0] = x.e[2];
    o.e[1] = x.e[3];
    o.e[2] = x.e[0];
    o.e[3] = x.e[1];
  }
  return o;
}
// sum of a number's squares, or of products
__device__ __forceinline__ float oct_dot(const Oct& a, const Oct& b) {
  uint64_t t = fmul2(a.e[0], b.e[0]);
  #pragma unroll
  for (int i = 1; i < 4; ++i) t = ffma2(a.e[i], b.e[i], t);
  return f2_lo(t) + f2_hi(t);
}
__device__ __forceinline__ float sum8(float x) {       // over the eight lanes of a head
  x += __shfl_xor_sync(0xffffffffu, x, 1);
  x += __shfl_xor_sync(0xffffffffu, x, 2);
  x += __shfl_xor_sync(0xffffffffu, x, 4);
  return x;
}
__device__ __forceinline__ float rope_weight(const void* w, int bf16, int d) {
  if (w == nullptr) return 1.0f;
  return bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(w)[d])
              : static_cast<const float*>(w)[d];
}

// Where a lane sits: eight lanes a head, four heads a step.
struct RopeLane {
  int sub, d0, d1;      // head of the step; dimensions of numbers 0-3 and 4-7
  int at0;              // place of numbers 0-3 in a table of 64 (4-7: at0 ^ 4)
  long long freq;       // pair `lane`'s turns a position, times 2^64 (without whole turns)
  float bad;            // 0, NaN where inv_freq is not finite
};
template <bool kInter>
__device__ __forceinline__ RopeLane rope_lane(const RopeParams& p, int lane) {
  RopeLane r;
  r.sub = lane >> 3;
  const int j = lane & 7;
  const bool halves = !kInter && j < p.rotary / 8;       // rotary is a multiple of 16
  const int lo = halves ? 4 * j : 8 * j, hi = halves ? 4 * j + p.rotary / 2 : 8 * j + 4;
  const bool odd = r.sub & 1;
  r.d0 = odd ? hi : lo;
  r.d1 = odd ? lo : hi;
  r.at0 = 8 * j + (odd ? 4 : 0);
  const float f = lane < (p.rotary >> 1) ? __ldg(p.inv_freq + lane) : 0.0f;
  const double turns = (double)f * 0.15915494309189533577;                  // 1 / (2 pi)
  r.freq = __double2ll_rn((turns - rint(turns)) * 18446744073709551616.0);  // 2^64
  r.bad = f - f;
  return r;
}

// C and S of a token in tables of 64: the numbers of lane j of an even head at 8 j
// (rope_table_dim).  Lane i computes pair i.
template <bool kInter>
__device__ __forceinline__ void rope_angles(const RopeParams& p, int pos, int lane,
                                            const RopeLane& me, float* sC, float* sS) {
  __syncwarp();                            // the last token's heads have read C and S
  if (lane < (p.rotary >> 1)) {
    // positions are whole numbers: whole turns leave the 64 bits at the top.  The lower
    // half counts too, as a signed number, so that an angle far below a turn keeps 24
    // bits (with the upper 32 alone one of 1e-7 had six).  Two conversions of 32 bits:
    // one of 64 took 2 % more with few heads a token.
    const unsigned long long turns = (unsigned long long)(long long)pos *
                                     (unsigned long long)me.freq;
    const float whole = (float)(int)((turns + 0x80000000ull) >> 32) * 4.656612873077392578e-10f;
    float s, c;
    sincospif(fmaf((float)(int)turns, 1.0842021724855044e-19f, whole) + me.bad, &s, &c);  // 2^-63
    s *= p.amplitude;
    c *= p.amplitude;
    const int a = kInter ? 2 * lane : (lane >> 2) * 8 + (lane & 3);
    const int b = kInter ? a + 1 : a + 4;
    sC[a] = c;
    sC[b] = c;
    sS[a] = -s;
    sS[b] = s;
  }
  __syncwarp();
}
__device__ __forceinline__ Oct oct_load(const float* table, int at0) {
  const ulonglong2 a = *reinterpret_cast<const ulonglong2*>(table + at0);
  const ulonglong2 b = *reinterpret_cast<const ulonglong2*>(table + (at0 ^ 4));
  return Oct{{a.x, a.y, b.x, b.y}};
}
// The dimension at place i of such a table.
template <bool kInter>
__device__ __forceinline__ int rope_table_dim(int i, int rotary) {
  if (kInter || i >= rotary) return i;
  return (i >> 3) * 4 + (i & 3) + ((i & 4) ? rotary / 2 : 0);
}

// A warp's ring of chunks: one lane issues the bulk copies, a barrier per stage
// counts their bytes; every wait is bounded (kWaitLimitNs).
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes,
                                          uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::
          "r"(smem_u32(dst)),
      "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}

// Heads [h0, h1) of one tensor of a token that a part works on: whole steps of
// four heads, spread over the parts.
__device__ __forceinline__ void rope_share(int heads, int part, int parts, int* h0, int* h1) {
  if (parts == 1) {
    *h0 = 0;
    *h1 = heads;
    return;
  }
  const int steps = (heads + 3) >> 2;
  *h0 = 4 * (int)((long long)steps * part / parts);
  *h1 = min(heads, 4 * (int)((long long)steps * (part + 1) / parts));
}

// A CTA works on one part (blockIdx.y) of the heads of its tokens; warp w of all
// those of the part takes tokens w, w + warps, ...
struct RopePart {
  int q0, q1, k0, k1;                      // heads of q, and of k and v
  int nq, nk;                              // steps of q, and of k (and of v)
  unsigned first, stride;                  // tokens
};
__device__ __forceinline__ RopePart rope_part(const RopeParams& p, int warp) {
  RopePart x;
  rope_share(p.heads_q, blockIdx.y, gridDim.y, &x.q0, &x.q1);
  rope_share(p.heads_kv, blockIdx.y, gridDim.y, &x.k0, &x.k1);
  x.nq = (x.q1 - x.q0 + 3) >> 2;
  x.nk = (x.k1 - x.k0 + 3) >> 2;
  x.first = blockIdx.x * kRopeWarps + warp;
  x.stride = gridDim.x * kRopeWarps;
  return x;
}

// A copy did not land within the wait limit: record it, and give those in flight
// (chunks used - 1 .. issued - 1) time to land before the CTA leaves its memory.
__device__ __forceinline__ void rope_give_up(const RopeParams& p, uint64_t* full, int used,
                                             int issued, int depth) {
  atomicCAS(p.err, 0, DEVERR_TIMEOUT_FWD + 9);
  for (int i = used - 1; i < issued; ++i) mbar_wait(&full[i % depth], (i / depth) & 1, nullptr);
}

template <bool kNorm, bool kInter, bool kWhole>
__global__ void __launch_bounds__(kRopeThreads, kRopeCtas)
attn_sink_rope_kernel(const __grid_constant__ RopeParams p) {
  constexpr int kDepth = kWhole ? kRopeWholeDepth : kRopeDepth;
  // a step of four heads may read three behind the last
  constexpr int kStage = (kWhole ? kRopeWhole + 4 : kRopeChunk) * 128;
  __shared__ __align__(16) float s_w[2][2][64];            // q, k: weight, the other number's
  __shared__ __align__(16) float s_cs[kRopeWarps][2][64];
  __shared__ __align__(128) uint8_t s_ring[kRopeWarps][kDepth][kStage];
  __shared__ __align__(8) uint64_t s_full[kRopeWarps][kDepth];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const RopeLane me = rope_lane<kInter>(p, lane);
  const int j8 = 8 * (lane & 7);
  if (kNorm) {
    const int which = tid >> 6, i = tid & 63;
    const void* w = which ? p.k_weight : p.q_weight;
    s_w[which][0][i] = rope_weight(w, p.weight_bf16, rope_table_dim<kInter>(i, p.rotary));
    s_w[which][1][i] =
        rope_weight(w, p.weight_bf16, rope_table_dim<kInter>(kInter ? i ^ 1 : i ^ 4, p.rotary));
  }
  float* sC = s_cs[warp][0];
  float* sS = s_cs[warp][1];
  for (int d = lane; d < 64; d += 32) {                    // the dimensions that pass
    sC[d] = 1.0f;
    sS[d] = 0.0f;
  }
  if (lane == 0) {
    for (int i = 0; i < kDepth; ++i) mbar_init(&s_full[warp][i], 1);
    fence_mbarrier_init();
  }
  __syncthreads();
  const RopePart x = rope_part(p, warp);
  const unsigned tokens = (unsigned)p.tokens;
  const bool with_kv = p.k_out != nullptr || p.slots != nullptr;
  const bool with_v = p.v_out != nullptr || p.slots != nullptr;
  unsigned t = x.first;
  if (t >= tokens || x.nq + (with_kv || with_v ? x.nk : 0) == 0) return;

  // The copies run ahead (lane 0): token ft, tensor fk of it (q, k, v), the next
  // heads' source and how many heads are left.
  unsigned ft = t;
  int fk = -1, left = 0, issued = 0;
  const __nv_bfloat16* src = nullptr;
  const int in_q = x.q1 - x.q0, in_k = with_kv ? x.k1 - x.k0 : 0;
  const int in_v = with_v ? x.k1 - x.k0 : 0;
  auto fetch = [&]() {
    if constexpr (kWhole) {
      if (ft >= tokens) return;
      const int st = issued % kDepth;
      uint8_t* to = s_ring[warp][st];
      uint64_t* bar = &s_full[warp][st];
      mbar_arrive_expect_tx(bar, (in_q + in_k + in_v) * 128);
      if (in_q > 0) bulk_load(to, p.q + (size_t)ft * p.q_stride + x.q0 * 64, in_q * 128, bar);
      to += in_q * 128;
      if (in_k > 0) bulk_load(to, p.k + (size_t)ft * p.k_stride + x.k0 * 64, in_k * 128, bar);
      to += in_k * 128;
      if (in_v > 0) bulk_load(to, p.v + (size_t)ft * p.v_stride + x.k0 * 64, in_v * 128, bar);
      ft += x.stride;
      ++issued;
      return;
    }
    while (left == 0) {
      if (++fk == 3) {
        fk = 0;
        ft += x.stride;
      }
      if (ft >= tokens) return;
      left = fk == 0 ? x.q1 - x.q0 : (fk == 1 ? with_kv : with_v) ? x.k1 - x.k0 : 0;
      src = fk == 0   ? p.q + (size_t)ft * p.q_stride + x.q0 * 64
            : fk == 1 ? p.k + (size_t)ft * p.k_stride + x.k0 * 64
                      : p.v + (size_t)ft * p.v_stride + x.k0 * 64;
    }
    const int n = min(left, kRopeChunk), st = issued % kDepth;
    mbar_arrive_expect_tx(&s_full[warp][st], n * 128);
    bulk_load(s_ring[warp][st], src, n * 128, &s_full[warp][st]);
    src += n * 64;
    left -= n;
    ++issued;
  };
  if (lane == 0)
    for (int i = 0; i < kDepth - 1; ++i) fetch();
  // The next chunk has landed; the stage before it may be filled again.
  int used = 0;
  bool ok = true;
  auto next = [&]() -> const uint8_t* {
    __syncwarp();                                          // the last chunk has been read
    if (lane == 0) fetch();
    const int st = used % kDepth;
    ok = mbar_wait_warp(&s_full[warp][st], (used / kDepth) & 1, nullptr);
    ++used;
    return s_ring[warp][st];
  };
  auto position = [&](unsigned t) {
    return lane < (p.rotary >> 1) ? __ldg(p.positions + (size_t)p.pair_axis[lane] * p.tokens + t)
                                  : 0;
  };
  int pos = position(t);
  long long slot = p.slots ? __ldg(p.slots + t) : -1;
  const size_t kv_row = (size_t)p.heads_kv * 64;
  while (ok) {
    rope_angles<kInter>(p, pos, lane, me, sC, sS);
    if (slot < -1 || slot >= p.cache_rows) {
      if (lane == 0 && p.slots) atomicCAS(p.err, 0, DEVERR_DECODE_INPUT);
      slot = -1;
    }
    const long long here = slot;
    // the next token's position and slot, on their way during this token's heads
    const unsigned ty = t + x.stride;
    if (ty < tokens) {
      pos = position(ty);
      if (p.slots) slot = __ldg(p.slots + ty);
    }
    const uint8_t* token = nullptr;                        // kWhole: the token's heads
    if constexpr (kWhole) {
      token = next();
      if (!ok) break;
    }
    #pragma unroll
    for (int which = 0; which < 2; ++which) {              // q, then k
      if (which && !with_kv) break;
      Oct a = oct_load(sC, me.at0), b = oct_load(sS, me.at0);
      if (kNorm) {
        const Oct w = oct_load(s_w[which][0], me.at0), wp = oct_load(s_w[which][1], me.at0);
        #pragma unroll
        for (int i = 0; i < 4; ++i) {
          a.e[i] = fmul2(a.e[i], w.e[i]);
          b.e[i] = fmul2(b.e[i], wp.e[i]);
        }
      }
      const int h0 = which ? x.k0 : x.q0;
      int heads = (which ? x.k1 : x.q1) - h0;              // left of this tensor
      __nv_bfloat16* dst = nullptr;
      __nv_bfloat16* dst2 = nullptr;
      if (which == 0) {
        dst = p.q_out + ((size_t)t * p.heads_q + h0 + me.sub) * 64;
      } else {
        if (p.k_out) dst = p.k_out + (size_t)t * kv_row + (h0 + me.sub) * 64;
        if (here >= 0) dst2 = p.k_cache + (size_t)here * kv_row + (h0 + me.sub) * 64;
      }
      while (heads > 0 && ok) {
        const uint8_t* at = (kWhole ? token + (which ? in_q * 128 : 0) : next()) + me.sub * 128;
        if (!ok) break;
        const int n = kWhole ? heads : min(heads, kRopeChunk);
        heads -= n;
        #pragma unroll 2
        for (int h = 0; h < n; h += 4, at += 512) {
          const uint2 r0 = *reinterpret_cast<const uint2*>(at + 2 * me.d0);
          const uint2 r1 = *reinterpret_cast<const uint2*>(at + 2 * me.d1);
          const Oct v = oct_from_bf16(r0, r1), o = oct_other<kInter>(v);
          uint64_t inv2 = 0;
          if (kNorm) {
            const float inv = rsqrtf(sum8(oct_dot(v, v)) * (1.0f / 64.0f) + p.eps);
            inv2 = f2(inv, inv);
          }
          uint32_t w[4];
          #pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint64_t z = ffma2(o.e[i], b.e[i], fmul2(v.e[i], a.e[i]));
            if (kNorm) z = fmul2(z, inv2);
            w[i] = f2_to_bf16x2(z);
          }
          if (h + me.sub < n) {                            // heads behind the last: stale bytes
            if (which == 0 || dst) {
              *reinterpret_cast<uint2*>(dst + me.d0) = make_uint2(w[0], w[1]);
              *reinterpret_cast<uint2*>(dst + me.d1) = make_uint2(w[2], w[3]);
            }
            if (which && dst2) {
              *reinterpret_cast<uint2*>(dst2 + me.d0) = make_uint2(w[0], w[1]);
              *reinterpret_cast<uint2*>(dst2 + me.d1) = make_uint2(w[2], w[3]);
            }
          }
          if (which == 0 || dst) dst += 256;
          if (which && dst2) dst2 += 256;
        }
      }
    }
    for (int heads = with_v ? x.k1 - x.k0 : 0, h0 = x.k0; heads > 0 && ok;) {
      const uint8_t* at = kWhole ? token + (in_q + in_k) * 128 : next();
      if (!ok) break;
      const int n = kWhole ? heads : min(heads, kRopeChunk);
      for (int h = me.sub; h < n; h += 4) {
        const uint4 r = *reinterpret_cast<const uint4*>(at + h * 128 + 2 * j8);
        const size_t off = (size_t)(h0 + h) * 64 + j8;
        if (p.v_out) *reinterpret_cast<uint4*>(p.v_out + (size_t)t * kv_row + off) = r;
        if (here >= 0) *reinterpret_cast<uint4*>(p.v_cache + (size_t)here * kv_row + off) = r;
      }
      heads -= n;
      h0 += n;
    }
    t = ty;
    if (t >= tokens) break;
  }
  if (!ok && lane == 0) rope_give_up(p, s_full[warp], used, issued, kDepth);
}

template <bool kNorm, bool kInter, bool kFp32, bool kWhole>
__global__ void __launch_bounds__(kRopeThreads, kRopeBwdCtas)
attn_sink_rope_bwd_kernel(const __grid_constant__ RopeParams p) {
  constexpr int kDyHead = kFp32 ? 256 : 128;               // bytes of a head of dy
  // heads of a stage, dy and then x; a step of four may read three behind the last
  // (of dy: from the x behind it)
  constexpr int kHeads = kWhole ? (kFp32 ? kRopeBwdWholeFp32 : kRopeBwdWhole) : kRopeBwdChunk;
  constexpr int kSlack = kWhole ? 3 : 0;
  constexpr int kDy = (kHeads + (kNorm ? 0 : kSlack)) * kDyHead;
  static_assert(!kNorm || !kWhole || kSlack * kDyHead <= kHeads * 128, "the x behind dy");
  constexpr int kDepth = kWhole ? kRopeWholeDepth : kRopeBwdDepth;
  __shared__ __align__(16) float s_w[2][64];
  __shared__ __align__(16) float s_cs[kRopeWarps][2][64];
  __shared__ __align__(16) float s_dw[2][kRopeWarps][32][8];   // each lane's sums, q and k
  __shared__ __align__(128) uint8_t
      s_ring[kRopeWarps][kDepth][kDy + (kNorm ? (kHeads + kSlack) * 128 : 0)];
  __shared__ __align__(8) uint64_t s_full[kRopeWarps][kDepth];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const RopeLane me = rope_lane<kInter>(p, lane);
  const int j8 = 8 * (lane & 7);
  if (kNorm) {
    s_w[tid >> 6][tid & 63] = rope_weight(tid >> 6 ? p.k_weight : p.q_weight, p.weight_bf16,
                                          rope_table_dim<kInter>(tid & 63, p.rotary));
    for (int i = 0; i < 8; ++i) s_dw[0][warp][lane][i] = s_dw[1][warp][lane][i] = 0.0f;
  }
  float* sC = s_cs[warp][0];
  float* sS = s_cs[warp][1];
  for (int d = lane; d < 64; d += 32) {
    sC[d] = 1.0f;
    sS[d] = 0.0f;
  }
  if (lane == 0) {
    for (int i = 0; i < kDepth; ++i) mbar_init(&s_full[warp][i], 1);
    fence_mbarrier_init();
  }
  __syncthreads();
  if (kNorm) grid_launch_dependents();                     // the sum of the weights' gradients
  const RopePart x = rope_part(p, warp);
  const unsigned tokens = (unsigned)p.tokens;
  const bool with_v = p.dv != nullptr;
  unsigned t = x.first, ft = t;
  bool ok = t < tokens && x.nq + x.nk > 0;
  const bool any = ok;
  // as in the forward kernel; a chunk of dv has no x
  int fk = -1, left = 0, issued = 0, used = 0;
  const char* dy = nullptr;
  const __nv_bfloat16* src = nullptr;
  const int in_q = x.q1 - x.q0, in_k = x.k1 - x.k0, in_v = with_v ? in_k : 0;
  auto fetch = [&]() {
    if constexpr (kWhole) {
      if (ft >= tokens) return;
      const int st = issued % kDepth;
      uint8_t* to = s_ring[warp][st];
      uint64_t* bar = &s_full[warp][st];
      auto load = [&](int at, const void* base, int heads, int h0, int n) {
        if (n > 0)
          bulk_load(to + at * kDyHead,
                    static_cast<const char*>(base) + ((size_t)ft * heads + h0) * kDyHead,
                    n * kDyHead, bar);
      };
      mbar_arrive_expect_tx(bar, (in_q + in_k + in_v) * kDyHead +
                                     (kNorm ? (in_q + in_k) * 128 : 0));
      load(0, p.dq, p.heads_q, x.q0, in_q);
      load(in_q, p.dk, p.heads_kv, x.k0, in_k);
      load(in_q + in_k, p.dv, p.heads_kv, x.k0, in_v);
      if (kNorm) {
        to += kDy;
        if (in_q > 0) bulk_load(to, p.q + (size_t)ft * p.q_stride + x.q0 * 64, in_q * 128, bar);
        to += in_q * 128;
        if (in_k > 0) bulk_load(to, p.k + (size_t)ft * p.k_stride + x.k0 * 64, in_k * 128, bar);
      }
      ft += x.stride;
      ++issued;
      return;
    }
    while (left == 0) {
      if (++fk == 3) {
        fk = 0;
        ft += x.stride;
      }
      if (ft >= tokens) return;
      left = fk == 0 ? x.q1 - x.q0 : fk == 1 || with_v ? x.k1 - x.k0 : 0;
      const int h0 = fk == 0 ? x.q0 : x.k0;
      dy = static_cast<const char*>(fk == 0 ? p.dq : fk == 1 ? p.dk : p.dv) +
           ((size_t)ft * (fk == 0 ? p.heads_q : p.heads_kv) + h0) * kDyHead;
      if (kNorm)
        src = (fk == 0 ? p.q + (size_t)ft * p.q_stride : p.k + (size_t)ft * p.k_stride) + h0 * 64;
    }
    const int n = min(left, kRopeBwdChunk), st = issued % kDepth;
    uint64_t* bar = &s_full[warp][st];
    const bool with_x = kNorm && fk < 2;
    mbar_arrive_expect_tx(bar, n * (kDyHead + (with_x ? 128 : 0)));
    bulk_load(s_ring[warp][st], dy, n * kDyHead, bar);
    if (with_x) bulk_load(s_ring[warp][st] + kDy, src, n * 128, bar);
    dy += n * kDyHead;
    if (kNorm) src += n * 64;
    left -= n;
    ++issued;
  };
  auto next = [&]() -> const uint8_t* {
    __syncwarp();
    if (lane == 0) fetch();
    const int st = used % kDepth;
    ok = mbar_wait_warp(&s_full[warp][st], (used / kDepth) & 1, nullptr);
    ++used;
    return s_ring[warp][st];
  };
  // four numbers of dy from dimension d of a head
  auto four = [&](const uint8_t* head, int d, uint64_t* lo, uint64_t* hi) {
    if (kFp32) {
      const ulonglong2 r = *reinterpret_cast<const ulonglong2*>(head + 4 * d);
      *lo = r.x;
      *hi = r.y;
    } else {
      const uint2 r = *reinterpret_cast<const uint2*>(head + 2 * d);
      *lo = bf16x2_to_f2(r.x);
      *hi = bf16x2_to_f2(r.y);
    }
  };
  auto position = [&](unsigned t) {
    return lane < (p.rotary >> 1) ? __ldg(p.positions + (size_t)p.pair_axis[lane] * p.tokens + t)
                                  : 0;
  };
  int pos = 0;
  if (any) {
    if (lane == 0)
      for (int i = 0; i < kDepth - 1; ++i) fetch();
    pos = position(t);
  }
  while (ok) {
    rope_angles<kInter>(p, pos, lane, me, sC, sS);
    const unsigned ty = t + x.stride;
    if (ty < tokens) pos = position(ty);
    const uint8_t* token = nullptr;        // kWhole: the token's heads
    if constexpr (kWhole) {
      token = next();
      if (!ok) break;
    }
    #pragma unroll 1
    for (int which = 0; which < 2; ++which) {
      const Oct c = oct_load(sC, me.at0), s = oct_load(sS, me.at0);
      Oct w, dw;
      if (kNorm) {
        w = oct_load(s_w[which], me.at0);
        dw = oct_load(&s_dw[which][warp][lane][0], 0);
      }
      const int h0 = which ? x.k0 : x.q0;
      int heads = (which ? x.k1 : x.q1) - h0;
      __nv_bfloat16* dst = (which ? p.dk_in + (size_t)t * p.dk_in_stride
                                  : p.dq_in + (size_t)t * p.dq_in_stride) + (h0 + me.sub) * 64;
      while (heads > 0 && ok) {
        const uint8_t* at = kWhole ? token : next();
        if (!ok) break;
        const int n = kWhole ? heads : min(heads, kRopeBwdChunk);
        heads -= n;
        const int first = (kWhole && which ? in_q : 0) + me.sub;
        const uint8_t* ax = at + kDy + first * 128;
        at += first * kDyHead;
        #pragma unroll 1
        for (int h = me.sub; h - me.sub < n; h += 4, at += 4 * kDyHead, ax += 512, dst += 256) {
          const bool on = h < n;           // heads behind the last: stale bytes
          Oct d, g;
          four(at, me.d0, &d.e[0], &d.e[1]);
          four(at, me.d1, &d.e[2], &d.e[3]);
          const Oct dp = oct_other<kInter>(d);
          #pragma unroll
          for (int i = 0; i < 4; ++i) {    // the transposed rotation: S negated
            const uint64_t m = fmul2(dp.e[i], s.e[i]);
            g.e[i] = ffma2(d.e[i], c.e[i], m ^ 0x8000000080000000ull);
          }
          if (kNorm) {
            const uint2 r0 = *reinterpret_cast<const uint2*>(ax + 2 * me.d0);
            const uint2 r1 = *reinterpret_cast<const uint2*>(ax + 2 * me.d1);
            const Oct v = oct_from_bf16(r0, r1);
            Oct hh;
            #pragma unroll
            for (int i = 0; i < 4; ++i) hh.e[i] = fmul2(g.e[i], w.e[i]);
            const float ss = sum8(oct_dot(v, v)), hx = sum8(oct_dot(hh, v));
            const float inv = rsqrtf(ss * (1.0f / 64.0f) + p.eps);
            const float back = -hx * (1.0f / 64.0f) * inv * inv;
            const uint64_t back2 = f2(back, back), inv2 = f2(inv, inv);
            #pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint64_t add = fmul2(g.e[i], inv2);
              if (on) dw.e[i] = ffma2(add, v.e[i], dw.e[i]);
              g.e[i] = fmul2(inv2, ffma2(v.e[i], back2, hh.e[i]));
            }
          }
          if (on) {
            *reinterpret_cast<uint2*>(dst + me.d0) =
                make_uint2(f2_to_bf16x2(g.e[0]), f2_to_bf16x2(g.e[1]));
            *reinterpret_cast<uint2*>(dst + me.d1) =
                make_uint2(f2_to_bf16x2(g.e[2]), f2_to_bf16x2(g.e[3]));
          }
        }
      }
      if (kNorm) {
        ulonglong2* o = reinterpret_cast<ulonglong2*>(&s_dw[which][warp][lane][0]);
        o[0] = make_ulonglong2(dw.e[0], dw.e[1]);
        o[1] = make_ulonglong2(dw.e[2], dw.e[3]);
      }
    }
    for (int heads = with_v ? x.k1 - x.k0 : 0, h0 = x.k0; heads > 0 && ok;) {
      const uint8_t* at = kWhole ? token + (in_q + in_k) * kDyHead : next();
      if (!ok) break;
      const int n = kWhole ? heads : min(heads, kRopeBwdChunk);
      for (int h = me.sub; h < n; h += 4) {
        uint64_t e[4];
        four(at + h * kDyHead, j8, &e[0], &e[1]);
        four(at + h * kDyHead, j8 + 4, &e[2], &e[3]);
        *reinterpret_cast<uint4*>(p.dv_in + (size_t)t * p.dv_in_stride + (size_t)(h0 + h) * 64 +
                                  j8) = make_uint4(f2_to_bf16x2(e[0]), f2_to_bf16x2(e[1]),
                                                   f2_to_bf16x2(e[2]), f2_to_bf16x2(e[3]));
      }
      heads -= n;
      h0 += n;
    }
    t = ty;
    if (t >= tokens) break;
  }
  if (any && !ok && lane == 0) rope_give_up(p, s_full[warp], used, issued, kDepth);
  if constexpr (kNorm) {
    // this CTA's weight gradients: every lane that holds a number, in order (odd
    // heads hold numbers 0-3 and 4-7 the other way round)
    __syncthreads();
    const int which = tid >> 6, i = tid & 63;
    float sum = 0.0f;
    for (int w = 0; w < kRopeWarps; ++w) {
      #pragma unroll
      for (int sub = 0; sub < 4; ++sub)
        sum += s_dw[which][w][8 * sub + (i >> 3)][(i & 7) ^ ((sub & 1) << 2)];
    }
    p.dw_part[((size_t)blockIdx.y * gridDim.x + blockIdx.x) * 128 + 64 * which +
              rope_table_dim<kInter>(i, p.rotary)] = sum;
  }
}

// The CTAs' partial weight gradients in a fixed order: thread (g, d) sums every
// eighth CTA's, then the eight sums are added in order.
constexpr int kRopeSumThreads = 1024;
struct RopeSum {
  const float* part;           // [CTAs][2][64]
  float* dwq;
  float* dwk;
  int ctas;
};
__global__ void __launch_bounds__(kRopeSumThreads)
attn_sink_rope_dw_kernel(const RopeSum p) {
  __shared__ float s[8][128];
  grid_dependency_wait();
  const int d = threadIdx.x & 127, g = threadIdx.x >> 7;
  float x = 0.0f;
  for (int c = g; c < p.ctas; c += 8) x += p.part[(size_t)c * 128 + d];
  s[g][d] = x;
  __syncthreads();
  if (g == 0) {
    #pragma unroll
    for (int i = 1; i < 8; ++i) x += s[i][d];
    (d < 64 ? p.dwq : p.dwk)[d & 63] = x;
  }
}

}  // namespace attn_sink
