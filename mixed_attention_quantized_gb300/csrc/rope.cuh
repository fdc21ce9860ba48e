// rope.cuh -- rotary positions: the table a kernel takes by value and the
// rotation of one 16-element item of a head.
//
// A head's first `rot` elements are rot/2 pairs (a_i, b_i); at position p
//     (a, b) -> m (a cos w - b sin w, b cos w + a sin w),   w = p f_i,
// with pair i = elements (i, i + rot/2) in the half layout and (2i, 2i + 1) in
// the interleaved one; elements past rot stay as they are.
//
// Angles: p f_i in fp32 is off by up to 2^-24 p f_i radians (0.02 at position
// 262144), so the table holds each frequency as a fraction of a turn in 64-bit
// fixed point, T_i = 2^64 f_i / 2 pi with the quotient a double (within 2^-55 for f_i <= 1),
// and p T_i mod 2^64 is the angle's fractional turn, off by |p| 2^-55 turns at
// most -- one wrapping integer multiply, no table of cosines to read.
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

#include "device_utils.cuh"
#include "internal.h"

namespace mixattn {

#ifdef __CUDACC__

// Cosine and sine of pair i at position pos, times the attention multiplier, rounded to fp32 once
// (within 1.5 half ulps; 2% of the sines and 0.6% of the cosines are not the nearest value): a rotated
// key that lies next to the border of two codes should not cross it for an angle's sake.  (With plain
// fp32 Taylor sums of the angle's upper 32 bits, off by up to 2^-23.4, 2048 tokens of 32 query and 8 kv
// heads took 13.2 us in the fused append and not 13.4; 29 against 21 of 25 million e4m3 keys were one
// code off.)
// The turn's nearest quarter gives the signs and which is which.  The rest is an angle within
// +-pi/4 as x + r, x the nearest fp32 and r what that leaves, so that
//   sin(x + r) = x + (x^3 S(x^2) + r (1 - x^2/2)),   cos(x + r) = w + (e - (x^2 - x2)/2 - r x + x^4 C(x^2))
// with x2 = x^2 rounded, w = 1 - x2/2 rounded and e what w leaves; S and C are Taylor sums whose next
// terms are below 2e-9 and 2e-10.  The multiplier is applied to both parts.
__device__ __forceinline__ float2 rope_cos_sin(const RopeTable& t, int32_t pos, int i) {
  const uint64_t turn = t.turn[i] * (uint64_t)(int64_t)pos;
  const uint32_t hi = (uint32_t)(turn >> 32);
  const uint32_t quarter = (hi + 0x20000000u) >> 30;
  const uint32_t d = hi - (quarter << 30);  // signed, 2^-32 turns
  // d's upper 24 bits, which are exact in fp32, and the rest of it with the 24 bits below, 2^-24 as large
  constexpr float kUnit = 1.4629180792671596e-9f, kUnitRest = -4.0709404e-17f;  // 2 pi 2^-32 and what fp32 leaves of it
  const float xh = (float)(int32_t)(d & 0xFFFFFF00u);
  const float xl = (float)__funnelshift_l((uint32_t)turn, d, 24);
  const float rest = fmaf(xh, kUnitRest, xl * (kUnit * 5.9604644775390625e-8f));
  const float x = fmaf(xh, kUnit, rest), r = fmaf(xh, kUnit, -x) + rest;
  const float x2 = __fmul_rn(x, x), h = 0.5f * x2;
  float s = fmaf(x2, 2.7557319e-6f, -1.9841270e-4f);
  s = fmaf(x2, s, 8.3333333e-3f);
  s = fmaf(x2, s, -1.6666667e-1f);
  s = fmaf(x2 * x, s, fmaf(-h, r, r));  // sine: x + s
  const float w = 1.f - h, e = (1.f - w) - h;
  float c = fmaf(x2, -2.7557319e-7f, 2.4801587e-5f);
  c = fmaf(x2, c, -1.3888889e-3f);
  c = fmaf(x2, c, 4.1666667e-2f);
  c = fmaf(x2 * x2, c, fmaf(-0.5f, fmaf(x, x, -x2), fmaf(-r, x, e)));  // cosine: w + c
  s = fmaf(x, t.mscale, fmaf(x, t.mscale_rest, s * t.mscale));
  c = fmaf(w, t.mscale, fmaf(w, t.mscale_rest, c * t.mscale));
  float co = (quarter & 1u) ? s : c, si = (quarter & 1u) ? c : s;
  co = ((quarter + 1u) & 2u) ? -co : co;
  si = (quarter & 2u) ? -si : si;
  return make_float2(co, si);
}

// First elements of the two 8-element chunks of item j (0 .. D/16 - 1) of a head:
// items below rot/16 hold 8 whole pairs, the others 16 elements to copy.
__device__ __forceinline__ void rope_item(const RopeTable& t, int j, int& e0, int& e1) {
  if (t.layout == MIXATTN_ROPE_HALF && 16 * j < t.rot) {
    e0 = 8 * j;
    e1 = e0 + t.rot / 2;
  } else {
    e0 = 16 * j;
    e1 = e0 + 8;
  }
}

// Item j's 16 values x0 (chunk e0), x1 (chunk e1) rotated in place; cs holds the
// (cos, sin) of its pairs 8j .. 8j+7.
__device__ __forceinline__ void rope_rotate(const RopeTable& t, const float2 (&cs)[8], int j, float (&x0)[8],
                                            float (&x1)[8]) {
  if (16 * j >= t.rot) return;
  if (t.layout == MIXATTN_ROPE_HALF) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float4 c = make_float4(cs[2 * k].x, cs[2 * k].y, cs[2 * k + 1].x, cs[2 * k + 1].y);
      const float a0 = x0[2 * k], b0 = x1[2 * k], a1 = x0[2 * k + 1], b1 = x1[2 * k + 1];
      x0[2 * k] = a0 * c.x - b0 * c.y;
      x1[2 * k] = b0 * c.x + a0 * c.y;
      x0[2 * k + 1] = a1 * c.z - b1 * c.w;
      x1[2 * k + 1] = b1 * c.z + a1 * c.w;
    }
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float(&x)[8] = k < 2 ? x0 : x1;
      const int o = 4 * (k & 1);
      const float4 c = make_float4(cs[2 * k].x, cs[2 * k].y, cs[2 * k + 1].x, cs[2 * k + 1].y);
      const float a0 = x[o], b0 = x[o + 1], a1 = x[o + 2], b1 = x[o + 3];
      x[o] = a0 * c.x - b0 * c.y;
      x[o + 1] = b0 * c.x + a0 * c.y;
      x[o + 2] = a1 * c.z - b1 * c.w;
      x[o + 3] = b1 * c.z + a1 * c.w;
    }
  }
}

__device__ __forceinline__ void half8_to_float(const uint4& w, float (&x)[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}

// A key or value element on its way into a quantised format: NaN counts as 0, values
// beyond the fp16 range saturate.
__device__ __forceinline__ float saturate_f16_range(float x) {
  return x != x ? 0.f : fminf(fmaxf(x, -65504.f), 65504.f);
}

__device__ __forceinline__ uint4 float8_to_half(const float (&x)[8]) {
  return make_uint4(pack_f16x2_out(x[0], x[1]), pack_f16x2_out(x[2], x[3]), pack_f16x2_out(x[4], x[5]),
                    pack_f16x2_out(x[6], x[7]));
}

// (cos, sin) of one token's pairs into shared memory, by the whole CTA (no barrier).
__device__ __forceinline__ void rope_fill(const RopeTable& t, int32_t pos, float2* cs) {
  for (int i = threadIdx.x; i < t.rot / 2; i += blockDim.x) cs[i] = rope_cos_sin(t, pos, i);
}

// Rotates the heads of one token, D elements each, by the whole CTA; cs is the token's.
template <int D>
__device__ __forceinline__ void rope_row(const RopeTable& t, const float2* cs, const uint16_t* x, uint16_t* out,
                                         int n_heads) {
  constexpr int IPH = D / 16;  // items per head
  for (int i = threadIdx.x; i < n_heads * IPH; i += blockDim.x) {
    const int h = i / IPH, j = i - h * IPH;
    int e0, e1;
    rope_item(t, j, e0, e1);
    const uint16_t* src = x + (int64_t)h * D;
    uint16_t* dst = out + (int64_t)h * D;
    uint4 w0 = *reinterpret_cast<const uint4*>(src + e0), w1 = *reinterpret_cast<const uint4*>(src + e1);
    if (16 * j < t.rot) {
      float2 c[8];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float4 v = reinterpret_cast<const float4*>(cs + 8 * j)[k];
        c[2 * k] = make_float2(v.x, v.y);
        c[2 * k + 1] = make_float2(v.z, v.w);
      }
      float x0[8], x1[8];
      half8_to_float(w0, x0);
      half8_to_float(w1, x1);
      rope_rotate(t, c, j, x0, x1);
      w0 = float8_to_half(x0);
      w1 = float8_to_half(x1);
    }
    *reinterpret_cast<uint4*>(dst + e0) = w0;
    *reinterpret_cast<uint4*>(dst + e1) = w1;
  }
}

#endif  // __CUDACC__

}  // namespace mixattn
