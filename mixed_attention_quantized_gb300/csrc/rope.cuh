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
// most -- one wrapping integer multiply, no table of cosines to read.  Its upper 32 bits are
// used: another 2^-32 of a turn (1.5e-9 radians), which is the larger part up to position 2^23.
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

#include "device_utils.cuh"
#include "internal.h"

namespace mixattn {

#ifdef __CUDACC__

// Cosine and sine of pair i at position pos, times the attention multiplier: the turn's
// nearest quarter gives the signs and which is which, the rest (an angle within +-pi/4) the
// Taylor sums to the 9th and 8th power, whose next terms are below 2e-9 and 3e-8; with the fp32
// steps both are within 2^-23.4 of the exact ones (over 8 million turns).
__device__ __forceinline__ float2 rope_cos_sin(const RopeTable& t, int32_t pos, int i) {
  const uint32_t turn = (uint32_t)((t.turn[i] * (uint64_t)(int64_t)pos) >> 32);
  const uint32_t quarter = (turn + 0x20000000u) >> 30;
  const float x = (float)(int32_t)(turn - (quarter << 30)) * 1.4629180792671596e-9f;  // 2 pi 2^-32
  const float x2 = x * x;
  float s = fmaf(x2, 2.7557319e-6f, -1.9841270e-4f);
  s = fmaf(x2, s, 8.3333333e-3f);
  s = fmaf(x2, s, -1.6666667e-1f);
  s = fmaf(x2 * x, s, x);
  float c = fmaf(x2, 2.4801587e-5f, -1.3888889e-3f);
  c = fmaf(x2, c, 4.1666667e-2f);
  c = fmaf(x2, c, -0.5f);
  c = fmaf(x2, c, 1.f);
  float co = (quarter & 1u) ? s : c, si = (quarter & 1u) ? c : s;
  co = ((quarter + 1u) & 2u) ? -co : co;
  si = (quarter & 2u) ? -si : si;
  return make_float2(co * t.mscale, si * t.mscale);
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
