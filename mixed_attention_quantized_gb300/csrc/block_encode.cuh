// block_encode.cuh -- the 32-element block encoders of the Q8_0 and Q4_0 formats,
// shared by the append kernels.
#pragma once

#include "device_utils.cuh"
#include "internal.h"

namespace mixattn {

__device__ __forceinline__ float h2f(uint16_t h) { return __half2float(__ushort_as_half(h)); }

// Encodes block b of plane row `row` (rows in [page][head][token] order, nb blocks each).
// Eight consecutive lanes hold the block, lane `sub` of them elements 4 sub .. 4 sub + 3;
// every lane of the warp takes part, and `store` says whether this block is written.
template <int FMT>
__device__ __forceinline__ void encode_block(uint8_t* quant, uint16_t* scale, const float (&v)[4], int64_t row, int64_t b,
                                             int nb, int sub, bool store) {
  if constexpr (FMT == MIXATTN_KV_Q8_0) {
    float amax = fmaxf(fmaxf(fabsf(v[0]), fabsf(v[1])), fmaxf(fabsf(v[2]), fabsf(v[3])));
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
    const float d = __fdiv_rn(amax, 127.0f);
    const float id = (d != 0.0f) ? __fdiv_rn(1.0f, d) : 0.0f;
    uint32_t packed = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int q = (int)roundf(__fmul_rn(v[i], id));
      packed |= (uint32_t)(uint8_t)(int8_t)q << (8 * i);
    }
    if (store) {
      *reinterpret_cast<uint32_t*>(quant + row * (int64_t)(nb * 32) + b * 32 + 4 * sub) = packed;
      if (sub == 0) scale[row * nb + b] = __half_as_ushort(__float2half_rn(d));
    }
  } else {  // Q4_0
    // element of largest magnitude, lowest index on ties
    float best_abs = -1.0f, best_val = 0.0f;
    int best_idx = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float m = fabsf(v[i]);
      if (m > best_abs) {
        best_abs = m;
        best_val = v[i];
        best_idx = 4 * sub + i;
      }
    }
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) {
      const float oa = __shfl_xor_sync(0xFFFFFFFFu, best_abs, o);
      const float ov = __shfl_xor_sync(0xFFFFFFFFu, best_val, o);
      const int oi = __shfl_xor_sync(0xFFFFFFFFu, best_idx, o);
      if (oa > best_abs || (oa == best_abs && oi < best_idx)) {
        best_abs = oa;
        best_val = ov;
        best_idx = oi;
      }
    }
    const float m = best_abs > 0.0f ? best_val : 0.0f;  // an all-zero block keeps m = +0
    const float d = __fdiv_rn(m, -8.0f);
    const float id = (d != 0.0f) ? __fdiv_rn(1.0f, d) : 0.0f;
    uint32_t q4 = 0;  // four nibbles, one per byte
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float s = __fadd_rn(__fmul_rn(v[i], id), 8.5f);
      int q = (int)truncf(s);
      q = q > 15 ? 15 : q;
      q4 |= (uint32_t)q << (8 * i);
    }
    // element k (lanes 0-3 of the 8) pairs with element k+16 (lanes 4-7)
    const uint32_t hi = __shfl_down_sync(0xFFFFFFFFu, q4, 4);
    if (store && sub < 4) {
      *reinterpret_cast<uint32_t*>(quant + row * (int64_t)(nb * 16) + b * 16 + 4 * sub) = q4 | (hi << 4);
    }
    if (store && sub == 0) scale[row * nb + b] = __half_as_ushort(__float2half_rn(d));
  }
}

}  // namespace mixattn
