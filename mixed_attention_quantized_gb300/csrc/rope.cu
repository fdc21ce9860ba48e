// rope.cu -- rotary positions of a step's tokens, alone or on the way into a
// block-format cache (the page-scaled formats: page_append.cu).
//
// Bytes set the floor (an fp16 element is read and written once, three flops and a
// shared cosine pair per pair), so the kernels are one pass of 16-byte loads and
// stores: a thread takes an item of 16 elements -- both halves of 8 pairs, wherever
// the layout puts them -- and every pair is rotated in registers.  One CTA takes one
// token, whose rot/2 cosine pairs it computes once for all its heads.  Measured: 2048 tokens of
// 32 heads of 128 6.4 us (33.6 MB, 5.2 TB/s), 16 tokens 2.2 us, which is a launch.
#include <cuda_runtime.h>

#include "block_encode.cuh"
#include "device_utils.cuh"
#include "internal.h"
#include "rope.cuh"

namespace mixattn {

namespace {

template <int D>
__global__ void __launch_bounds__(256) rope_kernel(const __grid_constant__ RopeTable t, TokenRows x, uint16_t* out,
                                                   int64_t out_stride, const int32_t* __restrict__ positions,
                                                   int n_heads) {
  __shared__ __align__(16) float2 cs[kMaxRotPairs];
  const int64_t tok = blockIdx.x;
  rope_fill(t, positions[tok], cs);
  __syncthreads();
  rope_row<D>(t, cs, x.x + tok * x.stride, out + tok * out_stride, n_heads);
}

struct RopeAppendArgs {
  TokenRows q, k, v;
  uint16_t* q_out;
  int64_t q_out_stride;
  const int32_t* positions;
  const int32_t* slots;
  uint8_t* k_quant;
  uint16_t* k_scale;
  uint8_t* v_quant;
  uint16_t* v_scale;
  int32_t hq, hkv, num_slots;
  unsigned int* err;
};

// The four elements at e .. e + 3 of a rotated head.  Groups of four never straddle a
// pair's halves (rot/2 is a multiple of 8).
template <int D>
__device__ __forceinline__ void rotated4(const RopeTable& t, const float2* cs, const uint16_t* head, int e,
                                         float (&v)[4]) {
  const uint2 raw = *reinterpret_cast<const uint2*>(head + e);
  v[0] = h2f(raw.x & 0xFFFFu);
  v[1] = h2f(raw.x >> 16);
  v[2] = h2f(raw.y & 0xFFFFu);
  v[3] = h2f(raw.y >> 16);
  if (e >= t.rot) return;
  if (t.layout == MIXATTN_ROPE_HALF) {
    const int half = t.rot / 2;
    const bool second = e >= half;
    const uint2 other = *reinterpret_cast<const uint2*>(head + (second ? e - half : e + half));
    const float w[4] = {h2f(other.x & 0xFFFFu), h2f(other.x >> 16), h2f(other.y & 0xFFFFu), h2f(other.y >> 16)};
    const int i = second ? e - half : e;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 c = cs[i + k];
      v[k] = second ? v[k] * c.x + w[k] * c.y : v[k] * c.x - w[k] * c.y;
    }
  } else {
#pragma unroll
    for (int k = 0; k < 4; k += 2) {
      const float2 c = cs[(e + k) / 2];
      const float a = v[k], b = v[k + 1];
      v[k] = a * c.x - b * c.y;
      v[k + 1] = b * c.x + a * c.y;
    }
  }
}

// One token's keys (ROT) or values into the cache: a warp takes four 32-element blocks
// at a time, lane l elements 4 (l % 8) .. + 3 of block l / 8.
template <int FMT, int D, bool ROT>
__device__ __forceinline__ void append_token(const RopeTable& t, const float2* cs, const uint16_t* x, uint8_t* quant,
                                             uint16_t* scale, int hkv, int32_t slot) {
  constexpr int NB = D / kBlock;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, n_warps = blockDim.x >> 5;
  const int sub = lane & 7;
  for (int b0 = 4 * warp; b0 < hkv * NB; b0 += 4 * n_warps) {  // the same trips for a whole warp
    const int blk = b0 + (lane >> 3);
    const bool in = blk < hkv * NB;
    const int g = in ? blk / NB : 0, b = in ? blk - g * NB : 0;
    float v[4] = {0.f, 0.f, 0.f, 0.f};
    const uint16_t* head = x + (int64_t)g * D;
    const int e = 32 * b + 4 * sub;
    const int64_t row = ((int64_t)(slot / kPage) * hkv + g) * kPage + slot % kPage;
    if constexpr (FMT == MIXATTN_KV_F16) {
      if (in) {
        uint2 w;
        if (ROT && e < t.rot) {
          rotated4<D>(t, cs, head, e, v);
          w = make_uint2(pack_f16x2_out(v[0], v[1]), pack_f16x2_out(v[2], v[3]));
        } else {
          w = *reinterpret_cast<const uint2*>(head + e);
        }
        *reinterpret_cast<uint2*>(quant + row * (2 * D) + 2 * e) = w;
      }
    } else {
      if (in) {
        if (ROT) {
          rotated4<D>(t, cs, head, e, v);
#pragma unroll
          for (int k = 0; k < 4; ++k) v[k] = saturate_f16_range(v[k]);
        } else {
          const uint2 raw = *reinterpret_cast<const uint2*>(head + e);
          v[0] = h2f(raw.x & 0xFFFFu);
          v[1] = h2f(raw.x >> 16);
          v[2] = h2f(raw.y & 0xFFFFu);
          v[3] = h2f(raw.y >> 16);
        }
      }
      encode_block<FMT>(quant, scale, v, row, b, NB, sub, in);
    }
  }
}

template <int FK, int FV, int D>
__global__ void __launch_bounds__(256) rope_append_kernel(const __grid_constant__ RopeTable t, RopeAppendArgs a) {
  __shared__ __align__(16) float2 cs[kMaxRotPairs];
  const int64_t tok = blockIdx.x;
  int32_t slot = a.slots[tok];
  rope_fill(t, a.positions[tok], cs);
  if (slot >= a.num_slots) {
    if (threadIdx.x == 0) set_device_error(a.err, MIXATTN_DEVERR_SLOT);
    slot = -1;
  }
  if (slot >= 0) append_token<FV, D, false>(t, cs, a.v.x + tok * a.v.stride, a.v_quant, a.v_scale, a.hkv, slot);
  __syncthreads();
  if (a.hq > 0)
    rope_row<D>(t, cs, a.q.x + tok * a.q.stride, a.q_out + tok * a.q_out_stride, a.hq);
  if (slot >= 0) append_token<FK, D, true>(t, cs, a.k.x + tok * a.k.stride, a.k_quant, a.k_scale, a.hkv, slot);
}

template <int FK, int FV>
cudaError_t launch_d(int d, int n, cudaStream_t s, const RopeTable& t, const RopeAppendArgs& a) {
  if (d == 64) rope_append_kernel<FK, FV, 64><<<n, 256, 0, s>>>(t, a);
  else rope_append_kernel<FK, FV, 128><<<n, 256, 0, s>>>(t, a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope(const RopeTable& t, const TokenRows& x, uint16_t* out, int64_t out_stride,
                        const int32_t* positions, int32_t n_tokens, int32_t n_heads, int32_t head_dim,
                        cudaStream_t s) {
  if (head_dim == 64) rope_kernel<64><<<n_tokens, 256, 0, s>>>(t, x, out, out_stride, positions, n_heads);
  else rope_kernel<128><<<n_tokens, 256, 0, s>>>(t, x, out, out_stride, positions, n_heads);
  return cudaGetLastError();
}

cudaError_t launch_rope_append(const mixattn_kv_cache& c, const RopeTable& t, int hq, const TokenRows& q,
                               uint16_t* q_out, int64_t q_out_stride, const TokenRows& k, const TokenRows& v,
                               const int32_t* positions, const int32_t* slots, int32_t n_new, unsigned int* err,
                               cudaStream_t s) {
  RopeAppendArgs a;
  a.q = q;
  a.k = k;
  a.v = v;
  a.q_out = q_out;
  a.q_out_stride = q_out_stride;
  a.positions = positions;
  a.slots = slots;
  a.k_quant = static_cast<uint8_t*>(c.k_quant);
  a.k_scale = static_cast<uint16_t*>(c.k_scale);
  a.v_quant = static_cast<uint8_t*>(c.v_quant);
  a.v_scale = static_cast<uint16_t*>(c.v_scale);
  a.hq = hq;
  a.hkv = c.num_kv_heads;
  a.num_slots = c.num_pages * kPage;
  a.err = err;
  const int d = c.head_dim, n = n_new;
  if (c.k_fmt == MIXATTN_KV_F16) return launch_d<MIXATTN_KV_F16, MIXATTN_KV_F16>(d, n, s, t, a);
  if (c.k_fmt == MIXATTN_KV_Q8_0) {
    if (c.v_fmt == MIXATTN_KV_Q8_0) return launch_d<MIXATTN_KV_Q8_0, MIXATTN_KV_Q8_0>(d, n, s, t, a);
    return launch_d<MIXATTN_KV_Q8_0, MIXATTN_KV_Q4_0>(d, n, s, t, a);
  }
  if (c.v_fmt == MIXATTN_KV_Q8_0) return launch_d<MIXATTN_KV_Q4_0, MIXATTN_KV_Q8_0>(d, n, s, t, a);
  return launch_d<MIXATTN_KV_Q4_0, MIXATTN_KV_Q4_0>(d, n, s, t, a);
}

}  // namespace mixattn
