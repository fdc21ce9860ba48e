// page_append.cu -- append into the page-scaled 8-bit formats (one fp32 scale per
// page of 32 tokens and kv head), the keys optionally rotated on the way in and the
// step's queries rotated in the same launch.
//
// The scale of a page covers tokens that arrive in different calls, so the unit of
// work is a (page, kv head, tensor): one warp holds every new row of that page in
// registers (one read of each new element), takes their maximum with the page's old
// scale, and writes their codes; when the scale grew it rounds the page's other codes
// again.  A page that gets its slot 0 is new and its old scale counts for nothing.
//
// Which warp owns a page has to come from the slot list alone (no scratch memory, so
// the call can be captured, replayed and run on any stream): a CTA takes a window of
// W consecutive tokens, enters their pages into a small hash table and looks through
// the whole list for tokens of those pages.  It owns the pages of which no earlier
// window has a token.  That search is n^2 / W list entries over the call, 8 KB per CTA
// at 2048 tokens.
#include <cuda_runtime.h>

#include "device_utils.cuh"
#include "internal.h"
#include "rope.cuh"

namespace mixattn {

namespace {

constexpr int kAppendThreads = 256;
constexpr int kAppendWarps = kAppendThreads / 32;
constexpr int kWindow = 32;  // most tokens of a window, so most pages of a CTA
constexpr int kHash = 64;

struct PageAppendArgs {
  TokenRows q, k, v;
  uint16_t* q_out;
  int64_t q_out_stride;
  const int32_t* positions;
  const int32_t* slots;
  uint8_t* codes[2];  // K, V [num_pages][hkv][32][D]
  float* scales[2];   // K, V [num_pages][hkv]
  int32_t n_new, window, heads_per_cta, head_groups, n_windows;
  int32_t hq, hkv, num_slots;
  unsigned int* err;
};

// Scale that a page needs for a largest magnitude amax (fp32, >= 0).
template <int FMT>
__device__ __forceinline__ float scale_for(float amax) {
  if (FMT == MIXATTN_KV_I8_PAGE) return __fdiv_rn(amax, 127.f);
  // the least power of two d with amax <= 448 d = 1.75 * 2^8 d; magnitudes below 2^-100 count as 0
  if (amax < 7.888609052210118e-31f) return 0.f;
  const uint32_t b = __float_as_uint(amax);
  return __uint_as_float(((b >> 23) - 8 + ((b & 0x7FFFFFu) > 0x600000u ? 1 : 0)) << 23);
}

// Codes of eight values at 1/d.
template <int FMT>
__device__ __forceinline__ uint2 encode8(const float (&x)[8], float inv) {
  uint32_t w[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float y[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) y[k] = __fmul_rn(x[4 * h + k], inv);
    if (FMT == MIXATTN_KV_I8_PAGE) {
      uint32_t r = 0;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int q = max(-127, min(127, __float2int_rn(y[k])));
        r |= (uint32_t)(uint8_t)(int8_t)q << (8 * k);
      }
      w[h] = r;
    } else {
      uint16_t lo, hi;
      asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(y[1]), "f"(y[0]));
      asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(y[3]), "f"(y[2]));
      w[h] = (uint32_t)lo | ((uint32_t)hi << 16);
    }
  }
  return make_uint2(w[0], w[1]);
}

// Eight codes as values.
template <int FMT>
__device__ __forceinline__ void decode8(const uint2& c, float (&x)[8]) {
  const uint32_t w[2] = {c.x, c.y};
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (FMT == MIXATTN_KV_I8_PAGE) {
#pragma unroll
      for (int k = 0; k < 4; ++k) x[4 * h + k] = (float)(int8_t)(w[h] >> (8 * k));
    } else {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        uint32_t f2;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(f2) : "h"((uint16_t)(w[h] >> (16 * k))));
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&f2));
        x[4 * h + 2 * k] = f.x;
        x[4 * h + 2 * k + 1] = f.y;
      }
    }
  }
}

// One (page, head, tensor), by one warp.  tok[32]: the new token of each of the page's
// slots, or -1.  ROT: cs_row(slot) is the shared (cos, sin) row of a new token.
template <int FMT, int D, bool ROT, typename CsRow>
__device__ __forceinline__ void append_page(const RopeTable& t, const CsRow& cs_row, const int32_t* tok,
                                            const TokenRows& x, uint8_t* codes, float* scale_p, int h) {
  constexpr int LPR = D / 16;        // lanes per row, an item of 16 elements each
  constexpr int RPS = 32 / LPR;      // rows per step
  constexpr int STEPS = kPage / RPS;
  const int lane = threadIdx.x & 31;
  const int j = lane % LPR, r0 = lane / LPR;
  int e0 = 16 * j, e1 = e0 + 8;
  if (ROT) rope_item(t, j, e0, e1);
  uint4 raw[STEPS][2];
#pragma unroll
  for (int s = 0; s < STEPS; ++s) {
    const int id = tok[s * RPS + r0];
    raw[s][0] = raw[s][1] = make_uint4(0u, 0u, 0u, 0u);
    if (id >= 0) {
      const uint16_t* src = x.x + (int64_t)id * x.stride + (int64_t)h * D;
      raw[s][0] = *reinterpret_cast<const uint4*>(src + e0);
      raw[s][1] = *reinterpret_cast<const uint4*>(src + e1);
    }
  }
  const bool fresh = tok[0] >= 0;
  float d_old = fresh ? 0.f : *scale_p;
  if (!(d_old >= 0.f && d_old < 1e30f)) d_old = 0.f;  // never written
  auto values = [&](int s, float(&x0)[8], float(&x1)[8]) {
    half8_to_float(raw[s][0], x0);
    half8_to_float(raw[s][1], x1);
    if (ROT) rope_rotate(t, cs_row(s * RPS + r0), j, x0, x1);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      x0[k] = saturate_f16_range(x0[k]);
      x1[k] = saturate_f16_range(x1[k]);
    }
  };
  float amax = 0.f;
#pragma unroll
  for (int s = 0; s < STEPS; ++s) {
    if (tok[s * RPS + r0] >= 0) {
      float x0[8], x1[8];
      values(s, x0, x1);
#pragma unroll
      for (int k = 0; k < 8; ++k) amax = fmaxf(amax, fmaxf(fabsf(x0[k]), fabsf(x1[k])));
    }
  }
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
  const float d = fmaxf(d_old, scale_for<FMT>(amax));
  const float inv = d > 0.f ? __fdiv_rn(1.f, d) : 0.f;
  const bool grown = !fresh && d > d_old;
  const float ratio = grown ? __fdiv_rn(d_old, d) : 1.f;
#pragma unroll
  for (int s = 0; s < STEPS; ++s) {
    const int slot = s * RPS + r0;
    uint8_t* row = codes + slot * D;
    if (tok[slot] >= 0) {
      float x0[8], x1[8];
      values(s, x0, x1);
      *reinterpret_cast<uint2*>(row + e0) = encode8<FMT>(x0, inv);
      *reinterpret_cast<uint2*>(row + e1) = encode8<FMT>(x1, inv);
    } else if (grown) {
      float x0[8];
      uint2* p0 = reinterpret_cast<uint2*>(row + e0);
      decode8<FMT>(*p0, x0);
      *p0 = encode8<FMT>(x0, ratio);
      uint2* p1 = reinterpret_cast<uint2*>(row + e1);
      decode8<FMT>(*p1, x0);
      *p1 = encode8<FMT>(x0, ratio);
    }
  }
  if (lane == 0 && (fresh || d != d_old)) *scale_p = d;
}

// Grid: first the append CTAs, [window][tensor][head group], then one CTA per token
// that rotates its queries.
template <int FMT, int D, bool ROT>
__global__ void __launch_bounds__(kAppendThreads) page_append_kernel(const __grid_constant__ RopeTable t,
                                                                     PageAppendArgs a) {
  __shared__ int32_t tbl[kWindow][kPage];  // new token of each slot of each page, -1: none
  __shared__ int32_t hash_key[kHash], hash_val[kHash];
  __shared__ int32_t page_id[kWindow];
  __shared__ int32_t not_mine[kWindow];
  __shared__ uint32_t rows[kWindow];       // mask of the page's new slots
  __shared__ int32_t n_pages;
  __shared__ int32_t row_tok[kPage];       // ROT: the batch's new tokens
  extern __shared__ __align__(16) float2 cs[];  // ROT: [rows of a batch][rot/2]
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int n_append = a.n_windows * 2 * a.head_groups;
  if (ROT && (int)blockIdx.x >= n_append) {
    const int64_t tok = blockIdx.x - n_append;
    rope_fill(t, a.positions[tok], cs);
    __syncthreads();
    rope_row<D>(t, cs, a.q.x + tok * a.q.stride, a.q_out + tok * a.q_out_stride, a.hq);
    return;
  }
  const int win = blockIdx.x / (2 * a.head_groups);
  const int unit = blockIdx.x - win * 2 * a.head_groups;
  const int tensor = unit & 1;
  const int h0 = (unit >> 1) * a.heads_per_cta, nh = min(a.heads_per_cta, a.hkv - h0);
  const int w0 = win * a.window, wn = min(a.window, a.n_new - w0);

  // ---- the window's pages ----
  for (int i = tid; i < kWindow * kPage; i += kAppendThreads) (&tbl[0][0])[i] = -1;
  if (tid < kHash) hash_key[tid] = -1;
  if (tid < kWindow) {
    not_mine[tid] = 0;
    rows[tid] = 0u;
  }
  __syncthreads();
  if (warp == 0) {
    int32_t slot = lane < wn ? a.slots[w0 + lane] : -1;
    if (slot >= a.num_slots) {
      set_device_error(a.err, MIXATTN_DEVERR_SLOT);
      slot = -1;
    }
    const int page = slot >= 0 ? slot / kPage : -1;
    const uint32_t same = __match_any_sync(0xFFFFFFFFu, page);
    const bool first = page >= 0 && (__ffs(same) - 1) == lane;
    const uint32_t firsts = __ballot_sync(0xFFFFFFFFu, first);
    if (first) {
      const int idx = __popc(firsts & ((1u << lane) - 1u));
      page_id[idx] = page;
      int h = page % kHash;
      while (atomicCAS(&hash_key[h], -1, page) != -1) h = (h + 1) % kHash;  // at most 32 keys in 64 places
      hash_val[h] = idx;
    }
    if (lane == 0) n_pages = __popc(firsts);
  }
  __syncthreads();
  const int np = n_pages;
  if (np == 0) return;
  // ---- their tokens, anywhere in the call; the last of several for one slot counts ----
  for (int i = tid; i < a.n_new; i += kAppendThreads) {
    const int32_t slot = a.slots[i];
    if (slot < 0 || slot >= a.num_slots) continue;
    const int page = slot / kPage;
    int h = page % kHash, key;
    while ((key = hash_key[h]) != -1 && key != page) h = (h + 1) % kHash;
    if (key == page) {
      const int idx = hash_val[h];
      atomicMax(&tbl[idx][slot % kPage], i);
      atomicOr(&rows[idx], 1u << (slot % kPage));
      if (i < w0) not_mine[idx] = 1;
    }
  }
  __syncthreads();
  // ---- the owned pages, in batches of at most 32 rows when cosines are shared ----
  const TokenRows& x = tensor == 0 ? a.k : a.v;
  const bool rot = ROT && tensor == 0;
  const int half = t.rot / 2;
  for (int p0 = 0; p0 < np;) {
    int p1 = p0, n_rows = 0;
    for (; p1 < np; ++p1) {
      const int r = not_mine[p1] ? 0 : __popc(rows[p1]);
      if (rot && p1 > p0 && n_rows + r > kPage) break;
      n_rows += r;
    }
    if (rot) {
      __syncthreads();  // the previous batch is done with cs
      int base = 0;
      for (int p = p0; p < p1; ++p) {
        if (not_mine[p]) continue;
        const uint32_t m = rows[p];
        if ((p & (kAppendWarps - 1)) == warp && ((m >> lane) & 1u))
          row_tok[base + __popc(m & ((1u << lane) - 1u))] = tbl[p][lane];
        base += __popc(m);
      }
      __syncthreads();
      for (int i = tid; i < n_rows * half; i += kAppendThreads) {
        const int r = i / half;
        cs[i] = rope_cos_sin(t, a.positions[row_tok[r]], i - r * half);
      }
      __syncthreads();
    }
    const int jobs = (p1 - p0) * nh;
    for (int job = warp; job < jobs; job += kAppendWarps) {
      const int pi = job / nh, p = p0 + pi, h = h0 + job - pi * nh;
      if (not_mine[p]) continue;
      const int64_t at = (int64_t)page_id[p] * a.hkv + h;
      uint8_t* codes = a.codes[tensor] + at * (kPage * D);
      float* scale = a.scales[tensor] + at;
      if (rot) {
        int base = 0;
        for (int b = p0; b < p; ++b) base += not_mine[b] ? 0 : __popc(rows[b]);
        const uint32_t m = rows[p];
        auto cs_row = [&](int slot) { return cs + (base + __popc(m & ((1u << slot) - 1u))) * half; };
        append_page<FMT, D, ROT>(t, cs_row, tbl[p], x, codes, scale, h);
      } else {
        auto no_row = [&](int) { return static_cast<const float2*>(nullptr); };
        append_page<FMT, D, false>(t, no_row, tbl[p], x, codes, scale, h);
      }
    }
    p0 = p1;
  }
}

template <int FMT, int D>
cudaError_t launch_d(const RopeTable* rope, const PageAppendArgs& a, int64_t n_ctas, cudaStream_t s) {
  if (rope) {
    const int smem = kPage * (rope->rot / 2) * (int)sizeof(float2);  // at most 16 KB
    page_append_kernel<FMT, D, true><<<(unsigned)n_ctas, kAppendThreads, smem, s>>>(*rope, a);
  } else {
    RopeTable none;
    none.rot = 0;
    page_append_kernel<FMT, D, false><<<(unsigned)n_ctas, kAppendThreads, 0, s>>>(none, a);
  }
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_page_append(const mixattn_kv_cache& c, const RopeTable* rope, int hq, const TokenRows& q,
                               uint16_t* q_out, int64_t q_out_stride, const TokenRows& k, const TokenRows& v,
                               const int32_t* positions, const int32_t* slots, int32_t n_new, unsigned int* err,
                               cudaStream_t s) {
  PageAppendArgs a;
  a.q = q;
  a.k = k;
  a.v = v;
  a.q_out = q_out;
  a.q_out_stride = q_out_stride;
  a.positions = positions;
  a.slots = slots;
  a.codes[0] = static_cast<uint8_t*>(c.k_quant);
  a.codes[1] = static_cast<uint8_t*>(c.v_quant);
  a.scales[0] = static_cast<float*>(c.k_scale);
  a.scales[1] = static_cast<float*>(c.v_scale);
  a.n_new = n_new;
  a.window = n_new >= 1024 ? 32 : 8;
  a.hq = hq;
  a.hkv = c.num_kv_heads;
  a.num_slots = c.num_pages * kPage;
  a.err = err;
  a.n_windows = (n_new + a.window - 1) / a.window;
  // heads per CTA: one warp each, fewer while the launch would leave SMs without work
  a.heads_per_cta = kAppendWarps;
  auto ctas = [&](int hpc) { return (int64_t)a.n_windows * 2 * ((a.hkv + hpc - 1) / hpc); };
  while (a.heads_per_cta > 1 && ctas(a.heads_per_cta) < 2 * 152) a.heads_per_cta /= 2;
  a.head_groups = (a.hkv + a.heads_per_cta - 1) / a.heads_per_cta;
  const int64_t n_ctas = ctas(a.heads_per_cta) + (rope && hq > 0 ? n_new : 0);
  if (n_ctas > INT32_MAX) return cudaErrorInvalidConfiguration;
  const bool d64 = c.head_dim == 64;
  if (c.k_fmt == MIXATTN_KV_I8_PAGE)
    return d64 ? launch_d<MIXATTN_KV_I8_PAGE, 64>(rope, a, n_ctas, s) : launch_d<MIXATTN_KV_I8_PAGE, 128>(rope, a, n_ctas, s);
  return d64 ? launch_d<MIXATTN_KV_E4M3_PAGE, 64>(rope, a, n_ctas, s) : launch_d<MIXATTN_KV_E4M3_PAGE, 128>(rope, a, n_ctas, s);
}

}  // namespace mixattn
