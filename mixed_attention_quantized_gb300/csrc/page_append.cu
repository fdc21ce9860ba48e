// page_append.cu -- append into the page-scaled 8-bit formats (one fp32 scale per
// page of 32 tokens and kv head), the keys optionally rotated on the way in and the
// step's queries rotated in the same launch.
//
// The scale of a page covers tokens that arrive in different calls, so the unit of
// work is a (page, kv head, tensor): the four warps of a CTA hold every new row of it in
// registers (one read of each new element), take their maximum with the page's old
// scale, and write their codes; when the scale grew they round the page's other codes
// again.  A page that gets its slot 0 is new and its old scale counts for nothing.
//
// Which CTA owns a page has to come from the slot list alone (no scratch memory, so
// the call can be captured, replayed and run on any stream): eight CTAs take a window
// of W consecutive tokens, enter its pages into a small hash table and look through
// the whole list for tokens of those pages; they own the pages of which no earlier
// window has a token.  Four of the eight take the keys' heads, four the values'.  In long
// calls the eight form a cluster that shares the search, each looking through an eighth
// and entering what it finds into all eight tables; in short ones, where a cluster's two
// barriers would cost more than the list, each looks through all of it.
//
// Bound: bytes (2 read and 1 written per new element), behind a launch and the search, which
// take about 4 us of each call (8201 tokens: 8500 of 27000 cycles pass before the first key or
// value is loaded).  Measured, 8 heads of 128: 64 tokens in pages of their own 4.1 us,
// 2048 in a row 7.4, 8201 15.4 (50 MB, 3.3 TB/s), 32768 65 (3.1 TB/s).  With rotated keys and 32 query
// heads, 2048 tokens 13.4, 8201 51.2; without queries 11.4 and 29.3.
#include <cooperative_groups.h>
#include <cuda_runtime.h>
#include <string.h>

#include "device_utils.cuh"
#include "internal.h"
#include "rope.cuh"

namespace mixattn {

namespace {

constexpr int kAppendThreads = 128;
constexpr int kSlices = 8;       // CTAs of a window
constexpr int kWindow = 128;     // most tokens of a window, so most pages of a CTA
constexpr int kHash = 256;
static_assert(kWindow <= kAppendThreads && kHash >= 2 * kWindow, "a thread per token of a window");
constexpr int kAppendCtas = 7;   // CTAs of an SM by registers; the rotary form at D = 128 holds
                                 // 35.9 KB of shared memory (tbl and cs 16 KB each), which lets 6 be
// New tokens from which the search is shared: at 1023 tokens in a row 5.5 us alone and 7.6 shared, at
// 2048 10.2 and 7.6.
constexpr int kClusterFrom = 1024;

struct PageAppendArgs {
  TokenRows q, k, v;
  uint16_t* q_out;
  int64_t q_out_stride;
  const int32_t* positions;
  const int32_t* slots;
  uint8_t* codes[2];  // K, V [num_pages][hkv][32][D]
  float* scales[2];   // K, V [num_pages][hkv]
  int32_t n_new, window, n_windows;
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

// Codes of eight values at 1/d.  I8: a sum with 1.5 * 2^23 rounds a magnitude below 2^22 to
// the nearest integer (ties to even) and leaves it, in two's complement, in the low byte;
// |x| <= 127 d (1 + 2^-23) keeps it within +-127.
template <int FMT>
__device__ __forceinline__ uint2 encode8(const float (&x)[8], float inv) {
  uint32_t w[2];
  // Products as sums with a -0 that the compiler does not know: it would fuse a plain paired product
  // with the paired sum behind it, which rounds once where the codes are defined by two roundings.
  const float zero = __fmul_rn(inv, -0.f);
  const uint64_t inv2 = f2_pack(inv, inv), zero2 = f2_pack(zero, zero);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint64_t y01 = ffma2(f2_pack(x[4 * h], x[4 * h + 1]), inv2, zero2), y23 = ffma2(f2_pack(x[4 * h + 2], x[4 * h + 3]), inv2, zero2);
    if (FMT == MIXATTN_KV_I8_PAGE) {
      y01 = fadd2(y01, f2_pack(12582912.f, 12582912.f));
      y23 = fadd2(y23, f2_pack(12582912.f, 12582912.f));
    }
    float y[4];
    f2_unpack(y01, y[0], y[1]);
    f2_unpack(y23, y[2], y[3]);
    if (FMT == MIXATTN_KV_I8_PAGE) {
      uint32_t q[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) q[k] = __float_as_uint(y[k]);
      w[h] = prmt(prmt(q[0], q[1], 0x0040u), prmt(q[2], q[3], 0x0040u), 0x5410u);
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
    uint32_t f[2];
    if (FMT == MIXATTN_KV_I8_PAGE) {
      s8x4_to_f16x2x2(w[h], f[0], f[1]);
    } else {
#pragma unroll
      for (int k = 0; k < 2; ++k)
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(f[k]) : "h"((uint16_t)(w[h] >> (16 * k))));
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&f[k]));
      x[4 * h + 2 * k] = v.x;
      x[4 * h + 2 * k + 1] = v.y;
    }
  }
}

// max(|a|, |b|, |c|), NaN if any is.
__device__ __forceinline__ float amax3_nan(float a, float b, float c) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// The largest of a value >= 0 (or NaN, which wins) over the CTA.
__device__ __forceinline__ float cta_max(float v, float* warp_max) {
  // non-negative floats and a NaN of clear sign compare like their bits
  const uint32_t m = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(v) & 0x7FFFFFFFu);
  if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = __uint_as_float(m);
  __syncthreads();
  uint32_t r = 0;
#pragma unroll
  for (int w = 0; w < kAppendThreads / 32; ++w) r = max(r, __float_as_uint(warp_max[w]));
  return __uint_as_float(r);
}

// One thread's share of a page: item j (16 elements, two chunks) of rows r0 + s RPS.
template <int D>
struct PageShare {
  static constexpr int LPR = D / 16;                // threads per row
  static constexpr int RPS = kAppendThreads / LPR;  // rows per step: 16 or 32
  static constexpr int STEPS = kPage / RPS;
};

// The new rows of one (page, head) as loaded: zeros where a slot gets no new token.
template <int D>
struct PageRaw {
  uint4 v[PageShare<D>::STEPS][2];
  float d_old;
};

// tok[32]: the new token of each of the page's slots, or -1.
template <int D, bool ROT>
__device__ __forceinline__ void load_page(PageRaw<D>& raw, const RopeTable& t, const int32_t* tok, const TokenRows& x,
                                          const float* scale_p, int h) {
  using P = PageShare<D>;
  const int j = threadIdx.x % P::LPR, r0 = threadIdx.x / P::LPR;
  int e0 = 16 * j, e1 = e0 + 8;
  if (ROT) rope_item(t, j, e0, e1);
#pragma unroll
  for (int s = 0; s < P::STEPS; ++s) {
    const int id = tok[s * P::RPS + r0];
    const uint16_t* src = x.x + (int64_t)max(id, 0) * x.stride + (int64_t)h * D;
    raw.v[s][0] = ldg_u128_pred(src + e0, id >= 0);
    raw.v[s][1] = ldg_u128_pred(src + e1, id >= 0);
  }
  raw.d_old = tok[0] >= 0 ? 0.f : *scale_p;
}

// One (page, head, tensor) by the CTA.  ROT: cs[(4 s + i) kAppendThreads] are the (cos, sin) of
// pairs 2i, 2i + 1 of this thread's item of step s.  warp_max: [2][warps].
template <int FMT, int D, bool ROT>
__device__ __forceinline__ void store_page(const PageRaw<D>& raw, const RopeTable& t, const float4* cs, const int32_t* tok,
                                           uint8_t* codes, float* scale_p, float* warp_max) {
  using P = PageShare<D>;
  const int j = threadIdx.x % P::LPR, r0 = threadIdx.x / P::LPR;
  int e0 = 16 * j, e1 = e0 + 8;
  if (ROT) rope_item(t, j, e0, e1);
  float x0[P::STEPS][8], x1[P::STEPS][8];
  float amax = 0.f;
#pragma unroll
  for (int s = 0; s < P::STEPS; ++s) {
    half8_to_float(raw.v[s][0], x0[s]);
    half8_to_float(raw.v[s][1], x1[s]);
    if (ROT) {
      float2 c[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 v = cs[(4 * s + i) * kAppendThreads];
        c[2 * i] = make_float2(v.x, v.y);
        c[2 * i + 1] = make_float2(v.z, v.w);
      }
      rope_rotate(t, c, j, x0[s], x1[s]);
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) amax = amax3_nan(amax, x0[s][k], x1[s][k]);
  }
  amax = cta_max(amax, warp_max);  // (every thread holds the old scale before any writes the new one)
  if (!(amax <= 65504.f)) {        // NaN, infinities or rotated values past the fp16 range: for all threads
    amax = 0.f;
#pragma unroll
    for (int s = 0; s < P::STEPS; ++s)
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        x0[s][k] = saturate_f16_range(x0[s][k]);
        x1[s][k] = saturate_f16_range(x1[s][k]);
        amax = amax3_nan(amax, x0[s][k], x1[s][k]);
      }
    amax = cta_max(amax, warp_max + kAppendThreads / 32);
  }
  const bool fresh = tok[0] >= 0;
  const float d_old = raw.d_old >= 0.f && raw.d_old < 1e30f ? raw.d_old : 0.f;  // (never written: anything)
  const float d = fmaxf(d_old, scale_for<FMT>(amax));
  const float inv = d > 0.f ? __fdiv_rn(1.f, d) : 0.f;
  const bool grown = !fresh && d > d_old;
  const float ratio = grown ? __fdiv_rn(d_old, d) : 1.f;
#pragma unroll
  for (int s = 0; s < P::STEPS; ++s) {
    const int slot = s * P::RPS + r0;
    uint8_t* row = codes + slot * D;
    uint2* p0 = reinterpret_cast<uint2*>(row + e0);
    uint2* p1 = reinterpret_cast<uint2*>(row + e1);
    if (tok[slot] >= 0) {
      const uint2 c0 = encode8<FMT>(x0[s], inv), c1 = encode8<FMT>(x1[s], inv);
      if (ROT) {
        *p0 = c0;
        *p1 = c1;
      } else {
        *reinterpret_cast<uint4*>(p0) = make_uint4(c0.x, c0.y, c1.x, c1.y);
      }
    } else if (grown) {
      decode8<FMT>(*p0, x0[s]);
      decode8<FMT>(*p1, x1[s]);
      *p0 = encode8<FMT>(x0[s], ratio);
      *p1 = encode8<FMT>(x1[s], ratio);
    }
  }
  if (threadIdx.x == 0 && (fresh || d != raw.d_old)) *scale_p = d;
}

// The jobs of one CTA: heads h0, h0 + 4, ... of every owned page.
template <int FMT, int D, bool ROT>
__device__ __forceinline__ void run_pages(const RopeTable& t, const PageAppendArgs& a, const TokenRows& x, int tensor,
                                          int h0, int np, const int32_t (*tbl)[kPage], const int32_t* page_id,
                                          const int32_t* not_mine, float* warp_max, float4* cs) {
  using P = PageShare<D>;
  auto next_page = [&](int p) {
    while (p < np && not_mine[p]) ++p;
    return p;
  };
  auto scale_of = [&](int p, int h) { return a.scales[tensor] + (int64_t)page_id[p] * a.hkv + h; };
  int p = next_page(0), h = h0;
  if (p >= np || h0 >= a.hkv) return;
  PageRaw<D> raw;
  load_page<D, ROT>(raw, t, tbl[p], x, scale_of(p, h), h);
  int cs_page = -1;
  for (int n = 0; p < np; ++n) {
    const int32_t* tok = tbl[p];
    if (ROT && cs_page != p) {  // this thread's pairs of its rows, shared by the heads (its own: no barrier)
      cs_page = p;
      const int j = threadIdx.x % P::LPR, r0 = threadIdx.x / P::LPR;
#pragma unroll
      for (int s = 0; s < P::STEPS; ++s) {
        const int id = tok[s * P::RPS + r0];
        if (id >= 0 && 16 * j < t.rot) {
          const int32_t pos = a.positions[id];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 u = rope_cos_sin(t, pos, 8 * j + 2 * i), v = rope_cos_sin(t, pos, 8 * j + 2 * i + 1);
            cs[(4 * s + i) * kAppendThreads] = make_float4(u.x, u.y, v.x, v.y);
          }
        }
      }
    }
    int pn = p, hn = h + 4;
    if (hn >= a.hkv) {
      hn = h0;
      pn = next_page(p + 1);
    }
    const PageRaw<D> now = raw;
    if (pn < np) load_page<D, ROT>(raw, t, tbl[pn], x, scale_of(pn, hn), hn);
    uint8_t* codes = a.codes[tensor] + ((int64_t)page_id[p] * a.hkv + h) * (kPage * D);
    // two areas of maxima in turn: a job's are read before the barrier of the next
    store_page<FMT, D, ROT>(now, t, cs, tok, codes, scale_of(p, h), warp_max + (n & 1) * (2 * kAppendThreads / 32));
    p = pn;
    h = hn;
  }
}

// Grid: the append CTAs, [window][slice], then one CTA per token that rotates its queries.
template <int FMT, int D, bool ROT, bool CLUSTER>
__global__ void __launch_bounds__(kAppendThreads, kAppendCtas) page_append_kernel(const __grid_constant__ RopeTable t,
                                                                     PageAppendArgs a) {
  using P = PageShare<D>;
  __shared__ int32_t tbl[kWindow][kPage];  // new token of each slot of each page, -1: none
  __shared__ int32_t hash_key[kHash], hash_val[kHash];
  __shared__ int32_t page_id[kWindow];
  __shared__ int32_t not_mine[kWindow];
  __shared__ uint32_t filter[2];           // bit (page mod 64) of every page of the window
  __shared__ float warp_max[4][kAppendThreads / 32];
  __shared__ __align__(16) float4 cs[ROT ? P::STEPS * 4 * kAppendThreads : 1];  // keys: [step][i][thread]; queries: [pair]
  const int tid = threadIdx.x;
  const int n_append = a.n_windows * kSlices;
  if (ROT && (int)blockIdx.x >= n_append) {
    const int64_t tok = blockIdx.x - n_append;
    if (tok >= a.n_new) return;  // (the grid is padded to whole clusters)
    float2* cs_q = reinterpret_cast<float2*>(cs);
    rope_fill(t, a.positions[tok], cs_q);
    __syncthreads();
    rope_row<D>(t, cs_q, a.q.x + tok * a.q.stride, a.q_out + tok * a.q_out_stride, a.hq);
    return;
  }
  const int win = blockIdx.x / kSlices, slice = blockIdx.x % kSlices;
  const int tensor = slice >> 2, h0 = slice & 3;  // heads h0, h0 + 4, ...
  if (!CLUSTER && h0 >= a.hkv) return;
  const int w0 = win * a.window, wn = min(a.window, a.n_new - w0);

  // ---- the window's pages ----
  // a page's place in the tables is the window index of its first token there, the same in
  // all CTAs of the window: a cluster's CTAs enter tokens into one another's tables
  for (int i = tid; i < a.window * kPage; i += kAppendThreads) (&tbl[0][0])[i] = -1;
  for (int i = tid; i < kHash; i += kAppendThreads) {
    hash_key[i] = -1;
    hash_val[i] = kWindow;
  }
  if (tid < 2) filter[tid] = 0u;
  __syncthreads();
  int my_page = -1, my_hash = 0;
  if (tid < wn) {
    const int32_t slot = a.slots[w0 + tid];
    if (slot >= a.num_slots) {
      set_device_error(a.err, MIXATTN_DEVERR_SLOT);
    } else if (slot >= 0) {
      my_page = slot / kPage;
      for (my_hash = my_page % kHash;; my_hash = (my_hash + 1) % kHash) {  // at most kWindow keys in twice as many places
        const int key = atomicCAS(&hash_key[my_hash], -1, my_page);
        if (key == -1 || key == my_page) break;
      }
      atomicMin(&hash_val[my_hash], tid);
      atomicOr(&filter[(my_page >> 5) & 1], 1u << (my_page & 31));
    }
  }
  const bool any = __syncthreads_or(my_page >= 0);
  if (tid < kWindow) {
    page_id[tid] = my_page;
    not_mine[tid] = !(my_page >= 0 && hash_val[my_hash] == tid);
  }
  if (CLUSTER) cooperative_groups::this_cluster().sync();
  else __syncthreads();
  if (!CLUSTER && !any) return;
  // ---- their tokens, anywhere in the call; the last of several for one slot counts ----
  const uint64_t filt = (uint64_t)filter[0] | ((uint64_t)filter[1] << 32);
  constexpr int kLoads = 8;  // list entries in flight per thread
  const int stride = CLUSTER ? kSlices * kAppendThreads : kAppendThreads;
  for (int i0 = (CLUSTER ? slice * kAppendThreads : 0) + tid; i0 < a.n_new; i0 += kLoads * stride) {
    int32_t slot[kLoads];
#pragma unroll
    for (int u = 0; u < kLoads; ++u) slot[u] = i0 + u * stride < a.n_new ? a.slots[i0 + u * stride] : -1;
#pragma unroll
    for (int u = 0; u < kLoads; ++u) {
      const int page = slot[u] >> 5;  // kPage == 32
      if (slot[u] < 0 || slot[u] >= a.num_slots || !((filt >> (page & 63)) & 1ull)) continue;
      int h = page % kHash, key;
      while ((key = hash_key[h]) != -1 && key != page) h = (h + 1) % kHash;
      if (key != page) continue;
      const int idx = hash_val[h], i = i0 + u * stride;
      int32_t* place = &tbl[idx][slot[u] % kPage];
      if (CLUSTER) {
        auto cl = cooperative_groups::this_cluster();
        for (int r = 0; r < kSlices; ++r) {
          atomicMax(cl.map_shared_rank(place, r), i);
          if (i < w0) atomicOr(cl.map_shared_rank(&not_mine[idx], r), 1);
        }
      } else {
        atomicMax(place, i);
        if (i < w0) not_mine[idx] = 1;
      }
    }
  }
  if (CLUSTER) cooperative_groups::this_cluster().sync();
  else __syncthreads();
  // ---- the owned pages: each job's rows are loaded before the job before it is done ----
  const TokenRows& x = tensor == 0 ? a.k : a.v;
  if (ROT && tensor == 0) run_pages<FMT, D, true>(t, a, x, tensor, h0, wn, tbl, page_id, not_mine, &warp_max[0][0], cs + tid);
  else run_pages<FMT, D, false>(t, a, x, tensor, h0, wn, tbl, page_id, not_mine, &warp_max[0][0], nullptr);
}

template <int FMT, int D, bool ROT>
cudaError_t launch_rot(const RopeTable& t, const PageAppendArgs& a, int64_t n_ctas, cudaStream_t s) {
  if (a.n_new < kClusterFrom) {
    page_append_kernel<FMT, D, ROT, false><<<(unsigned)n_ctas, kAppendThreads, 0, s>>>(t, a);
    return cudaGetLastError();
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((n_ctas + kSlices - 1) / kSlices * kSlices));
  cfg.blockDim = dim3(kAppendThreads);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = kSlices;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, page_append_kernel<FMT, D, ROT, true>, t, a);
}

template <int FMT, int D>
cudaError_t launch_d(const RopeTable* rope, const PageAppendArgs& a, int64_t n_ctas, cudaStream_t s) {
  if (rope) return launch_rot<FMT, D, true>(*rope, a, n_ctas, s);
  RopeTable none;
  memset(&none, 0, sizeof(none));
  return launch_rot<FMT, D, false>(none, a, n_ctas, s);
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
  // A decode step's tokens each have a page of their own: windows of one token spread them over
  // the SMs (64 tokens in 64 pages 4.1 us, with windows of eight 10.7; 200 7.8 and 11.8).  A prompt
  // fills a page with 32 tokens (512 in a row 9.1 us in windows of one, 4.8 of eight).  The count
  // alone does not tell one from the other: 300 tokens in 300 pages take 11.9 us in windows of eight
  // and 11.0 of one, from 512 on eight is faster for them too (15.4 and 16.8; 1000: 23.4 and 32.3).
  // From kClusterFrom on there are at most 120 windows, 960 CTAs, which seven an SM hold at once
  // (148 SMs or more; 2048 in a row 7.6 us with windows of 24, 9.6 with 64).  Not so the rotary
  // form at D = 128: six an SM are 912 of 152 SMs, and its queries' CTAs come on top.
  a.window = n_new > 256 ? 8 : 1;
  if (n_new >= kClusterFrom) a.window = min(kWindow, ((n_new + 119) / 120 + 7) / 8 * 8);
  a.hq = hq;
  a.hkv = c.num_kv_heads;
  a.num_slots = c.num_pages * kPage;
  a.err = err;
  a.n_windows = (n_new + a.window - 1) / a.window;
  const int64_t n_ctas = (int64_t)a.n_windows * kSlices + (rope && hq > 0 ? n_new : 0);
  if (n_ctas > INT32_MAX - kSlices) return cudaErrorInvalidConfiguration;
  const bool d64 = c.head_dim == 64;
  if (c.k_fmt == MIXATTN_KV_I8_PAGE)
    return d64 ? launch_d<MIXATTN_KV_I8_PAGE, 64>(rope, a, n_ctas, s) : launch_d<MIXATTN_KV_I8_PAGE, 128>(rope, a, n_ctas, s);
  return d64 ? launch_d<MIXATTN_KV_E4M3_PAGE, 64>(rope, a, n_ctas, s) : launch_d<MIXATTN_KV_E4M3_PAGE, 128>(rope, a, n_ctas, s);
}

}  // namespace mixattn
