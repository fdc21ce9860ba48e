// page_attention.cuh -- the mixed-batch attention step over the page-scaled 8-bit
// formats (one fp32 scale per page of 32 keys and kv head).
//
// With dk, dv a page's K and V scales and c_k, c_v its codes, a query sees
//     x_j = log2(e)/sqrt(D) dk (q . c_k) + log2 dv,    P'_j = 2^(x_j - m'),
//     O = sum_j P'_j c_v,   l = sum over pages (sum_j P'_j) / dv,   o = O / l,
// m' a running reference of the x_j.  The scale of V rides in the exponent, so a page
// costs one multiply-add per score whatever its scales are, the codes go to the tensor
// cores exactly as they are, and P' is at most 1 (or 2^slack) whatever the range of V.
// Partial results (m', O, l) of different key ranges merge as for a plain softmax.
//
// Decode tiles: a CTA of 8 warps takes a page range of one (row, kv head) for up to
// 8 (query, head) rows; each warp walks its pages 16 keys at a time through a cp.async
// ring, QK^T and PV on mma.sync m16n8k16 with the codes as exact fp16 operands:
//   I8_PAGE    u = q + 128 as the fp16 subnormal u 2^-24; the offset leaves the scores
//              through the accumulators' start, the values through one more MMA;
//   E4M3_PAGE  the code's exponent and mantissa shifted into fp16 places are its value
//              times 2^-8, subnormals included.
#pragma once

#include <mutex>

#include "attention_kernel.cuh"

namespace mixattn {

// Factor by which a code's fp16 operand is smaller than the code.
template <int F>
__device__ __forceinline__ constexpr float code_unit() {
  return F == MIXATTN_KV_I8_PAGE ? 16777216.f : 256.f;
}

// Bytes 0 and 2 (even) or 1 and 3 (odd) of a word of codes as fp16 operands.
template <int F>
__device__ __forceinline__ uint32_t codes_even(uint32_t w) {
  if (F == MIXATTN_KV_I8_PAGE) return q8_even(w);
  return ((w << 8) & 0x80008000u) | ((w << 7) & 0x3F803F80u);
}
template <int F>
__device__ __forceinline__ uint32_t codes_odd(uint32_t w) {
  if (F == MIXATTN_KV_I8_PAGE) return q8_odd(w);
  return (w & 0x80008000u) | ((w >> 1) & 0x3F803F80u);
}

template <int D>
struct PageDecodeSmem {
  static constexpr int kV = 16 * D;
  static constexpr int kStage = 32 * D;  // 16 keys of K, then of V
  static constexpr int kPerWarp = 16 + kMaxGroup * D;
  static constexpr int kMerge = kWarps * kPerWarp * 4;
  static constexpr int kStages = D == 128 ? 3 : 6;  // two CTAs per SM
  static constexpr int kTotal = (kWarps * kStages * kStage > kMerge ? kWarps * kStages * kStage : kMerge) + 16;
  static_assert(kTotal <= 113 * 1024, "two decode CTAs do not fit on an SM");
};

// One decode tile (see decode_tile in attention_kernel.cuh for the roles of the
// descriptor's fields): pages t.begin .. + t.count of kv head t.kvh for queries
// t.kv1 .. + t.nsplit of row t.row, G heads each.
template <int F, int D>
__device__ __forceinline__ void page_decode_tile(const AttnParams& p, const TileDesc& t, uint8_t* smem,
                                                 unsigned int* err, int half) {
  using S = PageDecodeSmem<D>;
  constexpr int KS = D / 16;
  constexpr int NS = S::kStages;
  constexpr bool kOff = F == MIXATTN_KV_I8_PAGE;
  using PL = LdsmPlan<D>;
  static_assert(PL::kCh >= 4, "rows of four or more 16-byte chunks");

  const int tid = threadIdx.x - half * kThreads, warp = tid >> 5, lane = tid & 31;
  const int r = lane >> 2, c = lane & 3;
  const int G = p.group;
  const int g = t.kvh;
  const RowInfo ri = p.rows[t.row];
  const int split = t.part;
  const int qg0 = t.kv1, nq = t.nsplit, R = nq * G;
  const int my_q = qg0 + (r < R ? (r >> p.log2_group) : 0), my_h = r & (G - 1);
  const int pos = ri.q_offset + my_q;
  const int lo = window_first_key(pos, p.window);
  const int mask_hi = ri.q_offset + qg0 + 1;
  const int mask_lo = window_first_key(ri.q_offset + qg0 + nq - 1, p.window);
  // keys past the group's last query belong to no row of the tile
  const int last_page = (ri.q_offset + qg0 + nq - 1) / kPage;
  const int n_here = min(t.count, last_page + 1 - t.begin);
  const int pg_base = n_here > 0 ? n_here / kWarps : 0, pg_rem = n_here > 0 ? n_here - pg_base * kWarps : 0;
  const int wp0 = t.begin + warp * pg_base + min(warp, pg_rem);
  const int n_pg = pg_base + (warp < pg_rem ? 1 : 0);  // at most 32
  const int n_mt = 2 * n_pg;

  float o_acc[KS][4];
#pragma unroll
  for (int i = 0; i < KS; ++i) o_acc[i][0] = o_acc[i][1] = o_acc[i][2] = o_acc[i][3] = 0.f;
  float corr[4] = {0.f, 0.f, 0.f, 0.f};  // I8_PAGE: -128 2^-24 sum of P', every row the same
  float m_run = -CUDART_INF_F, l_run = 0.f;

  const int32_t* pt_row = p.page_table + (int64_t)t.row * p.max_pages;
  const uint32_t ring_s = smem_u32(smem) + warp * (NS * S::kStage);
  int off[PL::kOffs];  // K and V rows have the same layout
#pragma unroll
  for (int i = 0; i < PL::kOffs; ++i) off[i] = PL::lane_off(i, lane);
  const int cpo0 = swz(16 * lane), cpo1 = swz(16 * lane + 512);

  // lane j holds page wp0 + j: its id, and its scales in the form the loop takes them
  const int my_pid = lane < n_pg ? pt_row[wp0 + lane] : 0;
  const bool pid_ok = my_pid >= 0 && my_pid < p.num_pages;
  const uint32_t page_ok = __ballot_sync(0xFFFFFFFFu, pid_ok);
  if (lane < n_pg && !pid_ok) set_device_error(err, MIXATTN_DEVERR_PAGE_ID);

  int st_issue = 0;
  auto issue = [&](int i) {
    if (i < n_mt) {
      const int pid = __shfl_sync(0xFFFFFFFFu, my_pid, i >> 1);
      if ((page_ok >> (i >> 1)) & 1u) {
        const uint32_t st = ring_s + st_issue * S::kStage;
        const int64_t at = ((int64_t)pid * p.hkv + g) * (kPage * D) + (16 * (i & 1) * D + 16 * lane);
        const uint8_t* kq = p.k_quant + at;
        const uint8_t* vq = p.v_quant + at;
#pragma unroll
        for (int k = 0; k < D / 32; ++k)
          cp_async16_s(st + ((k & 1) ? cpo1 : cpo0) + 512 * (k & ~1), kq + 512 * k);
#pragma unroll
        for (int k = 0; k < D / 32; ++k)
          cp_async16_s(st + S::kV + ((k & 1) ? cpo1 : cpo0) + 512 * (k & ~1), vq + 512 * k);
      }
    }
    cp_async_commit();
    st_issue = st_issue + 1 == NS ? 0 : st_issue + 1;
  };
#pragma unroll
  for (int i = 0; i < NS - 1; ++i) issue(i);

  float my_a = 0.f, my_b = 0.f, my_inv = 0.f;  // score factor, log2 dv, 1 / dv of the lane's page
  if (lane < n_pg && pid_ok) {
    const int64_t at = (int64_t)my_pid * p.hkv + g;
    const float dk = reinterpret_cast<const float*>(p.k_scale)[at];
    const float dv = reinterpret_cast<const float*>(p.v_scale)[at];
    my_a = dk * p.scale_log2 * code_unit<F>();
    my_b = dv > 0.f ? log2f(dv) : 0.f;  // a page of zeros: its codes are 0, any scale does
    my_inv = dv > 0.f ? __fdiv_rn(1.f, dv) : 1.f;
  }

  // Q as the A operand (tile row r; rows 8..15 zero): k-step 2b + j covers dims
  // 32b + 16j + 4c + {0, 2} (a0) and {1, 3} (a2), the order of a word's even and odd codes
  uint32_t qa[KS][2];
  float cb = 0.f;  // I8_PAGE: start of the scores, -128 2^-24 sum of q
  {
    const bool real = r < R;
    const uint16_t* qrow =
        static_cast<const uint16_t*>(p.q) + ((int64_t)(ri.q_start + my_q) * p.hq + (int64_t)g * G + my_h) * D;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      uint2 v = ldg_u64(qrow + 16 * ks + 4 * c);
      if (!real) v = make_uint2(0u, 0u);
      cb += (h2f_lo(v.x) + h2f_hi(v.x)) + (h2f_lo(v.y) + h2f_hi(v.y));
      qa[ks][0] = prmt(v.x, v.y, 0x5410u);
      qa[ks][1] = prmt(v.x, v.y, 0x7632u);
    }
    cb += __shfl_xor_sync(0xFFFFFFFFu, cb, 1);
    cb += __shfl_xor_sync(0xFFFFFFFFu, cb, 2);
    cb = kOff ? cb * (-128.f * 5.9604644775390625e-8f) : 0.f;
  }

  const int kv0 = 2 * c;  // the lane's keys: kv0, kv0 + 1, kv0 + 8, kv0 + 9
  int st_cons = 0;
  for (int i = 0; i < n_mt; ++i) {
    issue(i + NS - 1);
    cp_async_wait<NS - 1>();
    __syncwarp();
    const uint32_t st_s = ring_s + st_cons * S::kStage;
    st_cons = st_cons + 1 == NS ? 0 : st_cons + 1;
    const float a_pg = __shfl_sync(0xFFFFFFFFu, my_a, i >> 1);
    const float b_pg = __shfl_sync(0xFFFFFFFFu, my_b, i >> 1);
    const float inv_pg = __shfl_sync(0xFFFFFFFFu, my_inv, i >> 1);
    if ((page_ok >> (i >> 1)) & 1u) {
      const int key0 = (wp0 + (i >> 1)) * kPage + 16 * (i & 1);
      const bool partial = key0 + 16 > mask_hi || key0 < mask_lo;

      // ---------------- S = Q c_k^T ----------------
      float u0[4], u1[4];
      u0[0] = u0[1] = u1[0] = u1[1] = cb;
      u0[2] = u0[3] = u1[2] = u1[3] = 0.f;
#pragma unroll
      for (int h = 0; h < PL::kGroups; ++h) {
        uint32_t w0[4], w1[4];
        ldsm_group<D, false>(st_s, off, h, w0, w1);
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          const uint32_t a[4] = {qa[4 * h + m][0], 0u, qa[4 * h + m][1], 0u};
          const uint32_t b0[2] = {codes_even<F>(w0[m]), codes_odd<F>(w0[m])};
          const uint32_t b1[2] = {codes_even<F>(w1[m]), codes_odd<F>(w1[m])};
          mma_16816(u0, a, b0);
          mma_16816(u1, a, b1);
        }
      }

      // ---------------- softmax over the 16 keys (tile row r) ----------------
      float s[4] = {fmaf(u0[0], a_pg, b_pg), fmaf(u0[1], a_pg, b_pg), fmaf(u1[0], a_pg, b_pg), fmaf(u1[1], a_pg, b_pg)};
      if (partial) {
        auto seen = [&](int k) { return k <= pos && k >= lo; };
        s[0] = seen(key0 + kv0) ? s[0] : -CUDART_INF_F;
        s[1] = seen(key0 + kv0 + 1) ? s[1] : -CUDART_INF_F;
        s[2] = seen(key0 + kv0 + 8) ? s[2] : -CUDART_INF_F;
        s[3] = seen(key0 + kv0 + 9) ? s[3] : -CUDART_INF_F;
      }
      // the reference follows the maximum lazily: P' stays <= 2^8, so the sums of 8-bit
      // codes times P' stay far inside fp32 and P' inside fp16
      constexpr float kSlack = 8.f;
      float pm = fmax3(s[0], s[1], fmaxf(s[2], s[3]));
      if (__any_sync(0xFFFFFFFFu, pm > m_run + kSlack)) {
        pm = fmaxf(pm, __shfl_xor_sync(0xFFFFFFFFu, pm, 1));
        pm = fmaxf(pm, __shfl_xor_sync(0xFFFFFFFFu, pm, 2));
        const bool grow = pm > m_run + kSlack;
        const float alpha = grow ? ex2(m_run - pm) : 1.f;
        m_run = grow ? pm : m_run;
        l_run *= alpha;
        const float a_even = __shfl_sync(0xFFFFFFFFu, alpha, 8 * c);
        const float a_odd = __shfl_sync(0xFFFFFFFFu, alpha, 8 * c + 4);
#pragma unroll
        for (int i2 = 0; i2 < KS; ++i2) {
          o_acc[i2][0] *= a_even;
          o_acc[i2][1] *= a_odd;
          o_acc[i2][2] *= a_even;
          o_acc[i2][3] *= a_odd;
        }
        corr[0] *= a_even;
        corr[1] *= a_odd;
      }
      const float mref = m_run == -CUDART_INF_F ? 0.f : m_run;
      const float p0 = ex2(s[0] - mref), p1 = ex2(s[1] - mref);
      const float p8 = ex2(s[2] - mref), p9 = ex2(s[3] - mref);
      l_run = fmaf((p0 + p1) + (p8 + p9), inv_pg, l_run);

      // ---------------- O^T += c_v^T P' ----------------
      const uint32_t bq[2] = {pack_f16x2(p0, p1), pack_f16x2(p8, p9)};
      if (kOff) {
        constexpr uint32_t o2 = 0x80808080u;  // (-128, -128) 2^-24
        const uint32_t ao[4] = {o2, o2, o2, o2};
        mma_16816(corr, ao, bq);
      }
#pragma unroll
      for (int h = 0; h < PL::kGroups; ++h) {
        uint32_t w0[4], w1[4];
        ldsm_group<D, true>(st_s + S::kV, off, h, w0, w1);
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          const uint32_t a[4] = {codes_even<F>(w0[m]), codes_odd<F>(w0[m]), codes_even<F>(w1[m]), codes_odd<F>(w1[m])};
          mma_16816(o_acc[4 * h + m], a, bq);
        }
      }
    }
    __syncwarp();
  }
  cp_async_wait<0>();

  // ---------------- warp partial -> shared memory ----------------
  l_run += __shfl_xor_sync(0xFFFFFFFFu, l_run, 1);
  l_run += __shfl_xor_sync(0xFFFFFFFFu, l_run, 2);
  decode_sync(half);
  float* ws = reinterpret_cast<float*>(smem);
  float* wm = ws + warp * S::kPerWarp;  // m[8], l[8], O[8][D]
  const int h0 = 2 * c, h1 = 2 * c + 1;
  if (c == 0 && r < R) {
    wm[r] = m_run;
    wm[8 + r] = l_run;
  }
#pragma unroll
  for (int tt = 0; tt < KS; ++tt) {
    const int d_lo = 16 * tt + 2 * r, d_hi = d_lo + 1;  // rows r, r + 8: bytes 2r, 2r + 1 of chunk tt
    if (h0 < R) {
      wm[16 + h0 * D + d_lo] = (o_acc[tt][0] + corr[0]) * code_unit<F>();
      wm[16 + h0 * D + d_hi] = (o_acc[tt][2] + corr[0]) * code_unit<F>();
    }
    if (h1 < R) {
      wm[16 + h1 * D + d_lo] = (o_acc[tt][1] + corr[1]) * code_unit<F>();
      wm[16 + h1 * D + d_hi] = (o_acc[tt][3] + corr[1]) * code_unit<F>();
    }
  }
  decode_sync(half);

  // ---------------- merge the 8 warps, then the splits ----------------
  auto out_of = [&](int rr) {
    return static_cast<uint16_t*>(p.o) +
           ((int64_t)(ri.q_start + qg0 + (rr >> p.log2_group)) * p.hq + (int64_t)g * G + (rr & (G - 1))) * D;
  };
  const int n_out = R * D;
  const bool single = ri.n_splits == 1;
  const int slot_rows = p.slot_rows > 0 ? p.slot_rows : G;
  float* part = p.partials + (int64_t)(t.kv0 + split) * slot_rows * (D + 2);
  for (int idx = tid; idx < n_out; idx += kThreads) {
    const int h = idx / D, d = idx - h * D;
    float mmax = -CUDART_INF_F;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) mmax = fmaxf(mmax, ws[w * S::kPerWarp + h]);
    float lsum = 0.f, osum = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {  // a warp without keys holds m = -inf and zeros
      const float* x = ws + w * S::kPerWarp;
      const float sc = x[h] == -CUDART_INF_F ? 0.f : ex2(x[h] - mmax);
      lsum += sc * x[8 + h];
      osum += sc * x[16 + h * D + d];
    }
    if (single) {
      out_of(h)[d] = f16_out(osum / lsum);
    } else {
      part[h * D + d] = osum;
      if (d == 0) {
        part[slot_rows * D + 2 * h] = mmax;
        part[slot_rows * D + 2 * h + 1] = lsum;
      }
    }
  }
  if (single) return;
  __threadfence();
  decode_sync(half);
  __shared__ int s_last_of[2];
  int& s_last = s_last_of[half];
  if (tid == 0) {
    const unsigned prev = atomicAdd(&p.counters[t.kv0], 1u);
    s_last = (prev == (unsigned)(ri.n_splits - 1));
  }
  decode_sync(half);
  if (!s_last) return;
  __threadfence();
  const int ns = ri.n_splits;
  const int64_t stride = (int64_t)slot_rows * (D + 2);
  const float* parts = p.partials + (int64_t)t.kv0 * stride;
  for (int idx = tid; idx < n_out; idx += kThreads) {
    const int h = idx / D, d = idx - h * D;
    float mmax = -CUDART_INF_F;
    for (int s2 = 0; s2 < ns; ++s2) mmax = fmaxf(mmax, __ldcg(parts + s2 * stride + slot_rows * D + 2 * h));
    float lsum = 0.f, osum = 0.f;
    for (int s2 = 0; s2 < ns; ++s2) {
      const float* x = parts + s2 * stride;
      const float mx = __ldcg(x + slot_rows * D + 2 * h);
      const float sc = mx == -CUDART_INF_F ? 0.f : ex2(mx - mmax);
      lsum += sc * __ldcg(x + slot_rows * D + 2 * h + 1);
      osum += sc * __ldcg(x + h * D + d);
    }
    out_of(h)[d] = f16_out(osum / lsum);
  }
}

template <int F, int D>
__global__ void __launch_bounds__(kThreads, 2) page_decode_kernel(AttnParams p, unsigned int* err) {
  extern __shared__ __align__(1024) uint8_t smem[];
  page_decode_tile<F, D>(p, p.tiles[blockIdx.x + p.n_chunk_tiles], smem, err, 0);
}

template <int F, int D>
cudaError_t launch_page_attention_t(const AttnParams& p, unsigned int* err, cudaStream_t s) {
  if (p.n_chunk_tiles + p.n_decode_tiles == 0) return cudaSuccess;
  constexpr int kDec = PageDecodeSmem<D>::kTotal;
  {
    static std::mutex mu;
    static bool configured[kMaxDevices] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    std::lock_guard<std::mutex> lock(mu);
    if (!configured[dev]) {
      e = cudaFuncSetAttribute(page_decode_kernel<F, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, kDec);
      if (e != cudaSuccess) return e;
      configured[dev] = true;
    }
  }
  page_decode_kernel<F, D><<<p.n_decode_tiles, kThreads, kDec, s>>>(p, err);
  return cudaGetLastError();
}

}  // namespace mixattn
