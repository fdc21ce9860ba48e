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

// ===========================================================================
// Chunk tiles
// ===========================================================================
//
// A tile is 256 rows (256/G query tokens x G heads of one kv head) as two 128-row query
// tiles A and B that share every converted K and V tile of 128 keys.  Codes are exact in
// fp16, so one MMA a step does (the block formats' chunk tiles need a high and a low one),
// and a KV tile's four pages are the four 32-column chunks in which the softmax reads its
// scores: each chunk takes one (factor, offset) pair.  Roles of the 16 warps:
//   softmax A (warps 0-3) and B (4-7), thread = TMEM lane = query row: row maximum and
//     P' of S as fp16 over the scores already read; O rescaled only when a row's
//     maximum passed its reference by more than 2^8; then the output;
//   conversion (8-11): K and V codes from the cache planes, one tile ahead in
//     registers, as fp16 into 128-byte-swizzled operand tiles, two buffers each;
//   MMA (one thread of warp 12): PV_A(j-1) QK_A(j) PV_B(j-1) QK_B(j), so each query
//     tile's softmax runs beside the other's MMAs.
// The MMAs of one thread run in issue order and a commit covers all that were issued
// before it: S_A(j) complete therefore means that PV_A(j-1) is too (O may be rescaled),
// and QK_B(j) complete that K(j) and V(j-1) have been read.
// TMEM: S_A | S_B | O_A | O_B, 128 columns each, P' over the first half of its S.
// No role waits at a CTA barrier inside its loop; every wait is on an mbarrier, bounded,
// and a role that gives up leaves its loops, after which the others' waits run out.
template <int D>
struct PageChunkSmem {
  static constexpr int kTile = 128 * D * 2;  // fp16 [D/64][128 rows][128 B], swizzled
  static constexpr int kQ = 0;               // query tiles A, B
  static constexpr int kK = 2 * kTile;       // K(j) in buffer j % 2
  static constexpr int kV = 4 * kTile;
  static constexpr int kBar = 6 * kTile;
  static constexpr int kTotal = kBar + 256 + 1024;  // + slack for 1024-byte alignment
};

// Sixteen codes as two 16-byte chunks of fp16 values.
template <int F>
__device__ __forceinline__ void codes16_to_half(const uint4& c, uint4& lo, uint4& hi) {
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
  uint32_t o[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (F == MIXATTN_KV_I8_PAGE) {
      s8x4_to_f16x2x2(w[i], o[2 * i], o[2 * i + 1]);
    } else {
      asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.rn.f16x2.e4m3x2 %0, a;\n cvt.rn.f16x2.e4m3x2 %1, b;\n}"
          : "=r"(o[2 * i]), "=r"(o[2 * i + 1])
          : "r"(w[i]));
    }
  }
  lo = make_uint4(o[0], o[1], o[2], o[3]);
  hi = make_uint4(o[4], o[5], o[6], o[7]);
}

// mbar_wait for a whole warp: one answer for all lanes.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, unsigned int* err) {
  const bool ok = mbar_wait(bar, parity, err);
  return __all_sync(0xFFFFFFFFu, ok);
}

// The score factor, log2 dv and 1/dv of the page `pid` for kv head g.  A page outside the
// cache (or past the row's keys) gets the offset -inf: its keys weigh nothing.
struct PageTerms {
  float a, b, inv;
};
__device__ __forceinline__ PageTerms page_terms(const AttnParams& p, int pid, int g) {
  PageTerms r{1e-30f, -CUDART_INF_F, 0.f};
  if (pid >= 0 && pid < p.num_pages) {
    const int64_t at = (int64_t)pid * p.hkv + g;
    const float dk = reinterpret_cast<const float*>(p.k_scale)[at];
    const float dv = reinterpret_cast<const float*>(p.v_scale)[at];
    r.a = fmaxf(dk * p.scale_log2, 1e-30f);  // a page of zero keys: scores 0, and -inf stays -inf
    r.b = dv > 0.f ? log2f(dv) : 0.f;
    r.inv = dv > 0.f ? __fdiv_rn(1.f, dv) : 1.f;
  }
  return r;
}

template <int F, int D>
__device__ __forceinline__ void page_chunk_cta(const AttnParams& p, int cta, int n_ctas, uint8_t* smem_raw,
                                               unsigned int* err) {
  using L = PageChunkSmem<D>;
  constexpr uint32_t kTmemCols = 512, kOCol = 256;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kBar);
  uint64_t* q_ready = bars;       // [2] query tile A / B of the next tile written   (4 warps)
  uint64_t* qk_done = bars + 2;   // [2] S of A / B complete                          (commit)
  uint64_t* p_ready = bars + 4;   // [2] P' of A / B written, O rescaled              (4 warps)
  uint64_t* o_done = bars + 6;    // [2] the tile's last PV of A / B complete         (commit)
  uint64_t* k_ready = bars + 8;   // [2] K(jg) in buffer jg % 2                       (4 warps)
  uint64_t* v_ready = bars + 10;  // [2] V(jg) in buffer jg % 2                       (4 warps)
  uint64_t* kv_free = bars + 12;  // [2] K(jg) and V(jg-1) read                       (commit)
  uint64_t* mma_fin = bars + 14;  // every MMA of the CTA complete                    (commit)
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 15);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = p.group, lg = p.log2_group;
  const int n_rounds = (p.n_chunk_tiles + n_ctas - 1) / n_ctas;
  if (tid == 0) {
    for (int i = 0; i < 15; ++i) {
      const bool commits = (i >= 2 && i < 4) || (i >= 6 && i < 8) || i >= 12;
      mbar_init(bars + i, commits ? 1 : 4);
    }
    fence_mbar_init();
  }
  if (warp == 0) {
    tmem_alloc(tmem_slot, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp < 8) {
    // ======================= softmax A / B =======================
    const int gq = warp >> 2;
    const int row = tid & 127;
    const int tok = (gq * 128 + row) >> lg, head = row & (G - 1);
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t s_col = tmem + lane_base + 128 * gq;
    const uint32_t o_col = tmem + lane_base + kOCol + 128 * gq;
    const uint32_t ninf = __float_as_uint(-CUDART_INF_F);
    bool ok = true;
    uint32_t n_qk = 0, n_tile = 0;  // S tiles and chunk tiles this group has taken (barrier phases)
    // the CTA's next round >= k with a tile in which this query tile has rows
    auto next_round = [&](int k) {
      for (; k < n_rounds; ++k) {
        const int idx = chunk_tile_of(cta, k, n_ctas, p.n_chunk_tiles);
        if (idx >= 0 && (gq == 0 || p.tiles[idx].count * G > 128)) break;
      }
      return k;
    };
    auto write_q = [&](int k) {
      const TileDesc t = p.tiles[chunk_tile_of(cta, k, n_ctas, p.n_chunk_tiles)];
      const RowInfo ri = p.rows[t.row];
      const uint16_t* src = static_cast<const uint16_t*>(p.q) +
                            ((int64_t)(ri.q_start + t.begin + min(tok, t.count - 1)) * p.hq + (int64_t)t.kvh * G + head) * D;
      uint8_t* dst = smem + L::kQ + gq * L::kTile;
#pragma unroll
      for (int c = 0; c < D / 8; ++c) {
        const uint4 w = tok < t.count ? ldg_u128(src + 8 * c) : make_uint4(0u, 0u, 0u, 0u);
        *reinterpret_cast<uint4*>(dst + (c >> 3) * (128 * 128) + sw128_off(row, c & 7)) = w;
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&q_ready[gq]);
    };
    int k = next_round(0);
    if (k < n_rounds) write_q(k);
    while (ok && k < n_rounds) {
      const int idx = chunk_tile_of(cta, k, n_ctas, p.n_chunk_tiles);
      const TileDesc t = p.tiles[idx];
      const RowInfo ri = p.rows[t.row];
      const bool row_valid = tok < t.count;
      const int pos = ri.q_offset + t.begin + min(tok, t.count - 1);
      const int lo = window_first_key(pos, p.window);
      const int kv0 = t.kv0, n_kv = t.kv1 - t.kv0;
      const int n_pages = (min(ri.seq_len, ri.q_offset + t.begin + t.count) + kPage - 1) / kPage;
      const int32_t* pt_row = p.page_table + (int64_t)t.row * p.max_pages;
      // lane l holds the terms of page l % 4 of the tile: this one's, and the next one's page id
      auto pid_of = [&](int j) {
        const int pg = (kv0 + j) * kPagesPerKvTile + (lane & 3);
        return ldg_s32_or(pt_row + pg, j < n_kv && pg < n_pages, -1);
      };
      PageTerms next = page_terms(p, pid_of(0), t.kvh);
      int next_pid = pid_of(1);
      float m_run = -CUDART_INF_F, l_run = 0.f;
      for (int j = 0; j < n_kv; ++j) {
        const PageTerms mine = next;
        ok = warp_wait(&qk_done[gq], n_qk & 1, err);
        if (!ok) break;
        ++n_qk;
        tc_fence_after();
        if (j + 1 < n_kv) {
          next = page_terms(p, next_pid, t.kvh);
          next_pid = pid_of(j + 2);
        }
        const int kbase = (kv0 + j) * kChunkN;
        const bool diag = __any_sync(0xFFFFFFFFu, kbase + kChunkN - 1 > pos || kbase < lo);
        uint32_t a[32];
        // pass 1: the row's largest x of the tile
        float m_tile = -CUDART_INF_F;
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          tmem_ld32(s_col + 32 * c, a);
          const float ca = __shfl_sync(0xFFFFFFFFu, mine.a, c), cb = __shfl_sync(0xFFFFFFFFu, mine.b, c);
          tmem_wait_ld();
          if (diag) {
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (kbase + 32 * c + e > pos || kbase + 32 * c + e < lo) a[e] = ninf;
          }
          float mx0 = -CUDART_INF_F, mx1 = -CUDART_INF_F;
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            mx0 = fmax3(mx0, __uint_as_float(a[e]), __uint_as_float(a[e + 1]));
            mx1 = fmax3(mx1, __uint_as_float(a[e + 2]), __uint_as_float(a[e + 3]));
          }
          m_tile = fmaxf(m_tile, fmaf(fmaxf(mx0, mx1), ca, cb));
        }
        // the reference moves only when P' would pass 2^8: O is then rescaled (PV(j-1) is
        // complete, see above; a tile's first PV overwrites O)
        const bool grow = m_tile > m_run + 8.f;
        if (__any_sync(0xFFFFFFFFu, grow)) {
          const float alpha = grow ? ex2(m_run - m_tile) : 1.f;
          m_run = grow ? m_tile : m_run;
          l_run *= alpha;
          if (j > 0) {
            const uint64_t al2 = f2_pack(alpha, alpha);
#pragma unroll 1
            for (int ch = 0; ch < D / 32; ++ch) {
              tmem_ld32(o_col + 32 * ch, a);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 32; e += 2) {
                float y0, y1;
                f2_unpack(fmul2(f2_pack(__uint_as_float(a[e]), __uint_as_float(a[e + 1])), al2), y0, y1);
                a[e] = __float_as_uint(y0);
                a[e + 1] = __float_as_uint(y1);
              }
              tmem_st32(o_col + 32 * ch, a);
            }
          }
        }
        const float mref = m_run == -CUDART_INF_F ? 0.f : m_run;
        // pass 2: P' = 2^(x - m) as fp16 over the scores already read; sums in fp32
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          tmem_ld32(s_col + 32 * c, a);
          const float ca = __shfl_sync(0xFFFFFFFFu, mine.a, c);
          const float cb = __shfl_sync(0xFFFFFFFFu, mine.b, c) - mref;
          const float ci = __shfl_sync(0xFFFFFFFFu, mine.inv, c);
          const uint64_t ca2 = f2_pack(ca, ca), cb2 = f2_pack(cb, cb);
          tmem_wait_ld();
          if (diag) {
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (kbase + 32 * c + e > pos || kbase + 32 * c + e < lo) a[e] = ninf;
          }
          uint64_t sum_a = f2_pack(0.f, 0.f), sum_b = sum_a;
          uint32_t pk[16];
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            float x0, x1, x2, x3;
            f2_unpack(ffma2(f2_pack(__uint_as_float(a[e]), __uint_as_float(a[e + 1])), ca2, cb2), x0, x1);
            f2_unpack(ffma2(f2_pack(__uint_as_float(a[e + 2]), __uint_as_float(a[e + 3])), ca2, cb2), x2, x3);
            const float p0 = ex2(x0), p1 = ex2(x1), p2 = ex2(x2), p3 = ex2(x3);
            sum_a = fadd2(sum_a, f2_pack(p0, p1));
            sum_b = fadd2(sum_b, f2_pack(p2, p3));
            pk[e >> 1] = pack_f16x2(p0, p1);
            pk[(e >> 1) + 1] = pack_f16x2(p2, p3);
          }
          tmem_st16(s_col + 16 * c, pk);
          float s0, s1, s2, s3;
          f2_unpack(sum_a, s0, s1);
          f2_unpack(sum_b, s2, s3);
          l_run = fmaf((s0 + s1) + (s2 + s3), ci, l_run);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_ready[gq]);
      }
      if (!ok) break;
      // the next tile's Q (this tile's last QK is complete), then this tile's output
      const int kn = next_round(k + 1);
      if (kn < n_rounds) write_q(kn);
      ok = warp_wait(&o_done[gq], n_tile & 1, err);
      ++n_tile;
      if (!ok) break;
      tc_fence_after();
      uint16_t* dst = static_cast<uint16_t*>(p.o) +
                      ((int64_t)(ri.q_start + t.begin + tok) * p.hq + (int64_t)t.kvh * G + head) * D;
      if (t.nsplit == 1) {
        const float inv_l = 1.f / l_run;  // no key at all (every page bad): 0 / 0
#pragma unroll 1
        for (int ch = 0; ch < D / 32; ++ch) {
          uint32_t v[32];
          tmem_ld32(o_col + 32 * ch, v);
          tmem_wait_ld();
          if (row_valid) {
#pragma unroll
            for (int q4 = 0; q4 < 4; ++q4) {
              uint32_t w[4];
#pragma unroll
              for (int e = 0; e < 4; ++e)
                w[e] = pack_f16x2_out(__uint_as_float(v[8 * q4 + 2 * e]) * inv_l, __uint_as_float(v[8 * q4 + 2 * e + 1]) * inv_l);
              *reinterpret_cast<uint4*>(dst + 32 * ch + 8 * q4) = make_uint4(w[0], w[1], w[2], w[3]);
            }
          }
        }
      } else {
        // a piece of a cut tile leaves (m, l, O) of its rows; each warp's rows are merged by
        // the last piece's same warp to finish (a 4-bit ticket per warp, in the words of the
        // tile's first piece)
        const int64_t n_o = (int64_t)p.n_chunk_tiles * kPageChunkM * D;
        const int prow = gq * 128 + row;
        float* o_part = p.chunk_partials + ((int64_t)idx * kPageChunkM + prow) * D;
        float* ml_part = p.chunk_partials + n_o + ((int64_t)idx * kPageChunkM + prow) * 2;
        ml_part[0] = m_run;
        ml_part[1] = l_run;
#pragma unroll 1
        for (int ch = 0; ch < D / 32; ++ch) {
          uint32_t v[32];
          tmem_ld32(o_col + 32 * ch, v);
          tmem_wait_ld();
#pragma unroll
          for (int q4 = 0; q4 < 8; ++q4)
            *reinterpret_cast<uint4*>(o_part + 32 * ch + 4 * q4) =
                make_uint4(v[4 * q4], v[4 * q4 + 1], v[4 * q4 + 2], v[4 * q4 + 3]);
        }
        __threadfence();
        __syncwarp();
        const int first = idx - t.part;
        unsigned ticket = 0;
        if (lane == 0) ticket = (atomicAdd(&p.chunk_counters[first], 1u << (4 * warp)) >> (4 * warp)) & 15u;
        ticket = __shfl_sync(0xFFFFFFFFu, ticket, 0);
        if (ticket == (unsigned)(t.nsplit - 1)) {
          __threadfence();
          const float* ml0 = p.chunk_partials + n_o + ((int64_t)first * kPageChunkM + prow) * 2;
          const float* o0 = p.chunk_partials + ((int64_t)first * kPageChunkM + prow) * D;
          float m_all = -CUDART_INF_F;
          for (int q = 0; q < t.nsplit; ++q) m_all = fmaxf(m_all, __ldcg(ml0 + (int64_t)q * kPageChunkM * 2));
          float w[4], l_all = 0.f;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            w[q] = 0.f;
            if (q < t.nsplit) {
              const float mq = __ldcg(ml0 + (int64_t)q * kPageChunkM * 2);
              w[q] = mq == -CUDART_INF_F ? 0.f : ex2(mq - m_all);
              l_all += w[q] * __ldcg(ml0 + (int64_t)q * kPageChunkM * 2 + 1);
            }
          }
          const float inv_l = 1.f / l_all;
          if (row_valid) {
#pragma unroll 1
            for (int d0 = 0; d0 < D; d0 += 8) {
              float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                if (q >= t.nsplit || w[q] == 0.f) continue;  // (a piece without keys holds no O)
                const float* op = o0 + (int64_t)q * kPageChunkM * D + d0;
                const float4 x0 = __ldcg(reinterpret_cast<const float4*>(op));
                const float4 x1 = __ldcg(reinterpret_cast<const float4*>(op + 4));
                acc[0] += w[q] * x0.x; acc[1] += w[q] * x0.y; acc[2] += w[q] * x0.z; acc[3] += w[q] * x0.w;
                acc[4] += w[q] * x1.x; acc[5] += w[q] * x1.y; acc[6] += w[q] * x1.z; acc[7] += w[q] * x1.w;
              }
              *reinterpret_cast<uint4*>(dst + d0) =
                  make_uint4(pack_f16x2_out(acc[0] * inv_l, acc[1] * inv_l), pack_f16x2_out(acc[2] * inv_l, acc[3] * inv_l),
                             pack_f16x2_out(acc[4] * inv_l, acc[5] * inv_l), pack_f16x2_out(acc[6] * inv_l, acc[7] * inv_l));
            }
          }
        }
      }
      // O has been read: this warp's next p_ready lets the next tile's first PV overwrite it
      tc_fence_before();
      k = kn;
    }
  } else if (warp < 12) {
    // ======================= conversion of K and V =======================
    constexpr int CPR = D / 16;         // 16-byte code chunks of a key
    constexpr int KPI = 128 / CPR;      // keys between a thread's keys (16 or 32)
    constexpr int NI = kChunkN / KPI;   // keys of a thread per tile (8 or 4)
    const int t0 = tid - 256;
    const int cc = t0 % CPR, key0 = t0 / CPR;
    // destination of key key0 + i KPI: KPI is a multiple of 8, so the swizzle is the thread's own
    const uint32_t off0 = (uint32_t)((cc >> 2) * (128 * 128)) + sw128_off(key0, 2 * (cc & 3));
    const uint32_t off1 = (uint32_t)((cc >> 2) * (128 * 128)) + sw128_off(key0, 2 * (cc & 3) + 1);
    bool ok = true;
    int jg = 0;
    for (int k = 0; ok && k < n_rounds; ++k) {
      const int idx = chunk_tile_of(cta, k, n_ctas, p.n_chunk_tiles);
      if (idx < 0) continue;
      const TileDesc t = p.tiles[idx];
      const RowInfo ri = p.rows[t.row];
      const int key_end = min(ri.seq_len, ri.q_offset + t.begin + t.count);
      const int n_kv = t.kv1 - t.kv0;
      const int32_t* pt_row = p.page_table + (int64_t)t.row * p.max_pages;
      int pid[4];
      auto load_pids = [&](int j) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int pg = (t.kv0 + j) * kPagesPerKvTile + c;
          pid[c] = ldg_s32_or(pt_row + pg, j < n_kv && pg * kPage < key_end, kNoPage);
        }
      };
      auto load = [&](uint4(&raw)[NI], const uint8_t* plane, int j) {
        const int base = (t.kv0 + j) * kChunkN;
#pragma unroll
        for (int i = 0; i < NI; ++i) {
          const int key = key0 + i * KPI, c = (i * KPI) / kPage;  // key0 < KPI <= 32: the page is the loop's
          const int id = pid[c];
          const bool in = id >= 0 && id < p.num_pages;
          raw[i] = ldg_u128_pred(plane + (((int64_t)(in ? id : 0) * p.hkv + t.kvh) * kPage + (key & (kPage - 1))) * D + 16 * cc,
                                 in && base + key < key_end);
        }
      };
      auto store = [&](const uint4(&raw)[NI], uint8_t* dst) {
#pragma unroll
        for (int i = 0; i < NI; ++i) {
          uint4 x, y;
          codes16_to_half<F>(raw[i], x, y);
          *reinterpret_cast<uint4*>(dst + off0 + i * (KPI * 128)) = x;
          *reinterpret_cast<uint4*>(dst + off1 + i * (KPI * 128)) = y;
        }
        fence_proxy_async_smem();
        __syncwarp();
      };
      uint4 kr[NI], vr[NI];
      load_pids(0);
      load(kr, p.k_quant, 0);
      for (int j = 0; j < n_kv; ++j, ++jg) {
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (pid[c] != kNoPage && (pid[c] < 0 || pid[c] >= p.num_pages) && t0 == 0)
            set_device_error(err, MIXATTN_DEVERR_PAGE_ID);
        load(vr, p.v_quant, j);
        if (jg > 1) ok = warp_wait(&kv_free[jg & 1], (uint32_t)(((jg - 2) >> 1) & 1), err);
        if (!ok) break;
        store(kr, smem + L::kK + (jg & 1) * L::kTile);
        if (lane == 0) mbar_arrive(&k_ready[jg & 1]);
        load_pids(j + 1);
        if (j + 1 < n_kv) load(kr, p.k_quant, j + 1);
        if (jg > 1) ok = warp_wait(&kv_free[(jg - 1) & 1], (uint32_t)(((jg - 1) >> 1) & 1), err);
        if (!ok) break;
        store(vr, smem + L::kV + (jg & 1) * L::kTile);
        if (lane == 0) mbar_arrive(&v_ready[jg & 1]);
      }
    }
  } else if (tid == 384) {
    // ======================= MMA =======================
    constexpr uint32_t kIdescQK = idesc_f16_f32(128, kChunkN, false, false);
    constexpr uint32_t kIdescPV = idesc_f16_f32(128, D, false, true);
    const uint64_t dQ = sw128_desc(smem_u32(smem + L::kQ), 16, 1024);
    const uint64_t dK = sw128_desc(smem_u32(smem + L::kK), 16, 1024);
    const uint64_t dV = sw128_desc(smem_u32(smem + L::kV), kChunkN * 128, 1024);
    const uint32_t dVlo = (uint32_t)dV, dVhi = (uint32_t)(dV >> 32);
    bool ok = true;
    uint32_t n_p[2] = {0, 0}, n_tile[2] = {0, 0};
    int jg0 = 0;
    for (int k = 0; ok && k < n_rounds; ++k) {
      const int idx = chunk_tile_of(cta, k, n_ctas, p.n_chunk_tiles);
      if (idx < 0) continue;
      const TileDesc t = p.tiles[idx];
      const int n_kv = t.kv1 - t.kv0;
      const int n_q = t.count * G > 128 ? 2 : 1;
      for (int j = 0; ok && j <= n_kv; ++j) {
        const int jg = jg0 + j, st = jg & 1;
        for (int q = 0; ok && q < n_q; ++q) {
          const uint32_t s = tmem + 128 * q, o = tmem + kOCol + 128 * q;
          if (j > 0) {  // PV(j-1)
            const int jp = jg - 1;
            ok = mbar_wait(&p_ready[q], n_p[q] & 1, err) && mbar_wait(&v_ready[jp & 1], (uint32_t)((jp >> 1) & 1), err);
            if (!ok) break;
            ++n_p[q];
            tc_fence_after();
            const uint32_t vb = dVlo + (uint32_t)(((jp & 1) * L::kTile) >> 4);
#pragma unroll
            for (int kk = 0; kk < 8; ++kk) {
              const uint32_t boff = (uint32_t)(kk * 16 * 128) >> 4;
              if (kk == 0) tc_mma_ts_w(o, s, vb + boff, dVhi, kIdescPV, j > 1 ? 1u : 0u);
              else tc_mma_ts_w<1>(o, s + 8 * kk, vb + boff, dVhi, kIdescPV);
            }
            if (j == n_kv) tc_commit(&o_done[q]);
          }
          if (j < n_kv) {  // QK(j)
            if (j == 0) {
              ok = mbar_wait(&q_ready[q], n_tile[q] & 1, err);
              ++n_tile[q];
            }
            ok = ok && mbar_wait(&k_ready[st], (uint32_t)((jg >> 1) & 1), err);
            if (!ok) break;
            tc_fence_after();
            const uint64_t qa = dQ + (uint64_t)((q * L::kTile) >> 4), kb = dK + (uint64_t)((st * L::kTile) >> 4);
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) {
              const uint64_t off = (uint64_t)(((ks >> 2) * (128 * 128) + (ks & 3) * 32) >> 4);
              tc_mma_ss(s, qa + off, kb + off, kIdescQK, ks > 0 ? 1u : 0u);
            }
            tc_commit(&qk_done[q]);
          }
        }
        if (ok && j < n_kv) tc_commit(&kv_free[st]);
      }
      jg0 += n_kv;
    }
    // nothing this thread started may still run when TMEM is released
    tc_commit(mma_fin);
    mbar_wait(mma_fin, 0u, err);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

template <int F, int D>
__global__ void __launch_bounds__(kThreads, 2) page_decode_kernel(AttnParams p, unsigned int* err) {
  extern __shared__ __align__(1024) uint8_t smem[];
  page_decode_tile<F, D>(p, p.tiles[blockIdx.x + p.n_chunk_tiles], smem, err, 0);
}

// The fused launch: chunk CTAs, then decode CTAs of two tiles each.
template <int D>
struct PageFusedSmem {
  static constexpr int kHalf = (PageDecodeSmem<D>::kTotal + 1023) / 1024 * 1024;
  static constexpr int kBytes = PageChunkSmem<D>::kTotal > 2 * kHalf ? PageChunkSmem<D>::kTotal : 2 * kHalf;
  static_assert(kBytes <= 227 * 1024, "fused CTA does not fit in shared memory");
};

template <int F, int D>
__global__ void __launch_bounds__(kFusedThreads, 1) page_mixed_kernel(AttnParams p, unsigned int* err) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const int cta = blockIdx.x;
  if (cta < p.n_chunk_ctas) {
    page_chunk_cta<F, D>(p, cta, p.n_chunk_ctas, smem, err);
  } else {
    const int half = threadIdx.x >= kThreads ? 1 : 0;
    const int d = 2 * (cta - p.n_chunk_ctas) + half;
    if (d >= p.n_decode_tiles) return;
    page_decode_tile<F, D>(p, p.tiles[p.n_chunk_tiles + d], smem + half * PageFusedSmem<D>::kHalf, err, half);
  }
}

template <int F, int D>
cudaError_t launch_page_attention_t(const AttnParams& p, unsigned int* err, cudaStream_t s) {
  if (p.n_chunk_tiles + p.n_decode_tiles == 0) return cudaSuccess;
  constexpr int kDec = PageDecodeSmem<D>::kTotal, kFused = PageFusedSmem<D>::kBytes;
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
      if (e == cudaSuccess)
        e = cudaFuncSetAttribute(page_mixed_kernel<F, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, kFused);
      if (e != cudaSuccess) return e;
      configured[dev] = true;
    }
  }
  if (p.n_chunk_tiles == 0) {
    page_decode_kernel<F, D><<<p.n_decode_tiles, kThreads, kDec, s>>>(p, err);
  } else {
    AttnParams q = p;
    const bool persist = p.chunk_kv_tiles < kPersistMaxKvTiles * p.n_chunk_tiles;
    q.n_chunk_ctas = persist ? std::min(p.n_chunk_tiles, sm_count()) : p.n_chunk_tiles;
    const int n_ctas = q.n_chunk_ctas + (p.n_decode_tiles + 1) / 2;
    page_mixed_kernel<F, D><<<n_ctas, kFusedThreads, kFused, s>>>(q, err);
  }
  return cudaGetLastError();
}

}  // namespace mixattn
