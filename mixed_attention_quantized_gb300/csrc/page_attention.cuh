// page_attention.cuh -- the mixed-batch attention step over the page-scaled 8-bit
// formats (one fp32 scale per page of 32 keys and kv head).
//
// With dk, dv a page's K and V scales and c_k, c_v its codes, a query sees
//     x_j = log2(e)/sqrt(D) dk (q . c_k) + log2 dv,    P'_j = 2^(x_j - m'),
//     O = sum_j P'_j c_v,   l = sum over pages (sum_j P'_j) / dv,   o = O / l,
// m' a running reference of the x_j.  The scale of V rides in the exponent, so a page
// costs one multiply-add per score whatever its scales are, and the codes go to the tensor
// cores exactly as they are.  P' is rounded to fp16 there (2^-11 at most, as the probabilities of the
// block formats; for values of either sign 2e-4 of the output's size, beside 2e-4 of the output's own
// rounding -- exact ones would take a high and a low operand, twice the MMAs); l sums them in fp32.  The
// reference keeps the largest P' between 2^6 and 2^16, so that weights down to 2^-20 of it
// still have all 11 bits and those to 2^-30 some: a long tail under one dominant key counts in O
// as it does in l.
// Partial results (m', O, l) of different key ranges merge as for a plain softmax.
//
// Decode tiles: a CTA of 4 warps takes a page range of one (row, kv head) for up to
// 8 (query, head) rows; each warp walks its pages 16 keys at a time through a cp.async
// ring, on mma.sync m16n8k16: S^T = c_k Q^T with the 16 keys in the M rows and the tile's
// rows in N, P' turned by two movmatrix into the B operand of O^T += c_v^T P' (the page's
// scale is in the exponent, so there is one P' for all of a row's 32-element blocks).  The
// codes are exact fp16 operands:
//   I8_PAGE    u = q + 128 as the fp16 subnormal u 2^-24 (one or two logic operations a pair);
//              the offset leaves the scores through the accumulators' start, the values
//              through one more MMA;
//   E4M3_PAGE  cvt to fp16, two codes an instruction.
// Bound: HBM once the rows are long (16 rows of 30000 tokens, 8 kv heads of 128: 152 us, 6.5 TB/s;
// one session of 262144 tokens beside 15 short ones: 115 us, 97 at the copy rate), else the
// prologue and the merge (one row of 300 tokens 7.1 us, 16 rows of 8192 tokens 56 us; the loads
// alone take 49).  Keys in the M rows because eight query rows fill N exactly, where as M rows
// half of an m16 would be padding (with the rows in M and eight warps a tile: 16 rows of 8192
// tokens 66 us).
#pragma once

#include <mutex>

#include "attention_kernel.cuh"

namespace mixattn {

// Factor by which a code's fp16 operand is smaller than the code.
template <int F>
__device__ __forceinline__ constexpr float code_unit() {
  return F == MIXATTN_KV_I8_PAGE ? 16777216.f : 1.f;
}

__device__ __forceinline__ void e4m3x4_to_f16x2x2(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.rn.f16x2.e4m3x2 %0, a;\n cvt.rn.f16x2.e4m3x2 %1, b;\n}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}

// log2 dv and 1/dv of a page's V.  A page of zeros has no scale: its codes add nothing to O
// whatever stands in for it, and in l any pair (b, 2^-b) counts its keys rightly.  But b is part of
// the x that the reference m' follows, so it lies below that of every page with a value in it (fp16
// values: dv >= 2^-32): a zero page takes no bits of the others' P', and 2^60 times the sum of
// 2^31 P' below 2^16 is far inside fp32.
__device__ __forceinline__ float2 value_scale_terms(float dv) {
  return dv > 0.f ? make_float2(log2f(dv), __fdiv_rn(1.f, dv)) : make_float2(-60.f, 1152921504606846976.f);
}

// Four codes of one key (bytes 0 .. 3 of w) as the two k-pairs of an operand: codes 0, 2 and
// 1, 3 (I8_PAGE) or 0, 1 and 2, 3 (E4M3_PAGE).
template <int F>
__device__ __forceinline__ void key_pairs(uint32_t w, uint32_t& a, uint32_t& b) {
  if (F == MIXATTN_KV_I8_PAGE) {
    a = q8_even(w);
    b = q8_odd(w);
  } else {
    e4m3x4_to_f16x2x2(w, a, b);
  }
}

// Two elements of two keys (bytes 0, 1 of the first, 2, 3 of the second) as the pairs (first,
// second) of element 0 and of element 1.
template <int F>
__device__ __forceinline__ void value_pairs(uint32_t w, uint32_t& e0, uint32_t& e1) {
  if (F == MIXATTN_KV_I8_PAGE) {
    e0 = q8_even(w);
    e1 = q8_odd(w);
  } else {
    uint32_t x, y;
    e4m3x4_to_f16x2x2(w, x, y);
    e0 = prmt(x, y, 0x5410u);
    e1 = prmt(x, y, 0x7632u);
  }
}

// Transpose of an 8x8 matrix of 16-bit elements, one row's neighbouring pair per lane.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

constexpr int kPageThreads = 32 * kPageWarps;  // threads of a decode tile

template <int D>
struct PageDecodeSmem {
  static constexpr int kV = 16 * D;
  static constexpr int kStage = 32 * D;  // 16 keys of K, then of V
  static constexpr int kPerWarp = 16 + kMaxGroup * D;
  static constexpr int kMerge = kPageWarps * kPerWarp * 4;
  static constexpr int kStages = D == 128 ? 3 : 6;
  static constexpr int kRings = kPageWarps * kStages * kStage;
  static constexpr int kTotal = kRings > kMerge ? kRings : kMerge;
  static constexpr int kCtas = 16 / kPageWarps;  // CTAs per SM: 16 warps of 128 registers
  static_assert(kCtas * (kTotal + 1024) <= 227 * 1024, "the decode CTAs do not fit on an SM");
};

// Barrier over the warps of decode tile `part` of a CTA.
__device__ __forceinline__ void page_decode_sync(int part) {
  asm volatile("bar.sync %0, %1;" ::"r"(1 + part), "n"(kPageThreads) : "memory");
}

// One decode tile (see decode_tile in attention_kernel.cuh for the roles of the
// descriptor's fields): pages t.begin .. + t.count of kv head t.kvh for queries
// t.kv1 .. + t.nsplit of row t.row, G heads each.
template <int F, int D, bool TREE>
__device__ __forceinline__ void page_decode_tile(const AttnParams& p, const TileDesc& t, uint8_t* smem,
                                                 unsigned int* err, int sub) {
  using S = PageDecodeSmem<D>;
  constexpr int KS = D / 16;
  constexpr int NS = S::kStages;
  constexpr bool kOff = F == MIXATTN_KV_I8_PAGE;
  using PL = LdsmPlan<D>;
  static_assert(PL::kCh >= 4, "rows of four or more 16-byte chunks");

  const int tid = threadIdx.x - sub * kPageThreads, warp = tid >> 5, lane = tid & 31;
  const int r = lane >> 2, c = lane & 3;
  const int G = p.group;
  const int g = t.kvh;
  const RowInfo ri = p.rows[t.row];
  const int split = t.part;
  const int qg0 = t.kv1, nq = t.nsplit, R = nq * G;
  const int my_q = qg0 + (r < R ? (r >> p.log2_group) : 0), my_h = r & (G - 1);  // tile row r, whose Q this lane holds
  // the lane's scores are those of tile rows 2c and 2c + 1: their positions and window starts
  auto pos_of = [&](int row) { return ri.q_offset + qg0 + (row < R ? (row >> p.log2_group) : 0); };
  const int pos0 = pos_of(2 * c), pos1 = pos_of(2 * c + 1);
  int lo0 = window_first_key(pos0, p.window), lo1 = window_first_key(pos1, p.window);
  // a tree row's tokens see keys lo .. q_offset - 1 and those of their masks
  const int tree0 = TREE ? p.tree_starts[t.row] : -1;
  const bool tree = TREE && tree0 >= 0;
  TreeView tv0, tv1;
  if (tree) {
    tv0 = tree_view(p, ri, tree0, pos0 - ri.q_offset, lo0);
    tv1 = tree_view(p, ri, tree0, pos1 - ri.q_offset, lo1);
  }
  const int mask_hi = tree ? ri.q_offset : ri.q_offset + qg0 + 1;
  const int mask_lo = window_first_key(tree ? ri.seq_len - 1 : ri.q_offset + qg0 + nq - 1, p.window);
  // keys past the group's last query (of a tree, past the row) belong to no row of the tile
  const int last_key = tree ? ri.seq_len - 1 : ri.q_offset + qg0 + nq - 1;
  const int last_page = last_key / kPage;
  const int n_here = min(t.count, last_page + 1 - t.begin);
  const int pg_base = n_here > 0 ? n_here / kPageWarps : 0, pg_rem = n_here > 0 ? n_here - pg_base * kPageWarps : 0;
  const int wp0 = t.begin + warp * pg_base + min(warp, pg_rem);
  const int n_pg = pg_base + (warp < pg_rem ? 1 : 0);  // at most 32
  const int n_mt = 2 * n_pg;

  float o_acc[KS][4];
#pragma unroll
  for (int i = 0; i < KS; ++i) o_acc[i][0] = o_acc[i][1] = o_acc[i][2] = o_acc[i][3] = 0.f;
  float corr[4] = {0.f, 0.f, 0.f, 0.f};  // I8_PAGE: -128 2^-24 sum of P', every row the same
  float m0 = -CUDART_INF_F, m1 = -CUDART_INF_F, l0 = 0.f, l1 = 0.f;  // rows 2c, 2c + 1

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
    const float2 tv = value_scale_terms(dv);
    my_b = tv.x;
    my_inv = tv.y;
  }

  // Q as the B operand (column r: tile row r): k-step ks covers dims 16 ks + 4c .. + 3 in the
  // order of key_pairs
  uint32_t qa[KS][2];
  float cb0 = 0.f, cb1 = 0.f;  // I8_PAGE: start of the scores of rows 2c, 2c + 1: -128 2^-24 sum of q
  {
    const bool real = r < R;
    const uint16_t* qrow =
        static_cast<const uint16_t*>(p.q) + ((int64_t)(ri.q_start + my_q) * p.hq + (int64_t)g * G + my_h) * D;
    float sum = 0.f;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      uint2 v = ldg_u64(qrow + 16 * ks + 4 * c);
      if (!real) v = make_uint2(0u, 0u);
      sum += (h2f_lo(v.x) + h2f_hi(v.x)) + (h2f_lo(v.y) + h2f_hi(v.y));
      qa[ks][0] = kOff ? prmt(v.x, v.y, 0x5410u) : v.x;
      qa[ks][1] = kOff ? prmt(v.x, v.y, 0x7632u) : v.y;
    }
    if (kOff) {
      sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 1);
      sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 2);
      sum *= -128.f * 5.9604644775390625e-8f;
      cb0 = __shfl_sync(0xFFFFFFFFu, sum, 8 * c);
      cb1 = __shfl_sync(0xFFFFFFFFu, sum, 8 * c + 4);
    }
  }

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

      // ---------------- S^T = c_k Q^T: keys r and r + 8, rows 2c and 2c + 1 ----------------
      float u[4] = {cb0, cb1, cb0, cb1}, u2[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int h = 0; h < PL::kGroups; ++h) {
        uint32_t w0[4], w1[4];
        ldsm_group<D, false>(st_s, off, h, w0, w1);
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          uint32_t a[4];
          key_pairs<F>(w0[m], a[0], a[2]);
          key_pairs<F>(w1[m], a[1], a[3]);
          mma_16816((m & 1) ? u2 : u, a, qa[4 * h + m]);
        }
      }

      // ---------------- softmax over the 16 keys ----------------
      const float mr0 = m0 == -CUDART_INF_F ? 0.f : m0, mr1 = m1 == -CUDART_INF_F ? 0.f : m1;
      float x[4] = {fmaf(u[0] + u2[0], a_pg, b_pg - mr0), fmaf(u[1] + u2[1], a_pg, b_pg - mr1),
                    fmaf(u[2] + u2[2], a_pg, b_pg - mr0), fmaf(u[3] + u2[3], a_pg, b_pg - mr1)};
      uint32_t some = 0xFFFFFFFFu;  // keys that some row of a tree's tile sees; the others' page may have no scale
      if (partial) {
        const int k0 = key0 + r, k1 = k0 + 8;
        if (tree) {
          uint32_t v0 = tv0.bits(key0, p.tree_words), v1 = tv1.bits(key0, p.tree_words);
          some = __reduce_or_sync(0xFFFFFFFFu, v0 | v1);
          v0 >>= r;
          v1 >>= r;
          if (!(v0 & 1u) || k0 < lo0) x[0] = -CUDART_INF_F;
          if (!(v1 & 1u) || k0 < lo1) x[1] = -CUDART_INF_F;
          if (!(v0 & 256u) || k1 < lo0) x[2] = -CUDART_INF_F;
          if (!(v1 & 256u) || k1 < lo1) x[3] = -CUDART_INF_F;
        } else {
          if (k0 > pos0 || k0 < lo0) x[0] = -CUDART_INF_F;
          if (k0 > pos1 || k0 < lo1) x[1] = -CUDART_INF_F;
          if (k1 > pos0 || k1 < lo0) x[2] = -CUDART_INF_F;
          if (k1 > pos1 || k1 < lo1) x[3] = -CUDART_INF_F;
        }
      }
      // a reference is set 7 below the largest x and follows it lazily: P' stays <= 2^15, inside
      // fp16, and the sums of 8-bit codes times P' far inside fp32
      constexpr float kTop = 15.f, kSet = 7.f;
      float t0 = fmaxf(x[0], x[2]), t1 = fmaxf(x[1], x[3]);
      if (__any_sync(0xFFFFFFFFu, t0 > (m0 == -CUDART_INF_F ? m0 : kTop) || t1 > (m1 == -CUDART_INF_F ? m1 : kTop))) {
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
          t0 = fmaxf(t0, __shfl_xor_sync(0xFFFFFFFFu, t0, o));
          t1 = fmaxf(t1, __shfl_xor_sync(0xFFFFFFFFu, t1, o));
        }
        const bool g0 = t0 > (m0 == -CUDART_INF_F ? m0 : kTop), g1 = t1 > (m1 == -CUDART_INF_F ? m1 : kTop);
        t0 -= kSet;
        t1 -= kSet;
        const float n0 = g0 ? mr0 + t0 : m0, n1 = g1 ? mr1 + t1 : m1;
        const float al0 = g0 ? ex2(m0 - n0) : 1.f, al1 = g1 ? ex2(m1 - n1) : 1.f;
        if (g0) {
          x[0] -= t0;
          x[2] -= t0;
        }
        if (g1) {
          x[1] -= t1;
          x[3] -= t1;
        }
        m0 = n0;
        m1 = n1;
        l0 *= al0;
        l1 *= al1;
#pragma unroll
        for (int i2 = 0; i2 < KS; ++i2) {
          o_acc[i2][0] *= al0;
          o_acc[i2][1] *= al1;
          o_acc[i2][2] *= al0;
          o_acc[i2][3] *= al1;
        }
        corr[0] *= al0;
        corr[1] *= al1;
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = ex2(x[e]);
      const float inv = (some & 0xFFFFu) != 0u ? inv_pg : 0.f;
      l0 = fmaf(x[0] + x[2], inv, l0);
      l1 = fmaf(x[1] + x[3], inv, l1);

      // ---------------- O^T += c_v^T P' ----------------
      const uint32_t bq[2] = {transpose8x8(pack_f16x2(x[0], x[1])), transpose8x8(pack_f16x2(x[2], x[3]))};
      if (kOff) {
        constexpr uint32_t o2 = 0x80808080u;  // (-128, -128) 2^-24
        const uint32_t ao[4] = {o2, o2, o2, o2};
        mma_16816(corr, ao, bq);
      }
      uint32_t mk0 = 0xFFFFFFFFu, mk1 = 0xFFFFFFFFu;
      if (!kOff && partial) {  // codes of keys that no row sees may be NaN
        const int lo_first = window_first_key(tree ? ri.q_offset : ri.q_offset + qg0, p.window);
        auto any_row = [&](int k) {
          return (tree ? ((some >> (k - key0)) & 1u) != 0u : k <= last_key) && k >= lo_first;
        };
        const int k0 = key0 + 2 * c;
        mk0 = (any_row(k0) ? 0x0000FFFFu : 0u) | (any_row(k0 + 1) ? 0xFFFF0000u : 0u);
        mk1 = (any_row(k0 + 8) ? 0x0000FFFFu : 0u) | (any_row(k0 + 9) ? 0xFFFF0000u : 0u);
      }
#pragma unroll
      for (int h = 0; h < PL::kGroups; ++h) {
        uint32_t w0[4], w1[4];
        ldsm_group<D, true>(st_s + S::kV, off, h, w0, w1);
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          uint32_t a[4];
          value_pairs<F>(kOff ? w0[m] : w0[m] & mk0, a[0], a[1]);
          value_pairs<F>(kOff ? w1[m] : w1[m] & mk1, a[2], a[3]);
          mma_16816(o_acc[4 * h + m], a, bq);
        }
      }
    }
    __syncwarp();
  }
  cp_async_wait<0>();

  // ---------------- warp partial -> shared memory ----------------
#pragma unroll
  for (int o = 4; o < 32; o <<= 1) {
    l0 += __shfl_xor_sync(0xFFFFFFFFu, l0, o);
    l1 += __shfl_xor_sync(0xFFFFFFFFu, l1, o);
  }
  page_decode_sync(sub);
  float* ws = reinterpret_cast<float*>(smem);
  float* wm = ws + warp * S::kPerWarp;  // m[8], l[8], O[8][D]
  const int h0 = 2 * c, h1 = 2 * c + 1;
  if (r == 0) {  // (rows past R are never read)
    wm[h0] = m0;
    wm[h1] = m1;
    wm[8 + h0] = l0;
    wm[8 + h1] = l1;
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
  page_decode_sync(sub);

  // ---------------- merge the warps, then the splits ----------------
  // two neighbouring elements a thread: a warp's 64 belong to one row
  const int n_items = R * D / 2;
  const bool single = ri.n_splits == 1;
  const int slot_rows = p.slot_rows > 0 ? p.slot_rows : G;
  auto store = [&](int h, int d, float o0, float o1, float l) {
    uint16_t* out = static_cast<uint16_t*>(p.o) +
                    ((int64_t)(ri.q_start + qg0 + (h >> p.log2_group)) * p.hq + (int64_t)g * G + (h & (G - 1))) * D + d;
    if (tree && l == 0.f) l = CUDART_INF_F;  // (a drafted token that sees nothing gets zeros)
    *reinterpret_cast<uint32_t*>(out) = pack_f16x2_out(o0 / l, o1 / l);
  };
  const int64_t stride = (int64_t)slot_rows * (D + 2);
  float* part = p.partials + (int64_t)(t.kv0 + split) * stride;  // O [slot_rows][D], then (m, l) [slot_rows]
  for (int idx = tid; idx < n_items; idx += kPageThreads) {
    const int h = 2 * idx / D, d = 2 * idx - h * D;
    float mmax = -CUDART_INF_F;
#pragma unroll
    for (int w = 0; w < kPageWarps; ++w) mmax = fmaxf(mmax, ws[w * S::kPerWarp + h]);
    float l = 0.f, o0 = 0.f, o1 = 0.f;
#pragma unroll
    for (int w = 0; w < kPageWarps; ++w) {  // a warp without keys holds m = -inf and zeros
      const float* x = ws + w * S::kPerWarp;
      const float sc = x[h] == -CUDART_INF_F ? 0.f : ex2(x[h] - mmax);
      const float2 o = *reinterpret_cast<const float2*>(x + 16 + h * D + d);
      l += sc * x[8 + h];
      o0 += sc * o.x;
      o1 += sc * o.y;
    }
    if (single) {
      store(h, d, o0, o1, l);
    } else {
      *reinterpret_cast<float2*>(part + h * D + d) = make_float2(o0, o1);
      if (d == 0) *reinterpret_cast<float2*>(part + slot_rows * D + 2 * h) = make_float2(mmax, l);
    }
  }
  if (single) return;
  __threadfence();
  page_decode_sync(sub);
  __shared__ int s_last_of[16 / kPageWarps];
  int& s_last = s_last_of[sub];
  if (tid == 0) {
    const unsigned prev = atomicAdd(&p.counters[t.kv0], 1u);
    s_last = (prev == (unsigned)(ri.n_splits - 1));
  }
  page_decode_sync(sub);
  if (!s_last) return;
  __threadfence();
  const int ns = ri.n_splits;
  const float* parts = p.partials + (int64_t)t.kv0 * stride;
  for (int idx = tid; idx < n_items; idx += kPageThreads) {  // (whole warps: n_items is a multiple of 32)
    const int h = 2 * idx / D, d = 2 * idx - h * D;
    const float* mlp = parts + slot_rows * D + 2 * h;  // the row's (m, l) of split s at mlp + s stride
    float mmax = -CUDART_INF_F;
    for (int s2 = lane; s2 < ns; s2 += 32) mmax = fmaxf(mmax, __ldcg(mlp + s2 * stride));
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) mmax = fmaxf(mmax, __shfl_xor_sync(0xFFFFFFFFu, mmax, o));
    float l = 0.f, o0 = 0.f, o1 = 0.f;
    for (int b = 0; b < ns; b += 32) {  // lane s holds split b + s's weight
      float sc = 0.f;
      if (b + lane < ns) {
        const float2 ml = __ldcg(reinterpret_cast<const float2*>(mlp + (b + lane) * stride));
        sc = ml.x == -CUDART_INF_F ? 0.f : ex2(ml.x - mmax);
        l += sc * ml.y;
      }
      const int n = min(32, ns - b);
      const float* op = parts + b * stride + h * D + d;
#pragma unroll 8
      for (int s2 = 0; s2 < n; ++s2) {
        const float wgt = __shfl_sync(0xFFFFFFFFu, sc, s2);
        const float2 o = __ldcg(reinterpret_cast<const float2*>(op + s2 * stride));
        o0 += wgt * o.x;
        o1 += wgt * o.y;
      }
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, o);
    store(h, d, o0, o1, l);
  }
}

// ===========================================================================
// Chunk tiles
// ===========================================================================
//
// A tile is up to 256 rows (256/G query tokens x G heads of one kv head).  Codes are exact in
// fp16, so one MMA a step does (the block formats' chunk tiles need a high and a low one),
// and a KV tile's four pages are the four 32-column chunks of its scores: each takes one
// (factor, offset) pair.  Two softmax groups, 0 and 1, keep the tensor pipe busy in turn:
//   more than 128 rows: group q takes rows 128 q .. of every KV tile of 128 keys, both
//     reading each converted K and V tile;
//   at most 128 rows (a verify row, the end of a chunk): both take the same rows, group q
//     every second KV tile, and group 0 joins the two results at the end.
// Roles of the 16 warps:
//   softmax (warps 0-3 and 4-7), thread = TMEM lane = query row: one pass over its 128 scores,
//     a page's 32 at a time, against the row's reference m; P' as fp16 over the first half of
//     the page's own scores.  m is set 6 below the largest x of the row's first page (whose P' is
//     then 2^6 to fp32's last bits, no fp16 rounding: a row that sees one key gets its value), so the
//     sum of a page's P', which l needs anyway, is below the fp16 range unless one of its x passes
//     that one by 4 or more; where it is not, m moves before the P' are stored, by whole bits, and O and
//     the tile's P' so far are multiplied by a power of two;
//   conversion (K 8-11, V 13-15): codes loaded one KV tile ahead into registers, as fp16 into
//     128-byte-swizzled operand tiles, two buffers each of K and V; a K warp also writes its
//     page's terms (below);
//   MMA (one thread of warp 12): PV(j-1) and QK(j) of one group, then of the other.
// The MMAs of one thread run in issue order and a commit covers all that were issued
// before it: a group's S complete therefore means that its PV before it is too (O may be
// rescaled).  TMEM: S_0 | S_1 | O_0 | O_1, 128 columns each, P' of a page over its own scores.
// Every K warp takes part in every K tile and every V warp in every V tile, so nobody waits
// for a phase of a barrier that is not the next one.  (A parity says only which of two
// neighbouring phases is over.)
// A tile is cut into key ranges when its row alone cannot fill the SMs: a piece leaves (m, l, O) of
// its rows, and the last to finish joins them.
// Measured (8 kv heads of 128, four query heads each): the 2048-token chunk at 32768 keys beside
// four decode rows 0.92 ms, 64% of the dense rate, where a 256 x 128 unit takes ~3200 SM cycles for
// 2048 of MMAs.  What bounds it: two groups' MMAs take ~1550 cycles each where they are issued alone
// (16 of 64 cycles, each held up by operand reads and operand writes that share the 128 bytes a
// cycle of shared memory), and a group's scores and two hand-overs have to fit beside the other's.
// No role waits at a CTA barrier inside its loop; every wait is on an mbarrier, bounded,
// and a role that gives up leaves its loops, after which the others' waits run out.
template <int D>
struct PageChunkSmem {
  static constexpr int kTile = 128 * D * 2;  // fp16 [D/64][128 rows][128 B], swizzled
  static constexpr int kQ = 0;               // query tiles A, B
  static constexpr int kK = 2 * kTile;       // K(j) in buffer j % 2
  static constexpr int kV = 4 * kTile;
  static constexpr int kMl = 6 * kTile;      // (m, l) of group 1's rows
  static constexpr int kTerms = kMl + 1024;  // [4][4] terms of the pages of KV tile jg in slot jg % 4
  static constexpr int kBar = kTerms + 256;
  static constexpr int kOut = kBar + 256;    // 2 KB a softmax warp: 32 columns of its rows' output
  static constexpr int kTotal = kOut + 8 * 2048 + 1024;  // + slack for 1024-byte alignment
};

// Sixteen codes as two 16-byte chunks of fp16 values.
template <int F>
__device__ __forceinline__ void codes16_to_half(const uint4& c, uint4& lo, uint4& hi) {
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
  uint32_t o[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (F == MIXATTN_KV_I8_PAGE) s8x4_to_f16x2x2(w[i], o[2 * i], o[2 * i + 1]);
    else e4m3x4_to_f16x2x2(w[i], o[2 * i], o[2 * i + 1]);
  }
  lo = make_uint4(o[0], o[1], o[2], o[3]);
  hi = make_uint4(o[4], o[5], o[6], o[7]);
}

// mbar_wait for a whole warp: one answer for all lanes.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, unsigned int* err) {
  const bool ok = mbar_wait(bar, parity, err);
  return __all_sync(0xFFFFFFFFu, ok);
}

// The terms of a page: score factor, log2 dv and 1/dv.  A missing page (outside the cache, or
// past the row's keys) gets the offset -inf: its keys weigh nothing.
__device__ __forceinline__ float4 page_terms(float dk, float dv, bool there, float scale_log2) {
  const float2 tv = value_scale_terms(dv);
  return make_float4(fmaxf(dk * scale_log2, 1e-30f),  // a page of zero keys: scores 0, and -inf stays -inf
                     there ? tv.x : -CUDART_INF_F, tv.y, 0.f);
}

// A chunk row's reference: kChunkSet below the largest x when it is set, and moved to 6 to 7 below
// when the 32 P' of a page sum to kChunkTop (so one is 2^10.98 or more; none above 65504
// passes).  The page's largest fp16 P' as the test, by packed integer maxima, with 11 and 2^15: the
// chunk of 2048 tokens at 32768 keys 1160 -> 1200 us.
constexpr float kChunkSet = 6.f, kChunkTop = 65000.f, kChunkMoved = 10.9f;

// A row's D columns of O times alpha.
template <int D>
__device__ __forceinline__ void scale_output(uint32_t o_col, float alpha) {
  const uint64_t al2 = f2_pack(alpha, alpha);
#pragma unroll 1
  for (int ch = 0; ch < D / 16; ++ch) {
    uint32_t o[16];
    tmem_ld16(o_col + 16 * ch, o);
    tmem_wait_ld();
#pragma unroll
    for (int e = 0; e < 16; e += 2) {
      float y0, y1;
      f2_unpack(fmul2(f2_pack(__uint_as_float(o[e]), __uint_as_float(o[e + 1])), al2), y0, y1);
      o[e] = __float_as_uint(y0);
      o[e + 1] = __float_as_uint(y1);
    }
    tmem_st16(o_col + 16 * ch, o);
  }
}

// The P' of a KV tile's pages before c times 2^-up (whole bits), as two fp16 powers of two down to
// 2^-48: below 2^-40 no P' is left of it.
__device__ __forceinline__ void scale_weights(uint32_t s_col, int c, float up) {
  const float e_all = fmaxf(-up, -48.f), e_half = ceilf(0.5f * e_all);
  const float al_1 = ex2(e_half), al_2 = ex2(e_all - e_half);
  const uint32_t al_h = pack_f16x2(al_1, al_1), al_l = pack_f16x2(al_2, al_2);
  tmem_wait_st();  // the P' of the pages before are in place
#pragma unroll 1
  for (int b = 0; b < c; ++b) {
    uint32_t o[16];
    tmem_ld16(s_col + 32 * b, o);
    tmem_wait_ld();
#pragma unroll
    for (int e = 0; e < 16; ++e) o[e] = hmul2_u32(hmul2_u32(o[e], al_h), al_l);
    tmem_st16(s_col + 32 * b, o);
  }
}

// The softmax's rare step, for page c (32 scores at s_col + 32 c) of a warp in which some row's
// P' sum to kChunkTop, or which has rows without a reference: moves the references of the rows
// that need it, multiplies O (if there is one yet: `scale_o`), l and the P' of the KV tile's
// pages before c by the change, a power of two, and writes the page's P'.  Out of line, so
// that the common path stays short.  Returns (m, l).  The row sees scores c_first .. c_last of the
// page; TREE: those with a bit in `c_first` from c_last on.
template <int D, bool TREE>
__device__ __noinline__ float2 page_move_reference(uint32_t s_col, uint32_t o_col, int c, float4 tm, int c_first,
                                                   int c_last, float m_run, float l_run, bool scale_o) {
  auto in = [&](int e) {
    if (TREE) return (((uint32_t)c_first >> e) & 1u) != 0u && e >= c_last;
    return e >= c_first && e <= c_last;
  };
  const uint32_t sc = s_col + 32 * c;
  float mx = -CUDART_INF_F;
#pragma unroll 1
  for (int b = 0; b < 2; ++b) {
    uint32_t o[16];
    tmem_ld16(sc + 16 * b, o);
    tmem_wait_ld();
#pragma unroll
    for (int e = 0; e < 16; ++e)
      if (in(16 * b + e)) mx = fmaxf(mx, __uint_as_float(o[e]));
  }
  mx = fmaf(mx, tm.x, tm.y);
  const bool grow = mx > -CUDART_INF_F && (m_run == -CUDART_INF_F || mx >= m_run + kChunkMoved);
  const bool first = m_run == -CUDART_INF_F;
  const float up = grow ? (first ? 0.f : floorf(mx - m_run - kChunkSet)) : 0.f;  // whole bits
  const float m_new = grow ? (first ? mx - kChunkSet : m_run + up) : m_run;
  const float alpha = grow && first ? 0.f : ex2(-up);  // a power of two, or 0
  l_run *= alpha;
  if (scale_o) scale_output<D>(o_col, alpha);
  scale_weights(s_col, c, up);
  // the page's P', 16 scores at a time: their 8 words stay before the scores not yet read
  const float cb = tm.y - (m_new == -CUDART_INF_F ? 0.f : m_new);
  float l_page = 0.f;
#pragma unroll 1
  for (int b = 0; b < 2; ++b) {
    uint32_t o[16], w[8];
    tmem_ld16(sc + 16 * b, o);
    tmem_wait_ld();
#pragma unroll
    for (int e = 0; e < 16; e += 2) {
      const bool in0 = in(16 * b + e), in1 = in(16 * b + e + 1);
      const float p0 = in0 ? ex2(fmaf(__uint_as_float(o[e]), tm.x, cb)) : 0.f;
      const float p1 = in1 ? ex2(fmaf(__uint_as_float(o[e + 1]), tm.x, cb)) : 0.f;
      l_page += p0 + p1;
      w[e >> 1] = pack_f16x2(p0, p1);
    }
    tmem_st8(sc + 8 * b, w);
  }
  return make_float2(m_new, fmaf(l_page, tm.z, l_run));
}

// A chunk tile's output rows, D elements each, heads first, then tokens; written by a warp through
// its 2 KB of shared memory, so that a store has four lanes to a row.
struct PageRowsOut {
  uint8_t* stage;
  uint16_t* dst;  // row 0
  int n_rows, lg, hq;

  // columns d0 .. d0 + 31 of row row0 + lane, packed
  template <int D>
  __device__ __forceinline__ void put(int row0, int d0, const uint32_t (&w)[16]) const {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int c = 0; c < 4; ++c)
      *reinterpret_cast<uint4*>(stage + 64 * lane + 16 * (c ^ ((lane >> 1) & 3))) =
          make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = 8 * i + (lane >> 2), c = lane & 3, row = row0 + r;
      const uint4 x = *reinterpret_cast<const uint4*>(stage + 64 * r + 16 * (c ^ ((r >> 1) & 3)));
      if (row < n_rows)
        *reinterpret_cast<uint4*>(dst + ((int64_t)(row >> lg) * hq + (row & ((1 << lg) - 1))) * D + d0 + 8 * c) = x;
    }
    __syncwarp();
  }
};

static_assert(kPageMaxPieces <= 4, "a tile is cut from eight KV tiles on: its pieces have two or more");

// Joins the pieces of a cut chunk tile for units u, u + u_step, .. below u_end; unit i is 32 rows
// (block i / (D / 32)) by 32 columns.  o and ml: the first piece's partials.  Out of line, so that
// it takes no registers from the common path.
template <int D, bool TREE>
__device__ __noinline__ void page_merge_pieces(PageRowsOut out, const float* o, const float2* ml, int nsplit, int u,
                                               int u_end, int u_step, bool tree) {
  const int lane = threadIdx.x & 31;
#pragma unroll 1
  for (; u < u_end; u += u_step) {
    const int row0 = 32 * (u / (D / 32)), d0 = 32 * (u % (D / 32));
    const float* o_unit = o + (int64_t)row0 * D + 32 * d0 + 4 * lane;
    float2 s[kPageMaxPieces];
    float m_all = -CUDART_INF_F, l_all = 0.f;
#pragma unroll
    for (int q = 0; q < kPageMaxPieces; ++q) s[q] = __ldcg(ml + min(q, nsplit - 1) * kPageChunkM + row0 + lane);
#pragma unroll
    for (int q = 0; q < kPageMaxPieces; ++q) {
      if (q >= nsplit) s[q].x = -CUDART_INF_F;
      m_all = fmaxf(m_all, s[q].x);
    }
#pragma unroll
    for (int q = 0; q < kPageMaxPieces; ++q) {
      s[q].x = s[q].x == -CUDART_INF_F ? 0.f : ex2(s[q].x - m_all);
      if (q < nsplit) l_all += s[q].x * s[q].y;  // (NaN where a piece's scores are all NaN)
    }
    const float inv_l = TREE && tree && l_all == 0.f ? 0.f : 1.f / l_all;
    uint32_t x[16];
#pragma unroll
    for (int c0 = 0; c0 < 8; c0 += 4) {  // the loads of 16 columns together
      float4 y[kPageMaxPieces][4];
#pragma unroll
      for (int q = 0; q < kPageMaxPieces; ++q)
#pragma unroll
        for (int c = 0; c < 4; ++c)
          y[q][c] = __ldcg(reinterpret_cast<const float4*>(o_unit + min(q, nsplit - 1) * (kPageChunkM * D) + 128 * (c0 + c)));
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int q = 0; q < kPageMaxPieces; ++q) {
          if (s[q].x == 0.f) continue;  // (no key of the row in this piece, or no such piece: any value may stand there)
          acc.x += s[q].x * y[q][c].x; acc.y += s[q].x * y[q][c].y; acc.z += s[q].x * y[q][c].z; acc.w += s[q].x * y[q][c].w;
        }
        x[2 * (c0 + c)] = pack_f16x2_out(acc.x * inv_l, acc.y * inv_l);
        x[2 * (c0 + c) + 1] = pack_f16x2_out(acc.z * inv_l, acc.w * inv_l);
      }
    }
    out.put<D>(row0, d0, x);
  }
}

// The launches overlap the end of the kernel before them, which writes the tile list into the
// workspace: nothing of the workspace (nor the tensors, which earlier kernels may be writing)
// is touched before that grid is complete.
__device__ __forceinline__ void wait_for_upload() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

template <int F, int D, bool TREE>
__device__ __forceinline__ void page_chunk_cta(const AttnParams& p, int cta, int n_ctas, uint8_t* smem_raw,
                                               unsigned int* err) {
  using L = PageChunkSmem<D>;
  constexpr uint32_t kTmemCols = 512, kOCol = 256;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kBar);
  // by 4 warps each:
  uint64_t* q_ready = bars;        // [2] a group's query rows of its next tile written
  uint64_t* p_ready = bars + 2;    // [2] a group's P' written, O rescaled
  uint64_t* ml_ready = bars + 4;   // group 1's (m, l) in shared memory, its O complete
  uint64_t* joined = bars + 5;     // group 0 has read group 1's O
  uint64_t* k_ready = bars + 6;    // [2] K(jg) in buffer jg % 2
  // by 3 warps:
  uint64_t* v_ready = bars + 8;    // [2] V(jg) in buffer jg % 2
  // by a commit:
  uint64_t* qk_done = bars + 10;   // [2] a group's S complete
  uint64_t* o_done = bars + 12;    // [2] a group's last PV of the tile complete
  uint64_t* k_free = bars + 14;    // [2] K(jg) read
  uint64_t* v_free = bars + 16;    // [2] V(jg) read
  uint64_t* mma_fin = bars + 18;   // every MMA of the CTA complete
  constexpr int kNumBars = 19;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + kNumBars);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = p.group, lg = p.log2_group;
  const int n_rounds = (p.n_chunk_tiles + n_ctas - 1) / n_ctas;
  if (tid == 0) {
    for (int i = 0; i < kNumBars; ++i) mbar_init(bars + i, i < 8 ? 4 : (i < 10 ? 3 : 1));
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
  wait_for_upload();

  if (warp < 8) {
    // ======================= softmax groups =======================
    const int gq = warp >> 2;
    const int row = tid & 127;
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t s_col = tmem + lane_base + 128 * gq;
    const uint32_t o_col = tmem + lane_base + kOCol + 128 * gq;
    float2* ml = reinterpret_cast<float2*>(smem + L::kMl);
    bool ok = true;
    uint32_t n_qk = 0, n_tile = 0, n_join = 0;  // S tiles, chunk tiles, joined tiles so far (barrier phases)
    int jg0 = 0;  // KV tiles before the chunk tile, over all the CTA's (also those without this group)
    int jg_skip = 0;  // KV tiles of the tiles that next_round has passed over
    // the CTA's next round >= k with a tile in which this group takes part
    auto next_round = [&](int k) {
      for (; k < n_rounds; ++k) {
        const int idx = chunk_tile_of(cta, k, n_ctas, p.n_chunk_tiles);
        if (idx < 0) continue;
        if (gq == 0) break;
        const TileDesc& t = p.tiles[idx];
        if (t.count * G > 128 || t.kv1 - t.kv0 > 1) break;
        jg_skip += t.kv1 - t.kv0;
      }
      return k;
    };
    auto write_q = [&](int k) {
      const TileDesc t = p.tiles[chunk_tile_of(cta, k, n_ctas, p.n_chunk_tiles)];
      const RowInfo ri = p.rows[t.row];
      const int base = t.count * G > 128 ? gq * 128 : 0;
      const uint16_t* src = static_cast<const uint16_t*>(p.q) +
                            ((int64_t)(ri.q_start + t.begin) * p.hq + (int64_t)t.kvh * G) * D;
      uint8_t* dst = smem + L::kQ + gq * L::kTile;
      // a row's 16-byte chunks to neighbouring lanes, 2 or 4 rows a load (one row a lane is 32 lines
      // a load: 7500 cycles for the tile, and the page ids and K codes wait behind them)
      constexpr int CH = D / 8;
      const int c = lane % CH;
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        const int r = 32 * (warp & 3) + i * (32 / CH) + lane / CH, tok = (base + r) >> lg, h = (base + r) & (G - 1);
        const uint4 w = tok < t.count ? ldg_u128(src + ((int64_t)tok * p.hq + h) * D + 8 * c) : make_uint4(0u, 0u, 0u, 0u);
        *reinterpret_cast<uint4*>(dst + (c >> 3) * (128 * 128) + sw128_off(r, c & 7)) = w;
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&q_ready[gq]);
    };
    int k = next_round(0);
    if (k < n_rounds) write_q(k);
    while (ok && k < n_rounds) {
      jg0 += jg_skip;
      jg_skip = 0;
      const int idx = chunk_tile_of(cta, k, n_ctas, p.n_chunk_tiles);
      const TileDesc t = p.tiles[idx];
      const RowInfo ri = p.rows[t.row];
      const bool two = t.count * G > 128;  // each group its own rows; else each its own KV tiles
      const int prow = (two ? gq * 128 : 0) + row;
      const int tok = prow >> lg;
      const bool row_valid = tok < t.count;
      const bool idle = (prow & ~31) >= t.count * G;  // a warp whose rows are all past the tile's only keeps step
      const int pos = ri.q_offset + t.begin + min(tok, t.count - 1);
      int lo = window_first_key(pos, p.window);
      const int tree0 = TREE ? p.tree_starts[t.row] : -1;
      const bool tree = TREE && tree0 >= 0;
      TreeView tv;
      if (tree) tv = tree_view(p, ri, tree0, t.begin + min(tok, t.count - 1), lo);
      const int kv0 = t.kv0, n_kv = t.kv1 - t.kv0;
      const int j0 = two ? 0 : gq, dj = two ? 1 : 2;
      float m_run = -CUDART_INF_F, l_run = 0.f;
      for (int j = j0; j < n_kv; j += dj) {
        ok = warp_wait(&qk_done[gq], n_qk & 1, err);
        if (!ok) break;
        ++n_qk;
        tc_fence_after();
        if (idle) {  // (its P' rows are whatever was there: no other row's result reads them)
          __syncwarp();
          if (lane == 0) mbar_arrive(&p_ready[gq]);
          continue;
        }
        const float4* terms = reinterpret_cast<const float4*>(smem + L::kTerms) + 4 * ((jg0 + j) & 3);
        const int kbase = (kv0 + j) * kChunkN;
        // the first and last visible key of the row in this tile (usually 0 and 127)
        const int first = lo - kbase, last = (tree ? ri.q_offset - 1 : pos) - kbase;
        const bool diag = __any_sync(0xFFFFFFFFu, last < kChunkN - 1 || first > 0);
        float4 tn = terms[0];  // (a page ahead: a shared-memory load is slow beside the MMAs' reads)
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          const float4 tm = tn;
          tn = terms[(c + 1) & 3];
          // (TREE: the visible scores of the page as bits, and the first of them in the window)
          int c_first = first - 32 * c, c_last = last - 32 * c;
          if (TREE) {
            const int from = c_first;
            c_first = -1;
            if (tree) c_first = (int)tv.bits(kbase + 32 * c, p.tree_words);
            else if (c_last < 31) c_first = c_last < 0 ? 0 : (int)((2u << c_last) - 1u);
            c_last = from;
          }
          const uint32_t sc = s_col + 32 * c;
          uint32_t x[32], pk[16];
          tmem_ld32(sc, x);
          const float cb = tm.y - (m_run == -CUDART_INF_F ? 0.f : m_run);
          const uint64_t ca2 = f2_pack(tm.x, tm.x), cb2 = f2_pack(cb, cb);
          tmem_wait_ld();
          if (diag) {
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (TREE ? !(((uint32_t)c_first >> e) & 1u) || e < c_last : e < c_first || e > c_last)
                x[e] = __float_as_uint(-CUDART_INF_F);
          }
          uint64_t sum_a = f2_pack(0.f, 0.f), sum_b = sum_a;
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            float x0, x1, x2, x3;
            f2_unpack(ffma2(f2_pack(__uint_as_float(x[e]), __uint_as_float(x[e + 1])), ca2, cb2), x0, x1);
            f2_unpack(ffma2(f2_pack(__uint_as_float(x[e + 2]), __uint_as_float(x[e + 3])), ca2, cb2), x2, x3);
            const float p0 = ex2(x0), p1 = ex2(x1), p2 = ex2(x2), p3 = ex2(x3);
            sum_a = fadd2(sum_a, f2_pack(p0, p1));
            sum_b = fadd2(sum_b, f2_pack(p2, p3));
            pk[e >> 1] = pack_f16x2(p0, p1);
            pk[(e >> 1) + 1] = pack_f16x2(p2, p3);
          }
          float s0, s1;
          f2_unpack(fadd2(sum_a, sum_b), s0, s1);
          const float l_page = s0 + s1;
          // (infinity and NaN too; a row without a reference takes one with its first key)
          const bool over = !(l_page < kChunkTop) || m_run == -CUDART_INF_F;
          if (!__any_sync(0xFFFFFFFFu, over)) {
            tmem_st16(sc, pk);
            l_run = fmaf(l_page, tm.z, l_run);
            continue;
          }
          const float2 ml_new = page_move_reference<D, TREE>(s_col, o_col, c, tm, c_first, c_last, m_run, l_run, j > j0);
          m_run = ml_new.x;
          l_run = ml_new.y;
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_ready[gq]);
      }
      if (!ok) break;
      // the next tile's Q (the group's last QK of this tile is complete), then this tile's output
      jg0 += n_kv;
      const int kn = next_round(k + 1);
      if (kn < n_rounds) write_q(kn);
      ok = warp_wait(&o_done[gq], n_tile & 1, err);
      ++n_tile;
      if (!ok) break;
      tc_fence_after();
      const bool join = !two && n_kv > 1;
      const int row0 = prow & ~31;
      const PageRowsOut out{smem + L::kOut + 2048 * warp,
                            static_cast<uint16_t*>(p.o) + ((int64_t)(ri.q_start + t.begin) * p.hq + (int64_t)t.kvh * G) * D,
                            t.count * G, lg, p.hq};
      float* part = p.chunk_partials + (int64_t)idx * kPageChunkM * D;  // [32-row block][D / 4][row] of 4 columns
      float2* ml_part = reinterpret_cast<float2*>(p.chunk_partials + (int64_t)p.n_chunk_tiles * kPageChunkM * D) +
                        (int64_t)idx * kPageChunkM;
      if (join && gq == 1) {  // hand (m, l, O) to group 0 and wait until it has read them
        ml[row] = make_float2(m_run, l_run);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(ml_ready);
        ok = warp_wait(joined, n_join & 1, err);
        ++n_join;
        if (!ok) break;
        tc_fence_after();
      } else {
        float w0 = 1.f, w1 = 0.f;  // weights of the two groups' O
        if (join) {
          ok = warp_wait(ml_ready, n_join & 1, err);
          if (!ok) break;
          tc_fence_after();
          const float2 other = ml[row];
          const float m = fmaxf(m_run, other.x);
          w0 = m_run == -CUDART_INF_F ? 0.f : ex2(m_run - m);
          w1 = other.x == -CUDART_INF_F ? 0.f : ex2(other.x - m);
          l_run = l_run * w0 + other.y * w1;
          m_run = m;
        }
        // 16 columns of the tile's O, unnormalised
        auto o_chunk = [&](int ch, uint32_t(&v)[16]) {
          tmem_ld16(o_col + 16 * ch, v);
          if (join) {
            uint32_t u[16];
            tmem_ld16(o_col + 128 + 16 * ch, u);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e)
              v[e] = __float_as_uint(__uint_as_float(v[e]) * w0 + __uint_as_float(u[e]) * w1);
          } else {
            tmem_wait_ld();
          }
        };
        if (idle) {
        } else if (t.nsplit == 1) {
          // no key at all (every page bad): 0 / 0; a drafted token that sees nothing: zeros
          const float inv_l = tree && l_run == 0.f ? 0.f : 1.f / l_run;
#pragma unroll 1
          for (int ch = 0; ch < D / 16; ch += 2) {
            uint32_t w[16];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              uint32_t v[16];
              o_chunk(ch + h, v);
#pragma unroll
              for (int e = 0; e < 8; ++e)
                w[8 * h + e] = pack_f16x2_out(__uint_as_float(v[2 * e]) * inv_l, __uint_as_float(v[2 * e + 1]) * inv_l);
            }
            out.put<D>(row0, 16 * ch, w);
          }
        } else {  // a piece of a cut tile leaves (m, l, O) of its rows
          ml_part[prow] = make_float2(m_run, l_run);
#pragma unroll 1
          for (int ch = 0; ch < D / 16; ++ch) {
            uint32_t v[16];
            o_chunk(ch, v);
#pragma unroll
            for (int q4 = 0; q4 < 4; ++q4)
              *reinterpret_cast<uint4*>(part + (int64_t)row0 * D + 128 * (4 * ch + q4) + 4 * lane) =
                  make_uint4(v[4 * q4], v[4 * q4 + 1], v[4 * q4 + 2], v[4 * q4 + 3]);
          }
        }
        // O has been read: the groups' next p_ready lets the next tile's first PVs overwrite it
        tc_fence_before();
        __syncwarp();
        if (join) {
          if (lane == 0) mbar_arrive(joined);
          if (t.nsplit > 1) ok = warp_wait(joined, n_join & 1, err);  // (below, this warp speaks for the others)
          ++n_join;
          if (!ok) break;
        }
      }
      // The last piece to finish joins all: of a tile with rows in both groups each warp its own
      // rows, else all eight warps a share (every piece has two KV tiles or more, so both groups
      // are here for each).  A 4-bit ticket per warp, in the word of the tile's first piece; joined
      // in the pieces' order, whichever was last.
      if (t.nsplit > 1 && !(two && idle)) {
        __threadfence();
        __syncwarp();
        unsigned ticket = 0;
        if (lane == 0) ticket = (atomicAdd(&p.chunk_counters[idx - t.part], 1u << (4 * warp)) >> (4 * warp)) & 15u;
        ticket = __shfl_sync(0xFFFFFFFFu, ticket, 0);
        if (ticket == (unsigned)(t.nsplit - 1)) {
          __threadfence();
          constexpr int U = D / 32;
          const int u0 = two ? (row0 / 32) * U : warp, u_end = two ? u0 + U : ((t.count * G + 31) / 32) * U;
          page_merge_pieces<D, TREE>(out, part - (int64_t)t.part * kPageChunkM * D, ml_part - (int64_t)t.part * kPageChunkM, t.nsplit,
                               u0, u_end, two ? 1 : 8, tree);
        }
      }
      k = kn;
    }
  } else if (warp != 12) {
    // ======================= conversion: K warps 8-11, V warps 13-15 =======================
    constexpr int CPR = D / 16;           // 16-byte code chunks of a key
    constexpr int KPL = 32 / CPR;         // keys of a load (4 or 8)
    constexpr int NL = 48 / KPL;          // most loads of a warp and tile
    const bool is_v = warp >= 12;
    // the warp's keys of a tile: 32 each of K; 48, 40, 40 of V.  They lie in one or two pages,
    // the second's from load `turn` on.
    const int w = is_v ? warp - 13 : warp - 8;
    const int r0 = is_v ? (w == 0 ? 0 : 8 + 40 * w) : 32 * w;
    const int n_load = (is_v ? (w == 0 ? 48 : 40) : 32) / KPL;
    const int turn = (kPage - (r0 & (kPage - 1))) / KPL;
    // eight lanes write neighbouring chunks of two keys (of one, at D = 128, they would meet in banks)
    const int cc = (lane & 3) | (D == 128 ? lane >> 4 << 2 : 0), key0 = r0 + (D == 128 ? (lane >> 2) & 3 : lane >> 2);
    // the lane's two 16-byte places in row key0 of a tile; row key0 + 4 i flips chunk bit 2 for odd i
    const uint32_t off0 = (uint32_t)((cc >> 2) * (128 * 128)) + sw128_off(key0, 2 * (cc & 3));
    const uint32_t off1 = (uint32_t)((cc >> 2) * (128 * 128)) + sw128_off(key0, 2 * (cc & 3) + 1);
    const uint8_t* plane = (is_v ? p.v_quant : p.k_quant) + (key0 & (kPage - 1)) * D + 16 * cc;
    uint64_t* freed = is_v ? v_free : k_free;
    uint64_t* ready = is_v ? v_ready : k_ready;
    bool ok = true;
    int jg = 0;  // KV tiles so far, over the CTA's chunk tiles: buffers and barrier phases follow it
    for (int k = 0; ok && k < n_rounds; ++k) {
      const int idx = chunk_tile_of(cta, k, n_ctas, p.n_chunk_tiles);
      if (idx < 0) continue;
      const TileDesc t = p.tiles[idx];
      const RowInfo ri = p.rows[t.row];
      const bool tree = TREE && p.tree_starts[t.row] >= 0;  // (its tokens may see any other of the row)
      const int key_end = (tree ? ri.seq_len : min(ri.seq_len, ri.q_offset + t.begin + t.count)) -
                          t.kv0 * kChunkN;  // keys of the KV range
      const int n_kv = t.kv1 - t.kv0;
      const int32_t* pt_row = p.page_table + (int64_t)t.row * p.max_pages + t.kv0 * kPagesPerKvTile;
      // the ids of the warp's two pages of KV tile j
      auto pids_of = [&](int j) {
        const int pg = j * kPagesPerKvTile + r0 / kPage;
        return make_int2(ldg_s32_or(pt_row + pg, j < n_kv && pg * kPage < key_end, kNoPage),
                         ldg_s32_or(pt_row + pg + 1, j < n_kv && turn < n_load && (pg + 1) * kPage < key_end, kNoPage));
      };
      const TreeTileOf<TREE> tt = tree_tile<TREE>(p, ri, t);
      uint4 raw[NL];
      float dk = 0.f, dv = 1.f;
      bool there = false;
      auto load = [&](int j, int2 pid) {
        const bool in_a = pid.x >= 0 && pid.x < p.num_pages, in_b = pid.y >= 0 && pid.y < p.num_pages;
        if (((pid.x != kNoPage && !in_a) || (pid.y != kNoPage && !in_b)) && lane == 0)
          set_device_error(err, MIXATTN_DEVERR_PAGE_ID);
        const int64_t at_a = (int64_t)(in_a ? pid.x : 0) * p.hkv + t.kvh, at_b = (int64_t)(in_b ? pid.y : 0) * p.hkv + t.kvh;
        const uint8_t* src_a = plane + at_a * (kPage * D);
        const uint8_t* src_b = plane + (at_b - 1) * (kPage * D);  // (the offset below passes the page's end)
        const int valid = key_end - j * kChunkN - key0;            // the lane's keys that exist
        if (in_a && (turn >= n_load || in_b) && (j + 1) * kChunkN <= key_end) {
#pragma unroll
          for (int i = 0; i < NL; ++i)
            if (i < n_load) raw[i] = ldg_u128((i < turn ? src_a : src_b) + i * (KPL * D));
        } else {
#pragma unroll
          for (int i = 0; i < NL; ++i)
            if (i < n_load)
              raw[i] = ldg_u128_pred((i < turn ? src_a : src_b) + i * (KPL * D), (i < turn ? in_a : in_b) && i * KPL < valid);
        }
        if (!is_v) {
          there = in_a;
          dk = ldg_f32_or(p.k_scale, at_a, in_a, 0.f);
          dv = ldg_f32_or(p.v_scale, at_a, in_a, 1.f);
        }
      };
      // The loads reach one tile ahead, less than HBM's latency; each K warp's page of the tiles up
      // to kAhead ahead and its V are on their way to L2 before (16 rows of 16 tokens at
      // 30000 keys 394 -> 363 us; a long chunk, whose tiles share their keys, is as fast without).
      constexpr int kAhead = 4;
      auto ahead_id = [&](int j) {
        const int pg = j * kPagesPerKvTile + w;
        return ldg_s32_or(pt_row + pg, !is_v && j < n_kv && pg * kPage < key_end, kNoPage);
      };
      auto to_l2 = [&](int pid) {
        if (pid < 0 || pid >= p.num_pages) return;
        const int64_t at = (int64_t)pid * p.hkv + t.kvh;
        if (D == 128 || lane < 16) prefetch_l2(p.k_quant + at * (kPage * D) + 128 * (lane % (D / 4)));
        if (D == 128 || lane >= 16) prefetch_l2(p.v_quant + at * (kPage * D) + 128 * (lane % (D / 4)));
      };
      load(0, pids_of(0));
      int2 next_pid = pids_of(1);
      int ahead = kNoPage;
      if (!is_v) {
        const int id = ahead_id(1 + lane % kAhead);
#pragma unroll 1
        for (int i = 0; i < kAhead - 1; ++i) to_l2(__shfl_sync(0xFFFFFFFFu, id, i));
        ahead = __shfl_sync(0xFFFFFFFFu, id, kAhead - 1);
      }
      for (int j = 0; j < n_kv; ++j, ++jg) {
        if (jg > 1) ok = warp_wait(&freed[jg & 1], (uint32_t)(((jg - 2) >> 1) & 1), err);  // tile jg - 2 has been read
        if (!ok) break;
        uint8_t* dst = smem + (is_v ? L::kV : L::kK) + (jg & 1) * L::kTile;
#pragma unroll
        for (int i = 0; i < NL; ++i) {
          if (i < n_load) {
            uint4 x, y;
            codes16_to_half<F>(raw[i], x, y);
            const uint32_t flip = (KPL == 4 && (i & 1)) ? 64u : 0u;
            *reinterpret_cast<uint4*>(dst + (off0 ^ flip) + i * (KPL * 128)) = x;
            *reinterpret_cast<uint4*>(dst + (off1 ^ flip) + i * (KPL * 128)) = y;
          }
        }
        if constexpr (TREE) {
          // values that no token of a tree's tile sees: zeros over what was written; pages of such keys alone count
          // as missing (they may have no scale)
          const int page0 = j * kChunkN + (r0 & ~(kPage - 1));
          if (tt.tree && page0 + 2 * kPage > tt.ctx) {
            const uint32_t some_a = tree_union(tt, page0, lane), some_b = tree_union(tt, page0 + kPage, lane);
            if (!is_v && some_a == 0u) {
              there = false;
              dv = 1.f;
            }
#pragma unroll 1
            for (int i = 0; is_v && i < n_load; ++i) {
              if (((i < turn ? some_a : some_b) >> ((key0 + i * KPL) & (kPage - 1))) & 1u) continue;
              const uint32_t flip = (KPL == 4 && (i & 1)) ? 64u : 0u;
              *reinterpret_cast<uint4*>(dst + (off0 ^ flip) + i * (KPL * 128)) = make_uint4(0u, 0u, 0u, 0u);
              *reinterpret_cast<uint4*>(dst + (off1 ^ flip) + i * (KPL * 128)) = make_uint4(0u, 0u, 0u, 0u);
            }
          }
        }
        if (!is_v && lane == 0)
          reinterpret_cast<float4*>(smem + L::kTerms)[4 * (jg & 3) + w] = page_terms(dk, dv, there, p.scale_log2);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ready[jg & 1]);
        if (j + 1 < n_kv) {
          load(j + 1, next_pid);
          next_pid = pids_of(j + 2);
          if (!is_v) {
            to_l2(ahead);
            ahead = ahead_id(j + 1 + kAhead);
          }
        }
      }
    }
  } else {
    // ======================= MMA (lane 0; the other lanes help to wait) =======================
    constexpr uint32_t kIdescQK = idesc_f16_f32(128, kChunkN, false, false);
    constexpr uint32_t kIdescPV = idesc_f16_f32(128, D, false, true);
    const uint64_t dQ = sw128_desc(smem_u32(smem + L::kQ), 16, 1024);
    const uint64_t dK = sw128_desc(smem_u32(smem + L::kK), 16, 1024);
    const uint64_t dV = sw128_desc(smem_u32(smem + L::kV), kChunkN * 128, 1024);
    const uint32_t dVlo = (uint32_t)dV, dVhi = (uint32_t)(dV >> 32);
    bool ok = true;
    // Lane l waits for one of: K, V, P'_0, P'_1, Q_0, Q_1 (l = 0 .. 5); `seen` counts what it has
    // waited for, which gives the barrier (K, V: two in turn) and its parity.  One poll takes
    // as long for one barrier as for all of them, and a poll is ~170 cycles beside the MMAs.
    const uint32_t my_bar = smem_u32(lane == 0 ? k_ready : (lane == 1 ? v_ready : (lane < 4 ? p_ready + (lane & 1) : q_ready + (lane & 1))));
    const bool in_turn = lane < 2;
    uint32_t seen = 0;
    auto wait = [&](uint32_t mask) {
      const bool need = (mask >> lane) & 1u;
      const uint32_t bar = my_bar + (in_turn ? (seen & 1u) * 8u : 0u), parity = (in_turn ? seen >> 1 : seen) & 1u;
      for (uint32_t i = 0; i < (1u << 21); ++i) {
        const bool done = !need || mbar_try_wait_s(bar, parity);
        if (__all_sync(0xFFFFFFFFu, done)) {
          seen += need;
          return true;
        }
      }
      if (need) set_device_error(err, MIXATTN_DEVERR_TIMEOUT);
      return false;
    };
    int jg0 = 0;
    for (int k = 0; ok && k < n_rounds; ++k) {
      const int idx = chunk_tile_of(cta, k, n_ctas, p.n_chunk_tiles);
      if (idx < 0) continue;
      const TileDesc t = p.tiles[idx];
      const int n_kv = t.kv1 - t.kv0;
      const bool two = t.count * G > 128;
      const int dj = two ? 1 : 2;
      // two: PV_0(j-1) QK_0(j) PV_1(j-1) QK_1(j) for each j; else PV_q(j-2) QK_q(j), q = j % 2
      int j = 0, q = 0;
      const int n_steps = two ? 2 * (n_kv + 1) : n_kv + 2;
#pragma unroll 1
      for (int step = 0; step < n_steps; ++step) {
        const bool has_k = j < n_kv, has_v = j >= dj && j - dj < n_kv;
        const bool last_q = !two || q == 1, first_q = !two || q == 0;
        const int jg = jg0 + j, jv = jg - dj;
        uint32_t mask = (has_v ? 4u : 0u) << q;
        if (has_k && j < dj) mask |= 16u << q;
        if (first_q) mask |= (has_k ? 1u : 0u) | (has_v ? 2u : 0u);
        ok = wait(mask);
        if (!ok) break;
        if (lane == 0) {
          tc_fence_after();
          const uint32_t s_tm = tmem + 128 * q, o_tm = s_tm + kOCol;
          if (has_v) {
            const uint32_t vb = dVlo + (uint32_t)(((jv & 1) * L::kTile) >> 4);
#pragma unroll
            for (int kk = 0; kk < 8; ++kk) {  // keys 16 kk ..: columns 32 (kk / 2) + 8 (kk % 2) of S
              const uint32_t boff = (uint32_t)(kk * 16 * 128) >> 4;
              if (kk == 0) tc_mma_ts_w(o_tm, s_tm, vb + boff, dVhi, kIdescPV, j >= 2 * dj ? 1u : 0u);
              else tc_mma_ts_w<1>(o_tm, s_tm + 32 * (kk >> 1) + 8 * (kk & 1), vb + boff, dVhi, kIdescPV);
            }
          }
          if (has_k) {
            const uint64_t qa = dQ + (uint64_t)((q * L::kTile) >> 4), kb = dK + (uint64_t)(((jg & 1) * L::kTile) >> 4);
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) {
              const uint64_t off = (uint64_t)(((ks >> 2) * (128 * 128) + (ks & 3) * 32) >> 4);
              tc_mma_ss(s_tm, qa + off, kb + off, kIdescQK, ks > 0 ? 1u : 0u);
            }
          }
          if (has_k) tc_commit(&qk_done[q]);
          else if (has_v) tc_commit(&o_done[q]);
          if (last_q) {
            if (has_v) tc_commit(&v_free[jv & 1]);
            if (has_k) tc_commit(&k_free[jg & 1]);
          }
        }
        __syncwarp();
        j += last_q;
        q ^= 1;
      }
      jg0 += n_kv;
    }
    // nothing this thread started may still run when TMEM is released
    if (lane == 0) {
      tc_commit(mma_fin);
      mbar_wait(mma_fin, 0u, err);
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

template <int F, int D, bool TREE>
__global__ void __launch_bounds__(kPageThreads, PageDecodeSmem<D>::kCtas) page_decode_kernel(AttnParams p, unsigned int* err) {
  extern __shared__ __align__(1024) uint8_t smem[];
  wait_for_upload();
  page_decode_tile<F, D, TREE>(p, p.tiles[blockIdx.x + p.n_chunk_tiles], smem, err, 0);
}

constexpr double kChunkShare = 1.15, kHalf = 2000.0;

// The fused launch: chunk CTAs, then decode CTAs of several tiles each.
template <int D>
struct PageFusedSmem {
  static constexpr int kTiles = kFusedThreads / kPageThreads;
  static constexpr int kPart = (PageDecodeSmem<D>::kTotal + 1023) / 1024 * 1024;
  static constexpr int kBytes = PageChunkSmem<D>::kTotal > kTiles * kPart ? PageChunkSmem<D>::kTotal : kTiles * kPart;
  static_assert(kBytes <= 227 * 1024, "fused CTA does not fit in shared memory");
};

template <int F, int D, bool TREE>
__global__ void __launch_bounds__(kFusedThreads, 1) page_mixed_kernel(AttnParams p, unsigned int* err) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const int cta = blockIdx.x;
  if (cta < p.n_chunk_ctas) {  // (waits for the upload when its barriers and TMEM are set up)
    page_chunk_cta<F, D, TREE>(p, cta, p.n_chunk_ctas, smem, err);
  } else {
    using FS = PageFusedSmem<D>;
    const int sub = threadIdx.x / kPageThreads;
    const int d = FS::kTiles * (cta - p.n_chunk_ctas) + sub;
    if (d >= p.n_decode_tiles) return;
    wait_for_upload();
    page_decode_tile<F, D, TREE>(p, p.tiles[p.n_chunk_tiles + d], smem + sub * FS::kPart, err, sub);
  }
}

template <int F, int D, bool TREE = false>
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
      e = cudaFuncSetAttribute(page_decode_kernel<F, D, TREE>, cudaFuncAttributeMaxDynamicSharedMemorySize, kDec);
      if (e == cudaSuccess)
        e = cudaFuncSetAttribute(page_mixed_kernel<F, D, TREE>, cudaFuncAttributeMaxDynamicSharedMemorySize, kFused);
      if (e != cudaSuccess) return e;
      configured[dev] = true;
    }
  }
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  cfg.stream = s;
  if (p.n_chunk_tiles == 0) {
    cfg.gridDim = dim3(p.n_decode_tiles);
    cfg.blockDim = dim3(kPageThreads);
    cfg.dynamicSmemBytes = kDec;
    return cudaLaunchKernelEx(&cfg, page_decode_kernel<F, D, TREE>, p, err);
  }
  AttnParams q = p;
  const bool persist = p.chunk_kv_tiles < kPersistMaxKvTiles * p.n_chunk_tiles;
  q.n_chunk_ctas = persist ? std::min(p.n_chunk_tiles, sm_count()) : p.n_chunk_tiles;
  if (persist && p.n_decode_tiles > 0 && sm_count() < (1 << 20)) {  // (1 << 30: the device does not say)
    // Chunk tiles are bound by the SM, decode tiles by HBM: side by side each takes about the
    // time it needs anyway.  The chunk CTAs get the share of the SMs that lets both kinds end
    // together, and a little more (decode CTAs take over the SMs that they leave, not the
    // other way round).  Costs in SM cycles: a KV tile of 128 rows 2000, a page of decode 230.
    // A cost of 1300 / 1600 / 2000 / 2650: the serving mix 151 / 146 / 144 / 149 us, the verify
    // batch 246 / 239 / 221 / 222 us; a share of 1.3 for 1.15: 146 and 222 us.  The same at
    // head_dim 64, where 1400 to 4000 differ by 2% (16 rows of 8192 tokens beside a 2048-token chunk
    // 155 to 157 us, 48 beside one without history 126 to 128) and 1000 loses up to 40%.
    const double tc = kHalf * p.chunk_kv_halves, td = 230.0 * p.decode_pages;
    const int share = (int)(kChunkShare * sm_count() * tc / (tc + td)) + 1;
    q.n_chunk_ctas = std::min(q.n_chunk_ctas, share);
  }
  constexpr int kTiles = PageFusedSmem<D>::kTiles;
  cfg.gridDim = dim3(q.n_chunk_ctas + (p.n_decode_tiles + kTiles - 1) / kTiles);
  cfg.blockDim = dim3(kFusedThreads);
  cfg.dynamicSmemBytes = kFused;
  return cudaLaunchKernelEx(&cfg, page_mixed_kernel<F, D, TREE>, q, err);
}

}  // namespace mixattn
