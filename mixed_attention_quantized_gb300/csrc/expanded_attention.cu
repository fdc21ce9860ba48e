// expanded_attention.cu -- expanded latent attention of prompts and chunks: per head queries of
// [128 | 64], keys of [128 | 64] whose last 64 all heads share, values of 128; causal.
//
// A tile is up to 256 queries of one head, in two groups of 128 rows that share each KV tile of 128
// keys; a group has an MMA warp and four softmax warps (a row a thread) of its own:
//   MMA      PV(j-1), then S(j), each as soon as P(j-1) and the KV tile are there
//   softmax  S(j) -> P(j) as the page-scaled chunk tiles do it (page_attention.cuh): one pass against a
//            reference that seldom moves, 32 keys at a time, P over the first half of its own scores
// While one group's softmax runs the other's MMAs do.  TMEM: S_0 | S_1 | O_0 | O_1, 128 columns each.
// Shared memory: Q of both groups (96 KB) and a ring of eight 16 KB slots of 128 keys x 64 elements,
// three to a K tile (the third the shared position keys) and two to a V tile, loaded by TMA.
//
// Values past a row's last key belong to the next row and may be anything: a warp of its own zeroes
// them in the slots of the row's last KV tile before their MMAs.
//
// 2048 tokens behind 8192, 32 heads: 283 us (1.40 PFLOP/s), 302 in a long run, at the power limit. A step of both groups has 2768 cycles of MMAs, and
// the tensor pipe is 67 % active: the rest is the softmax's chain, the items' starts and ends. One MMA warp for
// both groups, issuing from lane 0, took 569 us.
#include "latent.h"
#include "page_attention.cuh"
#include "tma.cuh"

namespace mixattn {

namespace {

constexpr int kExpandedThreads = 32 * 12;  // softmax 0-7, MMA 8 and 9, TMA 10, zeroing 11
constexpr int kSlots = 8;

struct ExpandedSmem {
  static constexpr int kQ = 0;                        // [group][3][128 rows][128 B]
  static constexpr int kGroupQ = 3 * 16384;
  static constexpr int kRing = 2 * kGroupQ;
  static constexpr int kBar = kRing + kSlots * 16384;
  static constexpr int kTotal = kBar + 256 + 1024;    // + slack for 1024-byte alignment
  static_assert(kTotal <= 227 * 1024, "the tile does not fit in shared memory");
};

// The ring's slots in order: K(0) K(0) K(0) V(0) V(0) K(1) ...; t counts the CTA's KV tiles.
// K(t) takes the slots of K(t - 2)'s last and of V(t - 2), V(t) those of K(t - 1)'s first two.
__device__ __forceinline__ int k_slot(int t, int s) { return (5 * t + s) % kSlots; }
__device__ __forceinline__ int v_slot(int t, int s) { return (5 * t + 3 + s) % kSlots; }

// KV tiles of an item that a group takes part in: those with a key that its last query sees.
__device__ __forceinline__ int group_steps(const ExpandedItem& it, int group) {
  const int rows = min(it.count - 128 * group, 128);
  if (rows <= 0) return 0;
  const int last = it.pos + 128 * group + rows - 1;
  return max(0, min(it.kv1, last / kChunkN + 1) - it.kv0);
}

// A row's weights are P = 2^(scale (S - r) - m); its reference (m = -inf: none yet) and their sum.  Up to kLargeScore
// r is 0.  Beyond, m alone would not do: of scale S near 2^28 no fp32 number is closer than 16, and the weights about
// such an m overflow fp16 or vanish.  Those rows take a score as r, so that S - r is exact to fp32 where a weight counts, and
// all their blocks the rare step: subtracting r from every row's scores, 283 -> 321 us for the case above.
struct ExpandedRef {
  float r, m, l;
  // what the common path adds to scale S: NaN, and with it the sum of the block, where a block needs the rare step
  __device__ __forceinline__ float shift() const {
    return m == -CUDART_INF_F || r != 0.f ? CUDART_NAN_F : -m;
  }
};
constexpr float kLargeScore = 4194304.f;

// page_move_reference for these rows, which see the scores up to c_last of block c's 32.  A change of more bits than
// P' have starts again.
__device__ __noinline__ ExpandedRef move_reference(uint32_t s_col, uint32_t o_col, int c, float scale, int c_last,
                                                   ExpandedRef ref, bool scale_o) {
  const uint32_t sc = s_col + 32 * c;
  float mx = -CUDART_INF_F;
#pragma unroll 1
  for (int b = 0; b < 2; ++b) {
    uint32_t o[16];
    tmem_ld16(sc + 16 * b, o);
    tmem_wait_ld();
#pragma unroll
    for (int e = 0; e < 16; ++e)
      if (16 * b + e <= c_last) mx = fmaxf(mx, __uint_as_float(o[e]));
  }
  const bool first = ref.m == -CUDART_INF_F;
  const float top = fmaf(mx - ref.r, scale, -ref.m);  // exponent of the largest weight
  const bool grow = mx > -CUDART_INF_F && (first || top >= kChunkMoved);
  float up = 0.f, alpha = 1.f;
  if (grow && (first || top - kChunkSet > 40.f)) {
    up = first ? 0.f : top - kChunkSet;
    alpha = first ? 0.f : ex2(-up);
    const bool large = fabsf(mx * scale) >= kLargeScore;
    ref.r = large ? mx : 0.f;
    ref.m = large ? -kChunkSet : fmaf(mx, scale, -kChunkSet);
  } else if (grow) {
    up = floorf(top - kChunkSet);
    alpha = ex2(-up);  // a power of two
    ref.m += up;
    if (ref.r == 0.f && fabsf(ref.m) >= kLargeScore) {
      ref.m = fmaf(-mx, scale, ref.m);  // (the same reference: rounded once, at its small difference)
      ref.r = mx;
    }
  }
  ref.l *= alpha;
  if (scale_o) scale_output<kExpandedV>(o_col, alpha);
  scale_weights(s_col, c, up);
  // the block's P', 16 scores at a time: their 8 words stay before the scores not yet read
  const float cb = ref.m == -CUDART_INF_F ? 0.f : -ref.m;
  const uint64_t nr2 = f2_pack(-ref.r, -ref.r), scale2 = f2_pack(scale, scale), cb2 = f2_pack(cb, cb);
#pragma unroll 1
  for (int b = 0; b < 2; ++b) {
    uint32_t o[16], w[8];
    tmem_ld16(sc + 16 * b, o);
    tmem_wait_ld();
#pragma unroll
    for (int e = 0; e < 16; e += 2) {
      float p0, p1;
      f2_unpack(ffma2(fadd2(f2_pack(__uint_as_float(o[e]), __uint_as_float(o[e + 1])), nr2), scale2, cb2), p0, p1);
      p0 = 16 * b + e <= c_last ? ex2(p0) : 0.f;
      p1 = 16 * b + e + 1 <= c_last ? ex2(p1) : 0.f;
      ref.l += p0 + p1;
      w[e >> 1] = pack_f16x2(p0, p1);
    }
    tmem_st8(sc + 8 * b, w);
  }
  return ref;
}

// Four 16-byte pieces a lane: piece e of lane q and piece q of lane e of each four lanes change places.
__device__ __forceinline__ void transpose_pieces(uint32_t (&w)[16], int lane) {
#pragma unroll
  for (int s = 1; s <= 2; s <<= 1) {
    const bool up = (lane & s) != 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i & s) continue;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        uint32_t &a = w[4 * i + e], &b = w[4 * (i ^ s) + e];
        const uint32_t got = __shfl_xor_sync(0xFFFFFFFFu, up ? a : b, s);
        if (up) a = got;
        else b = got;
      }
    }
  }
}

// A warp's 32 rows of O from TMEM.  Four lanes write 64 bytes of a row together, of four rows (`rows` of which
// exist) in turn: a row a lane is 32 lines an instruction.  Out of line, or the softmax loop's code suffers: 2048
// queries behind 8192, 32 heads, 322 us with a row a lane, 330 with this in line, 311 as it is.
__device__ __noinline__ void write_out(uint32_t o_col, uint16_t* dst, int stride, float inv_l, int rows, int lane) {
  dst += 8 * (lane & 3);
#pragma unroll 1
  for (int ch = 0; ch < kExpandedV / 32; ++ch) {
    uint32_t v[32], w[16];
    tmem_ld32(o_col + 32 * ch, v);
    tmem_wait_ld();
#pragma unroll
    for (int e = 0; e < 16; ++e)
      w[e] = pack_f16x2_out(__uint_as_float(v[2 * e]) * inv_l, __uint_as_float(v[2 * e + 1]) * inv_l);
    transpose_pieces(w, lane);
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (e < rows)
        *reinterpret_cast<uint4*>(dst + (int64_t)e * stride + 32 * ch) = make_uint4(w[4 * e], w[4 * e + 1], w[4 * e + 2], w[4 * e + 3]);
  }
}

__device__ __noinline__ void write_part(uint32_t o_col, float* dst, int rows, int lane) {
  dst += 4 * (lane & 3);
#pragma unroll 1
  for (int ch = 0; ch < kExpandedV / 16; ++ch) {
    uint32_t v[16];
    tmem_ld16(o_col + 16 * ch, v);
    tmem_wait_ld();
    transpose_pieces(v, lane);
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (e < rows)
        *reinterpret_cast<uint4*>(dst + e * kExpandedV + 16 * ch) = make_uint4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
  }
}

__global__ void __launch_bounds__(kExpandedThreads, 1)
    expanded_kernel(const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap k_map,
                    const __grid_constant__ CUtensorMap kr_map, const __grid_constant__ CUtensorMap v_map,
                    const __grid_constant__ ExpandedParams p, unsigned int* err) {
  using L = ExpandedSmem;
  constexpr uint32_t kTmemCols = 512, kOCol = 256;
  constexpr int kD = kExpandedV;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kBar);
  uint64_t* k_full = bars;               // [2] K(t) in t % 2, by TMA
  uint64_t* v_full = bars + 2;           // [2] V(t), by TMA or (a row's last) by the zeroing warp
  uint64_t* k_empty = bars + 4;          // [2] by both MMA warps: K(t) read
  uint64_t* v_empty = bars + 6;          // [2] by both MMA warps: V(t) read
  uint64_t* tail = bars + 8;             // a row's last V tile loaded
  uint64_t* q_full = bars + 9;
  uint64_t* q_empty = bars + 10;         // by both MMA warps: the item's last S done
  uint64_t* s_full = bars + 11;          // [2] a group's S done (and its PV before)
  uint64_t* p_full = bars + 13;          // [2] by 4 warps: P written, O rescaled
  uint64_t* o_full = bars + 15;          // [2] a group's last PV of the item done
  uint64_t* o_free = bars + 17;          // [2] by 4 warps: O read
  uint64_t* fin = bars + 19;             // [2]
  constexpr int kNumBars = 21;
  static_assert(8 * kNumBars + 8 <= 256, "barrier area");
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + kNumBars);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < kNumBars; ++i) mbar_init(bars + i, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(k_empty + i, 2);
      mbar_init(v_empty + i, 2);
      mbar_init(p_full + i, 4);
      mbar_init(o_free + i, 4);
    }
    mbar_init(q_empty, 2);
    fence_mbar_init();
    tma_prefetch_map(&q_map);
    tma_prefetch_map(&k_map);
    tma_prefetch_map(&kr_map);
    tma_prefetch_map(&v_map);
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
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const ExpandedItem* items = p.list.at<ExpandedItem>(p.items);
  const int32_t* cta_first = p.list.at<int32_t>(p.cta_first);
  const int it0 = cta_first[blockIdx.x], it1 = cta_first[blockIdx.x + 1];

  if (warp < 8) {
    // ======================= softmax groups =======================
    const int gq = warp >> 2, row = tid & 127;
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t s_col = tmem + lane_base + 128 * gq, o_col = tmem + lane_base + kOCol + 128 * gq;
    const uint64_t ca2 = f2_pack(p.scale_log2, p.scale_log2);
    bool ok = true;
    uint32_t n_s = 0, n_o = 0;  // S tiles, outputs so far (barrier phases)
    for (int i = it0; ok && i < it1; ++i) {
      const ExpandedItem it = items[i];
      const int n = group_steps(it, gq);
      const int prow = 128 * gq + row;
      const int64_t part = (int64_t)it.slot + it.part;
      if (n == 0) {  // (a part past the group's last key, or a tile without the group)
        if (it.n_parts > 1) p.part_ml[part * kExpandedRows + prow] = make_float4(0.f, -CUDART_INF_F, 0.f, 0.f);
        continue;
      }
      const int pos = it.pos + min(prow, it.count - 1);
      ExpandedRef ref{0.f, -CUDART_INF_F, 0.f};
      for (int j = 0; j < n; ++j) {
        ok = warp_wait_fast(&s_full[gq], n_s & 1, err);
        if (!ok) break;
        ++n_s;
        tc_fence_after();
        const int last = pos - (it.kv0 + j) * kChunkN;  // the last visible key of the row in this tile
        const bool diag = __any_sync(0xFFFFFFFFu, last < kChunkN - 1);
#pragma unroll 2  // (not unrolled 295 us for the case above, wholly 291, two of 32 scores loaded as halves 331)
        for (int c = 0; c < 4; ++c) {
          const int c_last = last - 32 * c;
          const uint32_t sc = s_col + 32 * c;
          uint32_t x[32], pk[16];
          tmem_ld32(sc, x);
          const float cb = ref.shift();  // (kept from block to block 305 us for 301, in a long run of the case above)
          const uint64_t cb2 = f2_pack(cb, cb);
          tmem_wait_ld();
          if (diag) {
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (e > c_last) x[e] = __float_as_uint(-CUDART_INF_F);
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
          const float l_new = s0 + s1;
          if (!__any_sync(0xFFFFFFFFu, !(l_new < kChunkTop))) {
            tmem_st16(sc, pk);
            ref.l += l_new;
            continue;
          }
          ref = move_reference(s_col, o_col, c, p.scale_log2, c_last, ref, j > 0);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[gq]);
      }
      if (!ok) break;
      ok = warp_wait_fast(&o_full[gq], n_o & 1, err);
      ++n_o;
      if (!ok) break;
      tc_fence_after();
      const bool whole = it.n_parts == 1;
      const float inv_l = ref.l > 0.f ? 1.f / ref.l : 0.f;
      const int row0 = prow & ~3;
      if (whole)
        write_out(o_col, p.o + ((int64_t)(it.q_start + row0) * p.heads + it.head) * kD, p.heads * kD, inv_l, it.count - row0, lane);
      else
        write_part(o_col, p.part_o + (part * kExpandedRows + row0) * kD, it.count - row0, lane);
      if (!whole) p.part_ml[part * kExpandedRows + prow] = make_float4(ref.r, ref.m, ref.l, 0.f);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&o_free[gq]);
    }
  } else if (warp == 10) {
    // ======================= TMA (its elected lane) =======================
    int t = 0, n_item = 0, last_tail = -2;  // KV tiles and items so far; the last tail's KV tile
    bool ok = true;
    const uint32_t ring = smem_u32(smem + L::kRing);
    for (int i = it0; ok && i < it1; ++i) {
      const ExpandedItem it = items[i];
      const int n = max(group_steps(it, 0), group_steps(it, 1));
      if (n == 0) continue;
      if (n_item > 0) ok = warp_wait_fast(q_empty, (uint32_t)((n_item - 1) & 1), err);
      if (!ok) break;
      ++n_item;
      const int groups = it.count > 128 ? 2 : 1;
      if (elect_one()) {
        mbar_arrive_expect_tx(q_full, groups * L::kGroupQ);
        for (int g = 0; g < groups; ++g)
          for (int s = 0; s < 3; ++s)
            tma_load_3d(smem_u32(smem + L::kQ) + g * L::kGroupQ + s * 16384, &q_map, 64 * s, it.head, it.q_start + 128 * g,
                        smem_u32(q_full));
      }
      __syncwarp();
      for (int j = 0; j < n; ++j, ++t) {
        const int key = (it.kv0 + j) * kChunkN, y = it.k_start + key;
        if (t >= 2) ok = warp_wait_fast(&v_empty[t & 1], (uint32_t)(((t >> 1) - 1) & 1), err);
        if (!ok) break;
        if (elect_one()) {
          const uint32_t bar = smem_u32(&k_full[t & 1]);
          mbar_arrive_expect_tx(&k_full[t & 1], 3 * 16384);
          tma_load_3d(ring + k_slot(t, 0) * 16384, &k_map, 0, it.head, y, bar);
          tma_load_3d(ring + k_slot(t, 1) * 16384, &k_map, 64, it.head, y, bar);
          tma_load_2d(ring + k_slot(t, 2) * 16384, &kr_map, 0, y, bar);
        }
        __syncwarp();
        const bool is_tail = key + kChunkN > it.seq_len;
        if (t >= 1) ok = warp_wait_fast(&k_empty[(t - 1) & 1], (uint32_t)(((t - 1) >> 1) & 1), err);
        // (one tail at a time on its barrier; an earlier one than the last V tile has been read)
        if (ok && is_tail && last_tail == t - 1 && t > 0)
          ok = warp_wait_fast(&v_full[(t - 1) & 1], (uint32_t)(((t - 1) >> 1) & 1), err);
        if (!ok) {
          ++t;
          break;
        }
        if (elect_one()) {
          uint64_t* b = is_tail ? tail : &v_full[t & 1];
          mbar_arrive_expect_tx(b, 2 * 16384);
          tma_load_3d(ring + v_slot(t, 0) * 16384, &v_map, 0, it.head, y, smem_u32(b));
          tma_load_3d(ring + v_slot(t, 1) * 16384, &v_map, 64, it.head, y, smem_u32(b));
        }
        __syncwarp();
        if (is_tail) last_tail = t;
      }
    }
    // nothing asked for may still be on its way when the CTA ends (which, but for an error, it is not)
    for (int k = max(0, t - 2); k < t; ++k) {
      warp_wait_fast(&k_full[k & 1], (uint32_t)((k >> 1) & 1), err);
      if (ok || k < t - 1) warp_wait_fast(&v_full[k & 1], (uint32_t)((k >> 1) & 1), err);
    }
    if (n_item > 0) warp_wait_fast(q_full, (uint32_t)((n_item - 1) & 1), err);
  } else if (warp == 11) {
    // ======================= zeroing of a row's last V tile =======================
    bool ok = true;
    int t = 0;  // KV tiles before the item
    uint32_t n_tail = 0;
    for (int i = it0; ok && i < it1; ++i) {
      const ExpandedItem it = items[i];
      const int n = max(group_steps(it, 0), group_steps(it, 1));
      t += n;
      if (n > 0 && (it.kv0 + n) * kChunkN > it.seq_len) {
        const int valid = it.seq_len - (it.kv0 + n - 1) * kChunkN;  // keys of the tile that are the row's
        ok = warp_wait_fast(tail, n_tail & 1, err);
        if (!ok) break;
        ++n_tail;
        for (int s = 0; s < 2; ++s) {
          uint4* rows = reinterpret_cast<uint4*>(smem + L::kRing + v_slot(t - 1, s) * 16384);
          for (int k = 8 * valid + lane; k < 8 * kChunkN; k += 32) rows[k] = make_uint4(0u, 0u, 0u, 0u);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&v_full[(t - 1) & 1]);
      }
    }
  } else {
    // ======================= MMA (the elected lane of each group's warp) =======================
    constexpr uint32_t kIdescS = idesc_f16_f32(128, kChunkN, false, false);
    constexpr uint32_t kIdescO = idesc_f16_f32(128, 64, false, true);
    const int g = warp - 8;
    auto lo = [](uint64_t d) { return (uint32_t)d; };
    const uint32_t dQ = lo(sw128_desc(smem_u32(smem + L::kQ), 16, 1024)) + g * (L::kGroupQ >> 4);
    const uint32_t dK = lo(sw128_desc(smem_u32(smem + L::kRing), 16, 1024));
    const uint32_t dV = lo(sw128_desc(smem_u32(smem + L::kRing), 16384, 1024));  // (N = 64: one slab)
    constexpr uint32_t kHi = (1024u >> 4) | (1u << 14) | (2u << 29);              // the upper word of them all
    const uint32_t s_tm = tmem + 128 * g, o_tm = s_tm + kOCol;
    bool ok = true;
    int t = 0;
    uint32_t n_item = 0, n_p = 0, n_out = 0;
    const int first = __shfl_sync(0xFFFFFFFFu, it0, 0), end = __shfl_sync(0xFFFFFFFFu, it1, 0);
    for (int i = first; ok && i < end; ++i) {
      const ExpandedItem it = items[i];
      // (control flow and operands the same in all lanes, and known to be)
      const int mine = __shfl_sync(0xFFFFFFFFu, group_steps(it, g), 0);
      const int n = max(mine, __shfl_sync(0xFFFFFFFFu, group_steps(it, g ^ 1), 0));
      if (n == 0) continue;
      ok = warp_wait_fast(q_full, n_item & 1, err);
      for (int j = 0; ok && j <= n; ++j) {
        const int tv = t + j - 1, tk = t + j;
        if (j > 0) {
          ok = warp_wait_fast(&v_full[tv & 1], (uint32_t)((tv >> 1) & 1), err);
          if (ok && j <= mine) {
            ok = warp_wait_fast(&p_full[g], n_p & 1, err);
            ++n_p;
            if (ok && j == 1 && n_out > 0) ok = warp_wait_fast(&o_free[g], (n_out - 1) & 1, err);
            if (!ok) break;
            tc_fence_after();
            // (a V tile's two slabs need not be neighbours in the ring: MMAs of N = 64)
            if (elect_one()) {
              const uint32_t acc = j > 1 ? 1u : 0u;
#pragma unroll
              for (int s = 0; s < 2; ++s) {
                const uint32_t vd = dV + v_slot(tv, s) * (16384 >> 4);
#pragma unroll
                for (int k = 0; k < 8; ++k)  // keys 16 k ..: columns 32 (k / 2) + 8 (k % 2) of S
                  tc_mma_ts_w(o_tm + 64 * s, s_tm + 32 * (k >> 1) + 8 * (k & 1), vd + ((k * 16 * 128) >> 4), kHi, kIdescO,
                              k > 0 ? 1u : acc);
              }
              tc_commit(&v_empty[tv & 1]);
              if (j == mine) tc_commit(&o_full[g]);
            }
            __syncwarp();
            n_out += j == mine;
          } else if (ok && elect_one()) {
            mbar_arrive(&v_empty[tv & 1]);
          }
          __syncwarp();
          if (!ok) break;
        }
        if (j < n) {
          ok = warp_wait_fast(&k_full[tk & 1], (uint32_t)((tk >> 1) & 1), err);
          if (!ok) break;
          if (elect_one()) {
            if (j < mine) {
              tc_fence_after();
#pragma unroll
              for (int s = 0; s < 3; ++s) {
                const uint32_t kd = dK + k_slot(tk, s) * (16384 >> 4);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                  tc_mma_ss_w(s_tm, dQ + ((s * 16384 + 32 * k) >> 4), kHi, kd + ((32 * k) >> 4), kHi, kIdescS,
                              s + k > 0 ? 1u : 0u);
              }
              tc_commit(&s_full[g]);
              tc_commit(&k_empty[tk & 1]);
              if (j == n - 1) tc_commit(q_empty);
            } else {
              mbar_arrive(&k_empty[tk & 1]);
              if (j == n - 1) tc_commit(q_empty);  // (behind the group's last S)
            }
          }
          __syncwarp();
        }
      }
      t += n;
      ++n_item;
    }
    // nothing the lane started may still run when TMEM is released
    if (elect_one()) {
      tc_commit(fin + g);
      mbar_wait(fin + g, 0u, err);
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

// Joins the parts of cut tiles: a warp takes four queries, four elements a lane; the loads of a part
// wait for nothing but the cut.
constexpr int kJoinRows = 16;  // queries of a CTA

__global__ void __launch_bounds__(128) expanded_join_kernel(const __grid_constant__ ExpandedParams p) {
  wait_for_upload();
  constexpr int kPer = kExpandedRows / kJoinRows;
  const ExpandedCut cut = p.list.at<ExpandedCut>(p.cuts)[blockIdx.x / kPer];
  const int row = kJoinRows * (blockIdx.x % kPer) + 4 * (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (row >= cut.count) return;
  const float4* ml = p.part_ml + (int64_t)cut.slot * kExpandedRows + row;
  const float* src = p.part_o + ((int64_t)cut.slot * kExpandedRows + row) * kExpandedV + 4 * lane;
  float r[4], m[4], l[4];
  float4 o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    r[i] = 0.f;
    m[i] = -CUDART_INF_F;
    l[i] = 0.f;
    o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
#pragma unroll 2
  for (int q = 0; q < cut.n_parts; ++q) {
    float4 x[4], y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {  // (rows past the tile's are within the slot: any value may stand there)
      x[i] = ml[(int64_t)q * kExpandedRows + i];
      y[i] = __ldcs(reinterpret_cast<const float4*>(src + ((int64_t)q * kExpandedRows + i) * kExpandedV));
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (x[i].y == -CUDART_INF_F) {  // no key of the row in this part, a sum of 0: the same; or scores that are all NaN
        l[i] += x[i].z;
        continue;
      }
      // the part's reference above the one so far, in bits: the larger is kept (2^-inf: 0).  (An m beside an r of 0
      // may be large: it belongs into the product's rounding.)
      const float dr = x[i].x - r[i];
      const float d = m[i] == -CUDART_INF_F ? CUDART_INF_F
                      : r[i] == 0.f         ? fmaf(dr, p.scale_log2, -m[i]) + x[i].y
                                            : fmaf(dr, p.scale_log2, x[i].y) - m[i];
      const float a = ex2(fminf(-d, 0.f)), w = ex2(fminf(d, 0.f));
      if (d > 0.f) {
        r[i] = x[i].x;
        m[i] = x[i].y;
      }
      l[i] = l[i] * a + w * x[i].z;
      o[i].x = o[i].x * a + w * y[i].x;
      o[i].y = o[i].y * a + w * y[i].y;
      o[i].z = o[i].z * a + w * y[i].z;
      o[i].w = o[i].w * a + w * y[i].w;
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (row + i >= cut.count) break;
    const float inv = l[i] > 0.f ? 1.f / l[i] : l[i];
    *reinterpret_cast<uint2*>(p.o + ((int64_t)(cut.q_start + row + i) * p.heads + cut.head) * kExpandedV + 4 * lane) =
        make_uint2(pack_f16x2_out(o[i].x * inv, o[i].y * inv), pack_f16x2_out(o[i].z * inv, o[i].w * inv));
  }
}

}  // namespace

cudaError_t launch_expanded_attention(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& kr,
                                      const CUtensorMap& v, const ExpandedParams& p, unsigned int* err, cudaStream_t s) {
  {
    static std::mutex mu;
    static bool configured[kMaxDevices] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    std::lock_guard<std::mutex> lock(mu);
    if (!configured[dev]) {
      e = cudaFuncSetAttribute(expanded_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, ExpandedSmem::kTotal);
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
  cfg.gridDim = dim3(p.n_ctas);
  cfg.blockDim = dim3(kExpandedThreads);
  cfg.dynamicSmemBytes = ExpandedSmem::kTotal;
  cudaError_t e = cudaLaunchKernelEx(&cfg, expanded_kernel, q, k, kr, v, p, err);
  if (e != cudaSuccess || p.n_cuts == 0) return e;
  cfg.gridDim = dim3(p.n_cuts * (kExpandedRows / kJoinRows));
  cfg.blockDim = dim3(128);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, expanded_join_kernel, p);
}

}  // namespace mixattn
