// expanded_attention.cu -- expanded latent attention of prompts and chunks: per head queries of
// [128 | 64], keys of [128 | 64] whose last 64 all heads share, values of 128; causal.
//
// A tile is up to 256 queries of one head, in two groups of 128 rows that share each KV tile of 128
// keys. One MMA thread issues PV_0(j-1) QK_0(j) PV_1(j-1) QK_1(j), and while one group's MMAs run
// the other's softmax does: as the page-scaled chunk tiles (page_attention.cuh), whose softmax
// against a reference that seldom moves this shares, with TMA in place of the conversion warps.
// TMEM: S_0 | S_1 | O_0 | O_1, 128 columns each, P of 32 keys over the first half of their scores.
// Shared memory: Q of both groups (96 KB) and a ring of eight 16 KB slots of 128 keys x 64 elements,
// three to a K tile (the third the shared position keys) and two to a V tile.
//
// Values past a row's last key belong to the next row and may be anything: a warp of its own zeroes
// them in the slots of the row's last KV tile before their MMAs.
#include "latent.h"
#include "page_attention.cuh"
#include "tma.cuh"

namespace mixattn {

namespace {

constexpr int kExpandedThreads = 32 * 11;  // softmax 0-7, TMA 8, MMA 9, zeroing 10
constexpr int kSlots = 8;

struct ExpandedSmem {
  static constexpr int kQ = 0;                        // [group][3][128 rows][128 B]
  static constexpr int kGroupQ = 3 * 16384;
  static constexpr int kRing = 2 * kGroupQ;
  static constexpr int kBar = kRing + kSlots * 16384;
  static constexpr int kTotal = kBar + 256 + 1024;    // + slack for 1024-byte alignment
  static_assert(kTotal <= 227 * 1024, "the tile does not fit in shared memory");
};

// KV tiles of an item that a group takes part in: those with a key that its last query sees.
__device__ __forceinline__ int group_steps(const ExpandedItem& it, int group) {
  const int rows = min(it.count - 128 * group, 128);
  if (rows <= 0) return 0;
  const int last = it.pos + 128 * group + rows - 1;
  return max(0, min(it.kv1, last / kChunkN + 1) - it.kv0);
}

__global__ void __launch_bounds__(kExpandedThreads, 1)
    expanded_kernel(const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap k_map,
                    const __grid_constant__ CUtensorMap kr_map, const __grid_constant__ CUtensorMap v_map,
                    const ExpandedParams p, unsigned int* err) {
  using L = ExpandedSmem;
  constexpr uint32_t kTmemCols = 512, kOCol = 256;
  constexpr int kD = kExpandedV;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kBar);
  uint64_t* full = bars;                 // [8] slot loaded (a row's last V tile: and zeroed)
  uint64_t* empty = full + kSlots;       // [8] slot read, by a commit
  uint64_t* tail = empty + kSlots;       // [2] slots of a row's last V tile loaded
  uint64_t* q_full = tail + 2;
  uint64_t* q_empty = q_full + 1;        // the item's last S done
  uint64_t* s_full = q_empty + 1;        // [2] a group's S done (and its PV before)
  uint64_t* p_full = s_full + 2;         // [2] by 4 warps: P written, O rescaled
  uint64_t* o_full = p_full + 2;         // [2] a group's last PV of the item done
  uint64_t* o_free = o_full + 2;         // [2] by 4 warps: O read
  uint64_t* fin = o_free + 2;
  constexpr int kNumBars = 2 * kSlots + 2 + 2 + 8 + 1;
  static_assert(8 * kNumBars + 8 <= 256, "barrier area");
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + kNumBars);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < kNumBars; ++i) mbar_init(bars + i, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(p_full + i, 4);
      mbar_init(o_free + i, 4);
    }
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
  const int it0 = p.cta_first[blockIdx.x], it1 = p.cta_first[blockIdx.x + 1];

  if (warp < 8) {
    // ======================= softmax groups =======================
    const int gq = warp >> 2, row = tid & 127;
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t s_col = tmem + lane_base + 128 * gq, o_col = tmem + lane_base + kOCol + 128 * gq;
    const float4 tm = make_float4(p.scale_log2, 0.f, 1.f, 0.f);
    const uint64_t ca2 = f2_pack(tm.x, tm.x);
    bool ok = true;
    uint32_t n_s = 0, n_o = 0;  // S tiles, outputs so far (barrier phases)
    for (int i = it0; ok && i < it1; ++i) {
      const ExpandedItem it = p.items[i];
      const int n = group_steps(it, gq);
      const int prow = 128 * gq + row;
      const bool valid = prow < it.count;
      const int64_t part = (int64_t)it.slot + it.part;
      if (n == 0) {  // (a part past the group's last key, or a tile without the group)
        if (it.n_parts > 1) p.part_ml[part * kExpandedRows + prow] = make_float2(-CUDART_INF_F, 0.f);
        continue;
      }
      const int pos = it.pos + min(prow, it.count - 1);
      float m_run = -CUDART_INF_F, l_run = 0.f;
      for (int j = 0; j < n; ++j) {
        ok = warp_wait(&s_full[gq], n_s & 1, err);
        if (!ok) break;
        ++n_s;
        tc_fence_after();
        const int last = pos - (it.kv0 + j) * kChunkN;  // the last visible key of the row in this tile
        const bool diag = __any_sync(0xFFFFFFFFu, last < kChunkN - 1);
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          const int c_last = last - 32 * c;
          const uint32_t sc = s_col + 32 * c;
          uint32_t x[32], pk[16];
          tmem_ld32(sc, x);
          const float cb = m_run == -CUDART_INF_F ? 0.f : -m_run;
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
          const bool over = !(l_new < kChunkTop) || m_run == -CUDART_INF_F;
          if (!__any_sync(0xFFFFFFFFu, over)) {
            tmem_st16(sc, pk);
            l_run += l_new;
            continue;
          }
          const float2 ml = page_move_reference<kD, false>(s_col, o_col, c, tm, 0, c_last, m_run, l_run, j > 0);
          m_run = ml.x;
          l_run = ml.y;
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[gq]);
      }
      if (!ok) break;
      ok = warp_wait(&o_full[gq], n_o & 1, err);
      ++n_o;
      if (!ok) break;
      tc_fence_after();
      const bool whole = it.n_parts == 1;
      const float inv_l = l_run > 0.f ? 1.f / l_run : 0.f;
      uint16_t* dst = p.o + ((int64_t)(it.q_start + prow) * p.heads + it.head) * kD;
      float* o_part = p.part_o + (part * kExpandedRows + prow) * kD;
#pragma unroll 1
      for (int ch = 0; ch < kD / 16; ++ch) {
        uint32_t v[16];
        tmem_ld16(o_col + 16 * ch, v);
        tmem_wait_ld();
        if (!valid) continue;
        if (whole) {
          uint32_t w[8];
#pragma unroll
          for (int e = 0; e < 8; ++e)
            w[e] = pack_f16x2_out(__uint_as_float(v[2 * e]) * inv_l, __uint_as_float(v[2 * e + 1]) * inv_l);
          reinterpret_cast<uint4*>(dst + 16 * ch)[0] = make_uint4(w[0], w[1], w[2], w[3]);
          reinterpret_cast<uint4*>(dst + 16 * ch)[1] = make_uint4(w[4], w[5], w[6], w[7]);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            reinterpret_cast<uint4*>(o_part + 16 * ch)[e] = make_uint4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
        }
      }
      if (!whole) p.part_ml[part * kExpandedRows + prow] = make_float2(m_run, l_run);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&o_free[gq]);
    }
  } else if (warp == 8) {
    // ======================= TMA (one thread) =======================
    if (lane == 0) {
      int slot = 0, round = 0, n_item = 0;
      int tail_slot = -1, tail_round = 0;  // the last tail's second slot
      bool ok = true;
      auto take = [&] {  // the next slot, free
        if (round > 0) ok = mbar_wait(&empty[slot], (uint32_t)((round - 1) & 1), err);
        return ok;
      };
      auto next = [&] {
        if (++slot == kSlots) {
          slot = 0;
          ++round;
        }
      };
      for (int i = it0; ok && i < it1; ++i) {
        const ExpandedItem it = p.items[i];
        const int n = max(group_steps(it, 0), group_steps(it, 1));
        if (n == 0) continue;
        if (n_item > 0) ok = mbar_wait(q_empty, (uint32_t)((n_item - 1) & 1), err);
        if (!ok) break;
        ++n_item;
        const int groups = it.count > 128 ? 2 : 1;
        mbar_arrive_expect_tx(q_full, groups * L::kGroupQ);
        for (int g = 0; g < groups; ++g)
          for (int s = 0; s < 3; ++s)
            tma_load_3d(smem_u32(smem + L::kQ + g * L::kGroupQ + s * 16384), &q_map, 64 * s, it.head,
                        it.q_start + 128 * g, smem_u32(q_full));
        for (int j = 0; ok && j < n; ++j) {
          const int key = (it.kv0 + j) * kChunkN, y = it.k_start + key;
          for (int s = 0; s < 3; ++s) {
            if (!take()) break;
            const uint32_t dst = smem_u32(smem + L::kRing + slot * 16384), bar = smem_u32(&full[slot]);
            mbar_arrive_expect_tx(&full[slot], 16384);
            if (s < 2) tma_load_3d(dst, &k_map, 64 * s, it.head, y, bar);
            else tma_load_2d(dst, &kr_map, 0, y, bar);
            next();
          }
          const bool is_tail = key + kChunkN > it.seq_len;
          // (one tail at a time on its barriers)
          if (is_tail && tail_slot >= 0) ok = ok && mbar_wait(&full[tail_slot], (uint32_t)(tail_round & 1), err);
          for (int s = 0; ok && s < 2; ++s) {
            if (!take()) break;
            if (is_tail) {
              tail_slot = slot;
              tail_round = round;
            }
            uint64_t* b = is_tail ? &tail[s] : &full[slot];
            mbar_arrive_expect_tx(b, 16384);
            tma_load_3d(smem_u32(smem + L::kRing + slot * 16384), &v_map, 64 * s, it.head, y, smem_u32(b));
            next();
          }
        }
      }
      // nothing asked for may still be on its way when the CTA ends (which, but for an error, it is not)
      for (int k = 0; k < kSlots; ++k) {
        const int rd = k < slot ? round : round - 1;
        if (rd >= 0) mbar_wait(&full[k], (uint32_t)(rd & 1), err);
      }
      if (n_item > 0) mbar_wait(q_full, (uint32_t)((n_item - 1) & 1), err);
    }
    __syncwarp();
  } else if (warp == 10) {
    // ======================= zeroing of a row's last V tile =======================
    bool ok = true;
    int slot = 0;  // slots before the item
    uint32_t n_tail = 0;
    for (int i = it0; ok && i < it1; ++i) {
      const ExpandedItem it = p.items[i];
      const int n = max(group_steps(it, 0), group_steps(it, 1));
      if (n > 0 && (it.kv0 + n) * kChunkN > it.seq_len) {
        const int valid = it.seq_len - (it.kv0 + n - 1) * kChunkN;  // keys of the tile that are the row's
        for (int s = 0; ok && s < 2; ++s) {
          ok = warp_wait(&tail[s], n_tail & 1, err);
          if (!ok) break;
          const int at = (slot + 5 * (n - 1) + 3 + s) % kSlots;
          uint4* rows = reinterpret_cast<uint4*>(smem + L::kRing + at * 16384);
          for (int k = 8 * valid + lane; k < 8 * kChunkN; k += 32) rows[k] = make_uint4(0u, 0u, 0u, 0u);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&full[at]);
        }
        ++n_tail;
      }
      slot = (slot + 5 * n) % kSlots;
    }
  } else if (lane == 0) {
    // ======================= MMA (one thread) =======================
    constexpr uint32_t kIdescS = idesc_f16_f32(128, kChunkN, false, false);
    constexpr uint32_t kIdescO = idesc_f16_f32(128, 64, false, true);
    const uint64_t dQ = sw128_desc(smem_u32(smem + L::kQ), 16, 1024);
    const uint64_t dK = sw128_desc(smem_u32(smem + L::kRing), 16, 1024);
    const uint64_t dV = sw128_desc(smem_u32(smem + L::kRing), 16384, 1024);  // (N = 64: one slab)
    bool ok = true;
    int base = 0;             // slots before the item, over all the CTA's
    uint32_t n_item = 0, n_p[2] = {0, 0}, n_out[2] = {0, 0};
    auto wait_slot = [&](int k) { return mbar_wait(&full[k % kSlots], (uint32_t)((k / kSlots) & 1), err); };
    for (int i = it0; ok && i < it1; ++i) {
      const ExpandedItem it = p.items[i];
      const int ng[2] = {group_steps(it, 0), group_steps(it, 1)};
      const int n = max(ng[0], ng[1]);
      if (n == 0) continue;
      ok = mbar_wait(q_full, n_item & 1, err);
      for (int j = 0; ok && j <= n; ++j) {
        const int kb = base + 5 * j, vb = base + 5 * (j - 1) + 3;  // first slots of K(j), V(j - 1)
        bool k_here = false, v_here = false;
        for (int g = 0; ok && g < 2; ++g) {
          const uint32_t s_tm = tmem + 128 * g, o_tm = s_tm + kOCol;
          if (j > 0 && j <= ng[g]) {
            ok = mbar_wait(&p_full[g], n_p[g] & 1, err);
            ++n_p[g];
            if (ok && j == 1 && n_out[g] > 0) ok = mbar_wait(&o_free[g], (n_out[g] - 1) & 1, err);
            for (int s = 0; ok && !v_here && s < 2; ++s) ok = wait_slot(vb + s);
            v_here = true;
            if (!ok) break;
            tc_fence_after();
            // (the two slabs are separate MMAs of N = 64: they need not be neighbours in the ring)
#pragma unroll
            for (int s = 0; s < 2; ++s) {
              const uint64_t vd = dV + (uint64_t)((((vb + s) % kSlots) * 16384) >> 4);
#pragma unroll
              for (int kk = 0; kk < 8; ++kk) {  // keys 16 kk ..: columns 32 (kk / 2) + 8 (kk % 2) of S
                const uint64_t b = vd + (uint64_t)((kk * 16 * 128) >> 4);
                tc_mma_ts(o_tm + 64 * s, s_tm + 32 * (kk >> 1) + 8 * (kk & 1), b, kIdescO, j > 1 || kk > 0 ? 1u : 0u);
              }
            }
            if (j == ng[g]) {
              tc_commit(&o_full[g]);
              ++n_out[g];
            }
          }
          // (V(j - 1) is read when the last group that takes it is done)
          if (j > 0 && (g == 1 || j > ng[1]) && !(g == 1 && j > ng[1])) {
            for (int s = 0; s < 2; ++s) tc_commit(&empty[(vb + s) % kSlots]);
          }
          if (j < ng[g]) {
            for (int s = 0; ok && !k_here && s < 3; ++s) ok = wait_slot(kb + s);
            k_here = true;
            if (!ok) break;
            tc_fence_after();
#pragma unroll
            for (int s = 0; s < 3; ++s)
#pragma unroll
              for (int k = 0; k < 4; ++k)
                tc_mma_ss(s_tm, dQ + (uint64_t)((g * L::kGroupQ + s * 16384 + 32 * k) >> 4),
                          dK + (uint64_t)((((kb + s) % kSlots) * 16384 + 32 * k) >> 4), kIdescS, s + k > 0 ? 1u : 0u);
            tc_commit(&s_full[g]);
          }
        }
        if (!ok) break;
        if (j < n) {
          for (int s = 0; s < 3; ++s) tc_commit(&empty[(kb + s) % kSlots]);
        }
        if (j == n - 1) tc_commit(q_empty);
      }
      base += 5 * n;
      ++n_item;
    }
    // nothing this thread started may still run when TMEM is released
    tc_commit(fin);
    mbar_wait(fin, 0u, err);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// Joins the parts of cut tiles: a warp a query, four elements a lane.
__global__ void __launch_bounds__(128) expanded_join_kernel(const ExpandedParams p) {
  wait_for_upload();
  constexpr int kPer = kExpandedRows / 4;
  const ExpandedCut cut = p.cuts[blockIdx.x / kPer];
  const int row = 4 * (blockIdx.x % kPer) + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (row >= cut.count) return;
  const float2* ml = p.part_ml + (int64_t)cut.slot * kExpandedRows + row;
  const float* src = p.part_o + ((int64_t)cut.slot * kExpandedRows + row) * kExpandedV + 4 * lane;
  float m = -CUDART_INF_F, l = 0.f;
  for (int q = 0; q < cut.n_parts; ++q) m = fmaxf(m, ml[(int64_t)q * kExpandedRows].x);
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int q = 0; q < cut.n_parts; ++q) {
    const float2 x = ml[(int64_t)q * kExpandedRows];
    if (x.x == -CUDART_INF_F) continue;  // (no key of the row in this part: any value may stand there)
    const float w = ex2(x.x - m);
    const float4 y = *reinterpret_cast<const float4*>(src + (int64_t)q * kExpandedRows * kExpandedV);
    l += w * x.y;
    o.x += w * y.x;
    o.y += w * y.y;
    o.z += w * y.z;
    o.w += w * y.w;
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
  *reinterpret_cast<uint2*>(p.o + ((int64_t)(cut.q_start + row) * p.heads + cut.head) * kExpandedV + 4 * lane) =
      make_uint2(pack_f16x2_out(o.x * inv, o.y * inv), pack_f16x2_out(o.z * inv, o.w * inv));
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
  cfg.gridDim = dim3(p.n_cuts * (kExpandedRows / 4));
  cfg.blockDim = dim3(128);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, expanded_join_kernel, p);
}

}  // namespace mixattn
