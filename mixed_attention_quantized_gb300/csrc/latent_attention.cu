// latent_attention.cu -- absorbed latent attention: every (query, head) row of a token meets the
// cached rows [c | r] of 512 + 64 fp16 elements, whose first 512 are the values too:
//     S = q [c | r]^T,   P = 2^(scale (S - m) + 7),   O = sum P c,   o = O / sum P.
//
// The reference m is a score and not one times the scale: the differences that weigh something are then exact to
// fp32 however large the scores are.  (Of scale S near 2^28 no fp32 number is closer than 16: weights 2^(scale S - m')
// about such an m' overflow fp16 or vanish.)  An addition more a score, of two scores together: no slower.
//
// A CTA takes a tile of N (16, 32 or 64) rows and walks a range of the row's pages, 64 keys (two
// pages) a step, each loaded once into shared memory and used from there by both products:
//   S   [64 rows][64 keys]   = Q (A, rows of 576) x K^T (B): M = 64, rows past N unused; Q in TMEM as far
//                              as there is room (N = 64: 384 elements of 576, with one buffer of S), or its reads and those of K
//                              fill shared memory's bandwidth, and copies and barriers wait behind them
//   O^T [512 elements][N]   += c^T (A, the same bytes read MN-major) x P^T (B): four blocks of 128
// O^T rather than O because 64 rows of 512 fp32 would fill TMEM alone, and because N then follows
// the number of rows: 16 heads cost a quarter of the operand reads that 64 do.
//
// Roles: softmax (warps 0-3), loads (warps 4-7), MMA (the elected lanes of warps 8 and 9). A step's four
// 128-element units of c and its r come through rings of slots with barriers of their own, so that a
// unit is refilled as soon as its block of O^T is done.
//
// The loads are 16-byte cp.async by four warps, swizzled by address, and not TMA boxes: a box of 128-byte
// rows moves 49 bytes a ns and SM at most (7.4 TB/s over all, measured with 192 KB in flight an SM, from
// HBM and from L2 alike), these 130 from L2.
//
// Bound by HBM with 16 heads: 64 rows of 1024 to 16384 tokens 115 us (638 MB, 5.6 TB/s over all; a steady step
// 6.5 to 7.2, the rest is items' starts and the join).  By the chain of a step's latencies over a ring of 2.75 steps
// with 64-row tiles, tensor pipe 59 % active: 128 heads, a session of 131072 tokens and 31 short rows 125 us, 16
// trees of 6 298 us (0.82 PFLOP/s).  32-key steps: 127, 152 us (the third not measured) where these took 118, 146.
#include <mutex>

#include "latent.h"
#include "page_attention.cuh"

namespace mixattn {

namespace {

constexpr int kSoftmaxWarps = 4;
constexpr int kLoadWarps = 4;
constexpr int kMmaWarp = kSoftmaxWarps + kLoadWarps;
constexpr int kLatentThreads = 32 * (kMmaWarp + 2);
constexpr int kStepKeys = 64;  // keys of a step: two pages

template <int N>
struct LatentSmem {
  static constexpr int kSBuffers = N == 64 ? 1 : 2;
  static constexpr int kTmemSlabs = N == 64 ? 6 : (N == 32 ? 8 : 9);  // of a row's nine 64-element slabs, those held in TMEM
  static constexpr int kQSlab = N * 128;                 // 64 elements of N rows, swizzled
  static constexpr int kQ = 0;                           // the other slabs
  static constexpr int kP = kQ + (9 - kTmemSlabs) * kQSlab;          // [N][64 keys]
  static constexpr int kRope = (kP + N * 128 + 1023) / 1024 * 1024;  // 2 slots of [64 keys][64]
  static constexpr int kUnit0 = kRope + 2 * 8192;        // slots of [2][64 keys][64]
  static constexpr int kUnits = N == 64 ? 11 : 12;
  static constexpr int kStat = kUnit0 + kUnits * 16384;  // alpha[64], l[64]
  static constexpr int kBar = kStat + 512;
  static constexpr int kTotal = kBar + 512 + 1024;       // + slack for 1024-byte alignment
  static_assert(kTotal <= 227 * 1024, "the tile does not fit in shared memory");
};

// 16 lanes x 64 columns of 32-bit TMEM: register 4 j + 2 h + e holds row lane / 4 + 8 h, column
// 8 j + 2 (lane % 4) + e.
__device__ __forceinline__ void tmem_ld_16x64(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x8.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
        "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]),
        "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]),
        "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}

// The same layout the other way.
__device__ __forceinline__ void tmem_st_16x64(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x256b.x8.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]),
      "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]),
      "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_st_16x32(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x256b.x4.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

// What one tile of an item covers.
struct LatentTile {
  int f0, rows;           // first (query, head) row of the row's, rows here
  int n_keys;             // keys of the row up to the last that some query of the tile may see
  int n_pages;            // the item's pages with such keys
  bool there;
};

__device__ __forceinline__ LatentTile tile_of(const LatentParams& p, const LatentItem& it, const LatentRowInfo& ri,
                                              int member, int N) {
  LatentTile t;
  const int total = (ri.seq_len - ri.q_offset) * p.heads;
  t.f0 = (it.mt0 + member) * N;
  t.rows = min(N, total - t.f0);
  t.there = t.rows > 0;
  const int last = ri.tree_start >= 0 ? ri.seq_len - 1 : ri.q_offset + (t.f0 + max(t.rows, 1) - 1) / p.heads;
  t.n_keys = last + 1;
  t.n_pages = max(0, min(it.n_pages, last / kPage + 1 - it.page0));
  return t;
}

template <int N>
__global__ void __launch_bounds__(kLatentThreads, 1)
    latent_kernel(const __grid_constant__ LatentParams p, unsigned int* err) {
  using L = LatentSmem<N>;
  constexpr int NU = L::kUnits;
  // O^T blocks; one or two buffers of S, 64 rows in the lower 16 lanes of each warp's 32; the slabs of Q
  // held here, two elements a column, in the same lanes
  constexpr int QT = L::kTmemSlabs, SB = L::kSBuffers;
  constexpr uint32_t kOCol = 0, kSCol = 4 * N, kSBuf = 64, kQCol = kSCol + SB * kSBuf;
  constexpr uint32_t kTmemCols = 512;
  static_assert(kQCol + 32 * QT <= kTmemCols, "TMEM");
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kBar);
  // step g's keys in g % 4, by the copies of the load warps' lanes: units 0-2 and the position keys; unit 3,
  // whose slot is the last to be free
  uint64_t* full = bars;                   // [4]
  uint64_t* full3 = full + 4;              // [4]
  uint64_t* unit_empty = full3 + 4;        // [NU] by a commit: the unit's block of O^T done
  uint64_t* rope_empty = unit_empty + NU;  // [2] by a commit
  uint64_t* q_full = rope_empty + 2;       // by the softmax warps: the item's queries written
  uint64_t* s_full = q_full + 1;           // [SB] S(g) in buffer g % SB
  uint64_t* s_read = s_full + SB;          // [SB] by the softmax warps: S(g) read
  uint64_t* p_full = s_read + SB;          // by the softmax warps: P(g) written, O^T rescaled
  uint64_t* pv_done = p_full + 1;          // PV(g) done
  uint64_t* o_free = pv_done + 1;          // by the softmax warps: the item's O^T read
  uint64_t* q_asked = o_free + 1;          // by the softmax warps: the first item's queries are on their way
  uint64_t* fin = q_asked + 1;             // [2]
  constexpr int kNumBars = NU + 17 + 2 * SB;
  static_assert(8 * kNumBars + 8 <= 512, "barrier area");
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + kNumBars);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < kNumBars; ++i) mbar_init(bars + i, 1);
    for (int i = 0; i < 4; ++i) {
      mbar_init(full + i, 32 * (kLoadWarps - 1));
      mbar_init(full3 + i, 32);
    }
    for (int i = 0; i < SB; ++i) mbar_init(s_read + i, N / 16);  // (the warps with rows)
    mbar_init(p_full, kSoftmaxWarps);
    mbar_init(o_free, kSoftmaxWarps);
    mbar_init(q_full, kSoftmaxWarps);
    mbar_init(q_asked, kSoftmaxWarps);
    *abort_flag = 0;
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
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the item list is written by the grid before
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  const int team = blockIdx.x / p.team, member = blockIdx.x - team * p.team;
  const LatentItem* items = p.list.at<LatentItem>(p.items);
  const LatentRowInfo* row_list = p.list.at<LatentRowInfo>(p.rows);
  const int it0 = p.list.at<int32_t>(p.team_first)[team], it1 = p.list.at<int32_t>(p.team_first)[team + 1];

  if (warp >= kSoftmaxWarps && warp < kMmaWarp) {
    // ======================= load (warp w: unit w of every step) =======================
    const int w = warp - kSoftmaxWarps;
    int slot = w, round = 0, g = 0;
    bool ok = true;
    uint64_t* filled = w < 3 ? full : full3;
    const int ch = lane & 15, kk = lane >> 4;  // the lane's 16-byte chunk of a key's 256 bytes, and its key of two
    const uint32_t dst_lane = smem_u32(smem + L::kUnit0) + (ch >> 3) * 8192 + kk * 128;
    // position keys: warps 0 and 1 load a page's, chunk lane % 8 of keys lane / 8 + 4 q
    const int r_key = 32 * (w & 1) + (lane >> 3);
    const uint32_t r_dst = smem_u32(smem + L::kRope) + sw128_off(r_key, lane & 7);
    // The queries go first: behind the keys of 2.5 steps, asked for by every SM at once, they would take
    // 5 us, and nothing starts without them.
    if (it0 < it1) ok = warp_wait_fast(q_asked, 0u, err);
    for (int i = it0; ok && i < it1; ++i) {
      const LatentItem it = items[i];
      const LatentRowInfo ri = row_list[it.row];
      const LatentTile t = tile_of(p, it, ri, member, N);
      if (!t.there || t.n_pages == 0) continue;
      const int32_t* pt_row = p.page_table + (int64_t)it.row * p.max_pages + it.page0;
      const int n_steps = (t.n_pages + 1) / 2;
      int pid = -1;
      for (int s = 0; s < n_steps; ++s, ++g) {
        if ((s & 15) == 0) {  // lane l: page 2 s + l of the item
          pid = 2 * s + lane < t.n_pages ? pt_row[2 * s + lane] : -1;
          if (pid < 0 || pid >= p.num_pages) {
            if (2 * s + lane < t.n_pages) set_device_error(err, MIXATTN_DEVERR_PAGE_ID);
            pid = -1;
          }
        }
        const int ia = __shfl_sync(0xFFFFFFFFu, pid, (2 * s) & 31), ib = __shfl_sync(0xFFFFFFFFu, pid, (2 * s + 1) & 31);
        if (round > 0) ok = warp_wait_fast(&unit_empty[slot], (uint32_t)((round - 1) & 1), err);
        if (ok && w < 2 && g >= 2) ok = warp_wait_fast(&rope_empty[g & 1], (uint32_t)(((g >> 1) - 1) & 1), err);
        if (!ok) break;
        // Keys that no query of the tile sees, and those of a page that is not there, are zeros: what the
        // cache holds there may be anything, and 0 x NaN is not 0.
        const int key0 = kPage * (it.page0 + 2 * s);
        uint32_t seen_a = low_bits(t.n_keys - key0), seen_b = low_bits(t.n_keys - key0 - kPage);
        if (ri.tree_start >= 0 && key0 + kStepKeys > ri.q_offset) {
          seen_a = seen_b = 0;
          const int q1 = (t.f0 + t.rows - 1) / p.heads;
          for (int q = t.f0 / p.heads + lane; q <= q1; q += 32) {
            const uint32_t* tm = p.tree_mask + (int64_t)(ri.tree_start + q) * p.tree_words;
            seen_a |= tree_bits(tm, p.tree_words, ri.seq_len - ri.q_offset, key0 - ri.q_offset);
            seen_b |= tree_bits(tm, p.tree_words, ri.seq_len - ri.q_offset, key0 + kPage - ri.q_offset);
          }
          seen_a = __reduce_or_sync(0xFFFFFFFFu, seen_a);
          seen_b = __reduce_or_sync(0xFFFFFFFFu, seen_b);
        }
        if (ia < 0) seen_a = 0;
        if (ib < 0) seen_b = 0;
        const bool whole = (seen_a & seen_b) == 0xFFFFFFFFu;
        const uint16_t* pa = p.data + (int64_t)max(ia, 0) * (kPage * kLatentRow);
        const uint16_t* pb = p.data + (int64_t)max(ib, 0) * (kPage * kLatentRow);
        const uint16_t* sa = pa + kk * kLatentRow + 128 * w + 8 * ch;
        const uint16_t* sb = pb + kk * kLatentRow + 128 * w + 8 * ch;
        const uint32_t dst = dst_lane + slot * 16384;
        const uint16_t* rs = (w == 0 ? pa : pb) + (r_key & 31) * kLatentRow + kLatent + 8 * (lane & 7);
        const uint32_t rd = r_dst + (g & 1) * 8192;
        if (whole) {
          if (w < 2) {
#pragma unroll
            for (int q = 0; q < 8; ++q)  // (keys 4 apart: chunk bit 2 flips)
              cp_async16_s((rd ^ ((q & 1) << 6)) + q * 512, rs + q * (4 * kLatentRow));
          }
#pragma unroll
          for (int q = 0; q < 32; ++q)
            cp_async16_s(dst + q * 256 + (((ch & 7) ^ ((2 * q + kk) & 7)) << 4),
                         (q < 16 ? sa : sb) + (q & 15) * (2 * kLatentRow));
        } else {
          if (w < 2) {
#pragma unroll
            for (int q = 0; q < 8; ++q)
              cp_async16_or_zero((rd ^ ((q & 1) << 6)) + q * 512, rs + q * (4 * kLatentRow),
                                 (((w == 0 ? seen_a : seen_b) >> ((lane >> 3) + 4 * q)) & 1u) != 0u);
          }
#pragma unroll 4
          for (int q = 0; q < 32; ++q)
            cp_async16_or_zero(dst + q * 256 + (((ch & 7) ^ ((2 * q + kk) & 7)) << 4),
                               (q < 16 ? sa : sb) + (q & 15) * (2 * kLatentRow),
                               (((q < 16 ? seen_a : seen_b) >> (2 * (q & 15) + kk)) & 1u) != 0u);
        }
        cp_async_arrive(&filled[g & 3]);  // (taken again four steps on, long after its MMAs)
        slot += 4;
        if (slot >= NU) {
          slot -= NU;
          ++round;
        }
      }
      if (__any_sync(0xFFFFFFFFu, *abort_flag)) ok = false;
    }
    if (!ok && lane == 0) *abort_flag = 1;
    // nothing asked for may still be on its way when the CTA ends
    cp_async_wait_all();
  } else if (warp >= kMmaWarp) {
    // ======================= MMA: S (the first warp's elected lane), PV (the second's) =======================
    // (Two warps: one that did both would hold a PV that could run behind an S whose keys are still on
    // their way, and with it the slots for the keys after those.)
    constexpr uint32_t kIdescS = idesc_f16_f32(64, kStepKeys, false, false);
    constexpr uint32_t kIdescO = idesc_f16_f32(128, N, true, false);
    auto lo = [](uint64_t d) { return (uint32_t)d; };
    const uint32_t dQ = lo(sw128_desc(smem_u32(smem + L::kQ), 16, 1024));
    const uint32_t dP = lo(sw128_desc(smem_u32(smem + L::kP), 16, 1024));
    const uint32_t dR = lo(sw128_desc(smem_u32(smem + L::kRope), 16, 1024));
    const uint32_t dK = lo(sw128_desc(smem_u32(smem + L::kUnit0), 16, 1024));
    const uint32_t dV = lo(sw128_desc(smem_u32(smem + L::kUnit0), 8192, 1024));  // slabs of 64 elements 8 KB apart
    constexpr uint32_t kHi = (1024u >> 4) | (1u << 14) | (2u << 29);              // the upper word of them all
    const bool is_s = warp == kMmaWarp;
    bool ok = true;
    int g = 0, n_item = 0, slot = 0;
    const int first = __shfl_sync(0xFFFFFFFFu, it0, 0), end = __shfl_sync(0xFFFFFFFFu, it1, 0);
    for (int i = first; ok && i < end; ++i) {
      const LatentItem it = items[i];
      const LatentTile t = tile_of(p, it, row_list[it.row], member, N);
      // (control flow and operands the same in all lanes, and known to be)
      const int n_steps = __shfl_sync(0xFFFFFFFFu, t.there ? (t.n_pages + 1) / 2 : 0, 0);
      if (n_steps == 0) continue;
      if (is_s) {
        ok = warp_wait_fast(q_full, (uint32_t)(n_item & 1), err);
        for (int s = 0; ok && s < n_steps; ++s, ++g) {
          ok = warp_wait_fast(&full[g & 3], (uint32_t)((g >> 2) & 1), err);
          if (ok && g >= SB) ok = warp_wait_fast(&s_read[g % SB], (uint32_t)((g / SB - 1) & 1), err);
          if (!ok) break;
          fence_proxy_async_smem();  // (the copies are the generic proxy's)
          tc_fence_after();
          const uint32_t s_tm = tmem + kSCol + kSBuf * (g % SB);
          if (elect_one()) {
            const uint32_t rd = dR + (g & 1) * (8192 >> 4);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              if (QT == 9) tc_mma_ts_w(s_tm, tmem + kQCol + 256 + 8 * k, rd + ((32 * k) >> 4), kHi, kIdescS, k > 0 ? 1u : 0u);
              else tc_mma_ss_w(s_tm, dQ + (((8 - QT) * L::kQSlab + 32 * k) >> 4), kHi, rd + ((32 * k) >> 4), kHi, kIdescS, k > 0 ? 1u : 0u);
            }
            tc_commit(&rope_empty[g & 1]);
          }
          __syncwarp();
          // 128 elements of Q against a unit of the keys, those of Q in TMEM first
#pragma unroll 1
          for (int b = 0; b < 4; ++b) {
            if (b == 3) {
              ok = warp_wait_fast(&full3[g & 3], (uint32_t)((g >> 2) & 1), err);
              if (!ok) break;
              fence_proxy_async_smem();
              tc_fence_after();
            }
            const uint32_t kd = dK + slot * (16384 >> 4);
            if (2 * b < QT) {
              if (elect_one()) {
                const uint32_t qt = tmem + kQCol + 64 * b;
#pragma unroll
                for (int k = 0; k < 8; ++k)
                  tc_mma_ts_w(s_tm, qt + 8 * k, kd + (((k >> 2) * 8192 + 32 * (k & 3)) >> 4), kHi, kIdescS, 1u);
              }
            } else {
              if (elect_one()) {
                const uint32_t qd = dQ + (2 * b - QT) * (L::kQSlab >> 4);
#pragma unroll
                for (int k = 0; k < 8; ++k)
                  tc_mma_ss_w(s_tm, qd + (((k >> 2) * L::kQSlab + 32 * (k & 3)) >> 4), kHi,
                              kd + (((k >> 2) * 8192 + 32 * (k & 3)) >> 4), kHi, kIdescS, 1u);
              }
            }
            __syncwarp();
            if (++slot == NU) slot = 0;
          }
          if (!ok) break;
          if (elect_one()) tc_commit(&s_full[g % SB]);
          __syncwarp();
        }
      } else {
        for (int s = 0; ok && s < n_steps; ++s, ++g) {
          ok = warp_wait_fast(p_full, (uint32_t)(g & 1), err);
          if (ok && s == 0 && n_item > 0) ok = warp_wait_fast(o_free, (uint32_t)((n_item - 1) & 1), err);
          if (!ok) break;
          // (the keys landed before S(g), and were fenced there: by another thread, so once more here)
          fence_proxy_async_smem();
          tc_fence_after();
          const uint32_t acc = s > 0 ? 1u : 0u;
#pragma unroll 1
          for (int b = 0; b < 4; ++b) {
            if (elect_one()) {
              const uint32_t vd = dV + slot * (16384 >> 4), o_tm = tmem + kOCol + N * b;
#pragma unroll
              for (int k = 0; k < 4; ++k)
                tc_mma_ss_w(o_tm, vd + ((2048 * k) >> 4), kHi, dP + ((32 * k) >> 4), kHi, kIdescO, k > 0 ? 1u : acc);
              tc_commit(&unit_empty[slot]);
              if (b == 3) tc_commit(pv_done);
            }
            __syncwarp();
            if (++slot == NU) slot = 0;
          }
        }
      }
      ++n_item;
    }
    // nothing the lane started may still run when TMEM is released
    if (elect_one()) {
      if (!ok) *abort_flag = 1;
      tc_commit(is_s ? fin : fin + 1);
      mbar_wait(is_s ? fin : fin + 1, 0u, err);
    }
    __syncwarp();
  } else {
    // ======================= softmax =======================
    constexpr int kGroup = 32 * kSoftmaxWarps;
    constexpr float kTop = 15.f, kSet = 7.f;  // as page_decode_tile: P up to 2^15, set at 2^7
    const uint64_t scale2 = f2_pack(p.scale_log2, p.scale_log2), set2 = f2_pack(kSet, kSet);
    constexpr int kBarGroup = 1;
    const int r = lane >> 2, c = lane & 3;
    const bool rows_here = 16 * warp < N;  // the warp's 16 rows of S; every warp has 32 elements of each O^T block
    const uint32_t lane_base = (uint32_t)(32 * warp) << 16;
    float* alpha_s = reinterpret_cast<float*>(smem + L::kStat);
    float* l_s = alpha_s + 64;
    const int rr0 = 16 * warp + r;  // rows rr0 and rr0 + 8
    bool ok = true;
    int g = 0;
    // Writes the queries of the CTA's next item from i on that has work.  A quad of lanes takes 16
    // elements of a row: 32 bytes.
    auto write_q = [&](int i, bool first) {
      for (; i < it1; ++i) {
        const LatentItem it = items[i];
        const LatentRowInfo ri = row_list[it.row];
        const LatentTile t = tile_of(p, it, ri, member, N);
        if (!t.there || t.n_pages == 0) continue;
        if (rows_here) {
          const uint16_t* q0 = p.q + ((int64_t)ri.q_start * p.heads + t.f0 + rr0) * kLatentRow + 4 * c;
          const uint16_t* q1 = q0 + 8 * kLatentRow;
          const bool in0 = rr0 < t.rows, in1 = rr0 + 8 < t.rows;
          // (all loads together: behind the first keys' a load takes several us)
          uint32_t v[5][32];
#pragma unroll
          for (int b = 0; b < 5; ++b)  // 128 elements each, the last 64
#pragma unroll
            for (int j = 0; j < (b < 4 ? 8 : 4); ++j) {
              const uint2 x = ldg_u64_pred(q0 + 128 * b + 16 * j, in0), y = ldg_u64_pred(q1 + 128 * b + 16 * j, in1);
              v[b][4 * j] = x.x;
              v[b][4 * j + 1] = x.y;
              v[b][4 * j + 2] = y.x;
              v[b][4 * j + 3] = y.y;
            }
          if (first && lane == 0) mbar_arrive(q_asked);
          first = false;
#pragma unroll
          for (int b = 0; b < 5; ++b) {
            if (2 * b < QT) {
              if (b < 4) {
                tmem_st_16x64(tmem + lane_base + kQCol + 64 * b, v[b]);
              } else {
                uint32_t u[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) u[e] = v[b][e];
                tmem_st_16x32(tmem + lane_base + kQCol + 64 * b, u);
              }
            } else {
#pragma unroll
              for (int j = 0; j < (b < 4 ? 8 : 4); ++j) {
                // elements 16 (j % 4) + 4 c of slab 2 b + j / 4: half of chunk 2 (j % 4) + c / 2
                uint8_t* at = smem + L::kQ + (2 * b + (j >> 2) - QT) * L::kQSlab + 8 * (c & 1);
                *reinterpret_cast<uint2*>(at + sw128_off(rr0, 2 * (j & 3) + (c >> 1))) =
                    make_uint2(v[b][4 * j], v[b][4 * j + 1]);
                *reinterpret_cast<uint2*>(at + sw128_off(rr0 + 8, 2 * (j & 3) + (c >> 1))) =
                    make_uint2(v[b][4 * j + 2], v[b][4 * j + 3]);
              }
            }
          }
          tmem_wait_st();
          if (QT < 9) fence_proxy_async_smem();
        } else if (first && lane == 0) {
          mbar_arrive(q_asked);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(q_full);
        return;
      }
      if (first && lane == 0) mbar_arrive(q_asked);  // (no item with work)
    };
    write_q(it0, true);
    for (int i = it0; i < it1; ++i) {
      const LatentItem it = items[i];
      const LatentRowInfo ri = row_list[it.row];
      const LatentTile t = tile_of(p, it, ri, member, N);
      if (!t.there) continue;
      const int64_t part = (int64_t)it.slot + (int64_t)member * it.n_parts + it.part;
      if (t.n_pages == 0) {  // (a part past the tile's last key)
        if (tid < N) p.part_ml[part * N + tid] = make_float2(-CUDART_INF_F, 0.f);
        continue;
      }
      const int n_steps = (t.n_pages + 1) / 2;
      const bool tree = ri.tree_start >= 0;
      const int qi0 = (t.f0 + min(rr0, t.rows - 1)) / p.heads, qi1 = (t.f0 + min(rr0 + 8, t.rows - 1)) / p.heads;
      const int pos0 = ri.q_offset + qi0, pos1 = ri.q_offset + qi1;
      const int mask_hi = tree ? ri.q_offset : ri.q_offset + t.f0 / p.heads + 1;  // keys below: seen by every row
      const int n_nodes = ri.seq_len - ri.q_offset;
      const uint32_t* tm0 = tree ? p.tree_mask + (int64_t)(ri.tree_start + qi0) * p.tree_words : nullptr;
      const uint32_t* tm1 = tree ? p.tree_mask + (int64_t)(ri.tree_start + qi1) * p.tree_words : nullptr;
      const int32_t* pt_row = p.page_table + (int64_t)it.row * p.max_pages + it.page0;
      float m0 = -CUDART_INF_F, m1 = -CUDART_INF_F, l0 = 0.f, l1 = 0.f;
      uint32_t good = 0;
      bool stop = false;
      for (int s = 0; s < n_steps; ++s, ++g) {
        if ((s & 15) == 0) {
          const int pid = 2 * s + lane < t.n_pages ? pt_row[2 * s + lane] : -1;
          good = __ballot_sync(0xFFFFFFFFu, pid >= 0 && pid < p.num_pages);
        }
        const bool ok_a = (good >> ((2 * s) & 31)) & 1u, ok_b = (good >> ((2 * s + 1) & 31)) & 1u;
        float x[32];
        float al0 = 1.f, al1 = 1.f;
        bool need = false;
        if (rows_here) {
          ok = warp_wait_fast(&s_full[g % SB], (uint32_t)((g / SB) & 1), err) && ok;
          tc_fence_after();
          uint32_t v[32];
          tmem_ld_16x64(tmem + lane_base + kSCol + kSBuf * (g % SB), v);
          tmem_wait_ld();
          tc_fence_before();
          if (lane == 0) mbar_arrive(&s_read[g % SB]);
          const int key0 = kPage * (it.page0 + 2 * s);
          if (!ok_a || !ok_b || key0 + kStepKeys > mask_hi) {
            uint32_t vis[2][2];  // [row][page]
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int k0 = key0 + kPage * h;
              const uint32_t in = (h ? ok_b : ok_a) ? 0xFFFFFFFFu : 0u;
              if (tree) {
                vis[0][h] = tree_bits(tm0, p.tree_words, n_nodes, k0 - ri.q_offset) & in;
                vis[1][h] = tree_bits(tm1, p.tree_words, n_nodes, k0 - ri.q_offset) & in;
              } else {
                vis[0][h] = low_bits(pos0 + 1 - k0) & in;
                vis[1][h] = low_bits(pos1 + 1 - k0) & in;
              }
            }
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              const int j = e >> 2, col = 8 * (j & 3) + 2 * c + (e & 1);
              if (!((vis[(e >> 1) & 1][j >> 2] >> col) & 1u)) v[e] = __float_as_uint(-CUDART_INF_F);
            }
          }
          float t0 = -CUDART_INF_F, t1 = -CUDART_INF_F;
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            t0 = fmax3(t0, __uint_as_float(v[e]), __uint_as_float(v[e + 1]));
            t1 = fmax3(t1, __uint_as_float(v[e + 2]), __uint_as_float(v[e + 3]));
          }
          t0 = fmaxf(t0, __shfl_xor_sync(0xFFFFFFFFu, t0, 1));
          t1 = fmaxf(t1, __shfl_xor_sync(0xFFFFFFFFu, t1, 1));
          t0 = fmaxf(t0, __shfl_xor_sync(0xFFFFFFFFu, t0, 2));
          t1 = fmaxf(t1, __shfl_xor_sync(0xFFFFFFFFu, t1, 2));
          const bool g0 = m0 == -CUDART_INF_F ? t0 > m0 : (t0 - m0) * p.scale_log2 > kTop - kSet;
          const bool g1 = m1 == -CUDART_INF_F ? t1 > m1 : (t1 - m1) * p.scale_log2 > kTop - kSet;
          if (g0) {
            al0 = ex2((m0 - t0) * p.scale_log2);
            m0 = t0;
            l0 *= al0;
          }
          if (g1) {
            al1 = ex2((m1 - t1) * p.scale_log2);
            m1 = t1;
            l1 *= al1;
          }
          need = g0 || g1;
          const float n0 = m0 == -CUDART_INF_F ? 0.f : -m0, n1 = m1 == -CUDART_INF_F ? 0.f : -m1;
          const uint64_t n0_2 = f2_pack(n0, n0), n1_2 = f2_pack(n1, n1);
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            const uint64_t d = fadd2(f2_pack(__uint_as_float(v[e]), __uint_as_float(v[e + 1])), (e & 2) ? n1_2 : n0_2);
            f2_unpack(ffma2(d, scale2, set2), x[e], x[e + 1]);
            x[e] = ex2(x[e]);
            x[e + 1] = ex2(x[e + 1]);
          }
          float a0 = 0.f, a1 = 0.f;
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            a0 += x[e] + x[e + 1];
            a1 += x[e + 2] + x[e + 3];
          }
          l0 += a0;
          l1 += a1;
        }
        if (bar_any(kBarGroup, kGroup, need) && s > 0) {  // some row's reference moved: O^T takes the factor
          if (rows_here && c == 0) {
            alpha_s[rr0] = al0;
            alpha_s[rr0 + 8] = al1;
          }
          bar_any(kBarGroup, kGroup, false);
          ok = warp_wait_fast(pv_done, (uint32_t)((g - 1) & 1), err) && ok;
          tc_fence_after();
#pragma unroll 1
          for (int b = 0; b < 4 * N / 16; ++b) {
            uint32_t o[16];
            tmem_ld16(tmem + lane_base + kOCol + 16 * b, o);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e)
              o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha_s[(16 * b + e) % N]);
            tmem_st16(tmem + lane_base + kOCol + 16 * b, o);
          }
          tmem_wait_st();
        } else if (g > 0) {
          ok = warp_wait_fast(pv_done, (uint32_t)((g - 1) & 1), err) && ok;  // P(g - 1) has been read
        }
        if (rows_here) {
          uint8_t* p0 = smem + L::kP + rr0 * 128 + 4 * c;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            *reinterpret_cast<uint32_t*>(p0 + ((j ^ (rr0 & 7)) << 4)) = pack_f16x2(x[4 * j], x[4 * j + 1]);
            *reinterpret_cast<uint32_t*>(p0 + 1024 + ((j ^ (rr0 & 7)) << 4)) = pack_f16x2(x[4 * j + 2], x[4 * j + 3]);
          }
          fence_proxy_async_smem();
        }
        tc_fence_before();
        if (bar_any(kBarGroup, kGroup, !ok || *abort_flag)) {  // one decision for the group
          stop = true;
          break;
        }
        if (lane == 0) mbar_arrive(p_full);
      }
      if (stop) {
        *abort_flag = 1;
        break;
      }
      // the next item's queries: the last S of this one is done
      write_q(i + 1, false);
      // ---- the item's output ----
      ok = warp_wait_fast(pv_done, (uint32_t)((g - 1) & 1), err);
      tc_fence_after();
      l0 += __shfl_xor_sync(0xFFFFFFFFu, l0, 1);
      l1 += __shfl_xor_sync(0xFFFFFFFFu, l1, 1);
      l0 += __shfl_xor_sync(0xFFFFFFFFu, l0, 2);
      l1 += __shfl_xor_sync(0xFFFFFFFFu, l1, 2);
      if (rows_here && c == 0) {
        if (it.n_parts == 1) {
          l_s[rr0] = l0 > 0.f ? 1.f / l0 : 0.f;
          l_s[rr0 + 8] = l1 > 0.f ? 1.f / l1 : 0.f;
        } else {
          p.part_ml[part * N + rr0] = make_float2(m0, l0);
          p.part_ml[part * N + rr0 + 8] = make_float2(m1, l1);
        }
      }
      if (bar_any(kBarGroup, kGroup, !ok)) {
        *abort_flag = 1;
        break;
      }
      const int64_t row0 = (int64_t)ri.q_start * p.heads + t.f0;
      const int odd = lane & 1;
#pragma unroll 1
      for (int b = 0; b < 4 * N / 16; ++b) {
        const int d = 128 * (16 * b / N) + 32 * warp + lane, col0 = (16 * b) % N;
        uint32_t o[16];
        tmem_ld16(tmem + lane_base + kOCol + 16 * b, o);
        tmem_wait_ld();
        if (it.n_parts > 1) {  // four rows at a time, [element][row]: 512 bytes a warp and store
          uint4* dst = reinterpret_cast<uint4*>(p.part_o) + (part * (4 * N / 16) + b) * 512 + 32 * warp + lane;
#pragma unroll
          for (int e = 0; e < 4; ++e) dst[128 * e] = make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
          continue;
        }
        // lanes 2 k, 2 k + 1 hold two neighbouring elements of every row: the even lane takes both of
        // every other row, the odd one those of the rows between
#pragma unroll
        for (int e = 0; e < 16; e += 2) {
          const float mine = __uint_as_float(odd ? o[e + 1] : o[e]);
          const float other = __shfl_xor_sync(0xFFFFFFFFu, __uint_as_float(odd ? o[e] : o[e + 1]), 1);
          const int col = col0 + e + odd;
          if (col >= t.rows) continue;
          const float inv = l_s[col];
          *reinterpret_cast<uint32_t*>(p.o + (row0 + col) * kLatent + d - odd) =
              pack_f16x2_out((odd ? other : mine) * inv, (odd ? mine : other) * inv);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(o_free);
      bar_any(kBarGroup, kGroup, false);  // (l_s is written again by the next item)
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

// Joins the parts of cut tiles.  Most tiles have two to four: a CTA takes 128 elements of 16 rows, each half
// of its threads every second part, and all loads go out together, behind that of the cut.  Of a long row's
// many parts a CTA takes 32 elements, its eight warps every eighth part (one row of 8000 tokens, both kernels:
// 22.6 us with the former alone, 20.5 with both).
__global__ void __launch_bounds__(256) latent_join_kernel(const __grid_constant__ LatentParams p, int tile_rows) {
  extern __shared__ float weights[];  // [parts][16]
  __shared__ float inv_l[16];
  __shared__ float sums[7 * 16 * 32];  // [groups - 1][16][elements]
  wait_for_upload();
  const int n = tile_rows / 4;  // units of 16 rows by 128 elements
  const LatentCut cut = p.list.at<LatentCut>(p.cuts)[blockIdx.x / n];
  const int b = blockIdx.x % n, col0 = 16 * b % tile_rows, rows = cut.rows - col0;  // rows here
  if (rows <= 0) return;
  const int width = cut.quarter < 0 ? 128 : 32, groups = 256 / width;
  const int e0 = threadIdx.x % width, group = threadIdx.x / width, d = max(cut.quarter, 0) * 32 + e0;
  const float4* src = reinterpret_cast<const float4*>(p.part_o) + ((int64_t)cut.slot * n + b) * 512 + d;
  float4 y[2][4];
  auto load = [&](int q, float4(&x)[4]) {
    const float4* at = src + (int64_t)min(q, cut.n_parts - 1) * n * 512;
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = __ldcs(at + 128 * e);
  };
  load(group, y[0]);
  load(group + groups, y[1]);
  {
    // sixteen threads a row form its parts' weights; a part without a key of the row weighs nothing
    const int row = threadIdx.x >> 4, k = threadIdx.x & 15;
    const float2* ml = p.part_ml + (int64_t)cut.slot * tile_rows + col0 + row;
    auto part = [&](int q) {
      return row < rows && q < cut.n_parts ? ml[(int64_t)q * tile_rows] : make_float2(-CUDART_INF_F, 0.f);
    };
    const float2 first = part(k);
    float m = first.x, l = 0.f;
    for (int q = k + 16; q < cut.n_parts; q += 16) m = fmaxf(m, part(q).x);
#pragma unroll
    for (int o = 1; o < 16; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    for (int q = k; q < cut.n_parts; q += 16) {
      const float2 x = q == k ? first : part(q);
      const float w = x.x == -CUDART_INF_F ? 0.f : ex2((x.x - m) * p.scale_log2);
      weights[16 * q + row] = w;
      l += w * x.y;  // (0 of a part without a key of the row; NaN where its scores are NaN, whatever the part weighs)
    }
#pragma unroll
    for (int o = 1; o < 16; o <<= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, o);
    if (k == 0) inv_l[row] = l > 0.f ? 1.f / l : l;  // (0, or the NaN of a query that is one)
  }
  __syncthreads();
  float acc[16];
#pragma unroll
  for (int e = 0; e < 16; ++e) acc[e] = 0.f;
  auto add = [&](int q, const float4(&x)[4]) {
    const float4* w = reinterpret_cast<const float4*>(weights + 16 * q);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float4 f = w[e];
      // (where a part has no key of the row any value may stand)
      acc[4 * e] = fmaf(f.x, f.x != 0.f ? x[e].x : 0.f, acc[4 * e]);
      acc[4 * e + 1] = fmaf(f.y, f.y != 0.f ? x[e].y : 0.f, acc[4 * e + 1]);
      acc[4 * e + 2] = fmaf(f.z, f.z != 0.f ? x[e].z : 0.f, acc[4 * e + 2]);
      acc[4 * e + 3] = fmaf(f.w, f.w != 0.f ? x[e].w : 0.f, acc[4 * e + 3]);
    }
  };
#pragma unroll 1
  for (int q = group; q < cut.n_parts; q += 2 * groups) {
    add(q, y[0]);
    if (q + 2 * groups < cut.n_parts) load(q + 2 * groups, y[0]);
    if (q + groups < cut.n_parts) add(q + groups, y[1]);
    if (q + 3 * groups < cut.n_parts) load(q + 3 * groups, y[1]);
  }
  if (group > 0) {
#pragma unroll
    for (int e = 0; e < 16; ++e) sums[((group - 1) * 16 + e) * width + e0] = acc[e];
  }
  __syncthreads();
  if (group > 0) return;
  for (int g = 0; g < groups - 1; ++g) {
#pragma unroll
    for (int e = 0; e < 16; ++e) acc[e] += sums[(g * 16 + e) * width + e0];
  }
  const int odd = d & 1;
  uint16_t* dst = p.o + (cut.row0 + col0) * kLatent + 128 * (16 * b / tile_rows) + d - odd;
#pragma unroll
  for (int e = 0; e < 16; e += 2) {  // (as the attention kernel writes its output)
    const float mine = odd ? acc[e + 1] : acc[e];
    const float other = __shfl_xor_sync(0xFFFFFFFFu, odd ? acc[e] : acc[e + 1], 1);
    if (e + odd >= rows) continue;
    const float inv = inv_l[e + odd];
    *reinterpret_cast<uint32_t*>(dst + (int64_t)(e + odd) * kLatent) =
        pack_f16x2_out((odd ? other : mine) * inv, (odd ? mine : other) * inv);
  }
}

template <int N>
cudaError_t launch_n(const LatentParams& p, unsigned int* err, cudaStream_t s) {
  {
    static std::mutex mu;
    static bool configured[kMaxDevices] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    std::lock_guard<std::mutex> lock(mu);
    if (!configured[dev]) {
      e = cudaFuncSetAttribute(latent_kernel<N>, cudaFuncAttributeMaxDynamicSharedMemorySize, LatentSmem<N>::kTotal);
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
  cfg.gridDim = dim3(p.n_teams * p.team);
  cfg.blockDim = dim3(kLatentThreads);
  cfg.dynamicSmemBytes = LatentSmem<N>::kTotal;
  cudaError_t e = cudaLaunchKernelEx(&cfg, latent_kernel<N>, p, err);
  if (e != cudaSuccess || p.n_cuts == 0) return e;
  cfg.gridDim = dim3(p.n_cuts * (N / 4));
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = p.max_parts * 16 * sizeof(float);  // (at most one part a team: 10 KB)
  return cudaLaunchKernelEx(&cfg, latent_join_kernel, p, N);
}

}  // namespace

cudaError_t launch_latent_attention(int tile_rows, const LatentParams& p, unsigned int* err, cudaStream_t s) {
  if (tile_rows == 16) return launch_n<16>(p, err, s);
  if (tile_rows == 32) return launch_n<32>(p, err, s);
  return launch_n<64>(p, err, s);
}

}  // namespace mixattn
