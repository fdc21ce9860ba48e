// latent.cu -- the latent cache's entry points: append (with the positions' rotation), export, and
// the plans and launches of both attention forms.  See include/mixattn_latent.h.
#include <cuda_runtime.h>
#include <string.h>

#include <algorithm>
#include <new>
#include <vector>

#include "block_encode.cuh"
#include "device_utils.cuh"
#include "latent.h"
#include "plan_list.h"
#include "rope.cuh"

namespace mixattn {

namespace {

// ===========================================================================
// Append and export
// ===========================================================================

struct HeadRows {
  const uint16_t* x;
  int64_t token, head;
};

struct LatentAppendArgs {
  HeadRows q, q_out;
  TokenRows c, r;
  uint16_t* data;
  const int32_t* positions;
  const int32_t* slots;
  int32_t heads, num_slots, n_tokens, per_cta;
  unsigned int* err;
};

// Bound by bytes, so every load of a CTA is under way before its tokens' cosines are formed: a thread
// takes kAppendJobs jobs -- 16 bytes of a latent vector to copy, or 16 elements (both halves of 8
// pairs) of a position key or of a query head to rotate -- of the CTA's one to three tokens.
// 8201 tokens of 32 heads 20.5 us on the GPU (86 MB, 4.2 TB/s), 16 of 128 4.3 us; with 256 threads 22.7 and 4.3, with
// four jobs a thread 20.5 and 6.2, with one 24.7 and 4.3.  A prompt's CTAs come in waves (69 registers: seven of
// 128 threads an SM), each loads, angles, a barrier and stores, with nothing of the next token under way.
constexpr int kAppendJobs = 2, kAppendTokens = 3, kAppendThreads = 128;
static_assert((kAppendTokens + 1) * (kLatent / 8 + kLatentRope / 16) > kAppendJobs * kAppendThreads,
              "a CTA's jobs are those of more tokens");

__global__ void __launch_bounds__(kAppendThreads) latent_append_kernel(const __grid_constant__ RopeTable t,
                                                                       const __grid_constant__ LatentAppendArgs a) {
  __shared__ __align__(16) float2 cs[kAppendTokens][kLatentRope / 2];
  constexpr int kItems = kLatentRope / 16, kCopies = kLatent / 8;
  const int tok0 = blockIdx.x * a.per_cta, n_tok = min(a.per_cta, a.n_tokens - tok0);
  const int jobs = kCopies + kItems * (1 + a.heads);  // of a token: copies, its key, its queries
  int32_t pos = 0;
  if (threadIdx.x < kLatentRope / 2 * n_tok) pos = a.positions[tok0 + threadIdx.x / (kLatentRope / 2)];
  bool first = true;
  for (int i0 = blockIdx.y * kAppendJobs * kAppendThreads; i0 < jobs * n_tok;
       i0 += gridDim.y * kAppendJobs * kAppendThreads) {
    uint4 w0[kAppendJobs], w1[kAppendJobs];
    uint16_t* dst[kAppendJobs];
    int item[kAppendJobs], row[kAppendJobs];  // item < 0: a copy
#pragma unroll
    for (int u = 0; u < kAppendJobs; ++u) {
      const int i = i0 + kAppendThreads * u + threadIdx.x;
      dst[u] = nullptr;
      row[u] = i / jobs;
      const int k = i - row[u] * jobs;
      if (row[u] >= n_tok) continue;
      const int64_t tok = tok0 + row[u];
      const uint16_t* src;
      if (k < kCopies + kItems) {
        const int32_t slot = a.slots[tok];
        if (slot >= a.num_slots && k == 0) set_device_error(a.err, MIXATTN_DEVERR_SLOT);
        if (slot < 0 || slot >= a.num_slots) continue;
        dst[u] = a.data + (int64_t)slot * kLatentRow;
      }
      if (k < kCopies) {
        item[u] = -1;
        dst[u] += 8 * k;
        w0[u] = *reinterpret_cast<const uint4*>(a.c.x + tok * a.c.stride + 8 * k);
        continue;
      }
      item[u] = (k - kCopies) % kItems;
      if (k < kCopies + kItems) {
        src = a.r.x + tok * a.r.stride;
        dst[u] += kLatent;
      } else {
        const int h = (k - kCopies) / kItems - 1;
        src = a.q.x + tok * a.q.token + h * a.q.head;
        dst[u] = const_cast<uint16_t*>(a.q_out.x) + tok * a.q_out.token + h * a.q_out.head;
      }
      int e0, e1;
      rope_item(t, item[u], e0, e1);
      w0[u] = *reinterpret_cast<const uint4*>(src + e0);
      w1[u] = *reinterpret_cast<const uint4*>(src + e1);
    }
    if (first) {
      if (threadIdx.x < kLatentRope / 2 * n_tok)
        cs[threadIdx.x / (kLatentRope / 2)][threadIdx.x % (kLatentRope / 2)] =
            rope_cos_sin(t, pos, threadIdx.x % (kLatentRope / 2));
      __syncthreads();
      first = false;
    }
#pragma unroll
    for (int u = 0; u < kAppendJobs; ++u) {
      if (!dst[u]) continue;
      if (item[u] < 0) {
        *reinterpret_cast<uint4*>(dst[u]) = w0[u];
        continue;
      }
      int e0, e1;
      rope_item(t, item[u], e0, e1);
      float2 c[8];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float4 v = reinterpret_cast<const float4*>(&cs[row[u]][8 * item[u]])[q];
        c[2 * q] = make_float2(v.x, v.y);
        c[2 * q + 1] = make_float2(v.z, v.w);
      }
      float x0[8], x1[8];
      half8_to_float(w0[u], x0);
      half8_to_float(w1[u], x1);
      rope_rotate(t, c, item[u], x0, x1);
      *reinterpret_cast<uint4*>(dst[u] + e0) = float8_to_half(x0);
      *reinterpret_cast<uint4*>(dst[u] + e1) = float8_to_half(x1);
    }
  }
}

// A row a CTA, 16 bytes a thread: 8201 rows 8.4 us on the GPU (19 MB, 2.2 TB/s), 16 rows 4.2, a call 10 us of either.
__global__ void __launch_bounds__(96) latent_export_kernel(const uint16_t* data, const int32_t* slots, int32_t num_slots,
                                                           uint16_t* out, unsigned int* err) {
  const int32_t slot = slots[blockIdx.x];
  if (slot < 0 || slot >= num_slots) {
    if (threadIdx.x == 0) set_device_error(err, MIXATTN_DEVERR_SLOT);
    return;
  }
  if (threadIdx.x < kLatentRow / 8)
    reinterpret_cast<uint4*>(out + (int64_t)blockIdx.x * kLatentRow)[threadIdx.x] =
        *reinterpret_cast<const uint4*>(data + (int64_t)slot * kLatentRow + 8 * threadIdx.x);
}

// ===========================================================================
// Host helpers
// ===========================================================================

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

int check_latent_dims(const mixattn_latent_cache* c) {
  if (!c || c->num_pages <= 0 || c->latent_dim <= 0 || c->rope_dim <= 0) return MIXATTN_ERR_INVALID_ARG;
  if (c->page_size != kPage || c->latent_dim != kLatent || c->rope_dim != kLatentRope) return MIXATTN_ERR_UNSUPPORTED;
  if ((int64_t)c->num_pages * kPage > INT32_MAX) return MIXATTN_ERR_INVALID_ARG;
  return MIXATTN_OK;
}

int check_latent_cache(const mixattn_latent_cache* c) {
  const int st = check_latent_dims(c);
  if (st != MIXATTN_OK) return st;
  return c->data && aligned(c->data, 256) ? MIXATTN_OK : MIXATTN_ERR_INVALID_ARG;
}

constexpr int64_t kMaxStride = (int64_t)1 << 31;  // elements

// Vectors of `width` elements for n tokens of `heads` heads, none of which overlap.
bool check_heads(const mixattn_heads* h, int64_t n, int64_t heads, int64_t width) {
  if (!h || !h->x || !aligned(h->x, 16) || h->token_stride % 8 || h->head_stride % 8) return false;
  if (h->token_stride < 0 || h->head_stride < 0 || h->token_stride >= kMaxStride || h->head_stride >= kMaxStride)
    return false;
  const int64_t ts = h->token_stride, hs = h->head_stride;
  if (heads > 1 && hs < width) return false;
  if (n > 1 && ts < width) return false;
  if (n == 1 || heads == 1) return true;
  return ts >= (heads - 1) * hs + width || hs >= (n - 1) * ts + width;
}

int64_t heads_span(const mixattn_heads* h, int64_t n, int64_t heads, int64_t width) {  // bytes
  return 2 * ((n - 1) * h->token_stride + (heads - 1) * h->head_stride + width);
}

bool check_rows(const void* x, int64_t stride, int64_t width, int64_t n) {
  return x && aligned(x, 16) && stride % 8 == 0 && (n <= 1 || (stride >= width && stride < kMaxStride));
}

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                              const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                              CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn tensor_map_encoder() {
  static const EncodeFn fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &found) !=
            cudaSuccess ||
        found != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<EncodeFn>(p);
  }();
  return fn;
}

// fp16 tensor of `rank` dimensions (innermost first, strides of the others in elements), boxes of
// 64 elements swizzled by 128 bytes; elements outside read as zeros.
bool make_map(CUtensorMap* map, const void* base, int rank, const uint64_t* dims, const int64_t* strides,
              const uint32_t* box) {
  const EncodeFn fn = tensor_map_encoder();
  if (!fn) return false;
  cuuint64_t d[4], st[4];
  cuuint32_t b[4], one[4];
  for (int i = 0; i < rank; ++i) {
    d[i] = dims[i];
    b[i] = box[i];
    one[i] = 1;
    if (i > 0) st[i - 1] = (cuuint64_t)strides[i - 1] * 2;
  }
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, (cuuint32_t)rank, const_cast<void*>(base), d, st, b, one,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int sms_of_device() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) {
    cudaGetLastError();
    return 1;
  }
  return n;
}

// The sections of a plan's image, in order, 16-byte aligned, behind 256 bytes of workspace.
struct Image {
  std::vector<uint8_t> bytes;
  template <class T>
  size_t add(const std::vector<T>& v) {
    const size_t at = bytes.size();
    bytes.resize(align_up(at + sizeof(T) * v.size(), 16), 0);
    if (!v.empty()) memcpy(bytes.data() + at, v.data(), sizeof(T) * v.size());
    return 256 + at;
  }
};

// ===========================================================================
// Absorbed form: the tiling
// ===========================================================================

struct LatentTiling {
  Image image;
  size_t rows = 0, items = 0, team_first = 0, cuts = 0, part_o = 0, part_ml = 0, total = 0;
  int tile_rows = 16, team = 1, n_teams = 1, n_cuts = 0, max_parts = 0;
  int64_t total_q = 0;
  bool trees = false;
  int32_t tree_words = 0;
};

// Pages that an item costs beside its own: its queries' load, first step and output.
constexpr int kItemPages = 5;
// Pages of an item, at least, where a row is cut: a step's chain of latencies is about as long as a part's
// way through the join (one row of 300 tokens, 16 heads, with 2 / 4 / 6: 14.5 / 16.4 / 16.5 us, of 1000 14.6 /
// 14.5 / 16.5, of 8000 26.7 / 20.8 / 20.6; 64 rows of 500 to 2000, 128 heads 80 / 73 / 80).
int64_t min_item_pages(int64_t row_pages) { return row_pages <= 16 ? 2 : 4; }

// CTAs of a team, at most (128 heads: two tiles a token; trees of six, twelve).
constexpr int kMaxTeam = 16;

// A tile of more parts is joined by four times as many CTAs.
constexpr int kManyParts = 8;

int build_latent_tiling(const mixattn_latent_cache& c, int heads, int n_rows, const int32_t* kinds, const int32_t* seq,
                        const int32_t* off, int max_pages, int n_sm, LatentTiling* out) {
  if (n_rows <= 0 || !kinds || !seq || !off || max_pages <= 0) return MIXATTN_ERR_INVALID_ARG;
  LatentTiling& T = *out;
  std::vector<LatentRowInfo> rows(n_rows);
  int64_t total_q = 0, tree_nodes = 0, most = 0;
  for (int r = 0; r < n_rows; ++r) {
    const int64_t s = seq[r], o = off[r], nq = s - o;
    if (kinds[r] == MIXATTN_ROW_DECODE) {
      if (s < 1 || o != s - 1) return MIXATTN_ERR_INVALID_ARG;
    } else if (kinds[r] == MIXATTN_ROW_CHUNK || kinds[r] == MIXATTN_ROW_TREE) {
      if (o < 0 || o >= s) return MIXATTN_ERR_INVALID_ARG;
    } else {
      return MIXATTN_ERR_INVALID_ARG;
    }
    const int64_t n_pages = (s + kPage - 1) / kPage;
    if (n_pages > max_pages || n_pages > c.num_pages) return MIXATTN_ERR_INVALID_ARG;
    rows[r] = LatentRowInfo{(int32_t)total_q, (int32_t)s, (int32_t)o, -1};
    if (kinds[r] == MIXATTN_ROW_TREE) {
      if (nq > kMaxTreeNodes) return MIXATTN_ERR_UNSUPPORTED;
      rows[r].tree_start = (int32_t)tree_nodes;
      tree_nodes += nq;
      T.trees = true;
      T.tree_words = std::max<int32_t>(T.tree_words, (int32_t)((nq + 31) / 32));
    }
    total_q += nq;
    if (total_q > (INT32_MAX - 64 * kMaxTeam) / heads) return MIXATTN_ERR_INVALID_ARG;
    most = std::max(most, nq * heads);
  }
  T.total_q = total_q;
  // (the widest row sets all rows' tiles: 64 decode rows of 1024 to 16384 tokens, 16 heads, take 117 us on the GPU, with
  // one more of 4000 119, and with a row of five drafted tokens in its place 127)
  T.tile_rows = most <= 16 ? 16 : (most <= 32 ? 32 : 64);
  auto tiles_of = [&](int r) { return ((int64_t)(seq[r] - off[r]) * heads + T.tile_rows - 1) / T.tile_rows; };
  // pages that the tiles mt0 .. mt1 - 1 of a row read, at most
  auto pages_of = [&](int r, int64_t mt1) {
    const int64_t last_f = std::min<int64_t>(mt1 * T.tile_rows, (int64_t)(seq[r] - off[r]) * heads) - 1;
    const int64_t last = kinds[r] == MIXATTN_ROW_TREE ? seq[r] - 1 : off[r] + last_f / heads;
    return last / kPage + 1;
  };

  // A team's CTAs take neighbouring tiles of the same keys side by side, so that each key comes from
  // HBM once; a row of more tiles is passed over several times.  The size that keeps the SMs
  // busiest; the larger of two that are as good.
  int64_t max_tiles = 1;
  for (int r = 0; r < n_rows; ++r) max_tiles = std::max(max_tiles, tiles_of(r));
  double best = 0.0;
  for (int t = 1; t <= std::min<int64_t>({max_tiles, kMaxTeam, n_sm}); ++t) {
    double cost = 0.0;
    for (int r = 0; r < n_rows; ++r) cost += (double)((tiles_of(r) + t - 1) / t) * ((seq[r] + kPage - 1) / kPage + kItemPages);
    cost /= n_sm / t;
    if (t == 1 || cost < best * 1.02) {
      T.team = t;
      best = t == 1 ? cost : std::min(best, cost);
    }
  }
  T.n_teams = std::max(1, n_sm / T.team);

  // The passes' pages in a line, cut into one run for each team: every team the same number of pages
  // (an item counts kItemPages more), no item shorter than min_item_pages unless its row is.
  std::vector<LatentItem> items;
  std::vector<int32_t> team_first(1, 0);
  std::vector<LatentCut> cuts;
  int64_t slots = 0;
  double total = 0.0;
  for (int r = 0; r < n_rows; ++r)
    for (int64_t mt0 = 0; mt0 < tiles_of(r); mt0 += T.team) total += (double)pages_of(r, mt0 + T.team) + kItemPages;
  const double share = (total + (double)kItemPages * T.n_teams) / T.n_teams;
  double used = 0.0;  // of all teams so far: what one took too much or too little, the next ones even out
  int team = 0;
  auto next_team = [&] {
    team_first.push_back((int32_t)items.size());
    ++team;
  };
  auto empty = [&] { return team_first.back() == (int32_t)items.size(); };
  for (int r = 0; r < n_rows; ++r) {
    const int64_t n_tiles = tiles_of(r);
    for (int64_t mt0 = 0; mt0 < n_tiles; mt0 += T.team) {
      const int64_t n_pages = pages_of(r, mt0 + T.team), least = min_item_pages(n_pages);
      const size_t first = items.size();
      int64_t at = 0;
      while (at < n_pages) {
        const int64_t left = n_pages - at;
        const bool last_team = team == T.n_teams - 1;
        int64_t take = left;
        if (!last_team) {
          const int64_t room = (int64_t)(share * (team + 1) - used - kItemPages + 0.5);
          if (room < least && !empty()) {
            next_team();
            continue;
          }
          take = std::max<int64_t>(least, room) & ~(int64_t)1;  // whole steps
          if (left - take < least) take = left;
        }
        if (items.size() > (size_t)1 << 24) return MIXATTN_ERR_INVALID_ARG;
        items.push_back(LatentItem{r, (int32_t)mt0, (int32_t)at, (int32_t)take, 0, 1, 0, 0});
        at += take;
        used += (double)(take + kItemPages);
        if (!last_team && used >= share * (team + 1) - 1.0) next_team();
      }
      const int32_t parts = (int32_t)(items.size() - first);
      if (parts > 1) {
        for (int32_t q = 0; q < parts; ++q) {
          items[first + q].part = q;
          items[first + q].n_parts = parts;
          items[first + q].slot = (int32_t)slots;
        }
        for (int64_t m = 0; m < T.team && mt0 + m < n_tiles; ++m)
          for (int32_t quarter = parts > kManyParts ? 0 : -1; quarter < (parts > kManyParts ? 4 : 0); ++quarter)
            cuts.push_back(LatentCut{(int64_t)rows[r].q_start * heads + (mt0 + m) * T.tile_rows,
                                     (int32_t)std::min<int64_t>(T.tile_rows, (int64_t)(seq[r] - off[r]) * heads -
                                                                                 (mt0 + m) * T.tile_rows),
                                     (int32_t)(slots + m * parts), parts, quarter});
        slots += (int64_t)parts * T.team;
        T.max_parts = std::max<int>(T.max_parts, parts);
        if (slots > INT32_MAX) return MIXATTN_ERR_INVALID_ARG;
      }
    }
  }
  while ((int)team_first.size() <= T.n_teams) team_first.push_back((int32_t)items.size());
  // teams without work are not launched
  while (T.n_teams > 1 && team_first[T.n_teams - 1] == (int32_t)items.size()) {
    team_first.pop_back();
    --T.n_teams;
  }
  if ((int64_t)cuts.size() * T.tile_rows > INT32_MAX || items.size() > (size_t)1 << 24) return MIXATTN_ERR_INVALID_ARG;
  T.n_cuts = (int)cuts.size();
  T.rows = T.image.add(rows);
  T.items = T.image.add(items);
  T.team_first = T.image.add(team_first);
  T.cuts = T.image.add(cuts);
  T.part_o = align_up(256 + T.image.bytes.size(), 256);
  T.part_ml = align_up(T.part_o + (size_t)slots * T.tile_rows * kLatent * sizeof(float), 256);
  T.total = align_up(T.part_ml + (size_t)slots * T.tile_rows * sizeof(float2), 256);
  return MIXATTN_OK;
}

// ===========================================================================
// Expanded form: the tiling
// ===========================================================================

struct ExpandedTiling {
  Image image;
  size_t items = 0, cta_first = 0, cuts = 0, part_o = 0, part_ml = 0, total = 0;
  int n_ctas = 1, n_cuts = 0;
  int64_t total_q = 0, total_k = 0;
};

// What an item costs beside its KV tiles (a KV tile of one group costs 1), and its least KV tiles
// where a tile is cut.  4096 queries, 32 heads, with a cost of 2 / 3 / 5: 168 / 174 / 175 us, eight prompts of up to
// 900, 16 heads 34.3 / 34.3 / 42.
constexpr int kExpandedItemCost = 2, kMinItemTiles = 4;

constexpr int kMaxExpandedHeads = 1 << 16;  // an output token's elements (128 a head) then count in 32 bits

// The tiles' KV tiles in a line -- neighbouring blocks of queries of one head read the same keys --
// cut into one run of equal cost for each SM.
int build_expanded_tiling(int heads, int n_rows, const int32_t* seq, const int32_t* off, int n_sm,
                          ExpandedTiling* out) {
  if (n_rows <= 0 || !seq || !off) return MIXATTN_ERR_INVALID_ARG;
  ExpandedTiling& T = *out;
  std::vector<ExpandedItem> items;
  std::vector<int32_t> cta_first(1, 0);
  std::vector<ExpandedCut> cuts;
  auto weight = [](int64_t count) { return count > 128 ? 2 : 1; };
  auto kv_tiles = [](int64_t keys) { return (keys + kChunkN - 1) / kChunkN; };
  double total = 0.0;
  int64_t n_tiles = 0;
  for (int r = 0; r < n_rows; ++r) {
    const int64_t s = seq[r], o = off[r];
    if (o < 0 || o >= s) return MIXATTN_ERR_INVALID_ARG;
    for (int64_t b = 0; b < s - o; b += kExpandedRows, n_tiles += heads) {
      const int64_t count = std::min<int64_t>(kExpandedRows, s - o - b);
      total += heads * ((double)kv_tiles(o + b + count) * weight(count) + kExpandedItemCost);
    }
    T.total_q += s - o;
    T.total_k += s;
    if (T.total_q > INT32_MAX / heads || T.total_k > INT32_MAX / 2) return MIXATTN_ERR_INVALID_ARG;
  }
  if (heads > kMaxExpandedHeads) return MIXATTN_ERR_UNSUPPORTED;
  if (n_tiles > 1 << 28) return MIXATTN_ERR_INVALID_ARG;
  const double share = total / n_sm + kExpandedItemCost;
  double used = 0.0;  // of all so far: what one took too much or too little, the next ones even out
  int cta = 0;
  auto next_cta = [&] {
    cta_first.push_back((int32_t)items.size());
    ++cta;
  };
  auto empty = [&] { return cta_first.back() == (int32_t)items.size(); };
  int64_t slots = 0, q0 = 0, k0 = 0;
  for (int r = 0; r < n_rows; ++r) {
    const int64_t s = seq[r], o = off[r];
    for (int h = 0; h < heads; ++h) {
      for (int64_t b = 0; b < s - o; b += kExpandedRows) {
        const int64_t count = std::min<int64_t>(kExpandedRows, s - o - b), n = kv_tiles(o + b + count);
        const int w = weight(count);
        const size_t first = items.size();
        int64_t at = 0;
        while (at < n) {
          const bool last = cta == n_sm - 1;
          int64_t take = n - at;
          if (!last) {
            const int64_t room = (int64_t)((share * (cta + 1) - used - kExpandedItemCost) / w + 0.5);
            if (room < std::min<int64_t>(kMinItemTiles, take) && !empty()) {
              next_cta();
              continue;
            }
            const int64_t cut = std::max<int64_t>(kMinItemTiles, room);
            if (take - cut >= kMinItemTiles) take = cut;
          }
          items.push_back(ExpandedItem{(int32_t)(q0 + b), (int32_t)k0, h, (int32_t)count, (int32_t)(o + b), (int32_t)s,
                                       (int32_t)at, (int32_t)(at + take), 0, 1, 0, 0});
          at += take;
          used += (double)(take * w + kExpandedItemCost);
          if (!last && used >= share * (cta + 1) - 1.0) next_cta();
        }
        const int32_t parts = (int32_t)(items.size() - first);
        if (parts > 1) {
          for (int32_t q = 0; q < parts; ++q) {
            items[first + q].part = q;
            items[first + q].n_parts = parts;
            items[first + q].slot = (int32_t)slots;
          }
          cuts.push_back(ExpandedCut{(int32_t)(q0 + b), h, (int32_t)count, (int32_t)slots, parts, 0});
          slots += parts;
        }
      }
    }
    q0 += s - o;
    k0 += s;
  }
  while ((int)cta_first.size() <= cta + 1) cta_first.push_back((int32_t)items.size());
  // A CTA's items by their first keys: those that share a head then walk its keys side by side, and most come
  // from L2 (2048 queries behind 8192, 32 heads, 311 -> 295 us; behind 30000, 16 heads, 484 -> 437).
  for (int c = 0; c <= cta; ++c)
    std::stable_sort(items.begin() + cta_first[c], items.begin() + cta_first[c + 1],
                     [](const ExpandedItem& a, const ExpandedItem& b) { return a.kv0 < b.kv0; });
  T.n_ctas = cta + 1;
  if (T.n_ctas > 1 && cta_first[T.n_ctas - 1] == (int32_t)items.size()) --T.n_ctas;
  T.n_cuts = (int)cuts.size();
  T.items = T.image.add(items);
  T.cta_first = T.image.add(cta_first);
  T.cuts = T.image.add(cuts);
  T.part_o = align_up(256 + T.image.bytes.size(), 256);
  T.part_ml = align_up(T.part_o + (size_t)slots * kExpandedRows * kExpandedV * sizeof(float), 256);
  T.total = align_up(T.part_ml + (size_t)slots * kExpandedRows * sizeof(float4), 256);
  return MIXATTN_OK;
}

// The list into a run's parameters, or (a longer one) on its way into the workspace.
int take_image(PlanList& list, const Image& image, uint8_t* ws, cudaStream_t s, PlanImage* out) {
  out->image = ws + 256;
  out->here = image.bytes.size() <= sizeof(out->list);
  if (!out->here) return list.upload(ws + 256, image.bytes.size(), s);
  memcpy(out->list, image.bytes.data(), image.bytes.size());
  return list.note_capture(s);
}

bool valid_scale(double s) { return s >= 1e-20 && s <= 1e6; }  // (false for NaN)

constexpr double kLog2e = 1.4426950408889634;

}  // namespace

}  // namespace mixattn

using namespace mixattn;

struct mixattn_latent_plan {
  mixattn_latent_cache cache;
  int32_t heads = 0, max_pages = 0;
  double scale = 0.0;
  LatentTiling tiling;
  PlanList list;
};

struct mixattn_expanded_plan {
  int32_t heads = 0;
  double scale = 0.0;
  ExpandedTiling tiling;
  PlanList list;
};

extern "C" {

size_t mixattn_latent_cache_bytes(const mixattn_latent_cache* c) {
  if (check_latent_dims(c) != MIXATTN_OK) return 0;
  return (size_t)c->num_pages * kPage * kLatentRow * 2;
}

int mixattn_latent_append(const mixattn_latent_cache* cache, const mixattn_rope* rope, int32_t num_heads,
                          const mixattn_heads* q, const mixattn_heads* q_out, const void* c_new, int64_t c_stride,
                          const void* k_rope, int64_t k_stride, const int32_t* positions, const int32_t* slot_mapping,
                          int32_t n_new, mixattn_stream stream) {
  int st = check_latent_cache(cache);
  if (st != MIXATTN_OK) return st;
  if (!rope || num_heads < 0 || n_new < 0) return MIXATTN_ERR_INVALID_ARG;
  if (rope->table.rot != kLatentRope) return MIXATTN_ERR_INVALID_ARG;
  if (num_heads > 1 << 16) return MIXATTN_ERR_UNSUPPORTED;
  if (n_new == 0) return MIXATTN_OK;
  if (!positions || !slot_mapping || !aligned(positions, 4) || !aligned(slot_mapping, 4))
    return MIXATTN_ERR_INVALID_ARG;
  if (!check_rows(c_new, c_stride, kLatent, n_new) || !check_rows(k_rope, k_stride, kLatentRope, n_new))
    return MIXATTN_ERR_INVALID_ARG;
  LatentAppendArgs a = {};
  if (num_heads > 0) {
    if (!check_heads(q, n_new, num_heads, kLatentRope) || !check_heads(q_out, n_new, num_heads, kLatentRope))
      return MIXATTN_ERR_INVALID_ARG;
    const uint8_t *qa = static_cast<const uint8_t*>(q->x), *oa = static_cast<const uint8_t*>(q_out->x);
    const bool same = qa == oa && (n_new == 1 || q->token_stride == q_out->token_stride) &&
                      (num_heads == 1 || q->head_stride == q_out->head_stride);
    const int64_t qn = heads_span(q, n_new, num_heads, kLatentRope), on = heads_span(q_out, n_new, num_heads, kLatentRope);
    if (!same && oa < qa + qn && qa < oa + on) return MIXATTN_ERR_INVALID_ARG;
    a.q = HeadRows{static_cast<const uint16_t*>(q->x), q->token_stride, q->head_stride};
    a.q_out = HeadRows{static_cast<const uint16_t*>(q_out->x), q_out->token_stride, q_out->head_stride};
  }
  if ((st = pending_device_check()) != MIXATTN_OK) return st;
  a.err = device_error_address();
  if (!a.err) return MIXATTN_ERR_CUDA;
  a.c = TokenRows{static_cast<const uint16_t*>(c_new), c_stride};
  a.r = TokenRows{static_cast<const uint16_t*>(k_rope), k_stride};
  a.data = static_cast<uint16_t*>(cache->data);
  a.positions = positions;
  a.slots = slot_mapping;
  a.heads = num_heads;
  a.num_slots = cache->num_pages * kPage;
  // As many tokens a CTA as give its threads their jobs, once every SM has four CTAs; a token of many heads
  // goes to several.
  const int64_t jobs = kLatent / 8 + kLatentRope / 16 * (1 + (int64_t)num_heads), cap = kAppendJobs * kAppendThreads;
  const int64_t fit = std::max<int64_t>(1, std::min<int64_t>(cap / jobs, kAppendTokens));
  a.n_tokens = n_new;
  a.per_cta = (int32_t)std::max<int64_t>(1, std::min<int64_t>(fit, n_new / (4 * sms_of_device())));
  const dim3 grid((unsigned)((n_new + a.per_cta - 1) / a.per_cta),
                  (unsigned)std::min<int64_t>((a.per_cta * jobs + cap - 1) / cap, 1024));
  latent_append_kernel<<<grid, kAppendThreads, 0, static_cast<cudaStream_t>(stream)>>>(rope->table, a);
  return cudaGetLastError() == cudaSuccess ? MIXATTN_OK : MIXATTN_ERR_CUDA;
}

int mixattn_latent_export(const mixattn_latent_cache* cache, const int32_t* slots, int32_t n, void* out,
                          mixattn_stream stream) {
  int st = check_latent_cache(cache);
  if (st != MIXATTN_OK) return st;
  if (n < 0) return MIXATTN_ERR_INVALID_ARG;
  if (n == 0) return MIXATTN_OK;
  if (!slots || !out || !aligned(slots, 4) || !aligned(out, 16)) return MIXATTN_ERR_INVALID_ARG;
  if ((st = pending_device_check()) != MIXATTN_OK) return st;
  unsigned int* err = device_error_address();
  if (!err) return MIXATTN_ERR_CUDA;
  latent_export_kernel<<<n, 96, 0, static_cast<cudaStream_t>(stream)>>>(
      static_cast<const uint16_t*>(cache->data), slots, cache->num_pages * kPage, static_cast<uint16_t*>(out), err);
  return cudaGetLastError() == cudaSuccess ? MIXATTN_OK : MIXATTN_ERR_CUDA;
}

int mixattn_latent_plan_create(mixattn_latent_plan** plan_out, const mixattn_latent_cache* cache, int32_t num_heads,
                               double softmax_scale, int32_t n_rows, const int32_t* row_kinds, const int32_t* seq_lens,
                               const int32_t* q_offsets, int32_t max_pages, size_t* workspace_bytes) {
  if (!plan_out) return MIXATTN_ERR_INVALID_ARG;
  *plan_out = nullptr;
  int st = check_latent_cache(cache);
  if (st != MIXATTN_OK) return st;
  if (num_heads <= 0 || !valid_scale(softmax_scale)) return MIXATTN_ERR_INVALID_ARG;
  if (num_heads > 128) return MIXATTN_ERR_UNSUPPORTED;
  mixattn_latent_plan* p = new (std::nothrow) mixattn_latent_plan();
  if (!p) return MIXATTN_ERR_CUDA;
  p->cache = *cache;
  p->heads = num_heads;
  p->scale = softmax_scale;
  st = mixattn_latent_plan_update(p, n_rows, row_kinds, seq_lens, q_offsets, max_pages, workspace_bytes);
  if (st != MIXATTN_OK) {
    delete p;
    return st;
  }
  arm_device_check();
  *plan_out = p;
  return MIXATTN_OK;
}

int mixattn_latent_plan_update(mixattn_latent_plan* plan, int32_t n_rows, const int32_t* row_kinds,
                               const int32_t* seq_lens, const int32_t* q_offsets, int32_t max_pages,
                               size_t* workspace_bytes) {
  if (!plan) return MIXATTN_ERR_INVALID_ARG;
  if (plan->list.captured()) return MIXATTN_ERR_UNSUPPORTED;
  try {
    LatentTiling t;
    int st = build_latent_tiling(plan->cache, plan->heads, n_rows, row_kinds, seq_lens, q_offsets, max_pages,
                                 sms_of_device(), &t);
    if (st != MIXATTN_OK) return st;
    if ((st = plan->list.fill(t.image.bytes)) != MIXATTN_OK) return st;
    plan->max_pages = max_pages;
    plan->tiling = std::move(t);
  } catch (const std::bad_alloc&) {
    return MIXATTN_ERR_CUDA;
  }
  if (workspace_bytes) *workspace_bytes = plan->tiling.total;
  return MIXATTN_OK;
}

int mixattn_latent_run(const mixattn_latent_plan* plan_c, const void* q, const int32_t* page_table,
                       const uint32_t* tree_mask, int32_t mask_words, void* o, void* workspace,
                       size_t workspace_bytes, mixattn_stream stream) {
  mixattn_latent_plan* plan = const_cast<mixattn_latent_plan*>(plan_c);
  if (!plan || !q || !o || !page_table) return MIXATTN_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(o, 16) || !aligned(page_table, 4)) return MIXATTN_ERR_INVALID_ARG;
  const LatentTiling& T = plan->tiling;
  if (T.trees && (!tree_mask || !aligned(tree_mask, 4) || mask_words < T.tree_words)) return MIXATTN_ERR_INVALID_ARG;
  if (!workspace || !aligned(workspace, 256) || workspace_bytes < T.total) return MIXATTN_ERR_WORKSPACE;
  if (int st = pending_device_check()) return st;
  unsigned int* err = device_error_address();
  if (!err) return MIXATTN_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  LatentParams p;
  if (int st = take_image(plan->list, T.image, ws, s, &p.list)) return st;
  p.rows = (int32_t)(T.rows - 256);
  p.items = (int32_t)(T.items - 256);
  p.team_first = (int32_t)(T.team_first - 256);
  p.cuts = (int32_t)(T.cuts - 256);
  p.q = static_cast<const uint16_t*>(q);
  p.data = static_cast<const uint16_t*>(plan->cache.data);
  p.page_table = page_table;
  p.tree_mask = tree_mask;
  p.o = static_cast<uint16_t*>(o);
  p.part_o = reinterpret_cast<float*>(ws + T.part_o);
  p.part_ml = reinterpret_cast<float2*>(ws + T.part_ml);
  p.tree_words = mask_words;
  p.max_pages = plan->max_pages;
  p.num_pages = plan->cache.num_pages;
  p.heads = plan->heads;
  p.team = T.team;
  p.n_teams = T.n_teams;
  p.n_cuts = T.n_cuts;
  p.max_parts = T.max_parts;
  p.scale_log2 = (float)(plan->scale * kLog2e);
  return launch_latent_attention(T.tile_rows, p, err, s) == cudaSuccess ? MIXATTN_OK : MIXATTN_ERR_CUDA;
}

void mixattn_latent_plan_destroy(mixattn_latent_plan* plan) { delete plan; }

int mixattn_expanded_plan_create(mixattn_expanded_plan** plan_out, int32_t num_heads, double softmax_scale,
                                 int32_t n_rows, const int32_t* seq_lens, const int32_t* q_offsets,
                                 size_t* workspace_bytes) {
  if (!plan_out) return MIXATTN_ERR_INVALID_ARG;
  *plan_out = nullptr;
  if (num_heads <= 0 || !valid_scale(softmax_scale)) return MIXATTN_ERR_INVALID_ARG;
  mixattn_expanded_plan* p = new (std::nothrow) mixattn_expanded_plan();
  if (!p) return MIXATTN_ERR_CUDA;
  p->heads = num_heads;
  p->scale = softmax_scale;
  const int st = mixattn_expanded_plan_update(p, n_rows, seq_lens, q_offsets, workspace_bytes);
  if (st != MIXATTN_OK) {
    delete p;
    return st;
  }
  arm_device_check();
  *plan_out = p;
  return MIXATTN_OK;
}

int mixattn_expanded_plan_update(mixattn_expanded_plan* plan, int32_t n_rows, const int32_t* seq_lens,
                                 const int32_t* q_offsets, size_t* workspace_bytes) {
  if (!plan) return MIXATTN_ERR_INVALID_ARG;
  if (plan->list.captured()) return MIXATTN_ERR_UNSUPPORTED;
  try {
    ExpandedTiling t;
    int st = build_expanded_tiling(plan->heads, n_rows, seq_lens, q_offsets, sms_of_device(), &t);
    if (st != MIXATTN_OK) return st;
    if ((st = plan->list.fill(t.image.bytes)) != MIXATTN_OK) return st;
    plan->tiling = std::move(t);
  } catch (const std::bad_alloc&) {
    return MIXATTN_ERR_CUDA;
  }
  if (workspace_bytes) *workspace_bytes = plan->tiling.total;
  return MIXATTN_OK;
}

int mixattn_expanded_run(const mixattn_expanded_plan* plan_c, const mixattn_heads* q, const mixattn_heads* k,
                         const void* k_rope, int64_t k_rope_stride, const mixattn_heads* v, void* o, void* workspace,
                         size_t workspace_bytes, mixattn_stream stream) {
  mixattn_expanded_plan* plan = const_cast<mixattn_expanded_plan*>(plan_c);
  if (!plan || !o || !aligned(o, 16)) return MIXATTN_ERR_INVALID_ARG;
  const ExpandedTiling& T = plan->tiling;
  const int h = plan->heads;
  if (!check_heads(q, T.total_q, h, kExpandedQ) || !check_heads(k, T.total_k, h, kNopeDim) ||
      !check_heads(v, T.total_k, h, kExpandedV) || !check_rows(k_rope, k_rope_stride, kLatentRope, T.total_k))
    return MIXATTN_ERR_INVALID_ARG;
  if (!workspace || !aligned(workspace, 256) || workspace_bytes < T.total) return MIXATTN_ERR_WORKSPACE;
  if (int st = pending_device_check()) return st;
  unsigned int* err = device_error_address();
  if (!err) return MIXATTN_ERR_CUDA;
  // (a stride of one token or head is never used; a map wants one all the same)
  auto head_map = [&](CUtensorMap* m, const mixattn_heads* x, int64_t n, int width, uint32_t rows) {
    const uint64_t dims[3] = {(uint64_t)width, (uint64_t)h, (uint64_t)n};
    const int64_t strides[2] = {h > 1 ? x->head_stride : width, n > 1 ? x->token_stride : width};
    const uint32_t box[3] = {64, 1, rows};
    return make_map(m, x->x, 3, dims, strides, box);
  };
  CUtensorMap q_map, k_map, kr_map, v_map;
  const uint64_t dims[2] = {kLatentRope, (uint64_t)T.total_k};
  const int64_t strides[1] = {T.total_k > 1 ? k_rope_stride : kLatentRope};
  const uint32_t box[2] = {64, 128};
  if (!head_map(&q_map, q, T.total_q, kExpandedQ, 128) || !head_map(&k_map, k, T.total_k, kNopeDim, 128) ||
      !head_map(&v_map, v, T.total_k, kExpandedV, 128) || !make_map(&kr_map, k_rope, 2, dims, strides, box))
    return MIXATTN_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  ExpandedParams p;
  if (int st = take_image(plan->list, T.image, ws, s, &p.list)) return st;
  p.items = (int32_t)(T.items - 256);
  p.cta_first = (int32_t)(T.cta_first - 256);
  p.cuts = (int32_t)(T.cuts - 256);
  p.o = static_cast<uint16_t*>(o);
  p.part_o = reinterpret_cast<float*>(ws + T.part_o);
  p.part_ml = reinterpret_cast<float4*>(ws + T.part_ml);
  p.heads = h;
  p.n_ctas = T.n_ctas;
  p.n_cuts = T.n_cuts;
  p.scale_log2 = (float)(plan->scale * kLog2e);
  return launch_expanded_attention(q_map, k_map, kr_map, v_map, p, err, s) == cudaSuccess ? MIXATTN_OK
                                                                                          : MIXATTN_ERR_CUDA;
}

void mixattn_expanded_plan_destroy(mixattn_expanded_plan* plan) { delete plan; }

}  // extern "C"
