// latent.h -- structures shared by the host planners and the kernels of the latent-cache
// operators (mixattn_latent.h).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include "../../include/mixattn_latent.h"
#include "internal.h"

namespace mixattn {

constexpr int kLatent = 512, kLatentRope = 64, kLatentRow = kLatent + kLatentRope;
constexpr int kNopeDim = 128, kExpandedV = 128, kExpandedQ = kNopeDim + kLatentRope;

// A plan's list as its kernels take it: all but the largest go with the launch itself, with no upload in front
// (a call among others: 32 rows of 500 to 2000 tokens, 16 heads, 24.4 -> 19.5 us, two rows of up to 300 14.4 -> 10.6; five
// prompts of up to 900, 8 heads, 26.9 -> 22.5, two of up to 2000, 32 heads, 83.1 -> 78.4; a session of 131072 tokens and
// 31 short rows, 128 heads, 123.1 -> 118.2: no call slower for the longer parameters).  500 decode rows pass it.
constexpr int kInlineBytes = 24576;  // (parameters may have 32764)

struct PlanImage {
  const uint8_t* image;  // the list in the workspace
  int32_t here;          // it is below, and not there
  uint4 list[kInlineBytes / 16];

#ifdef __CUDACC__
  template <class T>
  __device__ __forceinline__ const T* at(int32_t offset) const {
    return reinterpret_cast<const T*>((here ? reinterpret_cast<const uint8_t*>(list) : image) + offset);
  }
#endif
};

// ---------------------------------------------------------------------------
// Absorbed form
// ---------------------------------------------------------------------------

struct LatentRowInfo {
  int32_t q_start, seq_len, q_offset;
  int32_t tree_start;  // first mask row of a tree row, -1 of others
};

// Pages page0 .. + n_pages of a row for the tiles mt0 .. + team - 1 of its (query, head) rows,
// one for each CTA of a team.  A tile whose keys lie in several items (n_parts > 1) leaves
// partial results in slots: member m's part p in slot + m * n_parts + p.
struct LatentItem {
  int32_t row, mt0, page0, n_pages, part, n_parts, slot, pad;
};

// A tile whose parts are to be joined.
struct LatentCut {
  int64_t row0;  // first (query, head) row of the output
  int32_t rows, slot, n_parts;
  int32_t quarter;  // -1: all of each 128 elements; 0 .. 3: 32 of them (tiles of many parts, four entries each)
};

struct LatentParams {
  int32_t rows, items, team_first, cuts;  // offsets in the list: LatentRowInfo, LatentItem, int32 [n_teams + 1], LatentCut
  const uint16_t* q;          // [total_q][heads][576]
  const uint16_t* data;       // the cache
  const int32_t* page_table;
  const uint32_t* tree_mask;
  uint16_t* o;
  float* part_o;    // [slots][tile rows / 4 units of 128 elements by 16 rows][4][128][4 rows], unnormalised
  float2* part_ml;  // [slots][tile rows]: reference (a score before the scale) and sum
  int32_t tree_words, max_pages, num_pages, heads, team, n_teams, n_cuts, max_parts;
  float scale_log2;
  PlanImage list;
};

// tile_rows: 16, 32 or 64 (query, head) rows a CTA
cudaError_t launch_latent_attention(int tile_rows, const LatentParams& p, unsigned int* err, cudaStream_t s);

// ---------------------------------------------------------------------------
// Expanded form
// ---------------------------------------------------------------------------

constexpr int kExpandedRows = 256;  // queries of a tile: two groups of 128

// KV tiles (128 keys) kv0 .. kv1 - 1 of one head's queries q_start .. + count; a tile whose keys
// lie in several items (n_parts > 1) leaves partial results in slots slot + part.
struct ExpandedItem {
  int32_t q_start, k_start;  // packed first query of the tile, packed first key of its row
  int32_t head, count;
  int32_t pos, seq_len;      // position of the first query; keys of the row
  int32_t kv0, kv1, part, n_parts, slot, pad;
};

struct ExpandedCut {
  int32_t q_start, head, count, slot, n_parts, pad;
};

struct ExpandedParams {
  int32_t items, cta_first, cuts;  // offsets in the list: ExpandedItem, int32 [n_ctas + 1], ExpandedCut
  uint16_t* o;
  float* part_o;    // [slots][256][128], unnormalised
  float4* part_ml;  // [slots][256]: reference (a score or 0, and bits above it) and sum
  int32_t heads, n_ctas, n_cuts;
  float scale_log2;
  PlanImage list;
};

cudaError_t launch_expanded_attention(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& kr,
                                      const CUtensorMap& v, const ExpandedParams& p, unsigned int* err, cudaStream_t s);

}  // namespace mixattn
