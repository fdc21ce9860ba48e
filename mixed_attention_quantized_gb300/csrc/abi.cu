// abi.cu -- host side of the C ABI: validation, the ForwardBatch planner and
// the launches.  See include/mixattn.h for the contract of every entry point.
//
// Page "自研RDNA高併發推論引擎 以AI Max+ 395為範例": §1 (chunk rows and decode
// rows share one ForwardBatch and one attention kernel; a prompt is fed one
// bounded chunk per round) and §2 (blocked Q8 / 4-bit KV modes).
#include <cuda_runtime.h>
#include <stdlib.h>
#include <string.h>

#include <algorithm>
#include <cmath>
#include <functional>
#include <mutex>
#include <new>
#include <queue>
#include <vector>

#include "../../include/mixattn_sched.h"
#include "internal.h"
#include "plan_list.h"

namespace mixattn {

// Per device: word 0 = OR of MIXATTN_DEVERR_* bits set by kernels; words 2-3 =
// device address of the host-mapped flag that kernels also set (0 until armed).
__device__ __align__(16) unsigned int g_device_error[4] = {0u, 0u, 0u, 0u};

namespace {

std::mutex g_err_mu;
unsigned int* g_err_word[kMaxDevices] = {};          // device address of g_device_error
volatile unsigned int* g_err_flag[kMaxDevices] = {};  // host view of the armed flag

// Address of this device's error block (kernels receive it as an argument).
unsigned int* error_word() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return nullptr;
  std::lock_guard<std::mutex> lock(g_err_mu);
  if (!g_err_word[dev]) {
    void* p = nullptr;
    if (cudaGetSymbolAddress(&p, g_device_error) != cudaSuccess) return nullptr;
    g_err_word[dev] = static_cast<unsigned int*>(p);
  }
  return g_err_word[dev];
}

}  // namespace

// Arms the host-mapped flag of the current device (once): a pinned, mapped
// word whose device address is stored in the error block, so kernels that set
// an error bit also set the flag and the next call sees it without touching
// the device.  The copy runs on a private non-blocking stream in relaxed
// capture mode, so it neither waits for nor disturbs the caller's streams.
// Failure leaves the device unarmed (calls then cannot report earlier checks,
// mixattn_device_error still can).
void arm_device_check() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return;
  if (!error_word()) return;
  std::lock_guard<std::mutex> lock(g_err_mu);
  if (g_err_flag[dev]) return;
  cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;
  if (cudaThreadExchangeStreamCaptureMode(&mode) != cudaSuccess) return;
  unsigned int* host = nullptr;
  void* dptr = nullptr;
  cudaStream_t st = nullptr;
  bool ok = cudaHostAlloc(reinterpret_cast<void**>(&host), 64, cudaHostAllocMapped | cudaHostAllocPortable) ==
            cudaSuccess;
  if (ok) {
    host[0] = 0u;
    reinterpret_cast<void**>(host)[1] = nullptr;
    ok = cudaHostGetDevicePointer(&dptr, host, 0) == cudaSuccess && dptr;
  }
  if (ok) {
    reinterpret_cast<void**>(host)[1] = dptr;  // the value copied into words 2-3
    ok = cudaStreamCreateWithFlags(&st, cudaStreamNonBlocking) == cudaSuccess;
  }
  if (ok) {
    ok = cudaMemcpyToSymbolAsync(g_device_error, reinterpret_cast<void**>(host) + 1, sizeof(void*),
                                 2 * sizeof(unsigned int), cudaMemcpyHostToDevice, st) == cudaSuccess &&
         cudaStreamSynchronize(st) == cudaSuccess;
  }
  if (st) cudaStreamDestroy(st);
  if (ok) {
    g_err_flag[dev] = host;
  } else {
    if (host) cudaFreeHost(host);
    cudaGetLastError();  // nothing of this is the caller's error
  }
  cudaThreadExchangeStreamCaptureMode(&mode);
}

// MIXATTN_ERR_DEVICE_CHECK when a kernel on the current device has set an error
// bit since the last clear (seen through the armed flag), else MIXATTN_OK.
int pending_device_check() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return MIXATTN_OK;
  volatile unsigned int* f = g_err_flag[dev];
  return (f && *f) ? MIXATTN_ERR_DEVICE_CHECK : MIXATTN_OK;
}

namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

bool valid_fmt(int f) {
  return f == MIXATTN_KV_F16 || f == MIXATTN_KV_Q8_0 || f == MIXATTN_KV_Q4_0 || page_scaled(f);
}

// Dimensions and formats only (no pointers).
int check_cache_dims(const mixattn_kv_cache* c) {
  if (!c) return MIXATTN_ERR_INVALID_ARG;
  if (c->num_pages <= 0 || c->num_kv_heads <= 0 || c->head_dim <= 0) return MIXATTN_ERR_INVALID_ARG;
  if (c->page_size != kPage) return MIXATTN_ERR_UNSUPPORTED;
  if (c->head_dim % kBlock != 0) return MIXATTN_ERR_INVALID_ARG;
  if (c->head_dim != 64 && c->head_dim != 128) return MIXATTN_ERR_UNSUPPORTED;
  if (!valid_fmt(c->k_fmt) || !valid_fmt(c->v_fmt)) return MIXATTN_ERR_INVALID_ARG;
  const bool kf = c->k_fmt == MIXATTN_KV_F16, vf = c->v_fmt == MIXATTN_KV_F16;
  if (kf != vf) return MIXATTN_ERR_UNSUPPORTED;  // fp16 pairs only with fp16
  // a page-scaled format pairs only with itself
  if ((page_scaled(c->k_fmt) || page_scaled(c->v_fmt)) && c->k_fmt != c->v_fmt) return MIXATTN_ERR_UNSUPPORTED;
  if ((int64_t)c->num_pages * kPage > INT32_MAX) return MIXATTN_ERR_INVALID_ARG;
  return MIXATTN_OK;
}

int check_cache(const mixattn_kv_cache* c) {
  int st = check_cache_dims(c);
  if (st != MIXATTN_OK) return st;
  if (!c->k_quant || !c->v_quant) return MIXATTN_ERR_INVALID_ARG;
  if (!aligned(c->k_quant, 256) || !aligned(c->v_quant, 256)) return MIXATTN_ERR_INVALID_ARG;
  if (c->k_fmt != MIXATTN_KV_F16 && (!c->k_scale || !aligned(c->k_scale, 256))) return MIXATTN_ERR_INVALID_ARG;
  if (c->v_fmt != MIXATTN_KV_F16 && (!c->v_scale || !aligned(c->v_scale, 256))) return MIXATTN_ERR_INVALID_ARG;
  return MIXATTN_OK;
}

cudaError_t dispatch_attention(int k_fmt, int v_fmt, int head_dim, const AttnParams& p, unsigned int* err,
                               cudaStream_t s) {
  if (p.tree_starts) {
    if (k_fmt == MIXATTN_KV_I8_PAGE) return launch_tree_attention_i8_page(head_dim, p, err, s);
    if (k_fmt == MIXATTN_KV_E4M3_PAGE) return launch_tree_attention_e4m3_page(head_dim, p, err, s);
    if (k_fmt == MIXATTN_KV_F16) return launch_tree_attention_f16_f16(head_dim, p, err, s);
    if (k_fmt == MIXATTN_KV_Q8_0 && v_fmt == MIXATTN_KV_Q8_0) return launch_tree_attention_q8_q8(head_dim, p, err, s);
    if (k_fmt == MIXATTN_KV_Q4_0 && v_fmt == MIXATTN_KV_Q4_0) return launch_tree_attention_q4_q4(head_dim, p, err, s);
    if (k_fmt == MIXATTN_KV_Q8_0) return launch_tree_attention_q8_q4(head_dim, p, err, s);
    return launch_tree_attention_q4_q8(head_dim, p, err, s);
  }
  if (k_fmt == MIXATTN_KV_I8_PAGE) return launch_attention_i8_page(head_dim, p, err, s);
  if (k_fmt == MIXATTN_KV_E4M3_PAGE) return launch_attention_e4m3_page(head_dim, p, err, s);
  if (k_fmt == MIXATTN_KV_F16) return launch_attention_f16_f16(head_dim, p, err, s);
  if (k_fmt == MIXATTN_KV_Q8_0 && v_fmt == MIXATTN_KV_Q8_0) return launch_attention_q8_q8(head_dim, p, err, s);
  if (k_fmt == MIXATTN_KV_Q4_0 && v_fmt == MIXATTN_KV_Q4_0) return launch_attention_q4_q4(head_dim, p, err, s);
  if (k_fmt == MIXATTN_KV_Q8_0) return launch_attention_q8_q4(head_dim, p, err, s);
  return launch_attention_q4_q8(head_dim, p, err, s);
}

// The tiling of one batch: the image uploaded to the workspace plus counts.
struct Tiling {
  std::vector<uint8_t> image;  // [rows | tiles | counters], from WorkspaceLayout::rows
  int32_t total_q = 0, n_chunk = 0, n_decode = 0;
  int32_t slot_rows = 0;       // rows of a decode partial slot
  int32_t chunk_kv_tiles = 0;  // KV tiles over all chunk tiles (their mean decides persistence)
  int64_t chunk_kv_halves = 0; // the same, a tile of more than 128 rows counted twice
  int32_t decode_pages = 0;    // pages over all decode tiles
  bool trees = false;          // any tree row
  int32_t tree_words = 0;      // mask words that the largest of them needs
  WorkspaceLayout L{};
};

// SMs of the current device (0 when it cannot be read: no chunk splitting).
int device_sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
  return n;
}

// Pieces per chunk tile of one chunk row: the key range of each of the row's
// tiles is cut into s pieces (s = 1..most) when that shortens the row's share of
// the launch, judged by placing the pieces heaviest first on the least-loaded
// of n_sm SMs (one chunk CTA per SM).  A piece costs its KV tiles plus one for
// its prologue and the merge; rows with a tile shorter than 8 KV tiles are
// never cut.
int chunk_split_factor(const std::vector<int64_t>& costs, int n_sm, int most) {
  if (n_sm <= 0 || costs.empty()) return 1;
  int64_t min_cost = costs[0];
  for (int64_t c : costs) min_cost = std::min(min_cost, c);
  if (min_cost < 8) return 1;
  auto makespan = [&](int s) {
    std::vector<int64_t> pieces;
    pieces.reserve(costs.size() * s);
    for (int64_t c : costs)
      for (int q = 0; q < s; ++q) pieces.push_back((c * (q + 1)) / s - (c * q) / s + (s > 1 ? 1 : 0));
    std::sort(pieces.begin(), pieces.end(), std::greater<int64_t>());
    std::priority_queue<int64_t, std::vector<int64_t>, std::greater<int64_t>> load;
    for (int i = 0; i < n_sm; ++i) load.push(0);
    int64_t span = 0;
    for (int64_t pc : pieces) {
      const int64_t l = load.top() + pc;
      load.pop();
      load.push(l);
      span = std::max(span, l);
    }
    return span;
  };
  int best = 1;
  int64_t best_span = makespan(1);
  for (int s = 2; s <= most; ++s) {
    const int64_t sp = makespan(s);
    if (sp * 20 < best_span * 19) {  // at least 5% shorter
      best = s;
      best_span = sp;
    }
  }
  return best;
}

int build_tiling(const mixattn_kv_cache& c, int hq, int n_rows, const int32_t* kinds, const int32_t* seq,
                 const int32_t* off, int max_pages, int n_sm, int window, Tiling* out) {
  if (n_rows <= 0 || !kinds || !seq || !off || max_pages <= 0 || window < 0) return MIXATTN_ERR_INVALID_ARG;
  if (hq <= 0 || hq % c.num_kv_heads != 0) return MIXATTN_ERR_INVALID_ARG;
  const int G = hq / c.num_kv_heads;
  if (G != 1 && G != 2 && G != 4 && G != 8) return MIXATTN_ERR_UNSUPPORTED;
  const int hkv = c.num_kv_heads;
  const int T = chunk_rows(c.k_fmt) / G;  // query tokens per chunk tile
  const int QPG = kMaxGroup / G;  // queries per decode-style tile of a verify row
  bool any_verify = false, any_tree = false;
  int64_t tree_nodes = 0, tree_words = 0;

  std::vector<RowInfo> rows(n_rows);
  std::vector<int32_t> tree_starts(n_rows, -1);
  struct Chunk {
    TileDesc t;
    int64_t kv_first;  // first KV tile the tile's queries can see
    int64_t cost;      // KV tiles from there to the last query's key
    int split;
  };
  std::vector<Chunk> chunks;
  std::vector<TileDesc> decodes;
  int64_t total_q = 0;
  for (int r = 0; r < n_rows; ++r) {
    const int64_t s = seq[r], o = off[r];
    if (kinds[r] == MIXATTN_ROW_DECODE) {
      if (s < 1 || o != s - 1) return MIXATTN_ERR_INVALID_ARG;
    } else if (kinds[r] == MIXATTN_ROW_CHUNK) {
      if (o < 0 || o >= s) return MIXATTN_ERR_INVALID_ARG;
    } else if (kinds[r] == MIXATTN_ROW_TREE) {
      if (o < 0 || o >= s) return MIXATTN_ERR_INVALID_ARG;
      // (the drafted tokens of a path then lie within one window)
      if (s - o > kMaxTreeNodes || (window > 0 && s - o > window)) return MIXATTN_ERR_UNSUPPORTED;
      any_tree = true;
      tree_starts[r] = (int32_t)tree_nodes;
      tree_nodes += s - o;
      tree_words = std::max<int64_t>(tree_words, (s - o + 31) / 32);
    } else {
      return MIXATTN_ERR_INVALID_ARG;
    }
    const bool tree = kinds[r] == MIXATTN_ROW_TREE;
    const int64_t n_pages = (s + kPage - 1) / kPage;
    if (n_pages > max_pages) return MIXATTN_ERR_INVALID_ARG;
    if (n_pages > c.num_pages) return MIXATTN_ERR_INVALID_ARG;
    rows[r].q_start = (int32_t)total_q;
    rows[r].seq_len = (int32_t)s;
    rows[r].q_offset = (int32_t)o;
    rows[r].n_splits = 0;
    const int64_t nq = s - o;
    // a short chunk row (speculative verify: q_len * G <= kVerifyMaxRows) runs like decode
    // rows, on split-K tiles of up to 8 (query, head) rows
    const bool verify = kinds[r] != MIXATTN_ROW_DECODE && nq * G <= kVerifyMaxRows;
    any_verify = any_verify || verify;
    if (kinds[r] != MIXATTN_ROW_DECODE && !verify) {
      const size_t first_chunk = chunks.size();
      for (int g = 0; g < hkv; ++g) {
        for (int64_t b = 0; b < nq; b += T) {
          Chunk ch;
          ch.t.row = r;
          ch.t.kvh = g;
          ch.t.begin = (int32_t)b;
          ch.t.count = (int32_t)std::min<int64_t>(T, nq - b);
          ch.t.kv0 = ch.t.kv1 = ch.t.part = 0;
          ch.t.nsplit = 1;
          // (a tree's tokens may see any other of the row, and sit at any depth)
          const int64_t key_end = tree ? s : std::min<int64_t>(s, o + b + ch.t.count);
          // a sliding window skips the KV tiles before the first query's first key
          ch.kv_first = window_first_key((int)(tree ? o : o + b), window) / kChunkN;
          ch.cost = (key_end + kChunkN - 1) / kChunkN - ch.kv_first;
          ch.split = 1;
          chunks.push_back(ch);
        }
      }
      // how far to cut this row's tiles depends on the row alone (and the GPU), so
      // a row's result does not depend on the rest of the batch
      std::vector<int64_t> costs;
      for (size_t i = first_chunk; i < chunks.size(); ++i) costs.push_back(chunks[i].cost);
      const int split = chunk_split_factor(costs, n_sm, page_scaled(c.k_fmt) ? kPageMaxPieces : 4);
      for (size_t i = first_chunk; i < chunks.size(); ++i) chunks[i].split = split;
    } else {
      // pages from the one holding the first query's window start (page 0 without a
      // window) to the last; the split size depends on the row alone
      const int64_t first_page = window_first_key((int)o, window) / kPage;
      const int64_t n_win = n_pages - first_page;
      const int pps =
          page_scaled(c.k_fmt) ? page_decode_pages_per_split((int)n_win) : decode_pages_per_split((int)n_win);
      const int ns = (int)((n_win + pps - 1) / pps);
      rows[r].n_splits = ns;
      // query groups innermost: the groups reading the same pages sit side by side in
      // the tile list (and so run at about the same time), and the pages they share
      // come from L2 after the first read; slots are numbered group-major
      const int64_t n_groups = (nq + QPG - 1) / QPG;
      for (int g = 0; g < hkv; ++g) {
        const int32_t base = (int32_t)decodes.size();
        for (int sp = 0; sp < ns; ++sp) {
          for (int64_t gi = 0; gi < n_groups; ++gi) {
            TileDesc t;
            t.row = r;
            t.kvh = g;
            t.begin = (int32_t)(first_page + (int64_t)sp * pps);
            t.count = (int32_t)std::min<int64_t>(pps, n_win - (int64_t)sp * pps);
            t.kv0 = base + (int32_t)(gi * ns);                            // partial slot of split 0
            t.kv1 = (int32_t)(gi * QPG);                                  // the group's first query
            t.part = sp;
            t.nsplit = (int32_t)std::min<int64_t>(QPG, nq - gi * QPG);  // the group's queries
            decodes.push_back(t);
          }
        }
      }
    }
    total_q += nq;
    if (total_q > INT32_MAX / std::max(hq, 1)) return MIXATTN_ERR_INVALID_ARG;
  }
  // heaviest chunk tiles first (they set the length of the launch), each cut
  // into `split` consecutive pieces of its key range; longest decode tiles first
  // too, so the last wave holds the short ones (each keeps its partial slot)
  std::stable_sort(chunks.begin(), chunks.end(), [](const Chunk& a, const Chunk& b) { return a.cost > b.cost; });
  std::stable_sort(decodes.begin(), decodes.end(),
                   [](const TileDesc& a, const TileDesc& b) { return a.count > b.count; });
  int64_t n_pieces = 0;
  bool any_split = false;
  for (const Chunk& ch : chunks) {
    n_pieces += ch.split;
    any_split = any_split || ch.split > 1;
  }
  const int64_t n_tiles = n_pieces + (int64_t)decodes.size();
  if (n_tiles > INT32_MAX / 2) return MIXATTN_ERR_INVALID_ARG;

  Tiling& T2 = *out;
  T2.total_q = (int32_t)total_q;
  T2.n_chunk = (int32_t)n_pieces;
  T2.n_decode = (int32_t)decodes.size();
  T2.slot_rows = any_verify ? kMaxGroup : G;
  T2.L = workspace_layout(n_rows, (int)n_tiles, T2.n_decode, T2.slot_rows, c.head_dim, any_split,
                          chunk_rows(c.k_fmt), any_tree);
  T2.trees = any_tree;
  T2.tree_words = (int32_t)tree_words;
  T2.image.assign(T2.L.upload_end - T2.L.rows, 0);
  memcpy(T2.image.data(), rows.data(), sizeof(RowInfo) * rows.size());
  TileDesc* td = reinterpret_cast<TileDesc*>(T2.image.data() + (T2.L.tiles - T2.L.rows));
  int64_t at = 0, kv_tiles = 0;
  T2.chunk_kv_halves = 0;
  for (size_t i = 0; i < chunks.size(); ++i) {
    const int64_t n_kv = chunks[i].cost, kv_first = chunks[i].kv_first;
    kv_tiles += n_kv;
    T2.chunk_kv_halves += n_kv * (chunks[i].t.count * G > 128 ? 2 : 1);
    const int split = chunks[i].split;
    for (int q = 0; q < split; ++q) {
      TileDesc t = chunks[i].t;
      t.kv0 = (int32_t)(kv_first + (n_kv * q) / split);
      t.kv1 = (int32_t)(kv_first + (n_kv * (q + 1)) / split);
      t.part = q;
      t.nsplit = split;
      td[at++] = t;
    }
  }
  for (size_t i = 0; i < decodes.size(); ++i) td[n_pieces + i] = decodes[i];
  T2.chunk_kv_tiles = (int32_t)std::min<int64_t>(kv_tiles, INT32_MAX);
  int64_t decode_pages = 0;
  for (const TileDesc& t : decodes) decode_pages += t.count;
  T2.decode_pages = (int32_t)std::min<int64_t>(decode_pages, INT32_MAX);
  if (any_tree)
    memcpy(T2.image.data() + (T2.L.tree_starts - T2.L.rows), tree_starts.data(), sizeof(int32_t) * n_rows);
  // counters stay zero: every run starts its split tickets from 0
  return MIXATTN_OK;
}

}  // namespace

// Copies n16 16-byte words of a plan's tile list from its mapped pinned buffer
// into the workspace.
static __global__ void upload_kernel(const uint4* __restrict__ src, uint4* __restrict__ dst, size_t n16) {
  // an attention kernel launched to overlap this one may start setting up (it waits for
  // this grid's end before it reads the list)
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  for (size_t i = blockIdx.x * (size_t)blockDim.x + threadIdx.x; i < n16; i += (size_t)gridDim.x * blockDim.x)
    dst[i] = src[i];
}

int PlanList::fill(const std::vector<uint8_t>& image) {
  // runs before this may still be copying from the pinned buffer
  if (!wait_for_copies()) return MIXATTN_ERR_CUDA;
  if (image.size() > cap_) {
    if (buf_) cudaFreeHost(buf_);
    buf_ = nullptr;
    dev_ = nullptr;
    cap_ = size_ = 0;
    const size_t cap = std::max<size_t>(image.size(), 4096);
    if (cudaHostAlloc(reinterpret_cast<void**>(&buf_), cap, cudaHostAllocMapped | cudaHostAllocPortable) !=
        cudaSuccess) {
      buf_ = nullptr;
      return MIXATTN_ERR_CUDA;
    }
    void* dv = nullptr;
    if (cudaHostGetDevicePointer(&dv, buf_, 0) != cudaSuccess || !dv) {
      cudaFreeHost(buf_);
      buf_ = nullptr;
      return MIXATTN_ERR_CUDA;
    }
    dev_ = static_cast<const uint8_t*>(dv);
    cap_ = cap;
  }
  memcpy(buf_, image.data(), image.size());
  size_ = image.size();
  return MIXATTN_OK;
}

// The tile list comes in through a small kernel reading the mapped pinned buffer
// rather than a copy-engine transfer, which would queue behind any large
// host-to-device copy the caller has in flight on another stream.
int PlanList::upload(uint8_t* dst, size_t bytes, cudaStream_t s) {
  if (!dev_ || bytes > size_) return MIXATTN_ERR_INVALID_ARG;  // (an update that failed left no list)
  const size_t n16 = bytes / 16;
  const int blocks = (int)std::min<size_t>((n16 + 255) / 256, 128);
  upload_kernel<<<blocks, 256, 0, s>>>(reinterpret_cast<const uint4*>(dev_), reinterpret_cast<uint4*>(dst), n16);
  if (cudaGetLastError() != cudaSuccess) return MIXATTN_ERR_CUDA;
  // a captured run replays whenever its graph does, so no event can tell when the buffer
  // is free: the plan then keeps its tile list (an event recorded into the graph would
  // also fail every later wait for it)
  cudaStreamCaptureStatus capture = cudaStreamCaptureStatusNone;
  if (cudaStreamIsCapturing(s, &capture) != cudaSuccess) return MIXATTN_ERR_CUDA;
  if (capture != cudaStreamCaptureStatusNone) {
    captured_ = true;
    return MIXATTN_OK;
  }
  return note_copy(s);
}

int PlanList::note_copy(cudaStream_t s) {
  int dev = 0;
  unsigned long long id = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaStreamGetId(s, &id) != cudaSuccess) return MIXATTN_ERR_CUDA;
  std::lock_guard<std::mutex> lock(mu_);
  Copy* c = nullptr;
  for (Copy& x : copies_)
    if (x.event && x.device == dev && x.stream == id) c = &x;
  for (Copy& x : copies_) {  // (an event belongs to the device it was made on)
    if (c) break;
    if (!x.event) {
      if (cudaEventCreateWithFlags(&x.event, cudaEventDisableTiming) != cudaSuccess) {
        x.event = nullptr;
        return MIXATTN_ERR_CUDA;
      }
      x.device = dev;
    }
    if (!x.recorded && x.device == dev) c = &x;
  }
  for (Copy& x : copies_) {
    if (c) break;
    if (x.device != dev) continue;
    if (cudaStreamWaitEvent(s, x.event, 0) != cudaSuccess) return MIXATTN_ERR_CUDA;
    c = &x;
  }
  if (!c)  // every place is another device's: nothing to note once it is done
    return cudaStreamSynchronize(s) == cudaSuccess ? MIXATTN_OK : MIXATTN_ERR_CUDA;
  if (cudaEventRecord(c->event, s) != cudaSuccess) return MIXATTN_ERR_CUDA;
  c->stream = id;
  c->recorded = true;
  return MIXATTN_OK;
}

bool PlanList::wait_for_copies() {
  std::lock_guard<std::mutex> lock(mu_);
  for (Copy& x : copies_) {
    if (x.recorded && cudaEventSynchronize(x.event) != cudaSuccess) return false;
    x.recorded = false;
  }
  return true;
}

int PlanList::note_capture(cudaStream_t s) {
  cudaStreamCaptureStatus capture = cudaStreamCaptureStatusNone;
  if (cudaStreamIsCapturing(s, &capture) != cudaSuccess) return MIXATTN_ERR_CUDA;
  if (capture != cudaStreamCaptureStatusNone) captured_ = true;
  return MIXATTN_OK;
}

PlanList::~PlanList() {
  wait_for_copies();
  for (Copy& x : copies_)
    if (x.event) cudaEventDestroy(x.event);
  if (buf_) cudaFreeHost(buf_);
}

// Address of this device's error word, for launchers in other translation units.
unsigned int* device_error_address() { return error_word(); }

}  // namespace mixattn

using namespace mixattn;

struct mixattn_plan {
  mixattn_kv_cache cache;
  int32_t hq = 0, group = 0, log2_group = 0, n_rows = 0, max_pages = 0;
  int32_t window = 0;  // sliding window of every run of the plan (0: full causal attention)
  Tiling tiling;
  PlanList list;       // pinned, mapped copy of tiling.image
};

namespace {

// Tokens' heads in device memory: 16-byte aligned rows of `width` elements every `stride`.
bool check_token_rows(const void* x, int64_t stride, int64_t width) {
  return x && aligned(x, 16) && stride >= width && stride % 8 == 0 && stride <= INT64_MAX / 4 / INT32_MAX;
}

// In place, or rows that share nothing (decided where both strides are equal; one
// token has no stride).
bool check_rotate_overlap(const void* x, int64_t xs, const void* out, int64_t os, int64_t width, int64_t n) {
  if (x == out && (xs == os || n == 1)) return true;
  if (x == out) return false;
  if (xs != os && n > 1) return true;
  const int64_t xa = (int64_t)reinterpret_cast<uintptr_t>(x), oa = (int64_t)reinterpret_cast<uintptr_t>(out);
  const int64_t step = 2 * xs, w = 2 * width, span = (n - 1) * step + w;
  if (oa >= xa + span || xa >= oa + span) return true;
  if (n == 1) return false;
  const int64_t m = ((oa - xa) % step + step) % step;  // where out's rows start between x's
  return m >= w && m + w <= step;
}

int plan_fill(mixattn_plan* p, int32_t n_rows, const int32_t* kinds, const int32_t* seq, const int32_t* off,
              int32_t max_pages, size_t* ws_bytes) {
  if (p->list.captured()) return MIXATTN_ERR_UNSUPPORTED;
  Tiling t;
  int st = build_tiling(p->cache, p->hq, n_rows, kinds, seq, off, max_pages, device_sm_count(), p->window, &t);
  if (st != MIXATTN_OK) return st;
  if ((st = p->list.fill(t.image)) != MIXATTN_OK) return st;
  p->n_rows = n_rows;
  p->max_pages = max_pages;
  p->tiling = std::move(t);
  if (ws_bytes) *ws_bytes = p->tiling.L.total;
  return MIXATTN_OK;
}

}  // namespace

extern "C" {

size_t mixattn_kv_cache_bytes(const mixattn_kv_cache* c, size_t plane_bytes_out[4]) {
  if (check_cache_dims(c) != MIXATTN_OK) return 0;
  const size_t rows = (size_t)c->num_pages * c->num_kv_heads * kPage;
  const size_t kq = rows * quant_row_bytes(c->k_fmt, c->head_dim);
  const size_t pages = (size_t)c->num_pages * c->num_kv_heads;
  const size_t ks = pages * scale_page_bytes(c->k_fmt, c->head_dim);
  const size_t vq = rows * quant_row_bytes(c->v_fmt, c->head_dim);
  const size_t vs = pages * scale_page_bytes(c->v_fmt, c->head_dim);
  if (plane_bytes_out) {
    plane_bytes_out[0] = kq;
    plane_bytes_out[1] = ks;
    plane_bytes_out[2] = vq;
    plane_bytes_out[3] = vs;
  }
  return kq + ks + vq + vs;
}

int mixattn_kv_append_quant(const mixattn_kv_cache* cache, const void* k_new, const void* v_new,
                            const int32_t* slot_mapping, int32_t n_new, mixattn_stream stream) {
  int st = check_cache(cache);
  if (st != MIXATTN_OK) return st;
  if (n_new < 0) return MIXATTN_ERR_INVALID_ARG;
  if (n_new == 0) return MIXATTN_OK;
  if (!k_new || !v_new || !slot_mapping) return MIXATTN_ERR_INVALID_ARG;
  if (!aligned(k_new, 16) || !aligned(v_new, 16) || !aligned(slot_mapping, 4)) return MIXATTN_ERR_INVALID_ARG;
  if ((st = pending_device_check()) != MIXATTN_OK) return st;
  unsigned int* err = error_word();
  if (!err) return MIXATTN_ERR_CUDA;
  cudaError_t e;
  if (page_scaled(cache->k_fmt)) {
    const int64_t stride = (int64_t)cache->num_kv_heads * cache->head_dim;
    e = launch_page_append(*cache, nullptr, 0, TokenRows{nullptr, 0}, nullptr, 0,
                           TokenRows{static_cast<const uint16_t*>(k_new), stride},
                           TokenRows{static_cast<const uint16_t*>(v_new), stride}, nullptr, slot_mapping, n_new, err,
                           static_cast<cudaStream_t>(stream));
  } else {
    e = launch_kv_append(*cache, k_new, v_new, slot_mapping, n_new, err, static_cast<cudaStream_t>(stream));
  }
  return e == cudaSuccess ? MIXATTN_OK : MIXATTN_ERR_CUDA;
}

int mixattn_rope_create(mixattn_rope** rope_out, const mixattn_rope_config* cfg) {
  if (!rope_out) return MIXATTN_ERR_INVALID_ARG;
  *rope_out = nullptr;
  if (!cfg || cfg->rot_dim <= 0 || cfg->rot_dim > 2 * kMaxRotPairs) return MIXATTN_ERR_INVALID_ARG;
  if (cfg->rot_dim % 16 != 0) return MIXATTN_ERR_UNSUPPORTED;
  if (cfg->layout != MIXATTN_ROPE_HALF && cfg->layout != MIXATTN_ROPE_INTERLEAVED) return MIXATTN_ERR_INVALID_ARG;
  auto finite = [](double x) { return std::isfinite(x); };
  if (!finite(cfg->base) || cfg->base <= 1.0) return MIXATTN_ERR_INVALID_ARG;
  if (!finite(cfg->mscale) || cfg->mscale < 0.0 || cfg->mscale > 1e4) return MIXATTN_ERR_INVALID_ARG;
  const int sc = cfg->scaling;
  if (sc < MIXATTN_ROPE_SCALE_NONE || sc > MIXATTN_ROPE_SCALE_BANDS) return MIXATTN_ERR_INVALID_ARG;
  if (sc != MIXATTN_ROPE_SCALE_NONE && (!finite(cfg->factor) || cfg->factor < 1e-6)) return MIXATTN_ERR_INVALID_ARG;
  if (sc == MIXATTN_ROPE_SCALE_RAMP && cfg->factor < 1.0) return MIXATTN_ERR_INVALID_ARG;
  if (sc == MIXATTN_ROPE_SCALE_RAMP || sc == MIXATTN_ROPE_SCALE_BANDS) {
    if (cfg->original_ctx <= 0 || !finite(cfg->low) || !finite(cfg->high) || cfg->low <= 0.0 || cfg->high <= cfg->low)
      return MIXATTN_ERR_INVALID_ARG;
  }
  mixattn_rope* r = new (std::nothrow) mixattn_rope();
  if (!r) return MIXATTN_ERR_CUDA;
  const int rot = cfg->rot_dim, pairs = rot / 2;
  const double two_pi = 6.283185307179586476925;
  double m = 1.0, lo = 0.0, hi = 0.0;
  if (sc == MIXATTN_ROPE_SCALE_RAMP) {
    // the pair whose wavelength fits `turns` times into the trained context
    auto pair_of = [&](double turns) {
      return rot * std::log(cfg->original_ctx / (turns * two_pi)) / (2.0 * std::log(cfg->base));
    };
    lo = std::max(std::floor(pair_of(cfg->high)), 0.0);
    hi = std::min(std::ceil(pair_of(cfg->low)), (double)(rot - 1));
    m = 0.1 * std::log(cfg->factor) + 1.0;
  }
  for (int i = 0; i < pairs; ++i) {
    double f = std::pow(cfg->base, -2.0 * i / rot);
    if (sc == MIXATTN_ROPE_SCALE_LINEAR) {
      f /= cfg->factor;
    } else if (sc == MIXATTN_ROPE_SCALE_RAMP) {
      const double t = std::min(1.0, std::max(0.0, (i - lo) / std::max(hi - lo, 1e-3)));
      f = f * (1.0 - t) + f / cfg->factor * t;
    } else if (sc == MIXATTN_ROPE_SCALE_BANDS) {
      const double turns = cfg->original_ctx * f / two_pi;
      const double t = std::min(1.0, std::max(0.0, (turns - cfg->low) / (cfg->high - cfg->low)));
      f = f * t + f / cfg->factor * (1.0 - t);
    }
    r->freq[i] = f;
    const double turn = f / two_pi - std::floor(f / two_pi);  // [0, 1): whole turns change nothing
    const double fixed = std::ldexp(turn, 64);  // < 2^64; an integer from 2^52 on
    r->table.turn[i] = (uint64_t)(fixed < 4503599627370496.0 ? std::floor(fixed + 0.5) : fixed);
  }
  r->mscale = cfg->mscale > 0.0 ? cfg->mscale : m;
  r->table.mscale = (float)r->mscale;
  r->table.mscale_rest = (float)(r->mscale - (double)r->table.mscale);
  r->table.rot = rot;
  r->table.layout = cfg->layout;
  *rope_out = r;
  return MIXATTN_OK;
}

void mixattn_rope_destroy(mixattn_rope* rope) { delete rope; }

int mixattn_rope_info(const mixattn_rope* rope, int32_t* rot_dim, double* frequencies, double* mscale) {
  if (!rope) return MIXATTN_ERR_INVALID_ARG;
  if (rot_dim) *rot_dim = rope->table.rot;
  if (frequencies) memcpy(frequencies, rope->freq, sizeof(double) * (rope->table.rot / 2));
  if (mscale) *mscale = rope->mscale;
  return MIXATTN_OK;
}

int mixattn_rope_apply(const mixattn_rope* rope, const void* x, int64_t x_stride, void* out, int64_t out_stride,
                       const int32_t* positions, int32_t n_tokens, int32_t n_heads, int32_t head_dim,
                       mixattn_stream stream) {
  if (!rope || n_tokens < 0 || n_heads <= 0) return MIXATTN_ERR_INVALID_ARG;
  if (head_dim != 64 && head_dim != 128) return MIXATTN_ERR_UNSUPPORTED;
  if (rope->table.rot > head_dim) return MIXATTN_ERR_INVALID_ARG;
  if (n_tokens == 0) return MIXATTN_OK;
  const int64_t width = (int64_t)n_heads * head_dim;
  if (!positions || !aligned(positions, 4)) return MIXATTN_ERR_INVALID_ARG;
  if (!check_token_rows(x, x_stride, width) || !check_token_rows(out, out_stride, width) ||
      !check_rotate_overlap(x, x_stride, out, out_stride, width, n_tokens))
    return MIXATTN_ERR_INVALID_ARG;
  cudaError_t e = launch_rope(rope->table, TokenRows{static_cast<const uint16_t*>(x), x_stride},
                              static_cast<uint16_t*>(out), out_stride, positions, n_tokens, n_heads, head_dim,
                              static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? MIXATTN_OK : MIXATTN_ERR_CUDA;
}

int mixattn_rope_append(const mixattn_kv_cache* cache, const mixattn_rope* rope, int32_t num_q_heads, const void* q,
                        int64_t q_stride, void* q_out, int64_t q_out_stride, const void* k_new, int64_t k_stride,
                        const void* v_new, int64_t v_stride, const int32_t* positions, const int32_t* slot_mapping,
                        int32_t n_new, mixattn_stream stream) {
  int st = check_cache(cache);
  if (st != MIXATTN_OK) return st;
  if (!rope || n_new < 0 || num_q_heads < 0) return MIXATTN_ERR_INVALID_ARG;
  if (rope->table.rot > cache->head_dim) return MIXATTN_ERR_INVALID_ARG;
  if (n_new == 0) return MIXATTN_OK;
  const int64_t kw = (int64_t)cache->num_kv_heads * cache->head_dim, qw = (int64_t)num_q_heads * cache->head_dim;
  if (!positions || !slot_mapping || !aligned(positions, 4) || !aligned(slot_mapping, 4))
    return MIXATTN_ERR_INVALID_ARG;
  if (!check_token_rows(k_new, k_stride, kw) || !check_token_rows(v_new, v_stride, kw)) return MIXATTN_ERR_INVALID_ARG;
  if (num_q_heads > 0 && (!check_token_rows(q, q_stride, qw) || !check_token_rows(q_out, q_out_stride, qw) ||
                          !check_rotate_overlap(q, q_stride, q_out, q_out_stride, qw, n_new)))
    return MIXATTN_ERR_INVALID_ARG;
  if ((st = pending_device_check()) != MIXATTN_OK) return st;
  unsigned int* err = error_word();
  if (!err) return MIXATTN_ERR_CUDA;
  const TokenRows qr{static_cast<const uint16_t*>(q), q_stride}, kr{static_cast<const uint16_t*>(k_new), k_stride},
      vr{static_cast<const uint16_t*>(v_new), v_stride};
  uint16_t* qo = static_cast<uint16_t*>(q_out);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = page_scaled(cache->k_fmt)
                      ? launch_page_append(*cache, &rope->table, num_q_heads, qr, qo, q_out_stride, kr, vr, positions,
                                           slot_mapping, n_new, err, s)
                      : launch_rope_append(*cache, rope->table, num_q_heads, qr, qo, q_out_stride, kr, vr, positions,
                                           slot_mapping, n_new, err, s);
  return e == cudaSuccess ? MIXATTN_OK : MIXATTN_ERR_CUDA;
}

int mixattn_kv_export_blocks(const mixattn_kv_cache* cache, int32_t which, const int32_t* slots, int32_t n,
                             void* out, mixattn_stream stream) {
  int st = check_cache(cache);
  if (st != MIXATTN_OK) return st;
  if ((which != 0 && which != 1) || n < 0) return MIXATTN_ERR_INVALID_ARG;
  if (n == 0) return MIXATTN_OK;
  if (!slots || !out || !aligned(slots, 4)) return MIXATTN_ERR_INVALID_ARG;
  if ((st = pending_device_check()) != MIXATTN_OK) return st;
  unsigned int* err = error_word();
  if (!err) return MIXATTN_ERR_CUDA;
  cudaError_t e = launch_kv_export(*cache, which, slots, n, out, err, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? MIXATTN_OK : MIXATTN_ERR_CUDA;
}

int mixattn_plan_create(mixattn_plan** plan_out, const mixattn_kv_cache* cache, int32_t num_q_heads,
                        int32_t n_rows, const int32_t* row_kinds, const int32_t* seq_lens,
                        const int32_t* q_offsets, int32_t max_pages, size_t* workspace_bytes) {
  return mixattn_plan_create_window(plan_out, cache, num_q_heads, 0, n_rows, row_kinds, seq_lens, q_offsets,
                                    max_pages, workspace_bytes);
}

int mixattn_plan_create_window(mixattn_plan** plan_out, const mixattn_kv_cache* cache, int32_t num_q_heads,
                               int32_t window, int32_t n_rows, const int32_t* row_kinds, const int32_t* seq_lens,
                               const int32_t* q_offsets, int32_t max_pages, size_t* workspace_bytes) {
  if (!plan_out) return MIXATTN_ERR_INVALID_ARG;
  *plan_out = nullptr;
  int st = check_cache(cache);
  if (st != MIXATTN_OK) return st;
  if (num_q_heads <= 0 || num_q_heads % cache->num_kv_heads) return MIXATTN_ERR_INVALID_ARG;
  if (window < 0) return MIXATTN_ERR_INVALID_ARG;
  arm_device_check();
  mixattn_plan* p = new mixattn_plan();
  p->cache = *cache;
  p->window = window;
  p->hq = num_q_heads;
  p->group = num_q_heads / cache->num_kv_heads;
  p->log2_group = 0;
  while ((1 << p->log2_group) < p->group) ++p->log2_group;
  st = plan_fill(p, n_rows, row_kinds, seq_lens, q_offsets, max_pages, workspace_bytes);
  if (st != MIXATTN_OK) {
    mixattn_plan_destroy(p);
    return st;
  }
  *plan_out = p;
  return MIXATTN_OK;
}

int mixattn_plan_update(mixattn_plan* plan, int32_t n_rows, const int32_t* row_kinds, const int32_t* seq_lens,
                        const int32_t* q_offsets, int32_t max_pages, size_t* workspace_bytes) {
  if (!plan) return MIXATTN_ERR_INVALID_ARG;
  return plan_fill(plan, n_rows, row_kinds, seq_lens, q_offsets, max_pages, workspace_bytes);
}

int mixattn_plan_info(const mixattn_plan* plan, int32_t* total_q, int32_t* n_chunk_tiles,
                      int32_t* n_decode_tiles) {
  if (!plan) return MIXATTN_ERR_INVALID_ARG;
  if (total_q) *total_q = plan->tiling.total_q;
  if (n_chunk_tiles) *n_chunk_tiles = plan->tiling.n_chunk;
  if (n_decode_tiles) *n_decode_tiles = plan->tiling.n_decode;
  return MIXATTN_OK;
}

int mixattn_run(const mixattn_plan* plan, const void* q, const int32_t* page_table, void* o, void* workspace,
                size_t workspace_bytes, mixattn_stream stream) {
  return mixattn_run_tree(plan, q, page_table, nullptr, 0, o, workspace, workspace_bytes, stream);
}

int mixattn_run_tree(const mixattn_plan* plan_c, const void* q, const int32_t* page_table, const uint32_t* tree_mask,
                     int32_t mask_words, void* o, void* workspace, size_t workspace_bytes, mixattn_stream stream) {
  mixattn_plan* plan = const_cast<mixattn_plan*>(plan_c);
  if (!plan) return MIXATTN_ERR_INVALID_ARG;
  if (!q || !o || !page_table) return MIXATTN_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(o, 16) || !aligned(page_table, 4)) return MIXATTN_ERR_INVALID_ARG;
  const bool trees = plan->tiling.trees;
  if (trees && (!tree_mask || !aligned(tree_mask, 4) || mask_words < plan->tiling.tree_words))
    return MIXATTN_ERR_INVALID_ARG;
  const WorkspaceLayout& L = plan->tiling.L;
  if (!workspace || !aligned(workspace, 256) || workspace_bytes < L.total) return MIXATTN_ERR_WORKSPACE;
  if (int st = pending_device_check()) return st;
  unsigned int* err = error_word();
  if (!err) return MIXATTN_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  if (int st = plan->list.upload(ws + L.rows, L.upload_end - L.rows, s)) return st;

  AttnParams p;
  const mixattn_kv_cache& c = plan->cache;
  p.q = q;
  p.o = o;
  p.k_quant = static_cast<const uint8_t*>(c.k_quant);
  p.k_scale = static_cast<const uint16_t*>(c.k_scale);
  p.v_quant = static_cast<const uint8_t*>(c.v_quant);
  p.v_scale = static_cast<const uint16_t*>(c.v_scale);
  p.page_table = page_table;
  p.rows = reinterpret_cast<const RowInfo*>(ws + L.rows);
  p.tiles = reinterpret_cast<const TileDesc*>(ws + L.tiles);
  p.counters = reinterpret_cast<uint32_t*>(ws + L.counters);
  p.partials = reinterpret_cast<float*>(ws + L.partials);
  p.chunk_partials = reinterpret_cast<float*>(ws + L.chunk_partials);
  p.chunk_counters = p.counters + plan->tiling.n_decode;
  p.max_pages = plan->max_pages;
  p.num_pages = c.num_pages;
  p.n_chunk_tiles = plan->tiling.n_chunk;
  p.chunk_kv_tiles = plan->tiling.chunk_kv_tiles;
  p.chunk_kv_halves = (int32_t)std::min<int64_t>(plan->tiling.chunk_kv_halves, INT32_MAX);
  p.n_decode_tiles = plan->tiling.n_decode;
  p.decode_pages = plan->tiling.decode_pages;
  p.hq = plan->hq;
  p.hkv = c.num_kv_heads;
  p.group = plan->group;
  p.log2_group = plan->log2_group;
  p.scale_log2 = (float)(1.4426950408889634 / std::sqrt((double)c.head_dim));
  p.window = plan->window;
  p.slot_rows = plan->tiling.slot_rows;
  if (trees) {
    p.tree_starts = reinterpret_cast<const int32_t*>(ws + L.tree_starts);
    p.tree_mask = tree_mask;
    p.tree_words = mask_words;
  }
  cudaError_t e = dispatch_attention(c.k_fmt, c.v_fmt, c.head_dim, p, err, s);
  return e == cudaSuccess ? MIXATTN_OK : MIXATTN_ERR_CUDA;
}

void mixattn_plan_destroy(mixattn_plan* plan) { delete plan; }

int mixattn_workspace_bytes(const mixattn_kv_cache* cache, int32_t num_q_heads, int32_t n_rows,
                            const int32_t* row_kinds, const int32_t* seq_lens, const int32_t* q_offsets,
                            int32_t max_pages, size_t* workspace_bytes) {
  int st = check_cache_dims(cache);
  if (st != MIXATTN_OK) return st;
  if (!workspace_bytes) return MIXATTN_ERR_INVALID_ARG;
  Tiling t;
  st = build_tiling(*cache, num_q_heads, n_rows, row_kinds, seq_lens, q_offsets, max_pages, device_sm_count(), 0,
                    &t);
  if (st != MIXATTN_OK) return st;
  *workspace_bytes = t.L.total;
  return MIXATTN_OK;
}

int mixattn_mixed_attention(const mixattn_kv_cache* cache, int32_t num_q_heads, const void* q,
                            const int32_t* page_table, int32_t max_pages, int32_t n_rows, const int32_t* seq_lens,
                            const int32_t* q_offsets, const int32_t* row_kinds, void* o, void* workspace,
                            size_t workspace_bytes, mixattn_stream stream) {
  // a replay would read the tile list of the plan that this call frees
  cudaStreamCaptureStatus capture = cudaStreamCaptureStatusNone;
  if (cudaStreamIsCapturing(static_cast<cudaStream_t>(stream), &capture) != cudaSuccess)
    cudaGetLastError();  // (the launch below reports what is wrong)
  else if (capture != cudaStreamCaptureStatusNone)
    return MIXATTN_ERR_UNSUPPORTED;
  mixattn_plan* plan = nullptr;
  int st = mixattn_plan_create(&plan, cache, num_q_heads, n_rows, row_kinds, seq_lens, q_offsets, max_pages,
                               nullptr);
  if (st != MIXATTN_OK) return st;
  st = mixattn_run(plan, q, page_table, o, workspace, workspace_bytes, stream);
  mixattn_plan_destroy(plan);  // waits for the tile-list copy only
  return st;
}

int64_t mixattn_device_error(int32_t clear) {
  unsigned int v = 0;
  if (cudaMemcpyFromSymbol(&v, g_device_error, sizeof(v)) != cudaSuccess) return MIXATTN_ERR_CUDA;
  if (clear) {
    const unsigned int z = 0;
    if (cudaMemcpyToSymbol(g_device_error, &z, sizeof(z)) != cudaSuccess) return MIXATTN_ERR_CUDA;
    int dev = 0;
    if (cudaGetDevice(&dev) == cudaSuccess && dev >= 0 && dev < kMaxDevices && g_err_flag[dev])
      *g_err_flag[dev] = 0u;
  }
  return (int64_t)v;
}

const char* mixattn_status_string(int32_t status) {
  switch (status) {
    case MIXATTN_OK: return "ok";
    case MIXATTN_ERR_INVALID_ARG: return "invalid argument";
    case MIXATTN_ERR_UNSUPPORTED: return "unsupported configuration";
    case MIXATTN_ERR_WORKSPACE: return "workspace missing, misaligned or too small";
    case MIXATTN_ERR_CUDA: return "CUDA runtime error";
    case MIXATTN_ERR_DEVICE_CHECK: return "device-side check failed";
    case MIXATTN_ERR_CLIENT_QUOTA: return "client quota: too many requests waiting for this client";
    default: return "unknown status";
  }
}

int32_t mixattn_version(void) { return 100; }

}  // extern "C"
