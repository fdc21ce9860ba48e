// plan_list.h -- what the plans of every kind share on the host: the tile list in a pinned,
// mapped buffer, its upload into a run's workspace, and the device checks.
#pragma once

#include <cuda_runtime.h>

#include <mutex>
#include <vector>

#include "internal.h"

// A rotary table (mixattn_rope_create).
struct mixattn_rope {
  double freq[mixattn::kMaxRotPairs] = {};
  double mscale = 1.0;
  mixattn::RopeTable table{};
};

namespace mixattn {

class PlanList {
 public:
  PlanList() = default;
  PlanList(const PlanList&) = delete;
  PlanList& operator=(const PlanList&) = delete;
  ~PlanList();

  // Replaces the list; waits until every run so far, on whatever stream, has copied the old one.
  int fill(const std::vector<uint8_t>& image);
  // Enqueues the copy of the list's first `bytes` (a multiple of 16) to `dst`.
  int upload(uint8_t* dst, size_t bytes, cudaStream_t s);
  // For a run that takes the list otherwise: only notes that it is captured, if it is.
  int note_capture(cudaStream_t s);
  // Some run was captured: replays read the pinned buffer at any time, so it keeps its list.
  bool captured() const { return captured_; }

 private:
  uint8_t* buf_ = nullptr;
  const uint8_t* dev_ = nullptr;  // the same buffer as the device sees it
  size_t cap_ = 0, size_ = 0;
  // The last copy on each stream that has made one since the list was filled; of more streams than
  // there are places, one waits for another's copy and stands for both.
  struct Copy {
    cudaEvent_t event = nullptr;
    int device = 0;
    unsigned long long stream = 0;
    bool recorded = false;
  };
  int note_copy(cudaStream_t s);
  bool wait_for_copies();
  static constexpr int kStreams = 8;
  Copy copies_[kStreams];
  std::mutex mu_;  // (host threads may run one plan at once)
  bool captured_ = false;
};

// Arms the device-check flag of the current device (once).
void arm_device_check();
// MIXATTN_ERR_DEVICE_CHECK when a kernel on the current device has set an error bit since the last clear.
int pending_device_check();
// Address of the current device's error word (NULL when it cannot be had).
unsigned int* device_error_address();

}  // namespace mixattn
