// plan_list.h -- what the plans of every kind share on the host: the tile list in a pinned,
// mapped buffer, its upload into a run's workspace, and the device checks.
#pragma once

#include <cuda_runtime.h>

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

  // Replaces the list; waits until the previous run has copied the old one.
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
  cudaEvent_t copied_ = nullptr;
  bool copy_recorded_ = false;
  bool captured_ = false;
};

// Arms the device-check flag of the current device (once).
void arm_device_check();
// MIXATTN_ERR_DEVICE_CHECK when a kernel on the current device has set an error bit since the last clear.
int pending_device_check();
// Address of the current device's error word (NULL when it cannot be had).
unsigned int* device_error_address();

}  // namespace mixattn
