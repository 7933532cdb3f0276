// Internal interface between the host-side checks of the norm and the clipping
// (hyb_clip_api.cpp) and their kernels (hyb_clip.hip).
#pragma once

#include <vector>

#include "../../include/hyb_clip.h"
#include "hyb_internal.h"

namespace hyb {

// Elements of a chunk: a workgroup's unit of work, within one row.
constexpr int64_t kClipChunk = 16384;
// Tensors of one launch (their table is a kernel argument, at most 4 KiB).
constexpr int kClipTensors = 64;
// Workgroups of one launch, at most.
constexpr int64_t kClipGroups = 2048;

// One launch: tensors first .. first + count - 1, its workgroups, and the
// first of its sums in the workspace.
struct ClipLaunch {
  int64_t first;
  int count;
  int64_t chunks, groups, sum0;
};
// The launches over the tensors, which all have elements; *sums is the number of
// partial sums.
std::vector<ClipLaunch> clip_plan(const std::vector<hyb_tensor>& tensors, int64_t* sums);

hipError_t launch_norm(const std::vector<hyb_tensor>& tensors, float* norm, double* ws, hipStream_t s);
hipError_t launch_clip(const std::vector<hyb_tensor>& tensors, float max_norm, float* norm, double* ws, hipStream_t s);

}  // namespace hyb
