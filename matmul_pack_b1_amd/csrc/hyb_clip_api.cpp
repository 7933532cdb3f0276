// Host side of the norm and the clipping (include/hyb_clip.h): argument checks
// and planning, then the launches.
#include <algorithm>
#include <exception>

#include "hyb_clip_internal.h"

namespace hyb {

std::vector<ClipLaunch> clip_plan(const std::vector<hyb_tensor>& tensors, int64_t* sums) {
  std::vector<ClipLaunch> plan;
  *sums = 0;
  for (size_t i = 0; i < tensors.size(); i += kClipTensors) {
    ClipLaunch l{int64_t(i), int(std::min<size_t>(kClipTensors, tensors.size() - i)), 0, 0, *sums};
    for (int j = 0; j < l.count; ++j) {
      const hyb_tensor& t = tensors[i + j];
      l.chunks += t.rows * ((t.cols + kClipChunk - 1) / kClipChunk);
    }
    l.groups = std::min(l.chunks, kClipGroups);
    *sums += l.groups;
    plan.push_back(l);
  }
  return plan;
}

}  // namespace hyb

namespace {

using hyb::fail;
using hyb::ok;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

int elem_size(int32_t dt) { return dt == HYB_F32 ? 4 : 2; }

struct Range {
  uintptr_t from, to;
};

// First and last byte of rows x cols elements with row stride ld.
Range range_of(const void* p, const hyb_tensor& t, int64_t ld) {
  const uintptr_t at = reinterpret_cast<uintptr_t>(p);
  return Range{at, at + uintptr_t(((t.rows - 1) * ld + t.cols) * elem_size(t.dtype))};
}

bool cross(const Range& a, const Range& b) { return a.from < b.to && b.from < a.to; }

// May rows of `cols` elements lie `ld` apart, and their addresses within 64 bits?
bool reach(int64_t rows, int64_t cols, int64_t ld) {
  return ld >= cols && ld <= (int64_t(1) << 40) && ld <= (int64_t(1) << 44) / (rows - 1);
}

// Checks the list and keeps the tensors that have elements, rows joined where
// they are contiguous.  Without `data` (sizes are asked for, of a norm or of a
// scaling) an `ldo` that no call could take counts as lda.
hyb_status read_list(int64_t count, const hyb_tensor* list, bool data, bool out, std::vector<hyb_tensor>* kept) {
  if (count < 0) return fail(HYB_ERR_SHAPE, "count = %lld is negative", (long long)count);
  if (count > 0 && !list) return fail(HYB_ERR_INVALID_ARG, "tensors is NULL");
  for (int64_t i = 0; i < count; ++i) {
    hyb_tensor t = list[i];
    if (t.dtype != HYB_F16 && t.dtype != HYB_BF16 && t.dtype != HYB_F32)
      return fail(HYB_ERR_DTYPE, "tensor %lld: dtype %d is not HYB_F16, HYB_BF16 or HYB_F32", (long long)i, t.dtype);
    if (t.rows < 0 || t.cols < 0 || t.rows > (int64_t(1) << 40) || t.cols > (int64_t(1) << 40) ||
        (t.rows > 0 && t.cols > (int64_t(1) << 40) / t.rows))
      return fail(HYB_ERR_SHAPE, "tensor %lld is %lld x %lld: need 0 <= rows, cols and at most 2^40 elements",
                  (long long)i, (long long)t.rows, (long long)t.cols);
    if (t.rows == 0 || t.cols == 0) continue;
    if (!data && t.rows > 1 && !reach(t.rows, t.cols, t.ldo)) t.ldo = t.lda;
    const int64_t most = int64_t(1) << 40;
    for (const int64_t ld : {t.lda, out ? t.ldo : t.lda})
      if (t.rows > 1 && (ld < t.cols || ld > most))
        return fail(HYB_ERR_INVALID_ARG, "tensor %lld: row stride %lld outside [%lld, 2^40]", (long long)i, (long long)ld,
                    (long long)t.cols);
      else if (t.rows > 1 && ld > (int64_t(1) << 44) / (t.rows - 1))  // (addresses stay within 64 bits)
        return fail(HYB_ERR_INVALID_ARG, "tensor %lld: %lld rows of stride %lld reach over 2^44 elements", (long long)i,
                    (long long)t.rows, (long long)ld);
    if (data && (!t.data || !aligned(t.data, elem_size(t.dtype))))
      return fail(HYB_ERR_INVALID_ARG, "tensor %lld: data is NULL or not aligned to its element", (long long)i);
    if (data && out && (!t.out || !aligned(t.out, elem_size(t.dtype))))
      return fail(HYB_ERR_INVALID_ARG, "tensor %lld: out is NULL or not aligned to its element", (long long)i);
    if (t.rows > 1 && t.lda == t.cols && (!out || t.ldo == t.cols)) {
      t.cols *= t.rows;
      t.rows = 1;
    }
    if (t.rows == 1) t.lda = t.ldo = t.cols;
    kept->push_back(t);
  }
  return HYB_OK;
}

// Outputs overlap nothing but, exactly, their own data.
hyb_status check_overlap(const std::vector<hyb_tensor>& list, const float* norm) {
  struct Item {
    Range r;
    size_t i;
    bool out;
  };
  std::vector<Item> items;
  for (size_t i = 0; i < list.size(); ++i) {
    const hyb_tensor& t = list[i];
    items.push_back({range_of(t.out, t, t.ldo), i, true});
    if (t.out != t.data)
      items.push_back({range_of(t.data, t, t.lda), i, false});
    else if (t.rows > 1 && t.lda != t.ldo)
      return fail(HYB_ERR_INVALID_ARG, "a tensor in place has two row strides");
  }
  const uintptr_t at = reinterpret_cast<uintptr_t>(norm);
  items.push_back({Range{at, at + 4}, list.size(), true});
  std::sort(items.begin(), items.end(), [](const Item& a, const Item& b) { return a.r.from < b.r.from; });
  // the reach of the inputs and of the outputs so far
  uintptr_t in = 0, out = 0;
  for (const Item& it : items) {
    if (it.r.from < out || (it.out && it.r.from < in))
      return fail(HYB_ERR_INVALID_ARG, "an output overlaps another tensor or the norm");
    uintptr_t& reach = it.out ? out : in;
    reach = std::max(reach, it.r.to);
  }
  return HYB_OK;
}

hyb_status check_ws(const void* ws, size_t bytes, size_t need) {
  if (bytes < need) return fail(HYB_ERR_INVALID_ARG, "workspace_bytes = %zu, this call needs %zu", bytes, need);
  if (need > 0 && (!ws || !aligned(ws, 16)))
    return fail(HYB_ERR_INVALID_ARG, "workspace is NULL or not 16-byte aligned");
  return HYB_OK;
}

// One call; `clip` false: the norm alone.
hyb_status run(int64_t count, const hyb_tensor* tensors, bool clip, float max_norm, float* norm, void* workspace,
               size_t workspace_bytes, void* stream) {
  std::vector<hyb_tensor> list;
  hyb_status st = read_list(count, tensors, true, clip, &list);
  if (st != HYB_OK) return st;
  if (!norm || !aligned(norm, 4)) return fail(HYB_ERR_INVALID_ARG, "norm is NULL or not 4-byte aligned");
  if (clip && !(max_norm >= 0.f)) return fail(HYB_ERR_INVALID_ARG, "max_norm must be 0 or more");
  if (clip && (st = check_overlap(list, norm)) != HYB_OK) return st;
  if (!clip) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(norm);
    for (const hyb_tensor& t : list)
      if (cross(range_of(t.data, t, t.lda), Range{at, at + 4}))
        return fail(HYB_ERR_INVALID_ARG, "norm overlaps a tensor");
  }
  int64_t sums;
  (void)hyb::clip_plan(list, &sums);
  if ((st = check_ws(workspace, workspace_bytes, size_t(sums) * 8)) != HYB_OK) return st;
  double* ws = static_cast<double*>(workspace);
  hipStream_t s = static_cast<hipStream_t>(stream);
  return hyb::hip_status(clip ? hyb::launch_clip(list, max_norm, norm, ws, s) : hyb::launch_norm(list, norm, ws, s),
                         clip ? "clip launch" : "norm launch");
}

// Host memory may run out on a long list: no exception leaves a C entry.
template <typename F>
hyb_status guarded(F f) {
  try {
    return f();
  } catch (const std::exception&) {
    return fail(HYB_ERR_INVALID_ARG, "out of host memory");
  }
}

}  // namespace

extern "C" {

hyb_status hyb_clip_workspace_size(int64_t count, const hyb_tensor* tensors, size_t* bytes) {
  return guarded([&] {
    std::vector<hyb_tensor> list;
    const hyb_status st = read_list(count, tensors, false, true, &list);
    if (st != HYB_OK) return st;
    if (!bytes) return fail(HYB_ERR_INVALID_ARG, "bytes is NULL");
    int64_t sums;
    (void)hyb::clip_plan(list, &sums);
    *bytes = size_t(sums) * 8;
    return ok();
  });
}

hyb_status hyb_norm(int64_t count, const hyb_tensor* tensors, float* norm, void* workspace, size_t workspace_bytes,
                    void* stream) {
  return guarded([&] { return run(count, tensors, false, 0.f, norm, workspace, workspace_bytes, stream); });
}

hyb_status hyb_clip(int64_t count, const hyb_tensor* tensors, float max_norm, float* norm, void* workspace,
                    size_t workspace_bytes, void* stream) {
  return guarded([&] { return run(count, tensors, true, max_norm, norm, workspace, workspace_bytes, stream); });
}

}  // extern "C"
