// Sixteen bytes that are used once, at any address aligned to 2: loaded and stored
// as what the caches need not keep.
#ifndef HYB_STREAM_H_
#define HYB_STREAM_H_

#include "hyb_panel.h"

namespace hyb {
namespace {

// Outputs of more bytes than the last-level cache holds go around it.  (Clipping lists of
// 512 MB, and a pass over the result, 490 us instead of 523; 256 MB 265 and 282; 128 MB
// 154 instead of 143.)
constexpr int64_t kStreamBytes = int64_t(256) << 20;

typedef uint32_t __attribute__((ext_vector_type(4), aligned(2))) any16_t;

__device__ __forceinline__ Bytes16 stream_load(const void* p) {
  const any16_t v = __builtin_nontemporal_load(static_cast<const any16_t*>(p));
  return Bytes16{{v[0], v[1], v[2], v[3]}};
}
__device__ __forceinline__ void stream_store(void* p, const Bytes16& b) {
  __builtin_nontemporal_store(any16_t{b.w[0], b.w[1], b.w[2], b.w[3]}, static_cast<any16_t*>(p));
}

}  // namespace
}  // namespace hyb
#endif  // HYB_STREAM_H_
