// Test infrastructure: stand-ins for the launchers of the 8-bit product and
// the cross entropy, beside those of sanitize_launch_stub.cpp, so that their
// host-side files can be built by the host compiler with the sanitizers.
// Every launcher reports hipErrorNoDevice.
#include "../matmul_pack_b1_amd/csrc/hyb_xent_internal.h"

namespace hyb {

hipError_t launch_f8_quantize(const void*, int, int64_t, int64_t, int64_t, int, const hyb_f8&, hipStream_t) {
  return hipErrorNoDevice;
}
hipError_t launch_f8_dequantize(const hyb_f8&, int64_t, int64_t, void*, int, int64_t, hipStream_t) {
  return hipErrorNoDevice;
}
bool f8_fused(int64_t, int64_t, int64_t, int) { return false; }
hipError_t launch_f8_fused(const hyb_f8&, int64_t, int64_t, const void*, int, int64_t, int64_t, void*, int, int64_t,
                           hipStream_t) {
  return hipErrorNoDevice;
}
hipError_t launch_f8_gemm(const hyb_f8&, int64_t, int64_t, const hyb_f8&, int64_t, void*, int, int64_t, float*,
                          hipStream_t, int64_t) {
  return hipErrorNoDevice;
}
hipError_t launch_xent(const hyb_head&, const XentPlan&, int64_t, const void*, int, int64_t, const int64_t*, int64_t,
                       float*, float*, char*, hipStream_t) {
  return hipErrorNoDevice;
}
hipError_t launch_xent_backward(const hyb_head&, const XentPlan&, int64_t, const void*, int, int64_t, const int64_t*,
                                int64_t, const float*, const float*, void*, int64_t, void*, int64_t, char*,
                                hipStream_t) {
  return hipErrorNoDevice;
}

}  // namespace hyb
