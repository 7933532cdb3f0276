// Test infrastructure: stand-ins for the launchers of the 4-bit weights, the
// gated projection and the clipping, beside those of sanitize_launch_stub.cpp, so
// that their host-side files can be built by the host compiler with the
// sanitizers.  Every launcher reports hipErrorNoDevice.
#include "../matmul_pack_b1_amd/csrc/hyb_clip_internal.h"
#include "../matmul_pack_b1_amd/csrc/hyb_gated_internal.h"
#include "../matmul_pack_b1_amd/csrc/hyb_q4_internal.h"

namespace hyb {

hipError_t launch_q4_quantize(const void*, int, int64_t, int64_t, int64_t, const hyb_q4&, hipStream_t) {
  return hipErrorNoDevice;
}
hipError_t launch_q4_dequantize(const hyb_q4&, int64_t, int64_t, void*, int, int64_t, hipStream_t) {
  return hipErrorNoDevice;
}
hipError_t launch_q4_product(const hyb_q4&, const hyb_q4*, int, int64_t, int64_t, const void*, int, int64_t, int64_t,
                             void*, int, int64_t, char*, hipStream_t) {
  return hipErrorNoDevice;
}
hipError_t launch_gated(const hyb_gated_pair&, const GatedPlan&, int, const void*, int, int64_t, const GatedForward&,
                        char*, hipStream_t) {
  return hipErrorNoDevice;
}
hipError_t launch_gated_backward(const hyb_gated_pair&, const GatedPlan&, int, const void*, int, int64_t,
                                 const GatedBackward&, char*, hipStream_t) {
  return hipErrorNoDevice;
}
hipError_t launch_norm(const std::vector<hyb_tensor>&, float*, double*, hipStream_t) { return hipErrorNoDevice; }
hipError_t launch_clip(const std::vector<hyb_tensor>&, float, float*, double*, hipStream_t) { return hipErrorNoDevice; }

}  // namespace hyb
