// Host routing of the 8-bit product: tile shape and cuts of k per product.
#include "hyb_f8_internal.h"

namespace hyb {

F8Route f8_route(int64_t n, int64_t k, int64_t m, int64_t cus) {
  const int64_t np = (n + 15) / 16, mp = (m + 15) / 16;
  if (mp <= 4) return F8Route{1, mp <= 1 ? 1 : mp <= 2 ? 2 : 4, 8, 1};
  const int64_t big = ((np + 15) / 16) * ((mp + 15) / 16);
  if (big >= cus) return F8Route{16, 16, 0, 1};
  return F8Route{8, 8, 0, 1};
}

size_t f8_workspace_bytes(const F8Route& r, int64_t n, int64_t m) {
  if (r.parts <= 1) return 0;
  const int64_t na = (n + 16 * r.ap - 1) / (16 * r.ap), nb = (m + 16 * r.bp - 1) / (16 * r.bp);
  return size_t(na * nb * r.parts) * r.ap * r.bp * 1024;
}

}  // namespace hyb
