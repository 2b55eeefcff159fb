// linattn_f16.hip -- linear attention by chunks, f16 storage (linattn_common.hpp).
#include <type_traits>

#include "linattn_common.hpp"

namespace lstm {
hipError_t launch_linattn_f16(const LinArgs& a, const LinTile& t, int many, int dma, unsigned groups, hipStream_t s) {
  return linattn_of<f16_t>(a, t, many, dma, groups, s);
}
}  // namespace lstm
