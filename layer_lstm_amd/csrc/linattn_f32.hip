// linattn_f32.hip -- linear attention by chunks, f32 storage (linattn_common.hpp).
#include <type_traits>

#include "linattn_common.hpp"

namespace lstm {
hipError_t launch_linattn_f32(const LinArgs& a, const LinTile& t, int many, int dma, unsigned groups, hipStream_t s) {
  return linattn_of<float>(a, t, many, dma, groups, s);
}
}  // namespace lstm
