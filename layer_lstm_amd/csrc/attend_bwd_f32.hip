// attend_bwd_f32.hip -- the cross attention backward for f32 storage.
#include "attend_bwd.hpp"

namespace lstm {

hipError_t launch_attend_bwd_f32(const AttendPlan& p, const AttendArgs& a, hipStream_t s) {
  return attend_bwd_dp<float>(p, a, s);
}

}  // namespace lstm
