// attend_bwd_f16.hip -- the cross attention backward for f16 storage.
#include "attend_bwd.hpp"

namespace lstm {

hipError_t launch_attend_bwd_f16(const AttendPlan& p, const AttendArgs& a, hipStream_t s) {
  return attend_bwd_dp<f16_t>(p, a, s);
}

}  // namespace lstm
