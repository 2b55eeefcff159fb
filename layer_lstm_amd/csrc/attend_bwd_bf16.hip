// attend_bwd_bf16.hip -- the cross attention backward for bf16 storage.
#include "attend_bwd.hpp"

namespace lstm {

hipError_t launch_attend_bwd_bf16(const AttendPlan& p, const AttendArgs& a, hipStream_t s) {
  return attend_bwd_dp<bf16_t>(p, a, s);
}

}  // namespace lstm
