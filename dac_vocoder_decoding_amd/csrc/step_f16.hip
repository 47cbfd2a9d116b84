// step_f16.hip -- step_kernels.h for this type of queries, keys and values.
#include "step_kernels.h"

namespace voc {

void go_step_f16(const StepArgs& a, const StepPlan& p, hipStream_t s) { go_step_type<EL_F16>(a, p, s); }

}  // namespace voc
