// step_plan.h -- how the norm, rotation and append of a step's tokens are cut
// into launches (heads_kernels.hip), and the launches for each type
// (step_f32.hip and the like).
#pragma once
#include "ops.h"

namespace voc {

// How a step's work is cut.
struct StepPlan {
  int g, mode, pages, parts, wpp, np, groups, per, run;
  bool page;  // by step_page_kernel
  int64_t workgroups;  // of a sequence
};

void go_step_f32(const StepArgs& a, const StepPlan& p, hipStream_t s);
void go_step_bf16(const StepArgs& a, const StepPlan& p, hipStream_t s);
void go_step_f16(const StepArgs& a, const StepPlan& p, hipStream_t s);

}  // namespace voc
