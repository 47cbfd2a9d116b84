// int_matmul.hip -- the 8-bit integer product without adapters.
#include "int_matmul.h"

namespace voc {

hipError_t launch_int_matmul(int dtype, const IntMatmulArgs& a, hipStream_t s, Form& form) {
  if (dtype == EL_F32)
    go_int_matmul<EL_F32, false>(a, s, form);
  else if (dtype == EL_BF16)
    go_int_matmul<EL_BF16, false>(a, s, form);
  else
    go_int_matmul<EL_F16, false>(a, s, form);
  return hipGetLastError();
}

}  // namespace voc
