// The kernels of q4_kernels.h for one type of X and one form (a source each, to
// compile side by side).
#include "q4_kernels.h"

namespace sgemm {
template hipError_t launch_q4_kernels<T_F16, 2>(const Q4Args& g, hipStream_t s);
}  // namespace sgemm
