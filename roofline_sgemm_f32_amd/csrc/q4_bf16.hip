// The kernels of q4_kernels.h for X of one type (compiled side by side).
#include "q4_kernels.h"

namespace sgemm {
template hipError_t launch_q4_xt<T_BF16>(const Q4Args& g, hipStream_t s);
}
