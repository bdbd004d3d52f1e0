// What the sources of the orthogonalised update share.
#pragma once
#include "kernels.h"

namespace sgemm {

// Sides of up to this many rows or columns take the small matrices' kernels
// (orthogonalize_small.hip).
constexpr int64_t kOrthoSmall = 64;
// All steps' coefficients, as a kernel's argument (SGEMM_ORTHO_MAX_STEPS).
struct SmallCoefficients {
    double v[3 * 64];
};
size_t ortho_small_bytes(int64_t batch, int64_t M, int64_t N);
hipError_t launch_ortho_small(const OrthoArgs& g, hipStream_t s);

}  // namespace sgemm
