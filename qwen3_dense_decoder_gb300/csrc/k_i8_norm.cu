// k_i8_norm.cu -- the RMS norm, after a residual's addition or without, in 8-bit
// integers: the kernels of i8_rows.cuh, in a unit of their own to compile beside
// the others.
#include "i8_rows.cuh"

namespace q3 {

cudaError_t launch_i8_norm(const Launch& L, const I8RowArgs& a, int type) { return launch_type<NORM>(L, a, type); }

}  // namespace q3
