// k_i8_rows.cu -- rows as they are and SwiGLU of gate and up rows, in 8-bit
// integers: the kernels of i8_rows.cuh.
#include "i8_rows.cuh"

namespace q3 {

cudaError_t launch_i8_quantize(const Launch& L, const I8RowArgs& a, int type) { return launch_type<QUANT>(L, a, type); }
cudaError_t launch_i8_swiglu(const Launch& L, const I8RowArgs& a, int type) { return launch_type<SWIGLU>(L, a, type); }

}  // namespace q3
