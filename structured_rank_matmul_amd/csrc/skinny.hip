// The streaming products of skinny_linear.h in bf16 and float32.
#include "skinny_linear.h"

namespace dyra {

template hipError_t launch_skinny<bf16, bf16, false>(const LinearArgs<bf16, bf16> &, hipStream_t);
template hipError_t launch_narrow<bf16, bf16, false>(const LinearArgs<bf16, bf16> &, hipStream_t);
template hipError_t launch_skinny<bf16, float, false>(const LinearArgs<bf16, float> &, hipStream_t);
template hipError_t launch_narrow<bf16, float, false>(const LinearArgs<bf16, float> &, hipStream_t);
template hipError_t launch_skinny<float, float, false>(const LinearArgs<float, float> &, hipStream_t);
template hipError_t launch_narrow<float, float, false>(const LinearArgs<float, float> &, hipStream_t);
template hipError_t launch_skinny<bf16, bf16, true>(const LinearArgs<bf16, bf16> &, hipStream_t);
template hipError_t launch_narrow<bf16, bf16, true>(const LinearArgs<bf16, bf16> &, hipStream_t);
template hipError_t launch_skinny<float, float, true>(const LinearArgs<float, float> &, hipStream_t);
template hipError_t launch_narrow<float, float, true>(const LinearArgs<float, float> &, hipStream_t);

}  // namespace dyra
