// The streaming products of skinny_linear.h on 8-bit integers.
#include "skinny_linear.h"

namespace dyra {

template hipError_t launch_skinny<i8, bf16, false>(const LinearArgs<i8, bf16> &, hipStream_t);
template hipError_t launch_narrow<i8, bf16, false>(const LinearArgs<i8, bf16> &, hipStream_t);
template hipError_t launch_skinny<i8, bf16, true>(const LinearArgs<i8, bf16> &, hipStream_t);
template hipError_t launch_narrow<i8, bf16, true>(const LinearArgs<i8, bf16> &, hipStream_t);
template hipError_t launch_skinny<i8, float, false>(const LinearArgs<i8, float> &, hipStream_t);
template hipError_t launch_narrow<i8, float, false>(const LinearArgs<i8, float> &, hipStream_t);
template hipError_t launch_skinny<i8, float, true>(const LinearArgs<i8, float> &, hipStream_t);
template hipError_t launch_narrow<i8, float, true>(const LinearArgs<i8, float> &, hipStream_t);

}  // namespace dyra
