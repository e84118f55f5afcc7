// The linear layer and the gated pair of linear_tile.h on 8-bit integers.
#include "linear_tile.h"

namespace dyra {

template hipError_t launch_linear<i8, bf16, false>(const LinearArgs<i8, bf16> &, hipStream_t);
template hipError_t launch_linear<i8, float, false>(const LinearArgs<i8, float> &, hipStream_t);
template hipError_t launch_linear<i8, bf16, true>(const LinearArgs<i8, bf16> &, hipStream_t);
template hipError_t launch_linear<i8, float, true>(const LinearArgs<i8, float> &, hipStream_t);
template hipError_t launch_split<bf16, false>(const LinearArgs<i8, bf16> &, const Split &, int32_t *, hipStream_t);
template hipError_t launch_split<bf16, true>(const LinearArgs<i8, bf16> &, const Split &, int32_t *, hipStream_t);
template hipError_t launch_split<float, false>(const LinearArgs<i8, float> &, const Split &, int32_t *, hipStream_t);
template hipError_t launch_split<float, true>(const LinearArgs<i8, float> &, const Split &, int32_t *, hipStream_t);

}  // namespace dyra
