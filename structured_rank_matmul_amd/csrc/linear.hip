// The linear layer and the gated pair of linear_tile.h in bf16 and float32.
#include "linear_tile.h"

namespace dyra {

template hipError_t launch_linear<bf16, bf16, false>(const LinearArgs<bf16, bf16> &, hipStream_t);
template hipError_t launch_linear<bf16, float, false>(const LinearArgs<bf16, float> &, hipStream_t);
template hipError_t launch_linear<float, float, false>(const LinearArgs<float, float> &, hipStream_t);
template hipError_t launch_linear<bf16, bf16, true>(const LinearArgs<bf16, bf16> &, hipStream_t);
template hipError_t launch_linear<float, float, true>(const LinearArgs<float, float> &, hipStream_t);

}  // namespace dyra
