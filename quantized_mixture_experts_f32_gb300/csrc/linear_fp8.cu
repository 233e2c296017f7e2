// linear_fp8.cu -- which kernel of qmoe_linear_fp8 takes a call.
#include "linear_fp8.cuh"

namespace qmoe {

cudaError_t linear_fp8_prepare() { return linear_pair_prepare(); }

cudaError_t launch_linear_fp8(const LinearArgs& a, int num_sms, cudaStream_t st) {
    if (a.T > 256) return launch_linear_pair(a, num_sms, st);
    return launch_linear_few(a, st);
}

}  // namespace qmoe
