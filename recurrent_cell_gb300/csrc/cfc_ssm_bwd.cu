#include "ssm_common.cuh"
namespace cfc {
cudaError_t launch_ssm_backward(const SsmArgs& g, const SsmGrads& r, cudaStream_t s) { return cudaErrorNotSupported; }
}
