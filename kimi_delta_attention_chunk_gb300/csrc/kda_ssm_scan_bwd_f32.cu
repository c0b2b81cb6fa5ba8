// Selective state space scan over prompts, backward: fp32 inputs (a translation unit of its own, so that
// the two compile side by side).
#include "kda_ssm_scan_bwd.cuh"

namespace kda {

cudaError_t ssm_scan_bwd_f32(const SsmScanParams& p, cudaStream_t st) { return dispatch<float, float>(p, st); }

}  // namespace kda
