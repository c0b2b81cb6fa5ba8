// Selective state space scan over prompts, backward: bf16 inputs, and the choice by type.
#include "kda_ssm_scan_bwd.cuh"

namespace kda {

cudaError_t ssm_scan_bwd_f32(const SsmScanParams& p, cudaStream_t st);

size_t ssm_scan_bwd_workspace(const SsmScanParams& p) {
    Scratch w;
    return carve(w, nullptr, chunk_count(p.total, chunk_of(p)), bwd_blocks(p), p);
}

cudaError_t ssm_scan_bwd(kda_dtype dt, kda_dtype gdt, const SsmScanParams& p, cudaStream_t st) {
    if (dt == KDA_F32) return ssm_scan_bwd_f32(p, st);
    if (gdt == KDA_F32) return dispatch<__nv_bfloat16, float>(p, st);
    return dispatch<__nv_bfloat16, __nv_bfloat16>(p, st);
}

}  // namespace kda
