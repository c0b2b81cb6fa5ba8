// Parameters and launchers of the recurrent layer's operators around the KDA kernels: the short
// convolution, the selective state space scan and the pages of a cache (internal to libkda.so;
// the public surface is include/kda.h).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/kda.h"

namespace kda {

struct ConvParams {
    const void* x;        // [total][ldx]
    int64_t ldx;
    const float* weight;  // [C][W]
    const float* bias;    // [C] or null
    int act;
    const void* initial;  // [N][W-1][C] or null
    const int32_t* cu;
    int T, N, C, W, total;
    void* y;              // [total][C]
    void* final_hist;     // [N][W-1][C] or null
    // backward
    const void* dy;       // [total][C], gradient type
    const void* dfinal;   // [N][W-1][C] or null, gradient type
    void* dx;             // [total][C], gradient type
    void* dinitial;       // [N][W-1][C] or null, gradient type
    float* dweight;       // [C][W]
    float* dbias;         // [C] or null
    float* partial;       // [ranges][C][W + 1]
};

cudaError_t short_conv_fwd(kda_dtype dt, const ConvParams& p, cudaStream_t st);
cudaError_t short_conv_bwd(kda_dtype dt, kda_dtype gdt, const ConvParams& p, cudaStream_t st);
// Floats of `partial` that short_conv_bwd may use.
size_t short_conv_bwd_partial(int total, int C, int W);

struct ConvStepParams {
    const void* x;        // [N][ldx]
    int64_t ldx;
    const float* weight;
    const float* bias;
    int act;
    void* history;        // [P][W-1][C]
    const int32_t* slots; // [N] or null
    int N, P, C, W;
    void* y;              // [N][C]
    int32_t* status;
};
cudaError_t short_conv_step(kda_dtype dt, const ConvStepParams& p, cudaStream_t st);

struct SsmStepParams {
    const void *u, *delta, *z;      // [N][ld*]; z may be null
    int64_t ldu, ldd, ldz;
    const void *Bm, *Cm;            // [N][ldb / ldc], G groups of S values a row
    int64_t ldb, ldc;
    const float *A, *D, *bias;      // [C][S], [C] or null, [C] or null
    int softplus;
    float* state;                   // [P][C][S]
    const int32_t* slots;           // [N] or null
    int N, P, C, G, S;
    void* y;                        // [N][C]
    int32_t* status;
};
cudaError_t ssm_step(kda_dtype dt, const SsmStepParams& p, cudaStream_t st);

struct SsmScanParams {
    const void *u, *delta, *z;      // [total][ld*]; z may be null
    int64_t ldu, ldd, ldz;
    const void *Bm, *Cm;            // [total][ldb / ldc], G groups of S values a row
    int64_t ldb, ldc;
    const float *A, *D, *bias;      // [C][S], [C] or null, [C] or null
    int softplus;
    const float* initial;           // [N][C][S] or null
    const int32_t* cu;
    int T, N, C, G, S, total;
    void* y;                        // [total][C]
    float* final_state;             // [N][C][S] or null
    // backward
    const void* dy;                 // [total][C], gradient type
    const float* dfinal;            // [N][C][S] or null
    void *du, *ddelta, *dz;         // [total][C], gradient type; dz null with z
    void *dB, *dC;                  // [total][G][S], gradient type
    float *dA, *dD, *dbias;         // [C][S], [C] or null, [C] or null
    float* dinitial;                // [N][C][S] or null
    void* ws;
};
// Device bytes a call needs at p's sizes (p.cu null or not matters, no pointer is followed).
size_t ssm_scan_workspace(const SsmScanParams& p);
cudaError_t ssm_scan_fwd(kda_dtype dt, const SsmScanParams& p, cudaStream_t st);
size_t ssm_scan_bwd_workspace(const SsmScanParams& p);
cudaError_t ssm_scan_bwd(kda_dtype dt, kda_dtype gdt, const SsmScanParams& p, cudaStream_t st);

cudaError_t pages_alloc(int32_t* refs, int P, int n, int32_t* out, int32_t* status, cudaStream_t st);
cudaError_t pages_free(int32_t* refs, int P, const int32_t* pages, int64_t n, int32_t* status, cudaStream_t st);
cudaError_t pages_fork(int32_t* tables, int32_t* lens, int S, int width, int page_tokens, int32_t* refs, int P,
                       const int32_t* parents, const int32_t* children, int n, int32_t* src, int32_t* dst,
                       int32_t* status, cudaStream_t st);
size_t pages_compact_workspace(int P);
cudaError_t pages_compact(int32_t* refs, int P, int32_t* tables, int64_t entries, int32_t* src, int32_t* dst, void* ws,
                          int32_t* status, cudaStream_t st);
size_t pages_copy_workspace(int P, int n);
cudaError_t pages_copy(void* pool, int P, int64_t page_bytes, const int32_t* src, const int32_t* dst, int n, void* ws,
                       int32_t* status, cudaStream_t st);

}  // namespace kda
