// Pieces that the group norm's kernels share: rows in pairs of fp32, the activation, and the last sums of the weights' gradients.
//
//     p = w (x - mean) rstd + b,  y = p or p sigmoid(p);  rstd = 1 / sqrt(var + eps)
//     dp = dy act'(p),  q = w dp,  xh = (x - mean) rstd:  dx = rstd (q - mean(q) - xh mean(q xh)),  dw = sum dp xh,  db = sum dp
#pragma once

#include "kda_clusters.cuh"
#include "kda_layer.h"
#include "kda_tc.cuh"

namespace kda {

// x / (1 + e^-x), and the slope of that, s + x s (1 - s).
__device__ __forceinline__ f2 silu2(f2 p) { return mul2(p, gate2(p)); }
__device__ __forceinline__ f2 silu_slope2(f2 p) {
    const f2 s = gate2(p);
    return fma2(mul2(p, s), fma2(s, both(-1.f), both(1.f)), s);
}
// VEC consecutive fp32 as pairs (of one: its upper half zero), `none` where there are none.
template <int VEC>
__device__ __forceinline__ void vec_pairs(const float* p, float none, f2 (&v)[(VEC + 1) / 2]) {
#pragma unroll
    for (int k = 0; k < (VEC + 1) / 2; ++k) v[k] = p ? pack(__ldg(p + 2 * k), 2 * k + 1 < VEC ? __ldg(p + 2 * k + 1) : 0.f) : both(none);
}

// dweight and dbias from partial sums [parts][2][C] (sum dp xh, then sum dp), 32 channels a block, in a fixed order.  The first 256 threads
// of a block call it.
__device__ __forceinline__ void norm_weight_sums(const float* partial, int parts, int C, float* dweight, float* dbias, int block) {
    __shared__ float sums[8][33];
    const int lane = threadIdx.x % 32, w = threadIdx.x / 32, c = block * 32 + lane;
#pragma unroll
    for (int v = 0; v < 2; ++v) {
        float* const to = v ? dbias : dweight;
        if (!to) continue;
        float s = 0.f;
        if (c < C) {
#pragma unroll 4
            for (int k = w; k < parts; k += 8) s += partial[((int64_t)k * 2 + v) * C + c];
        }
        tc::named_sync(1, 256);  // (the block may have more threads)
        sums[w][lane] = s;
        tc::named_sync(1, 256);
        if (w == 0 && c < C) {
            s = 0.f;
#pragma unroll
            for (int k = 0; k < 8; ++k) s += sums[k][lane];
            to[c] = s;
        }
    }
}
static __global__ void __launch_bounds__(256) norm_weights_kernel(const float* partial, int parts, int C, float* dweight, float* dbias) {
    tc::grid_dep_wait();
    norm_weight_sums(partial, parts, C, dweight, dbias, blockIdx.x);
}

cudaError_t norm_token_fwd(kda_dtype dt, const NormParams& p, cudaStream_t st);
size_t norm_token_bwd_workspace(const NormParams& p);
cudaError_t norm_token_bwd(kda_dtype dt, kda_dtype gdt, const NormParams& p, cudaStream_t st);

}  // namespace kda
