// Pieces that the selective state space kernels share.
#pragma once

#include "kda_segments.cuh"

namespace kda {

// log(1 + e) for 0 <= e <= 1 from log(1 + e) = 2 atanh(r), r = e / (2 + e) <= 1/3, by the series
// r + r^3/3 + r^5/5 + ...: the first term left out is below 2e-8 of the sum.  (A logarithm of the
// rounded 1 + e would lose the small e that ordinary step sizes have.)
__device__ __forceinline__ float log1p_unit(float e) {
    const float r = __fdividef(e, 2.0f + e), q = r * r;
    float s = 1.0f / 13.0f;
    s = fmaf(s, q, 1.0f / 11.0f);
    s = fmaf(s, q, 1.0f / 9.0f);
    s = fmaf(s, q, 1.0f / 7.0f);
    s = fmaf(s, q, 1.0f / 5.0f);
    s = fmaf(s, q, 1.0f / 3.0f);
    s = fmaf(s * q, r, r);
    return s + s;
}

// log(1 + e^x) = max(x, 0) + log(1 + e^-|x|)
__device__ __forceinline__ float softplus(float x) { return fmaxf(x, 0.0f) + log1p_unit(ex2(-kLog2e * fabsf(x))); }

// ---- which channels and tokens a block works on ------------------------------------------------

// Blocks of CH channels, none across two groups: block x is the (x % per_group)-th of its group.
struct ChannelBlocks {
    int per_group, group_size;
    __host__ __device__ ChannelBlocks(int C, int G, int CH) : per_group((C / G + CH - 1) / CH), group_size(C / G) {}
    __device__ __forceinline__ int group(int x) const { return x / per_group; }
    __device__ __forceinline__ int in_group(int x, int CH) const { return x % per_group * CH; }
};

}  // namespace kda
