// Pieces that the selective state space kernels share.
#pragma once

#include "kda_segments.cuh"

namespace kda {

// log(1 + e) for 0 <= e <= 1 from log(1 + e) = 2 atanh(r), r = e / (2 + e) <= 1/3, with atanh(r) =
// r + r^3 P(r^2) and P the cubic of least maximal relative error (4.5e-9), fitted to r^2 in [0, 1/9].
// (A logarithm of the rounded 1 + e would lose the small e that ordinary step sizes have.)
// softplus(x) = max(x, 0) + log(1 + e^-|x|), here for two values.
__device__ __forceinline__ f2 softplus2(f2 x) {
    float a, b;
    unpack(x, a, b);
    const float ea = ex2(-kLog2e * fabsf(a)), eb = ex2(-kLog2e * fabsf(b));
    const f2 r = mul2(pack(ea, eb), pack(rcp(2.0f + ea), rcp(2.0f + eb))), q = mul2(r, r);
    const auto both = [](float v) { return pack(v, v); };
    f2 s = fma2(both(0.14005993f), q, both(0.14000903f));
    s = fma2(s, q, both(0.20010764f));
    s = fma2(s, q, both(0.33333208f));
    s = fma2(mul2(s, q), r, r);
    return fma2(s, both(2.0f), pack(fmaxf(a, 0.0f), fmaxf(b, 0.0f)));
}
__device__ __forceinline__ float softplus(float x) {
    float a, b;
    unpack(softplus2(pack(x, x)), a, b);
    return a;
}

// ---- which channels and tokens a block works on ------------------------------------------------

// Blocks of CH channels, none across two groups: block x is the (x % per_group)-th of its group.
struct ChannelBlocks {
    int per_group, group_size;
    __host__ __device__ ChannelBlocks(int C, int G, int CH) : per_group((C / G + CH - 1) / CH), group_size(C / G) {}
    __device__ __forceinline__ int group(int x) const { return x / per_group; }
    __device__ __forceinline__ int in_group(int x, int CH) const { return x % per_group * CH; }
};

}  // namespace kda
