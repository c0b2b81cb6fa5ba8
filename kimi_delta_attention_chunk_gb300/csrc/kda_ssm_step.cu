// Single-token form of the selective state space scan, on a pool of states.
//
// Per row and channel c (group g(c)), with S states:
//     d = softplus(delta + bias),  h <- exp(d A[c]) h + d u B[g],  y = (C[g] . h + D u) (z sigmoid(z))
// The states are read and written once, 8 S bytes a channel against some ten bytes of the rest, so
// HBM bounds a full batch and latency a small one.  S / 4 lanes own a channel with four states each
// (one 16-byte load and store) and sum y with shuffles.
#include "kda_layer.h"
#include "kda_segments.cuh"
#include "kda_slots.cuh"
#include "kda_ssm.cuh"

namespace kda {

namespace {

constexpr int kThreads = 256;

// Four consecutive elements of a vector, in pairs; `wide`: as one piece.
template <typename T>
struct Four {
    T v[4];
    __device__ __forceinline__ void load(const T* p, bool wide) {
        if (wide) {
            typedef typename Bits<4 * sizeof(T)>::type Raw;
            *reinterpret_cast<Raw*>(v) = __ldg(reinterpret_cast<const Raw*>(p));
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) v[k] = __ldg(p + k);
        }
    }
};

// kRows rows of the batch a block: A is as many bytes as a row's states, and is fetched once for them.
// Everything that the rows need is requested before the first is worked on.
template <typename T, int S, int kRows>
__global__ void __launch_bounds__(kThreads) ssm_step_kernel(SsmStepParams p, bool wide) {
    constexpr int LP = S / 4, CH = kThreads / LP;
    const int row0 = blockIdx.x * kRows;
    const int lane = threadIdx.x % LP;
    const int c = blockIdx.y * CH + threadIdx.x / LP;
    const bool on = c < p.C;
    const int cc = on ? c : 0, g = cc / (p.C / p.G) * S + lane * 4;
    int page[kRows];
    float4 h[kRows];
    T u[kRows], dl[kRows], z[kRows];
    Four<T> Bv[kRows], Cv[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const int row = min(row0 + i, p.N - 1);
        page[i] = page_of_row(p.slots, row, p.P);
        h[i] = __ldcs(reinterpret_cast<const float4*>(p.state + ((int64_t)max(page[i], 0) * p.C + cc) * S + lane * 4));
        u[i] = __ldg(static_cast<const T*>(p.u) + row * p.ldu + cc);
        dl[i] = __ldg(static_cast<const T*>(p.delta) + row * p.ldd + cc);
        if (p.z) z[i] = __ldg(static_cast<const T*>(p.z) + row * p.ldz + cc);
        Bv[i].load(static_cast<const T*>(p.Bm) + row * p.ldb + g, wide);
        Cv[i].load(static_cast<const T*>(p.Cm) + row * p.ldc + g, wide);
    }
    const float4 A = *reinterpret_cast<const float4*>(p.A + (int64_t)cc * S + lane * 4);
    const float a[4] = {A.x, A.y, A.z, A.w};
    const float bias = p.bias ? __ldg(p.bias + cc) : 0.f, D = p.D ? __ldg(p.D + cc) : 0.f;
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const int row = row0 + i;
        if (row >= p.N) break;
        if (row_refused(p.slots, row, page[i], p.status)) continue;
        float d = to_f32<T>(dl[i]) + bias;
        if (p.softplus) d = softplus(d);
        const float uv = to_f32<T>(u[i]), du = d * uv, de = d * kLog2e;
        float v[4] = {h[i].x, h[i].y, h[i].z, h[i].w}, y = 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            v[k] = fmaf(ex2(de * a[k]), v[k], du * to_f32<T>(Bv[i].v[k]));
            y = fmaf(to_f32<T>(Cv[i].v[k]), v[k], y);
        }
        if (on) __stcs(reinterpret_cast<float4*>(p.state + ((int64_t)page[i] * p.C + c) * S + lane * 4), make_float4(v[0], v[1], v[2], v[3]));
#pragma unroll
        for (int o = LP / 2; o > 0; o >>= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
        if (on && lane == 0) {
            y = fmaf(D, uv, y);
            if (p.z) {
                const float zv = to_f32<T>(z[i]);
                y *= zv * sigmoid(zv);
            }
            static_cast<T*>(p.y)[(int64_t)row * p.C + c] = from_f32<T>(y);
        }
    }
}

template <typename T, int S>
cudaError_t launch(const SsmStepParams& p, cudaStream_t st) {
    constexpr int CH = kThreads / (S / 4);
    const int blocks = (p.C + CH - 1) / CH;
    const size_t piece = 4 * sizeof(T);
    const bool wide = (uintptr_t)p.Bm % piece == 0 && (uintptr_t)p.Cm % piece == 0 && p.ldb % 4 == 0 && p.ldc % 4 == 0;
    // four rows a block once that leaves the machine four blocks an SM, else one
    if ((int64_t)(p.N + 3) / 4 * blocks >= 4 * 152)
        ssm_step_kernel<T, S, 4><<<dim3((p.N + 3) / 4, blocks), kThreads, 0, st>>>(p, wide);
    else
        ssm_step_kernel<T, S, 1><<<dim3(p.N, blocks), kThreads, 0, st>>>(p, wide);
    return cudaGetLastError();
}

template <typename T>
cudaError_t dispatch(const SsmStepParams& p, cudaStream_t st) {
    if (p.S == 8) return launch<T, 8>(p, st);
    if (p.S == 16) return launch<T, 16>(p, st);
    if (p.S == 32) return launch<T, 32>(p, st);
    return launch<T, 64>(p, st);
}

}  // namespace

cudaError_t ssm_step(kda_dtype dt, const SsmStepParams& p, cudaStream_t st) {
    return dt == KDA_BF16 ? dispatch<__nv_bfloat16>(p, st) : dispatch<float>(p, st);
}

}  // namespace kda
