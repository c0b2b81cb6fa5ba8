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

// CPT channels of a thread: their state loads are all issued before the first is used.
template <typename T, int S, int CPT>
__global__ void __launch_bounds__(kThreads) ssm_step_kernel(SsmStepParams p) {
    constexpr int LP = S / 4, CH = kThreads / LP;
    const int row = blockIdx.x;
    const int page = page_of_row(p.slots, row, p.P);
    const int lane = threadIdx.x % LP;
    const int c0 = blockIdx.y * (CH * CPT) + threadIdx.x / LP;
    float4* state = reinterpret_cast<float4*>(p.state + (int64_t)max(page, 0) * p.C * S);
    float4 h[CPT];
#pragma unroll
    for (int i = 0; i < CPT; ++i) {
        const int c = c0 + i * CH;
        if (c < p.C) h[i] = __ldcs(state + (int64_t)c * LP + lane);
    }
    if (row_refused(p.slots, row, page, p.status)) return;
    const int per = p.C / p.G;
    const T* Bm = static_cast<const T*>(p.Bm) + row * p.ldb;
    const T* Cm = static_cast<const T*>(p.Cm) + row * p.ldc;
#pragma unroll
    for (int i = 0; i < CPT; ++i) {
        const int c = c0 + i * CH;
        const bool on = c < p.C;
        float y = 0.f, u = 0.f;
        if (on) {
            u = ld(static_cast<const T*>(p.u), row * p.ldu + c);
            float d = ld(static_cast<const T*>(p.delta), row * p.ldd + c);
            if (p.bias) d += p.bias[c];
            if (p.softplus) d = softplus(d);
            const int g = c / per * S + lane * 4;
            const float4 A = *reinterpret_cast<const float4*>(p.A + (int64_t)c * S + lane * 4);
            const float a[4] = {A.x, A.y, A.z, A.w};
            float v[4] = {h[i].x, h[i].y, h[i].z, h[i].w};
            const float du = d * u, dl = d * kLog2e;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                v[k] = fmaf(ex2(dl * a[k]), v[k], du * ld(Bm, g + k));
                y = fmaf(ld(Cm, g + k), v[k], y);
            }
            __stcs(state + (int64_t)c * LP + lane, make_float4(v[0], v[1], v[2], v[3]));
        }
#pragma unroll
        for (int o = LP / 2; o > 0; o >>= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
        if (on && lane == 0) {
            if (p.D) y = fmaf(p.D[c], u, y);
            if (p.z) {
                const float z = ld(static_cast<const T*>(p.z), row * p.ldz + c);
                y *= z * sigmoid(z);
            }
            static_cast<T*>(p.y)[(int64_t)row * p.C + c] = from_f32<T>(y);
        }
    }
}

template <typename T, int S>
cudaError_t launch(const SsmStepParams& p, cudaStream_t st) {
    constexpr int CH = kThreads / (S / 4);
    // four channels a thread once that still leaves the machine full (152 SMs of 8 blocks), else one
    if ((int64_t)p.N * ((p.C + 4 * CH - 1) / (4 * CH)) >= 152 * 8)
        ssm_step_kernel<T, S, 4><<<dim3(p.N, (p.C + 4 * CH - 1) / (4 * CH)), kThreads, 0, st>>>(p);
    else
        ssm_step_kernel<T, S, 1><<<dim3(p.N, (p.C + CH - 1) / CH), kThreads, 0, st>>>(p);
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
