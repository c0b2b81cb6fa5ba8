// Single-token form of the selective state space scan, on a pool of states.
//
// Per row and channel c (group g(c)), with S states:
//     d = softplus(delta + bias),  h <- exp(d A[c]) h + d u B[g],  y = (C[g] . h + D u) (z sigmoid(z))
// The states are read and written once, 8 S bytes a channel against some ten bytes of the rest, so
// HBM bounds a full batch and latency a small one.  S / 8 lanes own a channel with eight states each
// (one 32-byte load and store) and sum y with shuffles.  512 x 8192 x 16 bf16 by slot: 100 us, 5.7 TB/s, 84% of a copy's
// rate; one row of 4096 channels: 4.1 us, the launch and three dependent loads.
#include "kda_layer.h"
#include "kda_segments.cuh"
#include "kda_slots.cuh"
#include "kda_ssm.cuh"

namespace kda {

namespace {

constexpr int kThreads = 128;

// Eight fp32 in pairs, 32 bytes in one access.
struct Eight {
    f2 v[4];
    __device__ __forceinline__ void load(const float* p) {
        asm volatile("ld.global.L1::no_allocate.v4.b64 {%0, %1, %2, %3}, [%4];" : "=l"(v[0]), "=l"(v[1]), "=l"(v[2]), "=l"(v[3]) : "l"(p) : "memory");
    }
    // Of a page that is one (>= 0), without a branch.
    __device__ __forceinline__ void load_if(int page, const float* p) {
        asm volatile(
            "{\n.reg .pred q;\nsetp.ge.s32 q, %5, 0;\n"
            "@q ld.global.L1::no_allocate.v4.b64 {%0, %1, %2, %3}, [%4];\n}"
            : "=l"(v[0]), "=l"(v[1]), "=l"(v[2]), "=l"(v[3])
            : "l"(p), "r"(page)
            : "memory");
    }
    __device__ __forceinline__ void store(float* p) const {
        asm volatile("st.global.L1::no_allocate.v4.b64 [%0], {%1, %2, %3, %4};" ::"l"(p), "l"(v[0]), "l"(v[1]), "l"(v[2]), "l"(v[3]) : "memory");
    }
};

// Eight consecutive elements of a row of B or C; `wide`: by 16-byte pieces.
template <typename T>
struct EightOf {
    uint4 r[sizeof(T) / 2];
    __device__ __forceinline__ void load(const T* p, bool wide) {
        if (wide) {
#pragma unroll
            for (int i = 0; i < (int)sizeof(T) / 2; ++i) r[i] = __ldg(reinterpret_cast<const uint4*>(p) + i);
        } else {
            T* v = reinterpret_cast<T*>(r);
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = __ldg(p + k);
        }
    }
    __device__ __forceinline__ f2 pair(int i) const {
        const uint32_t* w = reinterpret_cast<const uint32_t*>(r);
        if constexpr (sizeof(T) == 2) return pack(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
        else return pack(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
    }
};

// kRows rows of the batch a block: A is as many bytes as a row's states, and is fetched once for them.
// Everything that the rows need is requested before the first is worked on.
template <typename T, int S, int kRows>
__global__ void __launch_bounds__(kThreads) ssm_step_kernel(SsmStepParams p, int blocks, bool wide) {
    constexpr int LP = S / 8, CH = kThreads / LP;
    // (the blocks of one page follow one another)
    const int row0 = (int)(blockIdx.x / blocks) * kRows;
    const int lane = threadIdx.x % LP;
    const int c = (int)(blockIdx.x % blocks) * CH + threadIdx.x / LP;
    const bool on = c < p.C;
    const int cc = on ? c : 0, g = cc / (p.C / p.G) * S + lane * 8;
    const int64_t per_page = (int64_t)p.C * S, at = (int64_t)cc * S + lane * 8;
    int page[kRows];
    Eight h[kRows];
    T u[kRows], dl[kRows], z[kRows];
    EightOf<T> Bv[kRows], Cv[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const int row = min(row0 + i, p.N - 1);
        page[i] = page_of_row(p.slots, row, p.P);
        // A row without a page loads none: the first page's own row may be writing it.  (By graph, one row of 4096 channels takes
        // 1.8 us with the predicate and 2.0 with the branch, which the other loads wait behind; 512 of 8192 100 and 98.4.)
        if constexpr (kRows == 1) {
            h[i].load_if(page[i], p.state + page[i] * per_page + at);
        } else {
            if (page[i] >= 0) h[i].load(p.state + page[i] * per_page + at);
        }
        u[i] = __ldg(static_cast<const T*>(p.u) + row * p.ldu + cc);
        dl[i] = __ldg(static_cast<const T*>(p.delta) + row * p.ldd + cc);
        if (p.z) z[i] = __ldg(static_cast<const T*>(p.z) + row * p.ldz + cc);
        Bv[i].load(static_cast<const T*>(p.Bm) + row * p.ldb + g, wide);
        Cv[i].load(static_cast<const T*>(p.Cm) + row * p.ldc + g, wide);
    }
    f2 A2[4];
#pragma unroll
    for (int k = 0; k < 4; k += 2) {
        const float4 x = __ldg(reinterpret_cast<const float4*>(p.A + at) + k / 2);
        A2[k] = pack(kLog2e * x.x, kLog2e * x.y);
        A2[k + 1] = pack(kLog2e * x.z, kLog2e * x.w);
    }
    const float bias = p.bias ? __ldg(p.bias + cc) : 0.f, D = p.D ? __ldg(p.D + cc) : 0.f;
    const unsigned refused = rows_refused<kRows>(p.slots, row0, p.N, page, p.status);
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const int row = row0 + i;
        if (row >= p.N || (refused >> i & 1)) continue;
        float d = to_f32<T>(dl[i]) + bias;
        if (p.softplus) d = softplus(d);
        const float uv = to_f32<T>(u[i]), du = d * uv;
        const f2 dd = pack(d, d), du2 = pack(du, du);
        f2 y2 = 0ull;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            h[i].v[k] = fma2(ex2_2(mul2(dd, A2[k])), h[i].v[k], mul2(du2, Bv[i].pair(k)));
            y2 = fma2(h[i].v[k], Cv[i].pair(k), y2);
        }
        if (on) h[i].store(p.state + page[i] * per_page + at);
        float y = sum2(y2);
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
    constexpr int CH = kThreads / (S / 8);
    const int blocks = (p.C + CH - 1) / CH;
    const int piece = 16 / (int)sizeof(T);
    const bool wide = kda_host::rows_aligned(p.Bm, p.ldb, piece) && kda_host::rows_aligned(p.Cm, p.ldc, piece);
    // two rows a block once that leaves the machine four blocks an SM, else one
    if ((int64_t)(p.N + 1) / 2 * blocks >= 4 * 152)
        ssm_step_kernel<T, S, 2><<<(unsigned)((int64_t)((p.N + 1) / 2) * blocks), kThreads, 0, st>>>(p, blocks, wide);
    else
        ssm_step_kernel<T, S, 1><<<(unsigned)((int64_t)p.N * blocks), kThreads, 0, st>>>(p, blocks, wide);
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
