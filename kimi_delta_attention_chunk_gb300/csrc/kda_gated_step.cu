// Single-token form of the gated linear recurrence, on a pool of states (the formulas stand in kda_gated.cuh).
//
// The states are read and written once, 8 bytes a channel next to 8 or 10 of the bf16 rows: HBM bounds a full batch, latency a small one.
// A thread has VEC channels of one row, everything it needs requested before the first value is worked on: 512 x 8192 bf16 with gates in 14.9 us
// (76% of the bytes at the copy rate), fp32 in 19.0 (93%), one row in 2.3.  Rows that are no whole pieces go channel by channel: 512 x 8190 in 29,
// bf16 and fp32.
#include "kda_gated.cuh"
#include "kda_slots.cuh"

namespace kda {

namespace {

constexpr int kThreads = 128;

template <typename T, int VEC>
__global__ void __launch_bounds__(kThreads) gated_step_kernel(GatedStepParams p, int blocks) {
    constexpr int N2 = (VEC + 1) / 2;
    const int row = (int)(blockIdx.x / blocks), c = ((int)(blockIdx.x % blocks) * kThreads + (int)threadIdx.x) * VEC;
    const bool on = c < p.C;
    const int cc = on ? c : 0;
    int page[1] = {page_of_row(p.slots, row, p.P)};
    Row<T, VEC> x, r, i, z;
    float h[VEC], lam[VEC];
    float* const state = p.state + (int64_t)max(page[0], 0) * p.C + cc;
    x.load(static_cast<const T*>(p.x) + row * p.ldx + cc);
    r.load(static_cast<const T*>(p.r) + row * p.ldr + cc);
    i.load(static_cast<const T*>(p.i) + row * p.ldi + cc);
    if (p.z) z.load(static_cast<const T*>(p.z) + row * p.ldz + cc);
    if constexpr (VEC > 1) {
#pragma unroll
        for (int k = 0; k < VEC; k += 4) {
            *reinterpret_cast<float4*>(lam + k) = __ldg(reinterpret_cast<const float4*>(p.lam + cc + k));
            // a row without a page reads none: the first page's own row may be writing it
            if (page[0] >= 0) *reinterpret_cast<float4*>(h + k) = *reinterpret_cast<const float4*>(state + k);
        }
    } else {
        lam[0] = __ldg(p.lam + cc);
        if (page[0] >= 0) h[0] = *state;
    }
    if (rows_refused<1>(p.slots, row, p.N, page, p.status)) return;
    f2 xv[N2], rv[N2], iv[N2], zv[N2], y[N2];
    x.to(xv);
    r.to(rv);
    i.to(iv);
    if (p.z) z.to(zv);
#pragma unroll
    for (int k = 0; k < N2; ++k) {
        const int k1 = VEC > 1 ? 2 * k + 1 : 0;
        const f2 rate = pack(gated_rate(lam[2 * k], p.decay), gated_rate(lam[k1], p.decay));
        const Decay d = Decay::of<false>(sigmoid2(rv[k]), rate);
        const f2 u = mul2(mul2(root2(d.m2), sigmoid2(iv[k])), xv[k]);
        const f2 hn = fma2(d.a, pack(h[2 * k], h[k1]), u);
        y[k] = p.z ? mul2(hn, mul2(zv[k], sigmoid2(zv[k]))) : hn;
        float a, b;
        unpack(hn, a, b);
        h[2 * k] = a;
        if (VEC > 1) h[k1] = b;
    }
    if (!on) return;
    if constexpr (VEC > 1) {
#pragma unroll
        for (int k = 0; k < VEC; k += 4) *reinterpret_cast<float4*>(state + k) = *reinterpret_cast<float4*>(h + k);
    } else {
        *state = h[0];
    }
    Row<T, VEC> out;
    out.from(y);
    out.store(static_cast<T*>(p.y) + (int64_t)row * p.C + c);
}

template <typename T, int VEC>
cudaError_t launch(const GatedStepParams& p, cudaStream_t st) {
    const int blocks = (p.C + kThreads * VEC - 1) / (kThreads * VEC);
    gated_step_kernel<T, VEC><<<(unsigned)((int64_t)p.N * blocks), kThreads, 0, st>>>(p, blocks);
    return cudaGetLastError();
}

}  // namespace

cudaError_t gated_step(kda_dtype dt, const GatedStepParams& p, cudaStream_t st) {
    using kda_host::rows_aligned;
    const int vec = dt == KDA_BF16 ? 8 : 4;
    const bool wide = p.C % vec == 0 && rows_aligned(p.x, p.ldx, vec) && rows_aligned(p.r, p.ldr, vec) && rows_aligned(p.i, p.ldi, vec) &&
                      rows_aligned(p.z, p.ldz, vec) && rows_aligned(p.y, p.C, vec) && rows_aligned(p.state, 0, vec) && rows_aligned(p.lam, 0, vec);
    if (dt == KDA_BF16) return wide ? launch<__nv_bfloat16, 8>(p, st) : launch<__nv_bfloat16, 1>(p, st);
    return wide ? launch<float, 4>(p, st) : launch<float, 1>(p, st);
}

}  // namespace kda
