// The gated linear recurrence's arithmetic, in pairs of channels, and what its kernels share.
//
// Per channel c with rate = decay softplus(lam):
//     s = rate sigmoid(r),  a = e^-s,  m = sqrt(1 - e^-2s),  u = m sigmoid(i) x,  h <- a h + u,  y = h silu(z)
#pragma once

#include "kda_layer.h"
#include "kda_segments.cuh"

namespace kda {

constexpr int kSms = 152;
constexpr int kGatedThreads = 256, kGatedWarps = kGatedThreads / 32;
constexpr int kGatedCh = 64;  // channels of a block: a pair a lane, 128 bytes of a bf16 row
constexpr int kMostCluster = 8;

__device__ __forceinline__ f2 both(float v) { return pack(v, v); }
__device__ __forceinline__ f2 neg2(f2 x) { return x ^ 0x8000000080000000ull; }
__device__ __forceinline__ float rsq(float x) {
    float y;
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// rate = decay log(1 + e^lam) of one channel (once a kernel: with the accurate functions).
__device__ __forceinline__ float gated_rate(float lam, float decay) { return decay * (fmaxf(lam, 0.f) + log1pf(expf(-fabsf(lam)))); }

// 1 + e^-x, for sigmoid(x) = 1 / it.  kBound: no more than 2^60, so that the product of two can be inverted; sigmoid then ends at
// 2^-60 where it would go on to zero.
template <bool kBound>
__device__ __forceinline__ f2 one_plus(f2 x) {
    f2 t = mul2(x, both(-kLog2e));
    if constexpr (kBound) {
        float a, b;
        unpack(t, a, b);
        t = pack(fminf(a, 60.f), fminf(b, 60.f));
    }
    return add2(ex2_2(t), both(1.f));
}
__device__ __forceinline__ f2 rcp2(f2 x) {
    float a, b;
    unpack(x, a, b);
    return pack(rcp(a), rcp(b));
}

// The decay of a pair of channels from sigmoid(r): a, and a^2 and m^2 = 1 - e^-2s.  Where s < 1/4, 1 - e^-2s would lose its leading bits
// (layers are initialised with a in 0.9 ... 0.999); it is 2 a sinh(s) there, with sinh(s) / s = 1 + s^2/6 + s^4/120 to 5e-8.
struct Decay {
    f2 a, m2;
    __device__ __forceinline__ Decay(f2 sr, f2 rate) {
        const f2 s = mul2(sr, rate);
        a = ex2_2(mul2(s, both(-kLog2e)));
        const f2 q = mul2(s, s);
        const f2 series = fma2(q, fma2(q, both(1.f / 120.f), both(1.f / 6.f)), both(1.f));
        const f2 small = mul2(mul2(mul2(a, s), both(2.f)), series), large = fma2(neg2(a), a, both(1.f));
        float s0, s1, x0, x1, y0, y1;
        unpack(s, s0, s1);
        unpack(small, x0, x1);
        unpack(large, y0, y1);
        m2 = pack(s0 < 0.25f ? x0 : y0, s1 < 0.25f ? x1 : y1);
    }
};
// 1 / m; m = m^2 / m.  (m^2 = 0, a closed gate: m = 0.)
__device__ __forceinline__ f2 inverse_root(f2 m2) {
    float a, b;
    unpack(m2, a, b);
    return pack(rsq(fmaxf(a, 1e-36f)), rsq(fmaxf(b, 1e-36f)));
}

// h -> A h + H.  Where a sequence begins inside (kCuts), A's sign bit is set and h does not reach the end, be it infinite or NaN.
struct __align__(16) Affine {
    f2 A, H;
};
__device__ __forceinline__ f2 pick(f2 sign, f2 set, f2 clear) {
    float s0, s1, a0, a1, b0, b1;
    unpack(sign, s0, s1);
    unpack(set, a0, a1);
    unpack(clear, b0, b1);
    return pack(__float_as_int(s0) < 0 ? a0 : b0, __float_as_int(s1) < 0 ? a1 : b1);
}
template <bool kCuts>
__device__ __forceinline__ f2 apply(f2 A, f2 H, f2 h) {
    const f2 on = fma2(A, h, H);
    if constexpr (kCuts) return pick(A, H, on);
    return on;
}
// `first`, then `then`.
template <bool kCuts>
__device__ __forceinline__ Affine follow(const Affine& first, const Affine& then) {
    Affine r;
    r.H = apply<kCuts>(then.A, then.H, first.H);
    r.A = mul2(first.A, then.A);
    if constexpr (kCuts) r.A = pick(then.A, then.A, r.A);
    return r;
}
__device__ __forceinline__ Affine identity() { return Affine{both(1.f), 0ull}; }

// ---- clusters: the blocks of one channel block work on consecutive tiles at a time ------------------------

__device__ __forceinline__ unsigned cluster_rank() {
    unsigned r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }
// Writes v to the place of `mine` (an address in this block's shared memory) in block `rank` of the cluster.
__device__ __forceinline__ void store_at(unsigned rank, void* mine, const Affine& v) {
    uint32_t to;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(to) : "r"((uint32_t)__cvta_generic_to_shared(mine)), "r"(rank));
    asm volatile("st.shared::cluster.v2.b64 [%0], {%1, %2};" ::"r"(to), "l"(v.A), "l"(v.H) : "memory");
}

// ---- tiles -------------------------------------------------------------------------------------------------

// Requests `rows` rows of `has` channels at `from`, ld apart, into a tile [..][kGatedCh], by pieces of VEC elements.
template <typename T, int TT, int VEC>
__device__ __forceinline__ void request_rows(T* tile, const T* from, int64_t ld, int rows, int has) {
    constexpr int PR = kGatedCh / VEC;
#pragma unroll
    for (int k = 0; k < TT * PR; k += kGatedThreads) {
        const int e = k + (int)threadIdx.x, r = e / PR, c = e % PR * VEC;
        if ((TT * PR % kGatedThreads == 0 || e < TT * PR) && r < rows && c < has) Row<T, VEC>::copy_async(tile + r * kGatedCh + c, from + r * ld + c);
    }
}
template <typename T>
__device__ __forceinline__ f2 pair_at(const T* shared) {
    Row<T, 2> p;
    p.from_shared(shared);
    f2 v[1];
    p.to(v);
    return v[0];
}
// Stores a pair of channels; kWhole: pairs are whole and aligned.  n: how many of the two there are.
template <typename T, bool kWhole>
__device__ __forceinline__ void store_pair(T* to, f2 x, int n) {
    if constexpr (kWhole) {
        Row<T, 2> p;
        const f2 v[1] = {x};
        p.from(v);
        if (n > 0) p.store(to);
    } else {
        float a, b;
        unpack(x, a, b);
        if (n > 0) to[0] = from_f32<T>(a);
        if (n > 1) to[1] = from_f32<T>(b);
    }
}
// A pair of fp32 states (any alignment of pairs); null: zeros.
__device__ __forceinline__ f2 state_pair(const float* p, int64_t at, int n) {
    return p ? pack(n > 0 ? __ldg(p + at) : 0.f, n > 1 ? __ldg(p + at + 1) : 0.f) : 0ull;
}
__device__ __forceinline__ void store_state(float* p, int64_t at, f2 h, int n) {
    float a, b;
    unpack(h, a, b);
    if (n > 0) p[at] = a;
    if (n > 1) p[at + 1] = b;
}

// Launches a kernel in clusters of `cluster` blocks.
template <typename... KArgs, typename... Args>
cudaError_t launch_clusters(void (*kern)(KArgs...), int64_t grid, int cluster, int smem, cudaStream_t st, Args... args) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = kGatedThreads;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = cluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, static_cast<KArgs>(args)...);
}

// Blocks of a cluster: as many as bring the call's blocks to about two an SM, no more than there are tiles.
inline int cluster_size(int64_t groups, int T, int tile) {
    int k = 1;
    while (k < kMostCluster && groups * k * 2 <= 2 * kSms && (int64_t)k * tile < T) k *= 2;
    return k;
}

// Whether rows of p can be read by pieces of `bytes`: every pointer, stride and the row's length.
inline bool gated_pieces(const GatedParams& p, int es, int bytes) {
    const void* rows[] = {p.x, p.r, p.i, p.z};
    const int64_t ld[] = {p.ldx, p.ldr, p.ldi, p.ldz};
    if ((int64_t)p.C * es % bytes != 0) return false;
    for (int k = 0; k < 4; ++k)
        if (rows[k] && ((uintptr_t)rows[k] % bytes != 0 || ld[k] * es % bytes != 0)) return false;
    return true;
}

}  // namespace kda
