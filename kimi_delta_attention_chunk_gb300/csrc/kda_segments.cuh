// Sequences packed along one token axis, as the convolution and scan kernels walk them, and
// vector access to rows.
//
// A kernel works on tiles of the flat token stream whose positions come from the host's sizes
// alone; where sequences begin and end inside a tile is read from cu_seqlens on the device.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "kda_common.cuh"

namespace kda {

// N sequences in a stream of `total` tokens: packed by cu (N + 1 offsets), or T tokens each.
struct SeqMap {
    const int32_t* cu;
    int N, T, total;

    __device__ __forceinline__ int begin(int n) const {
        return cu ? min(max(__ldg(cu + n), 0), total) : n * T;
    }
    __device__ __forceinline__ int end(int n) const { return begin(n + 1); }
    // Tokens outside [first, last) belong to no sequence.
    __device__ __forceinline__ int first() const { return N > 0 ? begin(0) : 0; }
    __device__ __forceinline__ int last() const { return N > 0 ? begin(N) : 0; }

    // How many sequences begin before token `key` (a whole warp calls it with one key).  A
    // search by 32 probes a round: two dependent loads up to 1024 sequences.  On offsets that
    // are not sorted it still ends and stays within [0, N].
    __device__ __forceinline__ int begun_before(int key) const {
        if (!cu) return key <= 0 || T <= 0 ? 0 : min(N, (key - 1) / T + 1);
        const int lane = threadIdx.x & 31;
        int lo = 0, hi = N;
        while (hi > lo) {
            const int step = (hi - lo + 31) / 32;
            const int at = lo + (lane + 1) * step - 1;
            const bool below = at < hi && begin(at) < key;
            const int cnt = __popc(__ballot_sync(0xffffffffu, below));
            const int next = min(hi, lo + (cnt + 1) * step - 1);
            lo = min(hi, lo + cnt * step);
            hi = max(lo, next);
            if (step == 1) break;
        }
        return lo;
    }
};

// The sequences of tokens [t0, t0 + TT): start[i] / end[i] is the sequence that token t0 + i
// is the first / last of, or -1.  carry: the sequence that token t0 continues (-1: none), which
// began at carry_start.  Behind the tile the sequence at hand runs on to token `until`: a tile
// that ends before it has no boundary and needs no look.
template <int TT>
struct TokenTile {
    int start[TT], end[TT];
    int carry, carry_start, n0, until;

    // Every thread of the block calls it; the block has to be past its last use of the tile.
    template <int NTH>
    __device__ __forceinline__ void build(const SeqMap& m, int t0) {
        const int tid = threadIdx.x;
        for (int i = tid; i < TT; i += NTH) start[i] = end[i] = -1;
        if (tid < 32) {
            const int n = m.begun_before(t0), n1 = m.begun_before(t0 + TT);
            if (tid == 0) {
                n0 = n;
                carry = -1;
                carry_start = t0;
                until = n1 > 0 ? m.end(n1 - 1) : t0;
            }
        }
        __syncthreads();
        const int first = n0;
        if (tid == 0 && first > 0) {
            const int e = m.end(first - 1);
            if (e > t0) {
                carry = first - 1;
                carry_start = min(m.begin(first - 1), t0);
                if (e - t0 <= TT) end[e - 1 - t0] = first - 1;
            }
        }
        for (int n = first + tid; n < m.N; n += NTH) {
            const int s = m.begin(n);
            if (s - t0 >= TT) break;
            const int e = m.end(n);
            if (s < t0 || e <= s) continue;
            start[s - t0] = n;
            if (e - t0 <= TT) end[e - 1 - t0] = n;
        }
        __syncthreads();
    }
};

// ---- rows of VEC elements ------------------------------------------------------------------

// load() reads data that no thread writes during the kernel, load_rw() any data.
template <typename T, int VEC>
struct Row;
template <>
struct Row<__nv_bfloat16, 8> {
    uint4 r;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { r = __ldg(reinterpret_cast<const uint4*>(p)); }
    __device__ __forceinline__ void load_rw(const __nv_bfloat16* p) { r = *reinterpret_cast<const uint4*>(p); }
    __device__ __forceinline__ void to(float* f) const {
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    __device__ __forceinline__ void from(const float* f) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 v = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&v);
        }
        r = make_uint4(w[0], w[1], w[2], w[3]);
    }
    __device__ __forceinline__ void store(__nv_bfloat16* p) const { *reinterpret_cast<uint4*>(p) = r; }
    __device__ __forceinline__ void zero() { r = make_uint4(0, 0, 0, 0); }
};
template <>
struct Row<float, 4> {
    float4 r;
    __device__ __forceinline__ void load(const float* p) { r = __ldg(reinterpret_cast<const float4*>(p)); }
    __device__ __forceinline__ void load_rw(const float* p) { r = *reinterpret_cast<const float4*>(p); }
    __device__ __forceinline__ void to(float* f) const { f[0] = r.x; f[1] = r.y; f[2] = r.z; f[3] = r.w; }
    __device__ __forceinline__ void from(const float* f) { r = make_float4(f[0], f[1], f[2], f[3]); }
    __device__ __forceinline__ void store(float* p) const { *reinterpret_cast<float4*>(p) = r; }
    __device__ __forceinline__ void zero() { r = make_float4(0.f, 0.f, 0.f, 0.f); }
};
template <>
struct Row<float, 8> {
    float4 a, b;
    __device__ __forceinline__ void load(const float* p) {
        a = __ldg(reinterpret_cast<const float4*>(p));
        b = __ldg(reinterpret_cast<const float4*>(p) + 1);
    }
    __device__ __forceinline__ void to(float* f) const {
        f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
        f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
    }
    __device__ __forceinline__ void from(const float* f) {
        a = make_float4(f[0], f[1], f[2], f[3]);
        b = make_float4(f[4], f[5], f[6], f[7]);
    }
    __device__ __forceinline__ void store(float* p) const {
        reinterpret_cast<float4*>(p)[0] = a;
        reinterpret_cast<float4*>(p)[1] = b;
    }
    __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
};
template <typename T>
struct Row<T, 1> {
    T r;
    __device__ __forceinline__ void load(const T* p) { r = __ldg(p); }
    __device__ __forceinline__ void load_rw(const T* p) { r = *p; }
    __device__ __forceinline__ void to(float* f) const { f[0] = to_f32<T>(r); }
    __device__ __forceinline__ void from(const float* f) { r = from_f32<T>(f[0]); }
    __device__ __forceinline__ void store(T* p) const { *p = r; }
    __device__ __forceinline__ void zero() { r = from_f32<T>(0.f); }
};

// 2^x by the special-function unit (relative error about 2^-22; 0 below the normal range).
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
constexpr float kLog2e = 1.4426950408889634f;
// 1 / (1 + e^-x).  e^-x may overflow to infinity: the quotient is then 0, as it should be.
__device__ __forceinline__ float sigmoid(float x) { return __frcp_rn(1.0f + ex2(-kLog2e * x)); }

}  // namespace kda

// Whether rows of VEC-element pieces can be used: base 16-byte aligned, row length and row
// stride whole pieces.
namespace kda_host {
inline bool rows_aligned(const void* p, int64_t ld, int vec) { return p == nullptr || (aligned16(p) && ld % vec == 0); }
}  // namespace kda_host
