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
// that ends before it has no boundary and needs no look.  plain: one sequence runs through the tile
// and on.  marks: the tokens (bits) that are the first or last of a sequence.
template <int TT>
struct TokenTile {
    int start[TT], end[TT];
    unsigned marks[2];
    int carry, carry_start, n0, until;
    bool plain;
    static_assert(TT <= 64, "one bit a token");

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
                plain = n > 0 && n1 == n && until > t0 + TT;
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
        if (tid < 64) {
            const bool mark = tid < TT && (start[tid < TT ? tid : 0] >= 0 || end[tid < TT ? tid : 0] >= 0);
            const unsigned b = __ballot_sync(0xffffffffu, mark);
            if (tid % 32 == 0) marks[tid / 32] = b;
        }
        __syncthreads();
    }

    // Whether tokens k ... k + N - 1 of the tile (within a half of it) lie inside one sequence.
    template <int N>
    __device__ __forceinline__ bool clear(int k) const {
        return (marks[k >> 5] >> (k & 31) & ((1u << N) - 1)) == 0;
    }
};

// ---- two fp32 values in one 64-bit register ------------------------------------------------

typedef unsigned long long f2;
__device__ __forceinline__ f2 pack(float a, float b) {
    f2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpack(f2 x, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x)); }
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
    f2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
    f2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
    f2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ float sum2(f2 x) {
    float a, b;
    unpack(x, a, b);
    return a + b;
}

// ---- rows of VEC elements ------------------------------------------------------------------

// VEC elements of a row as they lie in memory (VEC = 1, or 8 or 16 bytes).
template <int BYTES>
struct Bits;
template <> struct Bits<16> { typedef uint4 type; };
template <> struct Bits<8> { typedef uint2 type; };
template <> struct Bits<4> { typedef uint32_t type; };
template <> struct Bits<2> { typedef unsigned short type; };

// load() reads data that no thread writes during the kernel, load_rw() any data.
template <typename T, int VEC>
struct Row {
    static constexpr int kBytes = VEC * (int)sizeof(T);
    typedef typename Bits<kBytes>::type Raw;
    static constexpr int N2 = (VEC + 1) / 2;  // pairs (VEC = 1: one, its upper half zero)
    Raw r;
    __device__ __forceinline__ void load(const T* p) { r = __ldg(reinterpret_cast<const Raw*>(p)); }
    __device__ __forceinline__ void load_rw(const T* p) { r = *reinterpret_cast<const Raw*>(p); }
    __device__ __forceinline__ void store(T* p) const { *reinterpret_cast<Raw*>(p) = r; }
    __device__ __forceinline__ void zero() { r = Raw{}; }
    __device__ __forceinline__ void to(f2 (&v)[N2]) const {
        if constexpr (VEC == 1) {
            v[0] = pack(to_f32<T>(*reinterpret_cast<const T*>(&r)), 0.f);
        } else if constexpr (sizeof(T) == 2) {
            const uint32_t* w = reinterpret_cast<const uint32_t*>(&r);
#pragma unroll
            for (int i = 0; i < N2; ++i) v[i] = pack(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
        } else {
            const float* w = reinterpret_cast<const float*>(&r);
#pragma unroll
            for (int i = 0; i < N2; ++i) v[i] = pack(w[2 * i], w[2 * i + 1]);
        }
    }
    __device__ __forceinline__ void from(const f2 (&v)[N2]) {
        if constexpr (VEC == 1) {
            float a, b;
            unpack(v[0], a, b);
            const T x = from_f32<T>(a);
            r = *reinterpret_cast<const Raw*>(&x);
        } else if constexpr (sizeof(T) == 2) {
            uint32_t* w = reinterpret_cast<uint32_t*>(&r);
#pragma unroll
            for (int i = 0; i < N2; ++i) {
                float a, b;
                unpack(v[i], a, b);
                const __nv_bfloat162 x = __floats2bfloat162_rn(a, b);
                w[i] = *reinterpret_cast<const uint32_t*>(&x);
            }
        } else {
            float* w = reinterpret_cast<float*>(&r);
#pragma unroll
            for (int i = 0; i < N2; ++i) unpack(v[i], w[2 * i], w[2 * i + 1]);
        }
    }
    // Copies a row's piece into shared memory without waiting (two bytes: at once).
    static __device__ __forceinline__ void copy_async(void* shared, const T* p) {
        if constexpr (kBytes >= 4) {
            const uint32_t s = (uint32_t)__cvta_generic_to_shared(shared);
            if constexpr (kBytes == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(s), "l"(p) : "memory");
            else asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(s), "l"(p), "n"(kBytes) : "memory");
        } else {
            *reinterpret_cast<Raw*>(shared) = __ldg(reinterpret_cast<const Raw*>(p));
        }
    }
    __device__ __forceinline__ void from_shared(const void* shared) { r = *reinterpret_cast<const Raw*>(shared); }
};
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// 2^x and 1 / x by the special-function unit (relative errors about 2^-22 and 2^-23; subnormal
// numbers count as zero).
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
constexpr float kLog2e = 1.4426950408889634f;
// 1 / (1 + e^-x).  e^-x may overflow to infinity: the quotient is then 0, as it should be.
__device__ __forceinline__ float sigmoid(float x) { return rcp(1.0f + ex2(-kLog2e * x)); }
__device__ __forceinline__ f2 ex2_2(f2 x) {
    float a, b;
    unpack(x, a, b);
    return pack(ex2(a), ex2(b));
}
__device__ __forceinline__ f2 sigmoid2(f2 x) {
    float a, b;
    unpack(x, a, b);
    return pack(sigmoid(a), sigmoid(b));
}

}  // namespace kda

// Whether rows of VEC-element pieces can be used: base 16-byte aligned, row length and row
// stride whole pieces.
namespace kda_host {
inline bool rows_aligned(const void* p, int64_t ld, int vec) { return p == nullptr || (aligned16(p) && ld % vec == 0); }
}  // namespace kda_host
