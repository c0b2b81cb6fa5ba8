// The gated linear recurrence's arithmetic, in pairs of channels, and what its kernels share.
//
// Per channel c with rate = decay softplus(lam):
//     s = rate sigmoid(r),  a = e^-s,  m = sqrt(1 - e^-2s),  u = m sigmoid(i) x,  h <- a h + u,  y = h silu(z)
#pragma once

#include "kda_clusters.cuh"
#include "kda_layer.h"

namespace kda {

__device__ __forceinline__ float rsq(float x) {
    float y;
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// rate = decay log(1 + e^lam) of one channel (once a kernel: with the accurate functions).
__device__ __forceinline__ float gated_rate(float lam, float decay) { return decay * (fmaxf(lam, 0.f) + log1pf(expf(-fabsf(lam)))); }

// The decay of a pair of channels from sr = sigmoid(r): a = e^-s with s = rate sr, and m2 = 1 - a^2.  Below s = 1/4 (layers are
// initialised with a in 0.9 ... 0.999), with S = sinh(s) / s = 1 + s^2/6 + s^4/120 and K = (cosh(s) - 1) / s^2 = 1/2 + s^2/24 + s^4/720
// (both to 5e-8): a = 1 + (s^2 K - s S), off by its last rounding only, which a state remembers for 1/s tokens, and m2 = 2 a s S, where
// 1 - a^2 would lose its leading bits.  kSmall: rate < 1/4, so every s is (known once a kernel).
struct Decay {
    f2 a, m2;
    template <bool kSmall>
    static __device__ __forceinline__ Decay of(f2 sr, f2 rate) {
        Decay d;
        const f2 s = mul2(sr, rate), q = mul2(s, s);
        const f2 sinh2 = mul2(s, fma2(q, fma2(q, both(1.f / 60.f), both(1.f / 3.f)), both(2.f)));  // 2 sinh
        const f2 cosh = mul2(q, fma2(q, fma2(q, both(1.f / 720.f), both(1.f / 24.f)), both(0.5f)));
        d.a = add2(fma2(sinh2, both(-0.5f), cosh), both(1.f));
        d.m2 = mul2(d.a, sinh2);
        if constexpr (!kSmall) {
            const f2 e = ex2_2(mul2(s, both(-kLog2e)));
            float s0, s1, x0, x1, y0, y1;
            unpack(s, s0, s1);
            unpack(d.m2, x0, x1);
            unpack(fma2(mul2(e, e), both(-1.f), both(1.f)), y0, y1);
            d.m2 = pack(s0 < 0.25f ? x0 : y0, s1 < 0.25f ? x1 : y1);
            unpack(d.a, x0, x1);
            unpack(e, y0, y1);
            d.a = pack(s0 < 0.25f ? x0 : y0, s1 < 0.25f ? x1 : y1);
        }
        return d;
    }
};
__device__ __forceinline__ bool small_rate(f2 rate) {
    float a, b;
    unpack(rate, a, b);
    return fmaxf(a, b) < 0.25f;
}
// 1 / m; m = m^2 / m.  (m^2 = 0, a closed gate: m = 0.)
__device__ __forceinline__ f2 inverse_root(f2 m2) {
    float a, b;
    unpack(m2, a, b);
    return pack(rsq(fmaxf(a, 1e-36f)), rsq(fmaxf(b, 1e-36f)));
}
__device__ __forceinline__ f2 root2(f2 m2) {
    float a, b;
    unpack(m2, a, b);
    asm("sqrt.approx.ftz.f32 %0, %0;" : "+f"(a));
    asm("sqrt.approx.ftz.f32 %0, %0;" : "+f"(b));
    return pack(a, b);
}
// 1 - x
__device__ __forceinline__ f2 rest2(f2 x) { return fma2(x, both(-1.f), both(1.f)); }

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
__device__ __forceinline__ f2 shuffle2(f2 x, int with) { return __shfl_xor_sync(0xffffffffu, x, with); }
// From the maps of a warp's strips: `total` of all of them, and `before`, that of those which are walked before this lane's (forwards the
// ones in front, backwards those behind).
template <typename L, bool kCuts, bool kForwards>
__device__ __forceinline__ void join_strips(const Affine& mine, Affine& total, Affine& before) {
    total = mine;
    before = identity();
#pragma unroll
    for (int d = 1; d < L::kStrips; d *= 2) {
        const Affine other{shuffle2(total.A, d * L::kPairs), shuffle2(total.H, d * L::kPairs)};
        const bool second = ((L::strip() & d) != 0) == kForwards;  // the other strips are walked before these
        const Affine a = follow<kCuts>(other, total), b = follow<kCuts>(total, other), c = follow<kCuts>(other, before);
        total.A = second ? a.A : b.A;
        total.H = second ? a.H : b.H;
        before.A = second ? c.A : before.A;
        before.H = second ? c.H : before.H;
    }
}

// ---- packed sequences as a warp walks them, strip by strip ------------------------------------------------

// What a warp knows of the sequences at its strip.
template <int STRIP>
struct Marks {
    int start[STRIP], end[STRIP];  // the sequence that a token is the first / last of, or -1
};
template <int STRIP>
struct Walk {
    int sb = 0, se = 0;        // the sequence at hand: its first token, one behind its last
    bool wide = true, clear = true;  // no boundary in the cluster's tiles, in the strip; else the marks are set
    // The strip at s0, the cluster's tiles at [w0, w1).
    __device__ __forceinline__ void look(const Offsets& m, int s0, int w0, int w1, Marks<STRIP>& marks) {
        wide = clear = sb < w0 && w1 < se;
        if (s0 >= m.T) clear = true;
        if (wide || s0 >= m.T) return;
        const int n = m.begun_before(s0 + 1) - 1;
        sb = n >= 0 ? m.begin(n) : 0;
        se = n >= 0 ? m.end(n) : 0;
        clear = sb < s0 && s0 + STRIP < se;
        if (clear) return;
        const int lane = threadIdx.x & 31, behind = m.begun_before(s0 + STRIP);
        __syncwarp();
        for (int j = lane; j < STRIP; j += 32) marks.start[j] = marks.end[j] = -1;
        __syncwarp();
        for (int k = max(m.begun_before(s0) - 1, 0) + lane; k < behind; k += 32) {
            const int s = m.begin(k), e = m.end(k);
            if (e <= s) continue;
            if (s >= s0 && s < s0 + STRIP) marks.start[s - s0] = k;
            if (e > s0 && e <= s0 + STRIP) marks.end[e - 1 - s0] = k;
        }
        __syncwarp();
    }
};

// ---- clusters: the blocks of one channel block work on consecutive tiles at a time ------------------------

// Writes v to the place of `mine` (an address in this block's shared memory) in block `rank` of the cluster.
__device__ __forceinline__ void store_at(unsigned rank, void* mine, const Affine& v) {
    const uint32_t to = address_at(rank, mine);
    asm volatile("st.shared::cluster.v2.b64 [%0], {%1, %2};" ::"r"(to), "l"(v.A), "l"(v.H) : "memory");
}

// ---- tiles -------------------------------------------------------------------------------------------------

// How a warp's lanes lie on CH channels: a lane has a pair of them, and the warp 64 / CH strips of STRIP tokens, one behind the other.
// In shared memory a strip's rows are followed by one that is not used, so that the strips of a warp begin in different banks.
template <int CH, int STRIP>
struct Lanes {
    static constexpr int kPairs = CH / 2, kStrips = 64 / CH, kTokens = kStrips * STRIP;  // of a warp
    static constexpr int kPart = (kStrips == 1 ? STRIP : kStrips * (STRIP + 1)) * CH;    // elements of a warp's rows in shared memory
    static __device__ __forceinline__ int pair() { return threadIdx.x % kPairs; }
    static __device__ __forceinline__ int strip() { return threadIdx.x % 32 / kPairs; }
    static __device__ __forceinline__ int row(int token) { return kStrips == 1 ? token : token + token / STRIP; }
    // Where this lane's pair of its strip's first token is.
    static __device__ __forceinline__ int place() { return row(strip() * STRIP) * CH + 2 * pair(); }
};

// A lane's share of the rows of one tensor's tokens (L::kTokens rows of CH channels, copied by the warp that works on them), by pieces
// of VEC elements.  Tiles are asked for in turn, `step` tokens apart.
template <typename T, int CH, int STRIP, int VEC>
struct Feed {
    using L = Lanes<CH, STRIP>;
    static constexpr int R = L::kTokens;
    static constexpr int PR = CH / VEC;                 // pieces of a row
    static constexpr int N = R * PR / 32;               // pieces of a lane
    static constexpr int ROWS = PR < 32 ? 32 / PR : 1;  // rows between them (one row by several rounds: PR = 64)
    static_assert(R * PR % 32 == 0 && (PR <= 32 || PR == 64), "whole rounds");
    const T* at;         // the next tile's piece of this lane
    int64_t step, more, ld;  // elements to the next tile's, to the lane's next row's, and to the next row's
    __device__ __forceinline__ Feed(const void* base, int64_t ld, int64_t first_row, int c0, int step)
        : at(static_cast<const T*>(base) + (first_row + row()) * ld + c0 + col()), step(step * ld), more(ROWS * ld), ld(ld) {}
    static __device__ __forceinline__ int row() { return threadIdx.x % 32 / PR; }
    static __device__ __forceinline__ int col() { return threadIdx.x % 32 % PR * VEC; }
    // The next tile, all of whose rows and channels are there.
    __device__ __forceinline__ void request(T* tile) {
        if constexpr (PR <= 32 && VEC * sizeof(T) >= 4) {
            const T* from = at;
#pragma unroll
            for (int k = 0; k < N; ++k, from += more) Row<T, VEC>::copy_async(tile + L::row(row() + k * ROWS) * CH + col(), from);
            at += step;
        } else {
            request(tile, R, CH);
        }
    }
    // The next tile, of which `rows` rows are there (none: <= 0) and `has` channels.
    __device__ __forceinline__ void request(T* tile, int rows, int has) {
        const T* from = at;
        const int lines = rows < R ? rows : R;
        if constexpr (VEC * sizeof(T) < 4) {
            // no asynchronous copies of two bytes: sixteen loads of a lane on their way at a time, none of them conditional (what is not
            // there is copied from where something is)
            if (lines > 0) {
                constexpr int H = PR > 32 ? PR / 32 : 1, B = N < 16 ? N : 16;  // elements of a row, and of a batch
                static_assert(N % B == 0, "whole batches");
                const int there = has - 1 - col();
                from += min(0, there);
                from -= row() * ld;
#pragma unroll
                for (int q0 = 0; q0 < N; q0 += B) {
                    T v[B];
#pragma unroll
                    for (int q = 0; q < B; ++q)
                        v[q] = from[min(row() + (q0 + q) / H * ROWS, lines - 1) * ld + min((q0 + q) % H * 32, max(0, there))];
#pragma unroll
                    for (int q = 0; q < B; ++q) tile[L::row(row() + (q0 + q) / H * ROWS) * CH + col() + (q0 + q) % H * 32] = v[q];
                }
            }
            at += step;
            return;
        }
        for (int r = row(); r < lines; r += ROWS, from += more)
#pragma unroll
            for (int h = 0; h < (PR + 31) / 32; ++h) {
                const int c = col() + h * 32 * VEC;
                if (c < has) Row<T, VEC>::copy_async(tile + L::row(r) * CH + c, from + h * 32 * VEC);
            }
        at += step;
    }
};
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

// The rows that a block takes, [row0, row0 + T), and the tokens of them that count, [first, last).
struct Stretch {
    int64_t row0;
    int T, first, last;
};
// Sequence n of a stream by itself: from the state that is left to the backward pass before its first token.  kEdges: with the stream's
// rows that belong to no sequence.  A sequence without tokens has no rows, but for those.
template <bool kEdges>
__device__ __forceinline__ Stretch sequence_rows(const GatedParams& p, int n) {
    const int begin = min(max(__ldg(p.cu + n), 0), p.T), end = min(max(__ldg(p.cu + n + 1), begin), p.T);
    const int from = kEdges && n == 0 ? 0 : begin / kGatedBlock * kGatedBlock, to = kEdges && n == p.N - 1 ? p.T : end;
    const bool none = begin == end && !(kEdges && (n == 0 || (n == p.N - 1 && end < p.T)));
    return {from, none ? 0 : to - from, begin - from, end - from};
}

// Whether a sequence of the stream has more than `most` tokens (every thread of the block calls it).
__device__ __forceinline__ bool any_longer(const GatedParams& p, int most) {
    bool found = false;
#pragma unroll 4
    for (int n = threadIdx.x; n < p.N; n += blockDim.x) {
        const int begin = min(max(__ldg(p.cu + n), 0), p.T), end = min(max(__ldg(p.cu + n + 1), 0), p.T);
        found |= end - begin > most;
    }
    return __syncthreads_or(found) != 0;
}

// Sequences that are packed in one stream have blocks of their own, unless they are so short that these would be mostly idle (`mean`
// tokens), or one of them alone would take them more than twice as many steps as the stream takes as a whole, at `pace` and `stream` tokens a
// step.  Only the offsets say so, on the device: both kernels are launched.  A long sequence's own blocks return at once, and the stream's kernel,
// behind them, looks for one and does everything again or nothing (a block that has one sequence does not look at all the others).
// (bf16 with gates, 4096 channels, decays of 0.9 to 0.999, forward and backward: 16 sequences of 1 to 700 tokens 61 and 105 us with blocks of their own,
// 77 and 156 as one stream; 128 x 128 139 and 266, 242 and 572; 256 x 64 282 and 308, 263 and 595; 512 x 32 574 and 410, 269 and 596; 1024 x 16
// 1146 and 704, 273 and 659; one of 16129 among 15 of 17 302 and 1051, 172 and 398, and as chosen, with the look for it, 197 and 417)
inline bool gated_each(const GatedParams& p, int mean) { return p.cu && p.N > 0 && p.N <= p.T / mean; }
inline int longest_of(const GatedParams& p, int64_t pace, int64_t stream) {
    const int64_t most = (p.T + stream - 1) / stream * 2 * pace;
    return p.N > 1 && most < p.T ? (int)most : p.T;
}
// The blocks of a sequence: one where there is one an SM anyway.
template <typename K>
cudaError_t gated_cluster(ClusterRoom& room, K kern, int64_t groups, int T, int tile, int threads, int smem, int& cluster) {
    cluster = 1;
    return groups > kSms ? cudaSuccess : room.size_for(kern, groups, T, tile, threads, smem, cluster);
}

// Channels of a block. 64 where blocks of them that take a whole sequence each come to one and a half an SM (two run on one); else 32 where
// those do; else blocks share a sequence as a cluster whatever their width, and the widest rows cost least (1 x 16384 x 4096: 151, 155 and
// 171 us with 64, 32 and 16) as long as clusters of eight fill the machine (1 x 65536 x 512: 213, 155, 104).
// bf16 with gates, 4096 channels, B sequences of 2048, forward and backward with 64 | 32 | 16 channels:
//     2: 41.5 and 91.5 | 37.7 and 74.0 | 48.5 and 87.6      3: 66.8 and 137 | 56.6 and 115 | 68.9 and 127     4: 66.8 and 138 | 71.4 and 144 | 84.2 and 150
//     5: 98.2 and 216 | 88.3 and 180 | 104 and 189          7: 100 and 219 | 106 and 212 | 140 and 250        9: 127 and 269 | 136 and 279 | 180 and 326
// (5 sequences come to 320 blocks of 64 channels for 304 places, a second filling for sixteen: there the rule does not choose the best.)
inline int gated_channels(const GatedParams& p, int streams) {
    for (const int blocks : {1, kMostCluster})
        for (const int ch : {64, 32})
            if ((int64_t)((p.C + ch - 1) / ch) * streams * blocks >= kSms * 3 / 2) return ch;
    return 16;
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
