// Group norm with an activation, channels last, over each token's groups of channels (the formulas stand in kda_group_norm.cuh).
//
// Every row is read once and stays in registers between the statistics and the output: HBM bounds it, and instruction issue where
// pieces are small.  A team of lanes owns a group of channels (16 lanes of 16 bytes for 128 bf16 channels), teams lie side by side
// along a row, and a block walks down the rows with its weights, and backwards its share of dw and db, in registers.  Mean, then the
// sum of squares around it: two sums over a team, by shuffles up to 32 lanes and through shared memory beyond.  Groups of up to
// 16384 channels fit a block.
// bf16 with SiLU, 4096 x 12288: 96 groups of 128 channels 36 us forwards (84% of the bytes at the copy rate) and 66.5 backwards (68%: 30
// instructions an element at 2.6 a cycle, of 24 warps); one group 88 and 176, where a row's sums wait for one another.
#pragma once

#include <type_traits>

#include "kda_group_norm.cuh"

namespace kda {

namespace {

constexpr int kDeclared = 512;  // shared memory that a kernel declares, at most

// Which channels and rows the threads of a block have.
struct Teams {
    int lanes;    // of a team: a power of two up to 32, or whole warps
    int groups;   // side by side in a block
    int rows;     // rows that a block has at a time
    int threads;  // of a block
    bool wide_weights;
};

// A variant: R pieces of VEC elements a lane, blocks of up to NTH threads; LANES: teams of so many lanes that the group's pieces fill
// exactly and that fill the row's groups (0: any team).
template <int VEC_, int R_, int NTH_, int LANES_>
struct Variant {
    static constexpr int VEC = VEC_, R = R_, NTH = NTH_, LANES = LANES_, E = R * VEC, E2 = E / 2;
    static_assert(E % 2 == 0, "values go in pairs");
    // A thread's rows in shared memory, one of them at work and the others under way; with one, the next is asked for when this one is in
    // registers; two-byte pieces have no asynchronous copy and none.
    static constexpr int kSlots = VEC == 1 ? 0 : E <= 16 && NTH <= 512 ? 4 : 1;
    static constexpr bool kKeep = E <= 8;  // the weights: kept, or read again for every row
    // Backwards, dw and db of a thread's channels: in registers, or where they are many in shared memory.
    static constexpr bool kSharedSums = E > 16 || NTH > 512;
    static constexpr int kFwd = NTH != 256 ? 1 : E > 16 ? 2 : E > 8 ? 3 : 4, kBwd = NTH != 256 ? 1 : E > 8 ? 2 : 3;  // blocks an SM
};

// Sums of `N` values over every team.  Teams of more than a warp meet in shared memory, in a buffer of their own each time.
template <int LANES, int NTH>
struct TeamSum {
    static constexpr int W = NTH / 32;
    float (*buf)[W][2];  // [2]
    int lanes, turn = 0, from = 0;
    bool reads = false;  // of the warps' sums this lane reads one: entry `from`
    __device__ __forceinline__ TeamSum(float (*buf)[W][2], int lanes) : buf(buf), lanes(lanes) {
        if (LANES > 0 || lanes <= 32) return;
        const int w = threadIdx.x / 32, team = lanes / 32;
        reads = (int)threadIdx.x % W < team;
        from = w / team * team + threadIdx.x % W;
    }
    template <int N>
    __device__ __forceinline__ void operator()(float (&v)[N]) {
        if constexpr (LANES > 0) {
            all<LANES>(v);
        } else {
            if (lanes >= 32) {
                all<32>(v);
            } else {
#pragma unroll
                for (int o = 16; o > 0; o /= 2)
                    if (o < lanes)
#pragma unroll
                        for (int k = 0; k < N; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
            }
            if (lanes <= 32) return;
            if (threadIdx.x % 32 == 0)
#pragma unroll
                for (int k = 0; k < N; ++k) buf[turn][threadIdx.x / 32][k] = v[k];
            __syncthreads();
#pragma unroll
            for (int k = 0; k < N; ++k) v[k] = reads ? buf[turn][from][k] : 0.f;
            all<W>(v);
            turn ^= 1;
        }
    }
    template <int L, int N>
    static __device__ __forceinline__ void all(float (&v)[N]) {
        if constexpr (N == 2 && L >= 8) {  // half of the lanes sum the one, half the other
            const bool up = threadIdx.x & (L / 2);
            float mine = up ? v[1] : v[0];
            mine += __shfl_xor_sync(0xffffffffu, up ? v[0] : v[1], L / 2);
#pragma unroll
            for (int o = L / 4; o > 0; o /= 2) mine += __shfl_xor_sync(0xffffffffu, mine, o);
            const float other = __shfl_xor_sync(0xffffffffu, mine, L / 2);
            v[0] = up ? other : mine;
            v[1] = up ? mine : other;
            return;
        }
#pragma unroll
        for (int o = L / 2; o > 0; o /= 2)
#pragma unroll
            for (int k = 0; k < N; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
    }
};

// A thread's place: its group, its row among those that the block has at a time, and its pieces of the group.  Pair j of its values is
// half of a piece, or (VEC = 1) two pieces.
template <typename V>
struct Place {
    int g, rsub, cg, lane, lanes, first;
    __device__ __forceinline__ Place(const NormParams& p, const Teams& t) {
        lanes = V::LANES > 0 ? V::LANES : t.lanes;
        const int team = threadIdx.x / lanes;
        lane = threadIdx.x % lanes;
        g = blockIdx.x * t.groups + team % t.groups;
        rsub = team / t.groups;
        cg = p.C / p.G;
        first = g * cg + lane * V::VEC;
        if (V::LANES == 0 && g >= p.G) cg = first = 0;
    }
    __device__ __forceinline__ bool has(int k) const { return V::LANES > 0 || (lane + k * lanes) * V::VEC < cg; }
    // Channels between a thread's first piece and its k-th.
    __device__ __forceinline__ int apart(int k) const { return k * lanes * V::VEC; }
    // x where pair j has values, zeros elsewhere.
    __device__ __forceinline__ f2 masked(int j, f2 x) const {
        if constexpr (V::LANES > 0) return x;
        if constexpr (V::VEC > 1) return has(2 * j / V::VEC) ? x : 0ull;
        float a, b;
        unpack(x, a, b);
        return pack(has(2 * j) ? a : 0.f, has(2 * j + 1) ? b : 0.f);
    }
};

// A thread's pieces of a row from memory into pairs (zeros where there are none) and back.
template <typename V, typename T>
struct Pieces {
    Row<T, V::VEC> r[V::R];
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int k = 0; k < V::R; ++k) r[k].zero();
    }
    __device__ __forceinline__ void pairs(f2 (&v)[V::E2]) const {
        if constexpr (V::VEC == 1) {
#pragma unroll
            for (int j = 0; j < V::E2; ++j) {
                f2 a[1], b[1];
                r[2 * j].to(a);
                r[2 * j + 1].to(b);
                float x, y, none;
                unpack(a[0], x, none);
                unpack(b[0], y, none);
                v[j] = pack(x, y);
            }
        } else {
#pragma unroll
            for (int k = 0; k < V::R; ++k) {
                f2 a[V::VEC / 2];
                r[k].to(a);
#pragma unroll
                for (int e = 0; e < V::VEC / 2; ++e) v[k * (V::VEC / 2) + e] = a[e];
            }
        }
    }
    static __device__ __forceinline__ void store(const Place<V>& at, T* to, const f2 (&v)[V::E2]) {
#pragma unroll
        for (int k = 0; k < V::R; ++k) {
            if (!at.has(k)) continue;
            Row<T, V::VEC> out;
            if constexpr (V::VEC == 1) {
                float a, b;
                unpack(v[k / 2], a, b);
                const f2 one[1] = {pack(k % 2 ? b : a, 0.f)};
                out.from(one);
            } else {
                f2 a[V::VEC / 2];
#pragma unroll
                for (int e = 0; e < V::VEC / 2; ++e) a[e] = v[k * (V::VEC / 2) + e];
                out.from(a);
            }
            out.store(to + at.apart(k));
        }
    }
};

// A thread's own rows, every next-th element from `from` on: asked for ahead through shared memory (what a thread asks for it alone
// reads, so that no thread waits for another), or loaded when their turn comes.
template <typename V, typename T, int A>
struct Rows {
    static constexpr int kBytes = A * V::R * V::NTH * V::VEC * (int)sizeof(T);
    const T* from;
    int64_t next;
    T* mine;
    __device__ __forceinline__ Rows(const void* base, int64_t first, int64_t ld, int64_t step, const Place<V>& at, void* shared)
        : from(static_cast<const T*>(base) + first * ld + at.first), next(step * ld), mine(static_cast<T*>(shared) + threadIdx.x * V::VEC) {}
    __device__ __forceinline__ T* slot(int i, int k) const { return mine + ((A > 1 ? i % A : 0) * V::R + k) * V::NTH * V::VEC; }
    __device__ __forceinline__ void request(int i, const Place<V>& at) {
#pragma unroll
        for (int k = 0; k < V::R; ++k)
            if (at.has(k)) Row<T, V::VEC>::copy_async(slot(i, k), from + at.apart(k));
        from += next;
    }
    __device__ __forceinline__ void take(int i, const Place<V>& at, Pieces<V, T>& p) {
        if constexpr (A > 0) {
#pragma unroll
            for (int k = 0; k < V::R; ++k)
                if (at.has(k)) p.r[k].from_shared(slot(i, k));
                else p.r[k].zero();
        } else {
#pragma unroll
            for (int k = 0; k < V::R; ++k)
                if (at.has(k)) p.r[k].load(from + at.apart(k));
                else p.r[k].zero();
            from += next;
        }
    }
};

// 1 / sqrt(var + eps): the accurate function, for which subnormal numbers count and what is not a number (the variance around an infinite
// mean) stays so.
__device__ __forceinline__ float inverse_deviation(float m2, float inv_n, float eps) { return rsqrtf(fmaf(m2, inv_n, eps)); }

// One of the weights of a thread's channels in pairs, `none` without weights.
template <typename V>
__device__ __forceinline__ void weight_pairs(const float* p, float none, const Place<V>& at, bool wide, f2 (&v)[V::E2]) {
    if (!p) {
#pragma unroll
        for (int j = 0; j < V::E2; ++j) v[j] = both(none);
        return;
    }
    p += at.first;
    if constexpr (V::VEC >= 4) {
        if (wide) {
#pragma unroll
            for (int k = 0; k < V::R; ++k)
#pragma unroll
                for (int e = 0; e < V::VEC / 4; ++e) {
                    float4 x = make_float4(none, none, none, none);
                    if (at.has(k)) x = __ldg(reinterpret_cast<const float4*>(p + at.apart(k)) + e);
                    v[k * (V::VEC / 2) + 2 * e] = pack(x.x, x.y);
                    v[k * (V::VEC / 2) + 2 * e + 1] = pack(x.z, x.w);
                }
            return;
        }
    }
#pragma unroll
    for (int j = 0; j < V::E2; ++j) {
        const int k0 = V::VEC > 1 ? 2 * j / V::VEC : 2 * j, k1 = V::VEC > 1 ? k0 : k0 + 1, e = V::VEC > 1 ? 2 * j % V::VEC : 0;
        const float a = at.has(k0) ? __ldg(p + at.apart(k0) + e) : none, b = at.has(k1) ? __ldg(p + at.apart(k1) + (V::VEC > 1 ? e + 1 : 0)) : none;
        v[j] = pack(a, b);
    }
}
template <typename V>
struct Weights {
    f2 w[V::E2], b[V::E2];
    __device__ __forceinline__ Weights(const NormParams& p, const Place<V>& at, bool wide) {
        if constexpr (V::kKeep) read(p, at, wide);
    }
    __device__ __forceinline__ void read(const NormParams& p, const Place<V>& at, bool wide) {
        weight_pairs<V>(p.weight, 1.f, at, wide, w);
        weight_pairs<V>(p.bias, 0.f, at, wide, b);
    }
};

// The rows of a block: every step-th of `rows` from blockIdx.y * rows; how many turns have all of them, and how many there are (teams
// of more than a warp meet, so every thread takes as many).
struct Turns {
    int64_t step, first;
    int full, all;
    __device__ __forceinline__ Turns(const NormParams& p, const Teams& t, int rsub) {
        const int64_t start = (int64_t)blockIdx.y * t.rows, behind = p.total - start - (t.rows - 1);
        step = (int64_t)gridDim.y * t.rows;
        first = start + rsub;
        full = behind > 0 ? (int)((behind + step - 1) / step) : 0;
        all = p.total > start ? (int)((p.total - start + step - 1) / step) : 0;
    }
    __device__ __forceinline__ bool has(const NormParams& p, int i) const { return first + i * step < p.total; }
};

int pow2_at_least(int n) {
    int k = 1;
    while (k < n) k *= 2;
    return k;
}
template <typename V>
Teams teams_of(const NormParams& p) {
    const int pieces = p.C / p.G / V::VEC, lanes = (pieces + V::R - 1) / V::R;
    Teams t;
    t.lanes = lanes <= 32 ? pow2_at_least(lanes) : (lanes + 31) / 32 * 32;
    const int teams = t.lanes >= V::NTH ? 1 : V::NTH / t.lanes;  // in a block
    t.groups = teams < p.G ? teams : t.lanes <= 32 ? pow2_at_least(p.G) : p.G;
    if (t.groups > teams) t.groups = teams;
    if (t.lanes >= 32 && t.groups < p.G) {  // blocks side by side have as many each (17401 x 2575 in 5 groups: 3 and 2 for 4 and 1)
        const int x = (p.G + t.groups - 1) / t.groups;
        t.groups = (p.G + x - 1) / x;
    }
    t.rows = teams / t.groups;
    t.threads = (t.rows * t.groups * t.lanes + 31) / 32 * 32;
    t.wide_weights = kda_host::aligned16(p.weight) && kda_host::aligned16(p.bias);
    return t;
}
// Blocks along the rows: no more than the rows need, about `resident` an SM in all (and more where blocks are smaller and have no rows in
// shared memory).
template <typename V>
dim3 grid_of(const NormParams& p, const Teams& t, int resident) {
    if (V::kSlots == 0) resident = resident * V::NTH / t.threads;
    const int x = (p.G + t.groups - 1) / t.groups;
    int64_t y = ((int64_t)p.total + t.rows - 1) / t.rows;
    const int64_t most = (int64_t)kSms * resident / x;
    if (y > most) y = most;
    if (y < 1) y = 1;
    if (y > 65535) y = 65535;
    return dim3(x, (unsigned)y);
}

// f(a variant) for groups of `pieces` pieces of VEC elements: the fewest values a lane with which a group fits a warp, then a block of
// 256 threads, then one of 1024.
// (one element a piece, 8192 rows: groups of 1791 bf16 25 and 57 us with 8 values a lane, 29 and 86 with 16; fp32 30 and 60, 37 and 89)
template <int VEC, bool kBackward, typename F>
auto pick_variant(int pieces, int G, F f) {
    if constexpr (VEC >= 4) {
        // teams that are filled need no tests
        if (pieces == 16 && G % 16 == 0) return f(Variant<VEC, 1, 256, 16>{});
        if (pieces == 32 && G % 8 == 0) return f(Variant<VEC, 1, 256, 32>{});
        if (pieces == 8 && G % 32 == 0) return f(Variant<VEC, 1, 256, 8>{});
        if (pieces <= 32) return f(Variant<VEC, 1, 256, 0>{});
        if (pieces <= 512) return f(Variant<VEC, 2, 256, 0>{});
        // (bf16: forwards two rows an SM, backwards one with its sums in registers)
        constexpr int R = VEC == 8 && kBackward ? 2 : 4;
        if (pieces <= 1024) return f(Variant<VEC, R, 1024 / R, 0>{});
        return f(Variant<VEC, 16 / VEC, 1024, 0>{});
    } else if constexpr (VEC == 2) {
        if (pieces <= 32) return f(Variant<2, 1, 256, 0>{});
        if (pieces <= 128) return f(Variant<2, 4, 256, 0>{});
        if (pieces <= 2048) return f(Variant<2, 8, 256, 0>{});
        return f(Variant<2, 8, 1024, 0>{});
    } else {
        if (pieces <= 64) return f(Variant<1, 2, 256, 0>{});
        if (pieces <= 2048) return f(Variant<1, 8, 256, 0>{});
        if (pieces <= 4096) return f(Variant<1, 16, 256, 0>{});
        return f(Variant<1, 16, 1024, 0>{});
    }
}

}  // namespace

}  // namespace kda
