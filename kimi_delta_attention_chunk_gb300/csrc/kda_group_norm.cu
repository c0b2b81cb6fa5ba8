// Group norm with an activation, channels last, over each token's groups of channels (the formulas stand in kda_group_norm.cuh).
//
// Every row is read once and stays in registers between the statistics and the output: HBM bounds it.  A team of lanes owns a group
// of channels (16 lanes of 16 bytes for 128 bf16 channels), teams lie side by side along a row, and a block walks down the rows with its
// weights, and backwards its share of dw and db, in registers.  Mean, then the sum of squares around it: two sums over a team, by
// shuffles up to 32 lanes and through shared memory beyond.  Groups of up to 16384 channels fit a block.
#include <type_traits>

#include "kda_group_norm.cuh"

namespace kda {

namespace {

// Which channels and rows the threads of a block have.
struct Teams {
    int lanes;   // of a team: a power of two
    int groups;  // side by side in a block
    int rows;    // rows that a block has at a time
};

// A variant: R pieces of VEC elements a lane, NTH threads a block, teams of LANES lanes that the group's pieces fill exactly and that
// fill the row's groups (0: any team).
template <int VEC_, int R_, int NTH_, int LANES_>
struct Variant {
    static constexpr int VEC = VEC_, R = R_, NTH = NTH_, LANES = LANES_, N2 = (VEC + 1) / 2, E = R * VEC;
    // Rows of a thread under way in shared memory; where a row is four pieces and more its own loads are enough.
    static constexpr int kAhead = R <= 2 && NTH == 256 ? 4 : 1;
    // Backwards, dw and db of a thread's channels: in registers, or where they are many in shared memory.
    static constexpr bool kSharedSums = E > 16 || NTH != 256;
    static constexpr int kFwd = NTH != 256 ? 1 : E > 16 ? 3 : 4, kBwd = NTH != 256 ? 1 : E > 8 ? 2 : 3;  // blocks an SM
};

// Sums of `N` values over every team.  Teams of more than a warp meet in shared memory, in a buffer of their own each time.
template <int LANES, int NTH>
struct TeamSum {
    float (*buf)[NTH / 32][2];  // [2]
    int lanes, turn;
    template <int N>
    __device__ __forceinline__ void operator()(float (&v)[N]) {
        if constexpr (LANES > 0) {
#pragma unroll
            for (int o = LANES / 2; o > 0; o /= 2)
#pragma unroll
                for (int k = 0; k < N; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
            return;
        }
#pragma unroll
        for (int o = 16; o > 0; o /= 2)
            if (o < lanes)
#pragma unroll
                for (int k = 0; k < N; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
        if (lanes <= 32) return;
        const int w = threadIdx.x / 32, team = lanes / 32, w0 = w / team * team;
        if (threadIdx.x % 32 == 0)
#pragma unroll
            for (int k = 0; k < N; ++k) buf[turn][w][k] = v[k];
        __syncthreads();
#pragma unroll
        for (int k = 0; k < N; ++k) {
            v[k] = 0.f;
            for (int j = 0; j < team; ++j) v[k] += buf[turn][w0 + j][k];
        }
        turn ^= 1;
    }
};

// A thread's place: its group, its row among those that the block has at a time, and its pieces of the group.
template <typename V>
struct Place {
    int g, rsub, cg, lane, lanes;
    __device__ __forceinline__ Place(const NormParams& p, const Teams& t) {
        lanes = V::LANES > 0 ? V::LANES : t.lanes;
        const int team = threadIdx.x / lanes;
        lane = threadIdx.x % lanes;
        g = blockIdx.x * t.groups + team % t.groups;
        rsub = team / t.groups;
        cg = p.C / p.G;
        if (V::LANES == 0 && g >= p.G) cg = 0;
    }
    __device__ __forceinline__ bool has(int k) const { return V::LANES > 0 || (lane + k * lanes) * V::VEC < cg; }
    // (of a piece that is there)
    __device__ __forceinline__ int channel(int k) const { return g * cg + (lane + k * lanes) * V::VEC; }
};

// A thread's own pieces of the next rows, on their way through shared memory: what a thread asks for it alone reads, so that no thread
// waits for another.  (Two-byte pieces have no asynchronous copy: they are loaded when asked for.)
template <typename V, typename T>
struct Ring {
    static constexpr int kBytes = V::kAhead > 1 ? V::kAhead * V::R * V::NTH * V::VEC * (int)sizeof(T) : 0;
    T* mine;
    Row<T, V::VEC> now[V::kAhead > 1 ? 1 : V::R];
    __device__ __forceinline__ explicit Ring(void* shared) : mine(static_cast<T*>(shared) + threadIdx.x * V::VEC) {}
    __device__ __forceinline__ T* at(int row, int k) const { return mine + ((row % V::kAhead) * V::R + k) * V::NTH * V::VEC; }
    __device__ __forceinline__ void request(int row, int k, const T* from) {
        if constexpr (V::kAhead > 1) Row<T, V::VEC>::copy_async(at(row, k), from);
        else now[k].load(from);
    }
    __device__ __forceinline__ void take(int row, int k, f2 (&v)[V::N2]) const {
        if constexpr (V::kAhead > 1) {
            Row<T, V::VEC> r;
            r.from_shared(at(row, k));
            r.to(v);
        } else {
            now[k].to(v);
        }
    }
};

// 1 / sqrt(var + eps)
__device__ __forceinline__ float inverse_deviation(float m2, float inv_n, float eps) {
    float r;
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(fmaxf(fmaf(m2, inv_n, eps), 1e-37f)));
    return r;
}

// The weights of a thread's channels: kept where they are few, else read again for every row.
template <typename V>
struct Weights {
    static constexpr bool kKeep = V::E <= 8;
    f2 w[kKeep ? V::R : 1][V::N2], b[kKeep ? V::R : 1][V::N2];
    __device__ __forceinline__ void read(const NormParams& p, const Place<V>& at, int k, int to) {
        vec_pairs<V::VEC>(p.weight && at.has(k) ? p.weight + at.channel(k) : nullptr, 1.f, w[to]);
        vec_pairs<V::VEC>(p.bias && at.has(k) ? p.bias + at.channel(k) : nullptr, 0.f, b[to]);
    }
    __device__ __forceinline__ Weights(const NormParams& p, const Place<V>& at) {
        if constexpr (kKeep)
#pragma unroll
            for (int k = 0; k < V::R; ++k) read(p, at, k, k);
    }
    // Where piece k's are.
    __device__ __forceinline__ int of(const NormParams& p, const Place<V>& at, int k) {
        if constexpr (kKeep) return k;
        read(p, at, k, 0);
        return 0;
    }
};

// x - mean of a thread's pieces, zeros where there are none; the sum of squares.
template <typename V>
__device__ __forceinline__ float centre(f2 (&x)[V::R][V::N2], float mean, const Place<V>& at) {
    f2 a = 0ull;
#pragma unroll
    for (int k = 0; k < V::R; ++k)
#pragma unroll
        for (int e = 0; e < V::N2; ++e) {
            const f2 d = add2(x[k][e], pack(-mean, V::VEC == 1 ? 0.f : -mean));
            x[k][e] = at.has(k) ? d : 0ull;
            a = fma2(x[k][e], x[k][e], a);
        }
    return sum2(a);
}

template <typename T, typename V>
__global__ void __launch_bounds__(V::NTH, V::kFwd) norm_token_fwd_kernel(NormParams p, Teams t) {
    constexpr int R = V::R, N2 = V::N2, A = V::kAhead;
    __shared__ float buf[2][V::NTH / 32][2];
    extern __shared__ __align__(16) char shared[];
    TeamSum<V::LANES, V::NTH> sum{buf, t.lanes, 0};
    Ring<V, T> ring(shared);
    const Place<V> at(p, t);
    const float inv_n = 1.f / (float)(p.C / p.G);
    // this thread's rows: every step-th from `first`
    const int64_t step = (int64_t)gridDim.y * t.rows, first = (int64_t)blockIdx.y * t.rows + at.rsub;
    const int mine = first < p.total ? (int)((p.total - first + step - 1) / step) : 0;
    const int apart = at.lanes * V::VEC;  // channels between a thread's pieces
    const int64_t next_x = step * p.ldx, next_y = step * p.C;
    const T* from = static_cast<const T*>(p.x) + first * p.ldx + at.channel(0);
    auto request = [&](int i) {
        if (i < mine) {
#pragma unroll
            for (int k = 0; k < R; ++k)
                if (at.has(k)) ring.request(i, k, from + k * apart);
            from += next_x;
        }
        if constexpr (A > 1) copies_commit();
    };
#pragma unroll
    for (int i = 0; i < A - 1; ++i) request(i);
    Weights<V> weights(p, at);
    // (teams of more than a warp meet, so every thread of a block takes as many turns)
    const int turns = (int)((p.total - (int64_t)blockIdx.y * t.rows + step - 1) / step);
    T* to = static_cast<T*>(p.y) + first * p.C + at.channel(0);
    for (int i = 0; i < turns; ++i, to += next_y) {
        if constexpr (A > 1) copies_wait<A - 2>();
        else request(i);
        f2 x[R][N2], a = 0ull;
#pragma unroll
        for (int k = 0; k < R; ++k) {
            if (at.has(k)) {  // (behind the last row: whatever is there)
                ring.take(i, k, x[k]);
#pragma unroll
                for (int e = 0; e < N2; ++e) a = add2(a, x[k][e]);
            } else {
#pragma unroll
                for (int e = 0; e < N2; ++e) x[k][e] = 0ull;
            }
        }
        if constexpr (A > 1) request(i + A - 1);
        float s[1] = {sum2(a)};
        sum(s);
        s[0] = centre<V>(x, s[0] * inv_n, at);
        sum(s);
        if (i >= mine) continue;
        const f2 rstd = both(inverse_deviation(s[0], inv_n, p.eps));
#pragma unroll
        for (int k = 0; k < R; ++k) {
            const int wk = weights.of(p, at, k);
            f2 y[N2];
#pragma unroll
            for (int e = 0; e < N2; ++e) y[e] = fma2(mul2(x[k][e], rstd), weights.w[wk][e], weights.b[wk][e]);
            if (p.act) {
#pragma unroll
                for (int e = 0; e < N2; ++e) y[e] = silu2(y[e]);
            }
            Row<T, V::VEC> out;
            out.from(y);
            if (at.has(k)) out.store(to + k * apart);
        }
    }
}

// partial: [gridDim.y][2][C].
template <typename T, typename TG, typename V>
__global__ void __launch_bounds__(V::NTH, V::kBwd) norm_token_bwd_kernel(NormParams p, Teams t, float* partial) {
    constexpr int R = V::R, N2 = V::N2, A = V::kAhead, NTH = V::NTH;
    constexpr bool kShared = V::kSharedSums;
    __shared__ float buf[2][NTH / 32][2];
    extern __shared__ __align__(16) char shared[];
    TeamSum<V::LANES, NTH> sum{buf, t.lanes, 0};
    Ring<V, T> ring(shared);
    Ring<V, TG> ring_dy(shared + ring.kBytes);
    const Place<V> at(p, t);
    const float inv_n = 1.f / (float)(p.C / p.G);
    const int64_t step = (int64_t)gridDim.y * t.rows, first = (int64_t)blockIdx.y * t.rows + at.rsub;
    const int mine = first < p.total ? (int)((p.total - first + step - 1) / step) : 0;
    const int apart = at.lanes * V::VEC;
    const int64_t next_x = step * p.ldx, next_y = step * p.C;
    const T* from = static_cast<const T*>(p.x) + first * p.ldx + at.channel(0);
    const TG* from_dy = static_cast<const TG*>(p.dy) + first * p.C + at.channel(0);
    auto request = [&](int i) {
        if (i < mine) {
#pragma unroll
            for (int k = 0; k < R; ++k)
                if (at.has(k)) {
                    ring.request(i, k, from + k * apart);
                    ring_dy.request(i, k, from_dy + k * apart);
                }
            from += next_x;
            from_dy += next_y;
        }
        if constexpr (A > 1) copies_commit();
    };
#pragma unroll
    for (int i = 0; i < A - 1; ++i) request(i);
    Weights<V> weights(p, at);
    // dw and db of this thread's channels: in registers, or in shared memory [R N2][2][NTH], a single channel as it is, pairs as pairs
    using Sum = typename std::conditional<V::VEC == 1, float, f2>::type;
    f2 dw[kShared ? 1 : R][N2], db[kShared ? 1 : R][N2];
    auto sums_at = [&](int k, int e, int v, int thread) -> Sum& { return reinterpret_cast<Sum*>(shared)[((k * N2 + e) * 2 + v) * NTH + thread]; };
    auto as_pair = [](Sum s) {
        if constexpr (V::VEC == 1) return pack(s, 0.f);
        else return s;
    };
    auto put_sum = [](Sum& to, f2 s) {
        if constexpr (V::VEC == 1) {
            float none;
            unpack(s, to, none);
        } else {
            to = s;
        }
    };
#pragma unroll
    for (int k = 0; k < R; ++k)
#pragma unroll
        for (int e = 0; e < N2; ++e) {
            if constexpr (kShared) sums_at(k, e, 0, threadIdx.x) = sums_at(k, e, 1, threadIdx.x) = Sum(0);
            else dw[k][e] = db[k][e] = 0ull;
        }
    const int turns = (int)((p.total - (int64_t)blockIdx.y * t.rows + step - 1) / step);
    TG* to = static_cast<TG*>(p.dx) + first * p.C + at.channel(0);
    // kAll: all rows of the block are there
    auto turn = [&](int i, auto all) {
        constexpr bool kAll = decltype(all)::value;
        if constexpr (A > 1) copies_wait<A - 2>();
        else request(i);
        f2 x[R][N2], q[R][N2], a = 0ull;
#pragma unroll
        for (int k = 0; k < R; ++k) {
            if (at.has(k) && (kAll || i < mine)) {
                ring.take(i, k, x[k]);
                ring_dy.take(i, k, q[k]);
#pragma unroll
                for (int e = 0; e < N2; ++e) a = add2(a, x[k][e]);
            } else {
#pragma unroll
                for (int e = 0; e < N2; ++e) x[k][e] = q[k][e] = 0ull;
            }
        }
        if constexpr (A > 1) request(i + A - 1);
        float one[1] = {sum2(a)};
        sum(one);
        one[0] = centre<V>(x, one[0] * inv_n, at);
        sum(one);
        const f2 rstd = both(inverse_deviation(one[0], inv_n, p.eps));
        f2 m1 = 0ull, m2 = 0ull;
#pragma unroll
        for (int k = 0; k < R; ++k) {
            const int wk = weights.of(p, at, k);
#pragma unroll
            for (int e = 0; e < N2; ++e) x[k][e] = mul2(x[k][e], rstd);
            if (p.act) {
#pragma unroll
                for (int e = 0; e < N2; ++e) q[k][e] = mul2(q[k][e], silu_slope2(fma2(x[k][e], weights.w[wk][e], weights.b[wk][e])));
            }
#pragma unroll
            for (int e = 0; e < N2; ++e) {
                if constexpr (kShared) {
                    Sum &sw = sums_at(k, e, 0, threadIdx.x), &sb = sums_at(k, e, 1, threadIdx.x);
                    put_sum(sw, fma2(q[k][e], x[k][e], as_pair(sw)));
                    put_sum(sb, add2(q[k][e], as_pair(sb)));
                } else {
                    dw[k][e] = fma2(q[k][e], x[k][e], dw[k][e]);
                    db[k][e] = add2(q[k][e], db[k][e]);
                }
                q[k][e] = mul2(q[k][e], weights.w[wk][e]);
                m1 = add2(m1, q[k][e]);
                m2 = fma2(q[k][e], x[k][e], m2);
            }
        }
        float s[2] = {sum2(m1), sum2(m2)};
        sum(s);
        if (!kAll && i >= mine) return;
        const f2 n1 = both(-s[0] * inv_n), n2 = both(-s[1] * inv_n);
#pragma unroll
        for (int k = 0; k < R; ++k) {
            f2 dx[N2];
#pragma unroll
            for (int e = 0; e < N2; ++e) dx[e] = mul2(rstd, fma2(x[k][e], n2, add2(q[k][e], n1)));
            Row<TG, V::VEC> out;
            out.from(dx);
            if (at.has(k)) out.store(to + k * apart);
        }
        to += next_y;
    };
    const int64_t behind = p.total - (int64_t)blockIdx.y * t.rows - (t.rows - 1);  // rows from the block's last one on
    const int full = behind > 0 ? (int)((behind + step - 1) / step) : 0;
    for (int i = 0; i < full; ++i) turn(i, std::true_type{});
    for (int i = full; i < turns; ++i) turn(i, std::false_type{});
    tc::grid_dep_launch();
    if (!p.dweight && !p.dbias) return;
    // the block's rows side by side first
    copies_wait<0>();
    f2* const join = reinterpret_cast<f2*>(shared);
    const int row_threads = t.groups * at.lanes;  // threads of one row
#pragma unroll
    for (int v = 0; v < 2; ++v) {
        float* const out = partial + ((int64_t)blockIdx.y * 2 + v) * p.C;
#pragma unroll
        for (int k = 0; k < R; ++k) {
            f2 total[N2];
#pragma unroll
            for (int e = 0; e < N2; ++e) {
                if constexpr (kShared) total[e] = as_pair(sums_at(k, e, v, threadIdx.x));
                else total[e] = v ? db[k][e] : dw[k][e];
            }
            if (t.rows > 1) {
                __syncthreads();
                if constexpr (!kShared) {
#pragma unroll
                    for (int e = 0; e < N2; ++e) join[threadIdx.x * N2 + e] = total[e];
                    __syncthreads();
                }
                if (at.rsub == 0)
                    for (int r = 1; r < t.rows; ++r)
#pragma unroll
                        for (int e = 0; e < N2; ++e) {
                            const int other = threadIdx.x + r * row_threads;
                            total[e] = add2(total[e], kShared ? as_pair(sums_at(k, e, v, other)) : join[other * N2 + e]);
                        }
            }
            if (at.rsub == 0 && at.has(k)) {
#pragma unroll
                for (int e = 0; e < N2; ++e) {
                    float lo, hi;
                    unpack(total[e], lo, hi);
                    out[at.channel(k) + 2 * e] = lo;
                    if (2 * e + 1 < V::VEC) out[at.channel(k) + 2 * e + 1] = hi;
                }
            }
        }
    }
}

int pow2_at_least(int n) {
    int k = 1;
    while (k < n) k *= 2;
    return k;
}
template <typename V>
Teams teams_of(int pieces, int G) {
    Teams t;
    t.lanes = pow2_at_least((pieces + V::R - 1) / V::R);
    t.groups = pow2_at_least(G);
    if (t.groups > V::NTH / t.lanes) t.groups = V::NTH / t.lanes;
    t.rows = V::NTH / t.lanes / t.groups;
    return t;
}
// Blocks along the rows: no more than the rows need, about `resident` an SM in all.
dim3 grid_of(const NormParams& p, const Teams& t, int resident) {
    const int x = (p.G + t.groups - 1) / t.groups;
    int64_t y = ((int64_t)p.total + t.rows - 1) / t.rows;
    const int64_t most = (int64_t)kSms * resident / x;
    if (y > most) y = most;
    if (y < 1) y = 1;
    if (y > 65535) y = 65535;
    return dim3(x, (unsigned)y);
}

// f(a variant) for groups of `pieces` pieces of VEC elements: a warp has up to 128 pieces, a block of 256 threads up to 1024 (4096
// single elements), one of 1024 the rest.
template <int VEC, typename F>
auto pick_variant(int pieces, int G, F f) {
    if constexpr (VEC >= 4) {
        // teams that are filled need no tests
        if (pieces == 16 && G % 16 == 0) return f(Variant<VEC, 1, 256, 16>{});
        if (pieces == 32 && G % 8 == 0) return f(Variant<VEC, 1, 256, 32>{});
        if (pieces == 8 && G % 32 == 0) return f(Variant<VEC, 1, 256, 8>{});
        if (pieces <= 32) return f(Variant<VEC, 1, 256, 0>{});
        if (pieces <= 64) return f(Variant<VEC, 2, 256, 0>{});
        if (pieces <= 1024) return f(Variant<VEC, 4, 256, 0>{});
        return f(Variant<VEC, VEC == 4 ? 4 : 2, 1024, 0>{});
    } else {
        if (pieces <= 32) return f(Variant<1, 1, 256, 0>{});
        if (pieces <= 1024) return f(Variant<1, 4, 256, 0>{});
        if (pieces <= 4096) return f(Variant<1, 16, 256, 0>{});
        return f(Variant<1, 16, 1024, 0>{});
    }
}

template <typename T, int VEC>
cudaError_t launch_fwd(const NormParams& p, cudaStream_t st) {
    const int pieces = p.C / p.G / VEC;
    return pick_variant<VEC>(pieces, p.G, [&](auto variant) {
        using V = decltype(variant);
        const auto kern = norm_token_fwd_kernel<T, V>;
        constexpr int smem = Ring<V, T>::kBytes;
        static std::atomic<uint64_t> allowed;
    const cudaError_t e = allow_shared(kern, smem, allowed);
        if (e != cudaSuccess) return e;
        const Teams t = teams_of<V>(pieces, p.G);
        kern<<<grid_of(p, t, V::kFwd), V::NTH, smem, st>>>(p, t);
        return cudaGetLastError();
    });
}
template <typename T, typename TG, int VEC>
cudaError_t launch_bwd(const NormParams& p, cudaStream_t st) {
    const int pieces = p.C / p.G / VEC;
    return pick_variant<VEC>(pieces, p.G, [&](auto variant) {
        using V = decltype(variant);
        const auto kern = norm_token_bwd_kernel<T, TG, V>;
        constexpr int rings = Ring<V, T>::kBytes + Ring<V, TG>::kBytes;
        constexpr int sums = V::kSharedSums ? V::NTH * V::E * 8 : V::NTH * V::N2 * 8;
        static_assert(!V::kSharedSums || rings == 0, "the sums have the place");
        constexpr int smem = rings > sums ? rings : sums;
        static std::atomic<uint64_t> allowed;
    cudaError_t e = allow_shared(kern, smem, allowed);
        if (e != cudaSuccess) return e;
        const Teams t = teams_of<V>(pieces, p.G);
        const dim3 grid = grid_of(p, t, V::kBwd);
        float* const partial = static_cast<float*>(p.ws);
        kern<<<grid, V::NTH, smem, st>>>(p, t, partial);
        e = cudaGetLastError();
        if (e != cudaSuccess || (!p.dweight && !p.dbias)) return e;
        return tc::launch_dependent(norm_weights_kernel, (unsigned)((p.C + 31) / 32), 256, 0, st, (const float*)partial, (int)grid.y, p.C, p.dweight,
                                    p.dbias);
    });
}

}  // namespace

cudaError_t norm_token_fwd(kda_dtype dt, const NormParams& p, cudaStream_t st) {
    using kda_host::rows_aligned;
    const int vec = dt == KDA_BF16 ? 8 : 4, cg = p.C / p.G;
    const bool wide = cg % vec == 0 && rows_aligned(p.x, p.ldx, vec) && rows_aligned(p.y, p.C, vec);
    if (dt == KDA_BF16) return wide ? launch_fwd<__nv_bfloat16, 8>(p, st) : launch_fwd<__nv_bfloat16, 1>(p, st);
    return wide ? launch_fwd<float, 4>(p, st) : launch_fwd<float, 1>(p, st);
}

// The most blocks along the rows of the variants that p's channels allow (which one runs depends on the alignment).
template <int VEC>
size_t most_rows(const NormParams& p) {
    const int cg = p.C / p.G;
    if (cg % VEC != 0) return 0;
    return pick_variant<VEC>(cg / VEC, p.G, [&](auto variant) {
        using V = decltype(variant);
        return (size_t)grid_of(p, teams_of<V>(cg / VEC, p.G), V::kBwd).y;
    });
}
size_t norm_token_bwd_workspace(const NormParams& p) {
    size_t most = most_rows<1>(p);
    for (size_t n : {most_rows<8>(p), most_rows<4>(p)})
        if (n > most) most = n;
    return most * 2 * p.C * 4;
}

cudaError_t norm_token_bwd(kda_dtype dt, kda_dtype gdt, const NormParams& p, cudaStream_t st) {
    using kda_host::rows_aligned;
    const int vec = dt == KDA_BF16 && gdt == KDA_BF16 ? 8 : 4, cg = p.C / p.G;
    const bool wide = cg % vec == 0 && rows_aligned(p.x, p.ldx, dt == KDA_BF16 ? 8 : 4) && rows_aligned(p.dy, p.C, vec) && rows_aligned(p.dx, p.C, vec);
    if (dt == KDA_F32) return wide ? launch_bwd<float, float, 4>(p, st) : launch_bwd<float, float, 1>(p, st);
    if (gdt == KDA_F32) return wide ? launch_bwd<__nv_bfloat16, float, 4>(p, st) : launch_bwd<__nv_bfloat16, float, 1>(p, st);
    return wide ? launch_bwd<__nv_bfloat16, __nv_bfloat16, 8>(p, st) : launch_bwd<__nv_bfloat16, __nv_bfloat16, 1>(p, st);
}

}  // namespace kda
