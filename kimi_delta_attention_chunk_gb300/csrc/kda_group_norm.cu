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

// Sums of `N` values over every team.  Teams of more than a warp meet in shared memory, in a buffer of their own each time.
template <int N, int NTH>
struct TeamSum {
    float (*buf)[NTH / 32][N];  // [2]
    int lanes, turn;
    __device__ __forceinline__ void operator()(float (&v)[N]) {
        const int within = min(lanes, 32);
        for (int o = within / 2; o > 0; o >>= 1)
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

// A thread's place: its group, its row among those that the block has at a time, its first channel in the group and which of its R
// pieces are there.
template <int VEC, int R>
struct Place {
    int g, rsub, cg, lane, lanes;
    __device__ __forceinline__ Place(const NormParams& p, const Teams& t) {
        const int team = threadIdx.x / t.lanes;
        lane = threadIdx.x % t.lanes;
        lanes = t.lanes;
        g = blockIdx.x * t.groups + team % t.groups;
        rsub = team / t.groups;
        cg = p.C / p.G;
        if (g >= p.G) cg = 0;
    }
    __device__ __forceinline__ bool has(int k) const { return (lane + k * lanes) * VEC < cg; }
    // (of a piece that is there)
    __device__ __forceinline__ int channel(int k) const { return g * cg + (lane + k * lanes) * VEC; }
};

// A thread's own pieces of the next rows, on their way through shared memory: what a thread asks for it alone reads, so that no thread
// waits for another.  Two-byte pieces have no asynchronous copy: they are loaded when asked for.  Blocks of 1024 threads (groups of
// more than some thousand channels) load a row when its turn comes: their shared memory would not hold more, or has the sums.
template <int NTH>
constexpr int kAhead = NTH == 256 ? 4 : 1;  // rows under way, the one at hand among them
template <typename T, int VEC, int R, int NTH>
struct Ring {
    static constexpr int kRows = kAhead<NTH>;
    static constexpr int kBytes = kRows > 1 ? kRows * R * NTH * VEC * (int)sizeof(T) : 0;
    T* mine;
    Row<T, VEC> now[kRows > 1 ? 1 : R];
    __device__ __forceinline__ explicit Ring(void* shared) : mine(static_cast<T*>(shared) + threadIdx.x * VEC) {}
    __device__ __forceinline__ T* at(int row, int k) const { return mine + ((row % kRows) * R + k) * NTH * VEC; }
    __device__ __forceinline__ void request(int row, int k, const T* from) {
        if constexpr (kRows > 1) Row<T, VEC>::copy_async(at(row, k), from);
        else now[k].load(from);
    }
    __device__ __forceinline__ void take(int row, int k, f2 (&v)[(VEC + 1) / 2]) const {
        if constexpr (kRows > 1) {
            Row<T, VEC> r;
            r.from_shared(at(row, k));
            r.to(v);
        } else {
            now[k].to(v);
        }
    }
};
template <int NTH, int E>
constexpr int kResidentBwd = NTH != 256 ? 1 : E > 8 ? 2 : 3;

template <typename T, int VEC, int R, int NTH>
__global__ void __launch_bounds__(NTH, NTH == 256 ? 4 : 1) norm_token_fwd_kernel(NormParams p, Teams t) {
    constexpr int N2 = (VEC + 1) / 2;
    constexpr bool kKeep = R * VEC <= 16;
    __shared__ float buf[2][NTH / 32][1];
    extern __shared__ __align__(16) char shared[];
    TeamSum<1, NTH> sum{buf, t.lanes, 0};
    Ring<T, VEC, R, NTH> ring(shared);
    const Place<VEC, R> at(p, t);
    const float inv_n = 1.f / (float)(p.C / p.G);
    const int64_t step = (int64_t)gridDim.y * t.rows;
    const int64_t first = (int64_t)blockIdx.y * t.rows + at.rsub;
    auto request = [&](int i) {
        const int64_t row = first + i * step;
        if (row < p.total)
#pragma unroll
            for (int k = 0; k < R; ++k)
                if (at.has(k)) ring.request(i, k, static_cast<const T*>(p.x) + row * p.ldx + at.channel(k));
        copies_commit();
    };
#pragma unroll
    for (int i = 0; i < kAhead<NTH> - 1; ++i) request(i);
    f2 w[kKeep ? R : 1][N2], bias[kKeep ? R : 1][N2];
    if constexpr (kKeep) {
#pragma unroll
        for (int k = 0; k < R; ++k) {
            vec_pairs<VEC>(p.weight && at.has(k) ? p.weight + at.channel(k) : nullptr, 1.f, w[k]);
            vec_pairs<VEC>(p.bias && at.has(k) ? p.bias + at.channel(k) : nullptr, 0.f, bias[k]);
        }
    }
    // (teams of more than a warp meet, so every thread of a block takes as many turns)
    const int turns = (int)((p.total - (int64_t)blockIdx.y * t.rows + step - 1) / step);
    T* to = static_cast<T*>(p.y) + first * p.C;
    for (int i = 0; i < turns; ++i, to += step * p.C) {
        if constexpr (kAhead<NTH> > 1) copies_wait<kAhead<NTH> - 2>();
        else request(i);
        const bool here = first + i * step < p.total;
        f2 x[R][N2];
        f2 a = 0ull;
#pragma unroll
        for (int k = 0; k < R; ++k) {
            if (here && at.has(k)) {
                ring.take(i, k, x[k]);
#pragma unroll
                for (int e = 0; e < N2; ++e) a = add2(a, x[k][e]);
            } else {
#pragma unroll
                for (int e = 0; e < N2; ++e) x[k][e] = 0ull;
            }
        }
        if constexpr (kAhead<NTH> > 1) request(i + kAhead<NTH> - 1);
        float s[1] = {sum2(a)};
        sum(s);
        const float mean = s[0] * inv_n;
        a = 0ull;
#pragma unroll
        for (int k = 0; k < R; ++k)
#pragma unroll
            for (int e = 0; e < N2; ++e) {
                const f2 d = add2(x[k][e], pack(-mean, VEC == 1 ? 0.f : -mean));
                x[k][e] = at.has(k) ? d : 0ull;
                a = fma2(x[k][e], x[k][e], a);
            }
        s[0] = sum2(a);
        sum(s);
        const f2 rstd = both(rsqrtf(fmaf(s[0], inv_n, p.eps)));
#pragma unroll
        for (int k = 0; k < R; ++k) {
            if (!(here && at.has(k))) continue;
            if constexpr (!kKeep) {
                vec_pairs<VEC>(p.weight ? p.weight + at.channel(k) : nullptr, 1.f, w[0]);
                vec_pairs<VEC>(p.bias ? p.bias + at.channel(k) : nullptr, 0.f, bias[0]);
            }
            f2 y[N2];
#pragma unroll
            for (int e = 0; e < N2; ++e) y[e] = fma2(mul2(x[k][e], rstd), w[kKeep ? k : 0][e], bias[kKeep ? k : 0][e]);
            if (p.act) {
#pragma unroll
                for (int e = 0; e < N2; ++e) y[e] = silu2(y[e]);
            }
            Row<T, VEC> out;
            out.from(y);
            out.store(to + at.channel(k));
        }
    }
}

// partial: [gridDim.y][2][C].
template <typename T, typename TG, int VEC, int R, int NTH>
__global__ void __launch_bounds__(NTH, kResidentBwd<NTH, R * VEC>) norm_token_bwd_kernel(NormParams p, Teams t, float* partial) {
    constexpr int N2 = (VEC + 1) / 2;
    constexpr bool kKeep = R * VEC <= 8;
    __shared__ float buf[2][NTH / 32][2];
    extern __shared__ __align__(16) char shared[];
    f2* const join = reinterpret_cast<f2*>(shared);
    TeamSum<2, NTH> sum{buf, t.lanes, 0};
    Ring<T, VEC, R, NTH> ring(shared);
    Ring<TG, VEC, R, NTH> ring_dy(shared + ring.kBytes);
    const Place<VEC, R> at(p, t);
    const float inv_n = 1.f / (float)(p.C / p.G);
    const int64_t step = (int64_t)gridDim.y * t.rows;
    const int64_t first = (int64_t)blockIdx.y * t.rows + at.rsub;
    auto request = [&](int i) {
        const int64_t row = first + i * step;
        if (row < p.total)
#pragma unroll
            for (int k = 0; k < R; ++k)
                if (at.has(k)) {
                    ring.request(i, k, static_cast<const T*>(p.x) + row * p.ldx + at.channel(k));
                    ring_dy.request(i, k, static_cast<const TG*>(p.dy) + row * p.C + at.channel(k));
                }
        copies_commit();
    };
#pragma unroll
    for (int i = 0; i < kAhead<NTH> - 1; ++i) request(i);
    // dw and db of this thread's channels: in registers, or for large blocks in shared memory [R N2][2][NTH]
    constexpr bool kShared = NTH != 256;
    f2 w[kKeep ? R : 1][N2], bias[kKeep ? R : 1][N2], dw[kShared ? 1 : R][N2], db[kShared ? 1 : R][N2];
    // (a single channel as it is, pairs as pairs)
    using Sum = typename std::conditional<VEC == 1, float, f2>::type;
    auto sums_at = [&](int k, int e, int v, int thread) -> Sum& { return reinterpret_cast<Sum*>(shared)[((k * N2 + e) * 2 + v) * NTH + thread]; };
    auto as_pair = [](Sum s) {
        if constexpr (VEC == 1) return pack(s, 0.f);
        else return s;
    };
    auto put_sum = [](Sum& to, f2 s) {
        if constexpr (VEC == 1) {
            float none;
            unpack(s, to, none);
        } else {
            to = s;
        }
    };
#pragma unroll
    for (int k = 0; k < R; ++k) {
        if constexpr (kKeep) {
            vec_pairs<VEC>(p.weight && at.has(k) ? p.weight + at.channel(k) : nullptr, 1.f, w[k]);
            vec_pairs<VEC>(p.bias && at.has(k) ? p.bias + at.channel(k) : nullptr, 0.f, bias[k]);
        }
#pragma unroll
        for (int e = 0; e < N2; ++e) {
            if constexpr (kShared) sums_at(k, e, 0, threadIdx.x) = sums_at(k, e, 1, threadIdx.x) = Sum(0);
            else dw[k][e] = db[k][e] = 0ull;
        }
    }
    const int turns = (int)((p.total - (int64_t)blockIdx.y * t.rows + step - 1) / step);
    TG* to = static_cast<TG*>(p.dx) + first * p.C;
    for (int i = 0; i < turns; ++i, to += step * p.C) {
        if constexpr (kAhead<NTH> > 1) copies_wait<kAhead<NTH> - 2>();
        else request(i);
        const bool here = first + i * step < p.total;
        f2 x[R][N2], q[R][N2];
        f2 a = 0ull;
#pragma unroll
        for (int k = 0; k < R; ++k) {
            if (here && at.has(k)) {
                ring.take(i, k, x[k]);
                ring_dy.take(i, k, q[k]);
#pragma unroll
                for (int e = 0; e < N2; ++e) a = add2(a, x[k][e]);
            } else {
#pragma unroll
                for (int e = 0; e < N2; ++e) x[k][e] = q[k][e] = 0ull;
            }
        }
        if constexpr (kAhead<NTH> > 1) request(i + kAhead<NTH> - 1);
        float s[2] = {sum2(a), 0.f};
        sum(s);
        const float mean = s[0] * inv_n;
        a = 0ull;
#pragma unroll
        for (int k = 0; k < R; ++k)
#pragma unroll
            for (int e = 0; e < N2; ++e) {
                const f2 d = add2(x[k][e], pack(-mean, VEC == 1 ? 0.f : -mean));
                x[k][e] = at.has(k) ? d : 0ull;
                a = fma2(x[k][e], x[k][e], a);
            }
        s[0] = sum2(a);
        s[1] = 0.f;
        sum(s);
        const f2 rstd = both(rsqrtf(fmaf(s[0], inv_n, p.eps)));
        f2 m1 = 0ull, m2 = 0ull;
#pragma unroll
        for (int k = 0; k < R; ++k) {
            if constexpr (!kKeep) {
                vec_pairs<VEC>(p.weight && at.has(k) ? p.weight + at.channel(k) : nullptr, 1.f, w[0]);
                vec_pairs<VEC>(p.bias && at.has(k) ? p.bias + at.channel(k) : nullptr, 0.f, bias[0]);
            }
            const int kk = kKeep ? k : 0;
#pragma unroll
            for (int e = 0; e < N2; ++e) x[k][e] = mul2(x[k][e], rstd);
            if (p.act) {
#pragma unroll
                for (int e = 0; e < N2; ++e) q[k][e] = mul2(q[k][e], silu_slope2(fma2(x[k][e], w[kk][e], bias[kk][e])));
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
                q[k][e] = mul2(q[k][e], w[kk][e]);
                m1 = add2(m1, q[k][e]);
                m2 = fma2(q[k][e], x[k][e], m2);
            }
        }
        s[0] = sum2(m1);
        s[1] = sum2(m2);
        sum(s);
        const f2 n1 = both(-s[0] * inv_n), n2 = both(-s[1] * inv_n);
#pragma unroll
        for (int k = 0; k < R; ++k) {
            if (!(here && at.has(k))) continue;
            f2 dx[N2];
#pragma unroll
            for (int e = 0; e < N2; ++e) dx[e] = mul2(rstd, fma2(x[k][e], n2, add2(q[k][e], n1)));
            Row<TG, VEC> out;
            out.from(dx);
            out.store(to + at.channel(k));
        }
    }
    tc::grid_dep_launch();
    if (!p.dweight && !p.dbias) return;
    // the block's rows side by side first (where the last rows were on their way)
    copies_wait<0>();
    const int row_threads = t.groups * t.lanes;  // threads of one row
#pragma unroll
    for (int v = 0; v < 2; ++v) {
        float* const to = partial + ((int64_t)blockIdx.y * 2 + v) * p.C;
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
                            const int from = threadIdx.x + r * row_threads;
                            total[e] = add2(total[e], kShared ? as_pair(sums_at(k, e, v, from)) : join[from * N2 + e]);
                        }
            }
            if (at.rsub == 0 && at.has(k)) {
#pragma unroll
                for (int e = 0; e < N2; ++e) {
                    float a, b;
                    unpack(total[e], a, b);
                    to[at.channel(k) + 2 * e] = a;
                    if (2 * e + 1 < VEC) to[at.channel(k) + 2 * e + 1] = b;
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
// Teams for groups of `pieces` pieces, R of them a lane, in blocks of nth threads.
Teams teams_of(int pieces, int R, int G, int nth) {
    Teams t;
    t.lanes = pow2_at_least((pieces + R - 1) / R);
    t.groups = pow2_at_least(G);
    if (t.groups > nth / t.lanes) t.groups = nth / t.lanes;
    t.rows = nth / t.lanes / t.groups;
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

// ---- which variant: pieces a lane, threads a block ------------------------------------------

// f(R, NTH as constants) for groups of `pieces` pieces of VEC elements.
template <int N>
struct Int {
    static constexpr int value = N;
};
template <int VEC, typename F>
auto pick_variant(int pieces, F f) {
    if constexpr (VEC >= 4) {
        if (pieces <= 32) return f(Int<1>{}, Int<256>{});
        if (pieces <= 512) return f(Int<2>{}, Int<256>{});
        return f(Int<VEC == 4 ? 4 : 2>{}, Int<1024>{});
    } else {
        if (pieces <= 32) return f(Int<1>{}, Int<256>{});
        if (pieces <= 1024) return f(Int<4>{}, Int<256>{});
        return f(Int<16>{}, Int<1024>{});
    }
}
constexpr int resident_fwd(int nth) { return nth == 256 ? 4 : 1; }

template <typename T, int VEC>
cudaError_t launch_fwd(const NormParams& p, cudaStream_t st) {
    const int pieces = p.C / p.G / VEC;
    return pick_variant<VEC>(pieces, [&](auto r, auto nth) {
        constexpr int R = decltype(r)::value, NTH = decltype(nth)::value;
        const auto kern = norm_token_fwd_kernel<T, VEC, R, NTH>;
        constexpr int smem = Ring<T, VEC, R, NTH>::kBytes;
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        const Teams t = teams_of(pieces, R, p.G, NTH);
        kern<<<grid_of(p, t, resident_fwd(NTH)), NTH, smem, st>>>(p, t);
        return cudaGetLastError();
    });
}
template <typename T, typename TG, int VEC>
cudaError_t launch_bwd(const NormParams& p, cudaStream_t st) {
    const int pieces = p.C / p.G / VEC;
    return pick_variant<VEC>(pieces, [&](auto r, auto nth) {
        constexpr int R = decltype(r)::value, NTH = decltype(nth)::value;
        const auto kern = norm_token_bwd_kernel<T, TG, VEC, R, NTH>;
        constexpr int rings = Ring<T, VEC, R, NTH>::kBytes + Ring<TG, VEC, R, NTH>::kBytes;
        constexpr int joins = NTH == 256 ? NTH * ((VEC + 1) / 2) * 8 : NTH * R * VEC * 8;
        constexpr int smem = rings > joins ? rings : joins;
        cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        const Teams t = teams_of(pieces, R, p.G, NTH);
        const dim3 grid = grid_of(p, t, kResidentBwd<NTH, R * VEC>);
        float* const partial = static_cast<float*>(p.ws);
        kern<<<grid, NTH, smem, st>>>(p, t, partial);
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
size_t norm_token_bwd_workspace(const NormParams& p) {
    const int cg = p.C / p.G;
    size_t most = 0;
    auto look = [&](auto vec) {
        constexpr int VEC = decltype(vec)::value;
        if (cg % VEC != 0) return;
        const size_t y = pick_variant<VEC>(cg / VEC, [&](auto r, auto nth) {
            constexpr int R = decltype(r)::value, NTH = decltype(nth)::value;
            return (size_t)grid_of(p, teams_of(cg / VEC, R, p.G, NTH), kResidentBwd<NTH, R * VEC>).y;
        });
        if (y > most) most = y;
    };
    look(Int<8>{});
    look(Int<4>{});
    look(Int<1>{});
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
