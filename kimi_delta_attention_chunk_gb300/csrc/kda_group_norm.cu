// Group norm with an activation, channels last, over each token's groups of channels (the formulas stand in kda_group_norm.cuh).
//
// Every row is read once and stays in registers between the statistics and the output: HBM bounds it.  A team of lanes owns a group
// of channels (16 lanes of 16 bytes for 128 bf16 channels), teams lie side by side along a row, and a block walks down the rows with its
// weights, and backwards its share of dw and db, in registers.  Mean, then the sum of squares around it: two sums over a team, by
// shuffles up to 32 lanes and through shared memory beyond.  Groups of up to 16384 channels fit a block.
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

template <typename T, int VEC, int R, int U, int NTH>
__global__ void __launch_bounds__(NTH, NTH == 256 ? 3 : 1) norm_token_fwd_kernel(NormParams p, Teams t) {
    constexpr int N2 = (VEC + 1) / 2;
    constexpr bool kKeep = R * VEC <= 16;
    __shared__ float buf[2][NTH / 32][U];
    TeamSum<U, NTH> sum{buf, t.lanes, 0};
    const Place<VEC, R> at(p, t);
    const float inv_n = 1.f / (float)(p.C / p.G);
    f2 w[kKeep ? R : 1][N2], bias[kKeep ? R : 1][N2];
    if constexpr (kKeep) {
#pragma unroll
        for (int k = 0; k < R; ++k) {
            vec_pairs<VEC>(p.weight && at.has(k) ? p.weight + at.channel(k) : nullptr, 1.f, w[k]);
            vec_pairs<VEC>(p.bias && at.has(k) ? p.bias + at.channel(k) : nullptr, 0.f, bias[k]);
        }
    }
    const int64_t step = (int64_t)t.rows * U;
    for (int64_t base = blockIdx.y * step; base < p.total; base += gridDim.y * step) {
        Row<T, VEC> raw[U][R];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t row = base + u * t.rows + at.rsub;
#pragma unroll
            for (int k = 0; k < R; ++k) {
                if (row < p.total && at.has(k)) raw[u][k].load(static_cast<const T*>(p.x) + row * p.ldx + at.channel(k));
                else raw[u][k].zero();
            }
        }
        f2 x[U][R][N2];
        float s[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            f2 a = 0ull;
#pragma unroll
            for (int k = 0; k < R; ++k) {
                raw[u][k].to(x[u][k]);
#pragma unroll
                for (int e = 0; e < N2; ++e) a = add2(a, x[u][k][e]);
            }
            s[u] = sum2(a);
        }
        sum(s);
        float v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const float mean = s[u] * inv_n;
            f2 a = 0ull;
#pragma unroll
            for (int k = 0; k < R; ++k)
#pragma unroll
                for (int e = 0; e < N2; ++e) {
                    const f2 d = add2(x[u][k][e], pack(-mean, VEC == 1 ? 0.f : -mean));
                    x[u][k][e] = at.has(k) ? d : 0ull;
                    a = fma2(x[u][k][e], x[u][k][e], a);
                }
            v[u] = sum2(a);
        }
        sum(v);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t row = base + u * t.rows + at.rsub;
            const f2 rstd = both(rsqrtf(fmaf(v[u], inv_n, p.eps)));
#pragma unroll
            for (int k = 0; k < R; ++k) {
                if (!(row < p.total && at.has(k))) continue;
                if constexpr (!kKeep) {
                    vec_pairs<VEC>(p.weight ? p.weight + at.channel(k) : nullptr, 1.f, w[0]);
                    vec_pairs<VEC>(p.bias ? p.bias + at.channel(k) : nullptr, 0.f, bias[0]);
                }
                f2 y[N2];
#pragma unroll
                for (int e = 0; e < N2; ++e) {
                    y[e] = fma2(mul2(x[u][k][e], rstd), w[kKeep ? k : 0][e], bias[kKeep ? k : 0][e]);
                    if (p.act) y[e] = mul2(y[e], sigmoid2(y[e]));
                }
                Row<T, VEC> out;
                out.from(y);
                out.store(static_cast<T*>(p.y) + row * p.C + at.channel(k));
            }
        }
    }
}

// partial: [gridDim.y][2][C].
template <typename T, typename TG, int VEC, int R, int U, int NTH>
__global__ void __launch_bounds__(NTH, NTH == 256 ? 2 : 1) norm_token_bwd_kernel(NormParams p, Teams t, float* partial) {
    constexpr int N2 = (VEC + 1) / 2;
    constexpr bool kKeep = R * VEC <= 8;
    __shared__ float buf[2][NTH / 32][2 * U];
    __shared__ f2 join[NTH * N2];
    TeamSum<2 * U, NTH> sum{buf, t.lanes, 0};
    const Place<VEC, R> at(p, t);
    const float inv_n = 1.f / (float)(p.C / p.G);
    f2 w[kKeep ? R : 1][N2], bias[kKeep ? R : 1][N2], dw[R][N2], db[R][N2];
#pragma unroll
    for (int k = 0; k < R; ++k) {
        if constexpr (kKeep) {
            vec_pairs<VEC>(p.weight && at.has(k) ? p.weight + at.channel(k) : nullptr, 1.f, w[k]);
            vec_pairs<VEC>(p.bias && at.has(k) ? p.bias + at.channel(k) : nullptr, 0.f, bias[k]);
        }
#pragma unroll
        for (int e = 0; e < N2; ++e) dw[k][e] = db[k][e] = 0ull;
    }
    const int64_t step = (int64_t)t.rows * U;
    for (int64_t base = blockIdx.y * step; base < p.total; base += gridDim.y * step) {
        Row<T, VEC> raw[U][R];
        Row<TG, VEC> graw[U][R];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t row = base + u * t.rows + at.rsub;
#pragma unroll
            for (int k = 0; k < R; ++k) {
                if (row < p.total && at.has(k)) {
                    raw[u][k].load(static_cast<const T*>(p.x) + row * p.ldx + at.channel(k));
                    graw[u][k].load(static_cast<const TG*>(p.dy) + row * p.C + at.channel(k));
                } else {
                    raw[u][k].zero();
                    graw[u][k].zero();
                }
            }
        }
        f2 x[U][R][N2], q[U][R][N2];
        float s[2 * U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            f2 a = 0ull;
#pragma unroll
            for (int k = 0; k < R; ++k) {
                raw[u][k].to(x[u][k]);
#pragma unroll
                for (int e = 0; e < N2; ++e) a = add2(a, x[u][k][e]);
            }
            s[u] = sum2(a);
            s[U + u] = 0.f;
        }
        sum(s);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const float mean = s[u] * inv_n;
            f2 a = 0ull;
#pragma unroll
            for (int k = 0; k < R; ++k)
#pragma unroll
                for (int e = 0; e < N2; ++e) {
                    const f2 d = add2(x[u][k][e], pack(-mean, VEC == 1 ? 0.f : -mean));
                    x[u][k][e] = at.has(k) ? d : 0ull;
                    a = fma2(x[u][k][e], x[u][k][e], a);
                }
            s[u] = sum2(a);
        }
        sum(s);
        float rstd[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            rstd[u] = rsqrtf(fmaf(s[u], inv_n, p.eps));
            const f2 r2 = both(rstd[u]);
            f2 m1 = 0ull, m2 = 0ull;
#pragma unroll
            for (int k = 0; k < R; ++k) {
                graw[u][k].to(q[u][k]);
                if constexpr (!kKeep) {
                    vec_pairs<VEC>(p.weight && at.has(k) ? p.weight + at.channel(k) : nullptr, 1.f, w[0]);
                    vec_pairs<VEC>(p.bias && at.has(k) ? p.bias + at.channel(k) : nullptr, 0.f, bias[0]);
                }
#pragma unroll
                for (int e = 0; e < N2; ++e) {
                    const int kk = kKeep ? k : 0;
                    const f2 xh = mul2(x[u][k][e], r2);
                    x[u][k][e] = xh;
                    f2 dp = q[u][k][e];
                    if (p.act) dp = mul2(dp, silu_slope2(fma2(xh, w[kk][e], bias[kk][e])));
                    dw[k][e] = fma2(dp, xh, dw[k][e]);
                    db[k][e] = add2(dp, db[k][e]);
                    const f2 qq = mul2(dp, w[kk][e]);
                    q[u][k][e] = qq;
                    m1 = add2(m1, qq);
                    m2 = fma2(qq, xh, m2);
                }
            }
            s[u] = sum2(m1);
            s[U + u] = sum2(m2);
        }
        sum(s);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t row = base + u * t.rows + at.rsub;
            const f2 m1 = both(-s[u] * inv_n), m2 = both(-s[U + u] * inv_n), r2 = both(rstd[u]);
#pragma unroll
            for (int k = 0; k < R; ++k) {
                if (!(row < p.total && at.has(k))) continue;
                f2 dx[N2];
#pragma unroll
                for (int e = 0; e < N2; ++e) dx[e] = mul2(r2, fma2(x[u][k][e], m2, add2(q[u][k][e], m1)));
                Row<TG, VEC> out;
                out.from(dx);
                out.store(static_cast<TG*>(p.dx) + row * p.C + at.channel(k));
            }
        }
    }
    tc::grid_dep_launch();
    if (!p.dweight && !p.dbias) return;
    // the block's rows side by side first
    const int row_threads = t.groups * t.lanes;  // threads of one row
#pragma unroll
    for (int v = 0; v < 2; ++v) {
        float* const to = partial + ((int64_t)blockIdx.y * 2 + v) * p.C;
#pragma unroll
        for (int k = 0; k < R; ++k) {
            f2 total[N2];
#pragma unroll
            for (int e = 0; e < N2; ++e) total[e] = v ? db[k][e] : dw[k][e];
            if (t.rows > 1) {
                __syncthreads();
#pragma unroll
                for (int e = 0; e < N2; ++e) join[threadIdx.x * N2 + e] = total[e];
                __syncthreads();
                if (at.rsub == 0)
                    for (int r = 1; r < t.rows; ++r)
#pragma unroll
                        for (int e = 0; e < N2; ++e) total[e] = add2(total[e], join[(threadIdx.x + r * row_threads) * N2 + e]);
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
dim3 grid_of(const NormParams& p, const Teams& t, int U, int resident) {
    const int x = (p.G + t.groups - 1) / t.groups;
    int64_t y = ((int64_t)p.total + t.rows * U - 1) / (t.rows * U);
    const int64_t most = (int64_t)kSms * resident / x;
    if (y > most) y = most;
    if (y < 1) y = 1;
    if (y > 65535) y = 65535;
    return dim3(x, (unsigned)y);
}

// ---- which variant: pieces a lane, rows at a time, threads a block ------------------------------------------

// f(R, U, NTH as constants) for groups of `pieces` pieces of VEC elements.
template <int N>
struct Int {
    static constexpr int value = N;
};
template <int VEC, typename F>
auto pick_variant(int pieces, F f) {
    if constexpr (VEC >= 8) {
        if (pieces <= 32) return f(Int<1>{}, Int<2>{}, Int<256>{});
        if (pieces <= 512) return f(Int<2>{}, Int<1>{}, Int<256>{});
        return f(Int<2>{}, Int<1>{}, Int<1024>{});
    } else if constexpr (VEC == 4) {
        if (pieces <= 32) return f(Int<1>{}, Int<2>{}, Int<256>{});
        if (pieces <= 512) return f(Int<2>{}, Int<1>{}, Int<256>{});
        return f(Int<4>{}, Int<1>{}, Int<1024>{});
    } else {
        if (pieces <= 32) return f(Int<1>{}, Int<4>{}, Int<256>{});
        if (pieces <= 1024) return f(Int<4>{}, Int<1>{}, Int<256>{});
        return f(Int<16>{}, Int<1>{}, Int<1024>{});
    }
}

template <typename T, int VEC>
cudaError_t launch_fwd(const NormParams& p, cudaStream_t st) {
    const int pieces = p.C / p.G / VEC;
    return pick_variant<VEC>(pieces, [&](auto r, auto u, auto nth) {
        constexpr int R = decltype(r)::value, U = decltype(u)::value, NTH = decltype(nth)::value;
        const Teams t = teams_of(pieces, R, p.G, NTH);
        norm_token_fwd_kernel<T, VEC, R, U, NTH><<<grid_of(p, t, U, NTH == 256 ? 16 : 4), NTH, 0, st>>>(p, t);
        return cudaGetLastError();
    });
}
template <typename T, typename TG, int VEC>
cudaError_t launch_bwd(const NormParams& p, cudaStream_t st) {
    const int pieces = p.C / p.G / VEC;
    return pick_variant<VEC>(pieces, [&](auto r, auto u, auto nth) {
        constexpr int R = decltype(r)::value, U = decltype(u)::value, NTH = decltype(nth)::value;
        const Teams t = teams_of(pieces, R, p.G, NTH);
        const dim3 grid = grid_of(p, t, U, NTH == 256 ? 2 : 1);
        float* const partial = static_cast<float*>(p.ws);
        norm_token_bwd_kernel<T, TG, VEC, R, U, NTH><<<grid, NTH, 0, st>>>(p, t, partial);
        const cudaError_t e = cudaGetLastError();
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
        const size_t y = pick_variant<VEC>(cg / VEC, [&](auto r, auto u, auto nth) {
            constexpr int R = decltype(r)::value, U = decltype(u)::value, NTH = decltype(nth)::value;
            return (size_t)grid_of(p, teams_of(cg / VEC, R, p.G, NTH), U, NTH == 256 ? 2 : 1).y;
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
