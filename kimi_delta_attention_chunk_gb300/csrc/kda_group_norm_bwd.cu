// Group norm over each token's groups of channels: backward (how it works stands in kda_group_norm_token.cuh).
#include "kda_group_norm_token.cuh"

namespace kda {

namespace {

// The slots of x's and dy's rows (a variant's, or as many as the shared memory of its blocks has room for), and the bytes of these and of
// the sums that are held there.
template <typename T, typename TG, typename V>
struct Room {
    static constexpr int kSums = V::kSharedSums ? V::NTH * 8 * V::E : 0, kMost = 226 * 1024 / V::kBwd - 1024;
    static constexpr int slots(int n) { return n > 0 && n * V::E * V::NTH * (int)(sizeof(T) + sizeof(TG)) + kSums > kMost ? slots(n / 2) : n; }
    static constexpr int kSlots = slots(V::kSlots);
    static constexpr int kRings = Rows<V, T, kSlots>::kBytes + Rows<V, TG, kSlots>::kBytes;
};

// partial: [gridDim.y][2][C].
template <typename T, typename TG, typename V>
__global__ void __launch_bounds__(V::NTH, V::kBwd) norm_token_bwd_kernel(NormParams p, Teams t, float* partial) {
    using M = Room<T, TG, V>;
    constexpr int E2 = V::E2, A = M::kSlots, NTH = V::NTH;
    constexpr bool kShared = V::kSharedSums;
    __shared__ float buf[2][NTH / 32][2];
    static_assert(sizeof(buf) <= kDeclared, "what a launch allows for");
    extern __shared__ __align__(16) char shared[];
    TeamSum<V::LANES, NTH> sum(buf, t.lanes);
    const Place<V> at(p, t);
    const float inv_n = 1.f / (float)(p.C / p.G);
    const Turns turns(p, t, at.rsub);
    Rows<V, T, A> rows(p.x, turns.first, p.ldx, turns.step, at, shared);
    Rows<V, TG, A> grads(p.dy, turns.first, p.C, turns.step, at, shared + rows.kBytes);
    auto request = [&](int i) {
        if (i < turns.full || (i < turns.all && turns.has(p, i))) {
            rows.request(i, at);
            grads.request(i, at);
        }
        copies_commit();
    };
    if constexpr (A > 0)
#pragma unroll
        for (int i = 0; i < (A > 1 ? A - 1 : 1); ++i) request(i);
    Weights<V> weights(p, at, t.wide_weights);
    // dw and db of this thread's channels: in registers, or in shared memory [E2][2][NTH]
    f2 dw[kShared ? 1 : E2], db[kShared ? 1 : E2];
    f2* const sums = reinterpret_cast<f2*>(shared + (kShared ? M::kRings : 0));
#pragma unroll
    for (int j = 0; j < E2; ++j) {
        if constexpr (kShared) sums[(2 * j) * NTH + threadIdx.x] = sums[(2 * j + 1) * NTH + threadIdx.x] = 0ull;
        else dw[j] = db[j] = 0ull;
    }
    TG* to = static_cast<TG*>(p.dx) + turns.first * p.C + at.first;
    const int64_t next = turns.step * p.C;
    // kAll: all rows of the block are there
    auto turn = [&](int i, auto all) {
        const bool here = decltype(all)::value || turns.has(p, i);
        if constexpr (A > 0) copies_wait<(A > 1 ? A - 2 : 0)>();
        Pieces<V, T> raw;
        Pieces<V, TG> raw_dy;
        if (here) {
            rows.take(i, at, raw);
            grads.take(i, at, raw_dy);
        } else {
            raw.zero();
            raw_dy.zero();
        }
        if constexpr (A > 1) request(i + A - 1);
        f2 x[E2], q[E2], a = 0ull;
        raw.pairs(x);
#pragma unroll
        for (int j = 0; j < E2; ++j) a = add2(a, x[j]);
        float one[1] = {sum2(a)};
        sum(one);
        if constexpr (A == 1) request(i + 1);  // (behind the sum's barrier: the row is in registers)
        const f2 mean = both(-one[0] * inv_n);
        a = 0ull;
#pragma unroll
        for (int j = 0; j < E2; ++j) {
            x[j] = at.masked(j, add2(x[j], mean));
            a = fma2(x[j], x[j], a);
        }
        one[0] = sum2(a);
        sum(one);
        const f2 rstd = both(inverse_deviation(one[0], inv_n, p.eps));
        if constexpr (!V::kKeep) weights.read(p, at, t.wide_weights);
        raw_dy.pairs(q);
#pragma unroll
        for (int j = 0; j < E2; ++j) x[j] = mul2(x[j], rstd);
        if (p.act) {
#pragma unroll
            for (int j = 0; j < E2; ++j) q[j] = mul2(q[j], silu_slope2(fma2(x[j], weights.w[j], weights.b[j])));
        }
        f2 m1 = 0ull, m2 = 0ull;
#pragma unroll
        for (int j = 0; j < E2; ++j) {
            if constexpr (kShared) {
                f2 &sw = sums[(2 * j) * NTH + threadIdx.x], &sb = sums[(2 * j + 1) * NTH + threadIdx.x];
                sw = fma2(q[j], x[j], sw);
                sb = add2(q[j], sb);
            } else {
                dw[j] = fma2(q[j], x[j], dw[j]);
                db[j] = add2(q[j], db[j]);
            }
            q[j] = mul2(q[j], weights.w[j]);
            m1 = add2(m1, q[j]);
            m2 = fma2(q[j], x[j], m2);
        }
        float s[2] = {sum2(m1), sum2(m2)};
        sum(s);
        if (here) {
            const f2 n1 = both(-s[0] * inv_n), n2 = both(-s[1] * inv_n);
#pragma unroll
            for (int j = 0; j < E2; ++j) q[j] = mul2(rstd, fma2(x[j], n2, add2(q[j], n1)));
            Pieces<V, TG>::store(at, to, q);
        }
        to += next;
    };
    for (int i = 0; i < turns.full; ++i) turn(i, std::true_type{});
    for (int i = turns.full; i < turns.all; ++i) turn(i, std::false_type{});
    tc::grid_dep_launch();
    if (!p.dweight && !p.dbias) return;
    // the block's rows side by side first
    copies_wait<0>();
    const int row_threads = t.groups * at.lanes;  // threads of one row
#pragma unroll
    for (int v = 0; v < 2; ++v) {
        float* const out = partial + ((int64_t)blockIdx.y * 2 + v) * p.C + at.first;
#pragma unroll
        for (int j = 0; j < E2; ++j) {
            f2 total;
            if constexpr (kShared) total = sums[(2 * j + v) * NTH + threadIdx.x];
            else total = v ? db[j] : dw[j];
            if (t.rows > 1) {
                __syncthreads();
                const f2* join = sums + (2 * j + v) * NTH;
                if constexpr (!kShared) {
                    join = sums;
                    sums[threadIdx.x] = total;
                    __syncthreads();
                }
                if (at.rsub == 0)
                    for (int r = 1; r < t.rows; ++r) total = add2(total, join[threadIdx.x + r * row_threads]);
            }
            if (at.rsub != 0) continue;
            float lo, hi;
            unpack(total, lo, hi);
            const int k0 = V::VEC > 1 ? 2 * j / V::VEC : 2 * j, k1 = V::VEC > 1 ? k0 : k0 + 1, e = V::VEC > 1 ? 2 * j % V::VEC : 0;
            if (at.has(k0)) out[at.apart(k0) + e] = lo;
            if (at.has(k1)) out[at.apart(k1) + (V::VEC > 1 ? e + 1 : 0)] = hi;
        }
    }
}

template <typename T, typename TG, int VEC>
cudaError_t launch_bwd(const NormParams& p, cudaStream_t st) {
    return pick_variant<VEC, true>(p.C / p.G / VEC, p.G, [&](auto variant) {
        using V = decltype(variant);
        const auto kern = norm_token_bwd_kernel<T, TG, V>;
        using M = Room<T, TG, V>;
        constexpr int join = V::NTH * 8;  // (the joining of the rows' sums, where they are in registers)
        constexpr int smem = V::kSharedSums ? M::kRings + M::kSums : M::kRings > join ? M::kRings : join;
        static std::atomic<uint64_t> allowed;
        cudaError_t e = allow_shared(kern, kDeclared, smem, allowed);
        if (e != cudaSuccess) return e;
        const Teams t = teams_of<V>(p);
        const dim3 grid = grid_of<V>(p, t, V::kBwd);
        float* const partial = static_cast<float*>(p.ws);
        kern<<<grid, t.threads, smem, st>>>(p, t, partial);
        e = cudaGetLastError();
        if (e != cudaSuccess || (!p.dweight && !p.dbias)) return e;
        return tc::launch_dependent(norm_weights_kernel, (unsigned)((p.C + 31) / 32), 256, 0, st, (const float*)partial, (int)grid.y, p.C, p.dweight,
                                    p.dbias);
    });
}

}  // namespace

// The most blocks along the rows of the variants that p's channels allow (which one runs depends on the alignment).
template <int VEC>
size_t most_rows(const NormParams& p) {
    const int cg = p.C / p.G;
    if (cg % VEC != 0) return 0;
    return pick_variant<VEC, true>(cg / VEC, p.G, [&](auto variant) {
        using V = decltype(variant);
        return (size_t)grid_of<V>(p, teams_of<V>(p), V::kBwd).y;
    });
}
size_t norm_token_bwd_workspace(const NormParams& p) {
    size_t most = most_rows<1>(p);
    for (size_t n : {most_rows<8>(p), most_rows<4>(p), most_rows<2>(p)})
        if (n > most) most = n;
    return most * 2 * p.C * 4;
}

cudaError_t norm_token_bwd(kda_dtype dt, kda_dtype gdt, const NormParams& p, cudaStream_t st) {
    using kda_host::rows_aligned;
    const int vec = dt == KDA_BF16 && gdt == KDA_BF16 ? 8 : 4, es = dt == KDA_BF16 ? 2 : 4, gs = gdt == KDA_BF16 ? 2 : 4, cg = p.C / p.G;
    const bool wide = cg % vec == 0 && rows_aligned(p.x, p.ldx, dt == KDA_BF16 ? 8 : 4) && rows_aligned(p.dy, p.C, vec) && rows_aligned(p.dx, p.C, vec);
    const bool pairs = cg % 2 == 0 && p.ldx % 2 == 0 && (uintptr_t)p.x % (2 * es) == 0 && (uintptr_t)p.dy % (2 * gs) == 0 && (uintptr_t)p.dx % (2 * gs) == 0;
    if (dt == KDA_F32) return wide ? launch_bwd<float, float, 4>(p, st) : pairs ? launch_bwd<float, float, 2>(p, st) : launch_bwd<float, float, 1>(p, st);
    if (gdt == KDA_F32) {
        if (wide) return launch_bwd<__nv_bfloat16, float, 4>(p, st);
        return pairs ? launch_bwd<__nv_bfloat16, float, 2>(p, st) : launch_bwd<__nv_bfloat16, float, 1>(p, st);
    }
    if (wide) return launch_bwd<__nv_bfloat16, __nv_bfloat16, 8>(p, st);
    return pairs ? launch_bwd<__nv_bfloat16, __nv_bfloat16, 2>(p, st) : launch_bwd<__nv_bfloat16, __nv_bfloat16, 1>(p, st);
}

}  // namespace kda
