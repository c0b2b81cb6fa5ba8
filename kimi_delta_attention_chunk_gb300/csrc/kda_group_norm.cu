// Group norm over each token's groups of channels: forward (how it works stands in kda_group_norm_token.cuh).
#include "kda_group_norm_token.cuh"

namespace kda {

namespace {

template <typename T, typename V>
__global__ void __launch_bounds__(V::NTH, V::kFwd) norm_token_fwd_kernel(NormParams p, Teams t) {
    constexpr int E2 = V::E2, A = V::kSlots;
    __shared__ float buf[2][V::NTH / 32][2];
    static_assert(sizeof(buf) <= kDeclared, "what a launch allows for");
    extern __shared__ __align__(16) char shared[];
    TeamSum<V::LANES, V::NTH> sum(buf, t.lanes);
    const Place<V> at(p, t);
    const float inv_n = 1.f / (float)(p.C / p.G);
    const Turns turns(p, t, at.rsub);
    Rows<V, T, A> rows(p.x, turns.first, p.ldx, turns.step, at, shared);
    auto request = [&](int i) {
        if (i < turns.full || (i < turns.all && turns.has(p, i))) rows.request(i, at);
        copies_commit();
    };
    if constexpr (A > 0)
#pragma unroll
        for (int i = 0; i < (A > 1 ? A - 1 : 1); ++i) request(i);
    Weights<V> weights(p, at, t.wide_weights);
    T* to = static_cast<T*>(p.y) + turns.first * p.C + at.first;
    const int64_t next = turns.step * p.C;
    for (int i = 0; i < turns.all; ++i, to += next) {
        const bool here = i < turns.full || turns.has(p, i);
        if constexpr (A > 0) copies_wait<(A > 1 ? A - 2 : 0)>();
        Pieces<V, T> raw;
        if (here) rows.take(i, at, raw);
        else raw.zero();
        if constexpr (A > 1) request(i + A - 1);
        f2 x[E2], a = 0ull;
        raw.pairs(x);
#pragma unroll
        for (int j = 0; j < E2; ++j) a = add2(a, x[j]);
        float s[1] = {sum2(a)};
        sum(s);
        if constexpr (A == 1) request(i + 1);  // (behind the sum's barrier: the row is in registers)
        const f2 mean = both(-s[0] * inv_n);
        a = 0ull;
#pragma unroll
        for (int j = 0; j < E2; ++j) {
            x[j] = at.masked(j, add2(x[j], mean));
            a = fma2(x[j], x[j], a);
        }
        s[0] = sum2(a);
        sum(s);
        if (!here) continue;
        const f2 rstd = both(inverse_deviation(s[0], inv_n, p.eps));
        if constexpr (!V::kKeep) weights.read(p, at, t.wide_weights);
#pragma unroll
        for (int j = 0; j < E2; ++j) x[j] = fma2(mul2(x[j], rstd), weights.w[j], weights.b[j]);
        if (p.act) {
#pragma unroll
            for (int j = 0; j < E2; ++j) x[j] = silu2(x[j]);
        }
        Pieces<V, T>::store(at, to, x);
    }
}

template <typename T, int VEC>
cudaError_t launch_fwd(const NormParams& p, cudaStream_t st) {
    return pick_variant<VEC, false>(p.C / p.G / VEC, p.G, [&](auto variant) {
        using V = decltype(variant);
        const auto kern = norm_token_fwd_kernel<T, V>;
        constexpr int smem = Rows<V, T, V::kSlots>::kBytes;
        static std::atomic<uint64_t> allowed;
        const cudaError_t e = allow_shared(kern, kDeclared, smem, allowed);
        if (e != cudaSuccess) return e;
        const Teams t = teams_of<V>(p);
        kern<<<grid_of<V>(p, t, V::kFwd), t.threads, smem, st>>>(p, t);
        return cudaGetLastError();
    });
}
}  // namespace

cudaError_t norm_token_fwd(kda_dtype dt, const NormParams& p, cudaStream_t st) {
    using kda_host::rows_aligned;
    const int vec = dt == KDA_BF16 ? 8 : 4, es = dt == KDA_BF16 ? 2 : 4, cg = p.C / p.G;
    const bool wide = cg % vec == 0 && rows_aligned(p.x, p.ldx, vec) && rows_aligned(p.y, p.C, vec);
    const bool pairs = cg % 2 == 0 && p.ldx % 2 == 0 && (uintptr_t)p.x % (2 * es) == 0 && (uintptr_t)p.y % (2 * es) == 0;
    if (dt == KDA_BF16) return wide ? launch_fwd<__nv_bfloat16, 8>(p, st) : pairs ? launch_fwd<__nv_bfloat16, 2>(p, st) : launch_fwd<__nv_bfloat16, 1>(p, st);
    return wide ? launch_fwd<float, 4>(p, st) : pairs ? launch_fwd<float, 2>(p, st) : launch_fwd<float, 1>(p, st);
}

}  // namespace kda
