// Gated linear recurrence over prompts: forward (the formulas stand in kda_gated.cuh).
//
// An element costs 2 bytes of x, r, i, z and y each in bf16, four exponentials, two reciprocals and a root: HBM and instruction issue
// are near one another.  The recurrence is affine in h, so tokens are taken a tile at a time by a whole block: a warp has a strip
// of the tile's tokens and a lane a pair of channels, whose decays and inputs stay in registers; the strips' maps h -> A h + H go
// through shared memory, every warp folds those before it, and walks its tokens once more (one multiply-add each) from the true
// state.  Every row is read once, by asynchronous copies some tiles ahead.
// Where sequences and channels alone do not fill the machine, up to eight blocks of a cluster take consecutive tiles at a time and hand their
// tiles' maps to one another through distributed shared memory: one cluster barrier a tile, nothing read twice, sums in a fixed order.
#include <type_traits>

#include "kda_gated.cuh"
#include "kda_tc.cuh"

namespace kda {

namespace {

template <typename T>
constexpr int kStripOf = sizeof(T) == 2 ? 8 : 4;  // tokens of a warp's strip
template <typename T>
constexpr int kTileOf = kGatedWarps * kStripOf<T>;
constexpr int kStages = 3;

template <typename T, bool kRows>
constexpr int kTensors = kRows ? 4 : 3;
template <typename T, bool kRows>
constexpr int kSmem = kStages * kTensors<T, kRows> * kTileOf<T> * kGatedCh * (int)sizeof(T);

// kPacked: sequences by offsets, else a stream for each batch row.  kRows: y and the final states, else only the states that the
// backward pass starts from.
template <typename T, int VEC, bool kPacked, bool kRows>
__global__ void __launch_bounds__(kGatedThreads, 2) gated_fwd_kernel(GatedParams p, int cluster, int blocks, bool whole_pairs) {
    constexpr int STRIP = kStripOf<T>, TT = kTileOf<T>, NT = kTensors<T, kRows>, TILE = TT * kGatedCh;
    extern __shared__ __align__(128) char shared[];
    T* const stage0 = reinterpret_cast<T*>(shared);
    __shared__ Affine strips[kGatedWarps][32];
    __shared__ Affine peers[2][kMostCluster][32];
    __shared__ TokenTile<kPacked ? TT : 1> tile;

    const int lane = threadIdx.x % 32, w = threadIdx.x / 32;
    const int rank = cluster > 1 ? (int)cluster_rank() : 0;
    const int group = blockIdx.x / cluster, b = group / blocks, c0 = group % blocks * kGatedCh;
    const int has = min(kGatedCh, p.C - c0), c = c0 + 2 * lane, n2 = min(2, p.C - c);  // pairs of this lane: 2, 1 or none (<= 0)
    const SeqMap m{p.cu, p.N, p.T, p.T};
    const int first = kPacked ? m.first() : 0, last = kPacked ? m.last() : p.T;
    const int steps = (int)(((int64_t)p.T + TT * cluster - 1) / (TT * cluster));
    const int64_t row0 = (int64_t)b * p.T;

    auto request = [&](int it) {
        const int t0 = (it * cluster + rank) * TT;
        const int rows = it < steps ? min(TT, p.T - t0) : 0;
        T* const to = stage0 + it % kStages * (NT * TILE);
        if (rows > 0) {
#pragma unroll
            for (int v = 0; v < NT; ++v) {
                const void* base = v == 0 ? p.x : v == 1 ? p.r : v == 2 ? p.i : p.z;
                const int64_t ld = v == 0 ? p.ldx : v == 1 ? p.ldr : v == 2 ? p.ldi : p.ldz;
                if (v == 3 && !base) continue;
                request_rows<T, TT, VEC>(to + v * TILE, static_cast<const T*>(base) + (row0 + t0) * ld + c0, ld, rows, has);
            }
        }
        copies_commit();
    };
#pragma unroll
    for (int s = 0; s < kStages - 1; ++s) request(s);

    const f2 rate = pack(n2 > 0 ? gated_rate(__ldg(p.lam + c), p.decay) : 0.f, n2 > 1 ? gated_rate(__ldg(p.lam + c + 1), p.decay) : 0.f);
    // sequences without tokens hand their states on
    if (kRows && p.final_state) {
        const int warps = kGatedWarps * cluster;
        for (int n0 = (w * cluster + rank) * 32; n0 < p.N; n0 += warps * 32) {
            if (!kPacked && p.T > 0) break;
            const int n = n0 + lane;
            unsigned empty = __ballot_sync(0xffffffffu, n < p.N && (!kPacked || m.end(n) <= m.begin(n)));
            for (; empty; empty &= empty - 1) {
                const int64_t at = (int64_t)(n0 + __ffs(empty) - 1) * p.C + c;
                store_state(p.final_state, at, state_pair(p.initial, at, n2), n2);
            }
        }
    }
    f2 carry = kPacked ? 0ull : state_pair(p.initial, (int64_t)b * p.C + c, n2);
    if (cluster > 1) {  // everyone's shared memory is there
        cluster_arrive();
        cluster_wait();
    }

    int until = 0;  // no boundary before this token
    for (int it = 0; it < steps; ++it) {
        const int t0 = (it * cluster + rank) * TT, rows = min(TT, p.T - t0);  // rows <= 0: nothing, behind the end
        copies_wait<kStages - 2>();
        __syncthreads();  // the tile is there, and everyone is past the one before
        request(it + kStages - 1);
        bool clear = true;  // no boundary in this warp's strip
        if constexpr (kPacked) {
            const bool plain = t0 + TT < until;  // (the same in the whole block)
            if (!plain && rows > 0) {
                tile.template build<kGatedThreads>(m, t0);
                until = tile.until;
                clear = tile.plain || tile.template clear<STRIP>(w * STRIP);
            }
        }
        const T* const in = stage0 + it % kStages * (NT * TILE) + w * STRIP * kGatedCh + 2 * lane;
        f2 a[STRIP], u[STRIP], gate[STRIP];
#pragma unroll
        for (int j = 0; j < STRIP; ++j) {
            const f2 x = pair_at(in + j * kGatedCh), r = pair_at(in + TILE + j * kGatedCh), i = pair_at(in + 2 * TILE + j * kGatedCh);
            const Decay d(rcp2(one_plus<false>(r)), rate);
            a[j] = d.a;
            f2 si;
            if (kRows && p.z) {
                const f2 z = pair_at(in + 3 * TILE + j * kGatedCh), di = one_plus<true>(i), dz = one_plus<true>(z);
                const f2 inv = rcp2(mul2(di, dz));
                si = mul2(inv, dz);
                gate[j] = mul2(z, mul2(inv, di));
            } else {
                si = rcp2(one_plus<false>(i));
                gate[j] = both(1.f);
            }
            u[j] = mul2(mul2(mul2(d.m2, inverse_root(d.m2)), si), x);
        }
        if (rows < TT) {
#pragma unroll
            for (int j = 0; j < STRIP; ++j)
                if (w * STRIP + j >= rows) a[j] = both(1.f), u[j] = 0ull;
        }
        if (kPacked && !clear) {
#pragma unroll
            for (int j = 0; j < STRIP; ++j) {
                const int n = tile.start[w * STRIP + j];
                if (n >= 0) {
                    if (p.initial) u[j] = fma2(a[j], state_pair(p.initial, (int64_t)n * p.C + c, n2), u[j]);
                    a[j] = both(-1.f);
                }
            }
        }
        Affine mine{a[0], u[0]};
#pragma unroll
        for (int j = 1; j < STRIP; ++j) mine = follow<kPacked>(mine, Affine{a[j], u[j]});
        strips[w][lane] = mine;
        __syncthreads();
        Affine before = identity(), total = identity();
#pragma unroll
        for (int k = 0; k < kGatedWarps; ++k) {
            if (k == w) before = total;
            total = follow<kPacked>(total, strips[k][lane]);
        }
        f2 h = carry;
        if (cluster > 1) {
            const int buf = it & 1;
            if (w < cluster) store_at(w, &peers[buf][rank][lane], total);
            cluster_arrive();
            cluster_wait();
            for (int k = 0; k < cluster; ++k) {
                if (k == rank) h = carry;
                const Affine e = peers[buf][k][lane];
                carry = apply<kPacked>(e.A, e.H, carry);
            }
        } else {
            carry = apply<kPacked>(total.A, total.H, carry);
        }
        h = apply<kPacked>(before.A, before.H, h);
        if (p.states && w * STRIP % kGatedBlock == 0 && w * STRIP < rows) {
            const bool begins = t0 + w * STRIP == 0 || (kPacked && !clear && tile.start[w * STRIP] >= 0);
            const int64_t block = (int64_t)b * ((p.T + kGatedBlock - 1) / kGatedBlock) + (t0 + w * STRIP) / kGatedBlock;
            store_state(p.states, block * p.C + c, begins ? 0ull : h, n2);
        }
        if constexpr (kRows) {
            T* const to = static_cast<T*>(p.y) + (row0 + t0 + w * STRIP) * p.C + c;
#pragma unroll
            for (int j = 0; j < STRIP; ++j) {
                h = apply<kPacked>(a[j], u[j], h);
                const int t = t0 + w * STRIP + j;
                if (w * STRIP + j < rows && t >= first && t < last) {
                    const f2 y = mul2(h, gate[j]);
                    if (whole_pairs) store_pair<T, true>(to + (int64_t)j * p.C, y, n2);
                    else store_pair<T, false>(to + (int64_t)j * p.C, y, n2);
                }
                if (p.final_state) {
                    const int n = kPacked ? (clear ? -1 : tile.end[w * STRIP + j]) : (t == p.T - 1 ? b : -1);
                    if (n >= 0) store_state(p.final_state, (int64_t)n * p.C + c, h, n2);
                }
            }
        }
    }
}

template <typename T, int VEC, bool kPacked, bool kRows>
cudaError_t launch(const GatedParams& p, bool whole_pairs, cudaStream_t st) {
    const int blocks = (p.C + kGatedCh - 1) / kGatedCh;
    const int64_t groups = (int64_t)blocks * p.B;
    const int cluster = cluster_size(groups, p.T, kTileOf<T>);
    return launch_clusters(gated_fwd_kernel<T, VEC, kPacked, kRows>, groups * cluster, cluster, kSmem<T, kRows>, st, p, cluster, blocks,
                           whole_pairs);
}
template <typename T, int VEC, bool kRows>
cudaError_t launch_packed(const GatedParams& p, bool whole_pairs, cudaStream_t st) {
    return p.cu ? launch<T, VEC, true, kRows>(p, whole_pairs, st) : launch<T, VEC, false, kRows>(p, whole_pairs, st);
}
template <typename T, int VEC>
cudaError_t launch_rows(const GatedParams& p, bool whole_pairs, cudaStream_t st) {
    return p.y || p.final_state ? launch_packed<T, VEC, true>(p, whole_pairs, st) : launch_packed<T, VEC, false>(p, whole_pairs, st);
}

}  // namespace

cudaError_t gated_scan_fwd(kda_dtype dt, const GatedParams& p, cudaStream_t st) {
    const int es = dt == KDA_BF16 ? 2 : 4;
    const bool whole_pairs = p.C % 2 == 0 && (uintptr_t)p.y % (2 * es) == 0;
    if (dt == KDA_BF16) {
        if (gated_pieces(p, es, 16)) return launch_rows<__nv_bfloat16, 8>(p, whole_pairs, st);
        if (gated_pieces(p, es, 4)) return launch_rows<__nv_bfloat16, 2>(p, whole_pairs, st);
        return launch_rows<__nv_bfloat16, 1>(p, whole_pairs, st);
    }
    if (gated_pieces(p, es, 16)) return launch_rows<float, 4>(p, whole_pairs, st);
    return launch_rows<float, 1>(p, whole_pairs, st);
}

}  // namespace kda
