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

constexpr int kWarps = 8, kThreads = 32 * kWarps;
template <typename T>
constexpr int kStripOf = sizeof(T) == 2 ? 16 : 8;  // tokens of a strip
template <typename T>
constexpr int kTileOf = kWarps * kStripOf<T>;
// x, r, i and z of every warp's strip.  The next strip's x, r and i are asked for when the first walk is done with this one's, z before it.
template <typename T, bool kRows>
constexpr int kSmem = (kRows ? 4 : 3) * kTileOf<T> * kGatedCh * (int)sizeof(T);

// kPacked: sequences by offsets, else a stream for each batch row.  kRows: y and the final states, else only the states that the
// backward pass starts from.  VEC: elements of a piece of x, r, i and z; with more than one, pairs of channels of y are whole and aligned.
template <typename T, int VEC, bool kPacked, bool kRows>
__global__ void __launch_bounds__(kThreads, 2) gated_fwd_kernel(GatedParams p, int cluster, int blocks) {
    constexpr int STRIP = kStripOf<T>, TT = kTileOf<T>, PART = STRIP * kGatedCh;
    extern __shared__ __align__(128) char shared[];
    __shared__ Affine maps[2][kWarps][32];
    __shared__ Affine peers[2][kMostCluster][32];
    __shared__ f2 ends[2][32];
    __shared__ Marks<kPacked ? STRIP : 1> all_marks[kWarps];
    __shared__ int32_t offsets[kPacked ? kCachedOffsets : 1];

    const int lane = threadIdx.x % 32, w = __shfl_sync(0xffffffffu, threadIdx.x / 32, 0);
    const int rank = cluster > 1 ? (int)cluster_rank() : 0;
    const int group = blockIdx.x / cluster, b = group / blocks, c0 = group % blocks * kGatedCh;
    const int c = c0 + 2 * lane, has = p.C - c0, n2 = min(2, p.C - c);  // channels of this lane: 2, 1 or none (<= 0)
    const Offsets m(p.cu, p.N, p.T, offsets);
    const int first = kPacked ? m.first() : 0, last = kPacked ? m.last() : p.T;
    const int stride = TT * cluster;  // tokens between a block's tiles
    const int steps = (int)(((int64_t)p.T + stride - 1) / stride);
    const int64_t row0 = (int64_t)b * p.T;
    int s0 = rank * TT + w * STRIP;  // this strip's first token

    // this warp's rows: x, r, i and z [4][STRIP][64]
    T* const mine = reinterpret_cast<T*>(shared) + w * (kRows ? 4 : 3) * PART;
    Feed<T, STRIP, VEC> fx(p.x, p.ldx, row0 + s0, c0, stride), fr(p.r, p.ldr, row0 + s0, c0, stride), fi(p.i, p.ldi, row0 + s0, c0, stride);
    Feed<T, STRIP, VEC> fz(p.z, p.ldz, row0 + s0, c0, stride);
    auto request = [&](int rows) {
        if (rows >= STRIP && has >= kGatedCh) {
            fx.request(mine);
            fr.request(mine + PART);
            fi.request(mine + 2 * PART);
        } else if (rows > 0) {
            fx.request(mine, rows, has);
            fr.request(mine + PART, rows, has);
            fi.request(mine + 2 * PART, rows, has);
        }
        copies_commit();
    };
    request(p.T - s0);

    const f2 rate = pack(n2 > 0 ? gated_rate(__ldg(p.lam + c), p.decay) : 0.f, n2 > 1 ? gated_rate(__ldg(p.lam + c + 1), p.decay) : 0.f);
    const bool small = __all_sync(0xffffffffu, small_rate(rate)) != 0;
    // sequences without tokens hand their states on
    if (kRows && p.final_state) {
        const int warps = kWarps * cluster;
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
    if (w == 0) ends[0][lane] = carry;
    if (cluster > 1) {  // everyone's shared memory is there
        cluster_arrive<false>();
        cluster_wait();
    }

    Walk<kPacked ? STRIP : 1> walk;
    const Marks<kPacked ? STRIP : 1>& marks = all_marks[w];
    T* to = static_cast<T*>(p.y) + (row0 + s0) * p.C + c;
    for (int it = 0; it < steps; ++it, s0 += stride, to += (int64_t)stride * p.C) {
        const int buf = it & 1;
        if (kRows && p.z) {
            if (p.T - s0 >= STRIP && has >= kGatedCh) fz.request(mine + 3 * PART);
            else fz.request(mine + 3 * PART, p.T - s0, has);
        }
        copies_commit();
        if constexpr (kPacked) walk.look(m, s0, it * stride, (it + 1) * stride, all_marks[w]);
        const bool wide = walk.wide, clear = walk.clear;
        // the first walk: decays and inputs, and the strip's map
        copies_wait<1>();
        __syncwarp();
        const T* const in = mine + 2 * lane;
        f2 a[STRIP], u[STRIP];
        auto first_walk = [&](auto small_rates) {
#pragma unroll
            for (int j = 0; j < STRIP; ++j) {
                const f2 x = pair_at(in + j * kGatedCh), r = pair_at(in + PART + j * kGatedCh), i = pair_at(in + 2 * PART + j * kGatedCh);
                const Decay d = Decay::of<decltype(small_rates)::value>(gate2(r), rate);
                a[j] = d.a;
                u[j] = mul2(mul2(root2(d.m2), gate2(i)), x);
            }
        };
        if (small) first_walk(std::true_type{});
        else first_walk(std::false_type{});
        __syncwarp();
        request(p.T - s0 - stride);
        if (s0 + STRIP > p.T) {
#pragma unroll
            for (int j = 0; j < STRIP; ++j)
                if (s0 + j >= p.T) a[j] = both(1.f), u[j] = 0ull;
        }
        Affine map{a[0], u[0]};
        if (!kPacked || clear) {
#pragma unroll
            for (int j = 1; j < STRIP; ++j) map = follow<false>(map, Affine{a[j], u[j]});
        } else {
#pragma unroll
            for (int j = 0; j < STRIP; ++j) {
                const int n = marks.start[j];
                if (n >= 0) {
                    if (p.initial) u[j] = fma2(a[j], state_pair(p.initial, (int64_t)n * p.C + c, n2), u[j]);
                    a[j] = both(-1.f);
                }
                map = j ? follow<true>(map, Affine{a[j], u[j]}) : Affine{a[j], u[j]};
            }
        }
        maps[buf][w][lane] = map;
        __syncthreads();
        // the state before the strip: between the blocks by their tiles' maps, then by the strips before
        auto fold = [&](auto cuts) {
            constexpr bool kCuts = decltype(cuts)::value;
            f2 h;
            if (cluster > 1) {
                if (w == 0) {
                    Affine total = map;
#pragma unroll
                    for (int k = 1; k < kWarps; ++k) total = follow<kCuts>(total, maps[buf][k][lane]);
                    for (int k = 0; k < cluster; ++k) store_at(k, &peers[buf][rank][lane], total);
                    cluster_arrive<true>();
                } else {
                    cluster_arrive<false>();
                }
                cluster_wait();
#pragma unroll
                for (int k = 0; k < kMostCluster; ++k)
                    if (k < cluster) {
                        if (k == rank) h = carry;
                        const Affine e = peers[buf][k][lane];
                        carry = apply<kCuts>(e.A, e.H, carry);
                    }
            } else {
                h = ends[buf][lane];
            }
#pragma unroll
            for (int k = 0; k < kWarps - 1; ++k)
                if (k < w) {
                    const Affine e = maps[buf][k][lane];
                    h = apply<kCuts>(e.A, e.H, h);
                }
            return h;
        };
        f2 h = !kPacked || wide ? fold(std::false_type{}) : fold(std::true_type{});
        static_assert(kGatedBlock % STRIP == 0, "blocks begin at strips");
        if (p.states && s0 % kGatedBlock == 0 && s0 < p.T) {
            const bool begins = s0 == 0 || (kPacked && !clear && marks.start[0] >= 0);
            const int64_t block = (int64_t)b * ((p.T + kGatedBlock - 1) / kGatedBlock) + s0 / kGatedBlock;
            store_state(p.states, block * p.C + c, begins ? 0ull : h, n2);
        }
        if constexpr (kRows) {
            copies_wait<1>();  // z
            __syncwarp();
            const T* const zin = mine + 3 * PART + 2 * lane;
            if (VEC > 1 && (!kPacked || clear) && s0 >= first && s0 + STRIP <= last) {
                // all of the strip's tokens are of one sequence
                T* at = to;
                auto second_walk = [&](auto gated) {
#pragma unroll
                    for (int j = 0; j < STRIP; ++j, at += p.C) {
                        h = fma2(a[j], h, u[j]);
                        f2 y = h;
                        if constexpr (decltype(gated)::value) {
                            const f2 z = pair_at(zin + j * kGatedCh);
                            y = mul2(h, mul2(z, gate2(z)));
                        }
                        store_pair<T, true>(at, y, n2);
                    }
                };
                if (p.z) second_walk(std::true_type{});
                else second_walk(std::false_type{});
                if (!kPacked && p.final_state && s0 + STRIP == p.T) store_state(p.final_state, (int64_t)b * p.C + c, h, n2);
            } else {
#pragma unroll
                for (int j = 0; j < STRIP; ++j) {
                    h = apply<kPacked>(a[j], u[j], h);
                    const int t = s0 + j;
                    if (t >= first && t < last) {
                        const f2 z = pair_at(zin + j * kGatedCh);
                        store_pair<T, false>(to + (int64_t)j * p.C, p.z ? mul2(h, mul2(z, gate2(z))) : h, n2);
                    }
                    if (p.final_state) {
                        const int n = kPacked ? (clear ? -1 : marks.end[j]) : (t == p.T - 1 ? b : -1);
                        if (n >= 0) store_state(p.final_state, (int64_t)n * p.C + c, h, n2);
                    }
                }
            }
            __syncwarp();
        } else {
#pragma unroll
            for (int j = 0; j < STRIP; ++j) h = apply<kPacked>(a[j], u[j], h);
        }
        if (cluster == 1 && w == kWarps - 1) ends[buf ^ 1][lane] = h;
    }
}

template <typename T, int VEC, bool kPacked, bool kRows>
cudaError_t launch(const GatedParams& p, cudaStream_t st) {
    const int blocks = (p.C + kGatedCh - 1) / kGatedCh;
    const int64_t groups = (int64_t)blocks * p.B;
    const auto kern = gated_fwd_kernel<T, VEC, kPacked, kRows>;
    constexpr int smem = kSmem<T, kRows>;
    static ClusterRoom room;
    static std::atomic<uint64_t> allowed;
    const cudaError_t e = allow_shared(kern, smem, allowed);
    if (e != cudaSuccess) return e;
    const int cluster = room.size_for(kern, groups, p.T, kTileOf<T>, kThreads, smem);
    return launch_clusters(kern, groups * cluster, cluster, kThreads, smem, st, p, cluster, blocks);
}
template <typename T, int VEC, bool kRows>
cudaError_t launch_packed(const GatedParams& p, cudaStream_t st) {
    return p.cu ? launch<T, VEC, true, kRows>(p, st) : launch<T, VEC, false, kRows>(p, st);
}
template <typename T, int VEC>
cudaError_t launch_rows(const GatedParams& p, cudaStream_t st) {
    return p.y || p.final_state ? launch_packed<T, VEC, true>(p, st) : launch_packed<T, VEC, false>(p, st);
}

}  // namespace

cudaError_t gated_scan_fwd(kda_dtype dt, const GatedParams& p, cudaStream_t st) {
    const int es = dt == KDA_BF16 ? 2 : 4;
    const bool pairs = p.C % 2 == 0 && (uintptr_t)p.y % (2 * es) == 0;
    if (dt == KDA_BF16) {
        if (pairs && gated_pieces(p, es, 16)) return launch_rows<__nv_bfloat16, 8>(p, st);
        if (pairs && gated_pieces(p, es, 4)) return launch_rows<__nv_bfloat16, 2>(p, st);
        return launch_rows<__nv_bfloat16, 1>(p, st);
    }
    if (pairs && gated_pieces(p, es, 16)) return launch_rows<float, 4>(p, st);
    if (pairs && gated_pieces(p, es, 8)) return launch_rows<float, 2>(p, st);
    return launch_rows<float, 1>(p, st);
}

}  // namespace kda
