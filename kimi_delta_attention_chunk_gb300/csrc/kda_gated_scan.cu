// Gated linear recurrence over prompts: forward (the formulas stand in kda_gated.cuh).
//
// An element costs 2 bytes of x, r, i, z and y each in bf16, three exponentials (a fourth where rates are large), three reciprocals and a root
// (one exponential and one reciprocal fewer without z): HBM, instruction issue and the special functions are near one another.  The
// recurrence is affine in h, so tokens are taken a tile at a time by a whole block: a lane has a strip of the tile's tokens and a pair of
// channels, whose decays and inputs stay in registers; the strips' maps h -> A h + H are folded over a warp by shuffles and over the block
// in shared memory, and every lane walks its tokens once more (one multiply-add each) from the true state.  Every row is read once, by
// asynchronous copies of the warp that works on it, a tile ahead.
// A block has 64, 32 or 16 channels of one sequence and the machine is filled with sequences and channels as far as these go (gated_channels);
// where they do not, up to eight blocks of a cluster take consecutive tiles and hand their tiles' maps to one another through
// distributed shared memory: one cluster barrier a tile, nothing read twice, sums in a fixed order.  Sequences that are packed have blocks
// of their own or are walked as one stream with maps that are cut where one begins (gated_each).
// bf16 with gates, 4096 channels, decays of 0.9 to 0.999: 7 x 2048 tokens in 100 us (88% of the bytes at the copy rate), 2 x 8192 in 138 (73%),
// one of 16384, four blocks to a cluster, in 150 (67%; a barrier of the cluster and a fold of four tiles every 512 tokens); with decays of 0.1
// to 0.7 (rates above 1/4) 115 and 169.  Leaving `states` adds 1 to 2 us.  fp32: 4 x 2048 in 99 (all of the copy rate).
// Two blocks of 128 registers a thread fill an SM: 16 warps that issue 2.0 instructions a cycle.  They wait on fixed latencies (1.1 cycles an
// instruction) and on the queue to shared memory and the special functions (1.0): seven special functions an element keep their pipe busy 51%
// of the time, 60% on the busiest SMs.  And 2 x 4096 tokens come to 256 blocks for 304 places: 104 SMs have two and 48 have one, active for
// 92,000 to 144,000 cycles, 127,000 on average.
// Slower when built: a warp of its own that folds while others work ahead (189), the exchange behind the next tile's gates
// (226: twice the code, and it waits for instructions), strips of 8 tokens with three blocks an SM (180), the output gates computed
// while the maps travel (160), maps that are padded with identities instead of tested (158).
#include <type_traits>

#include "kda_gated.cuh"
#include "kda_tc.cuh"

namespace kda {

namespace {

constexpr int kWarps = 8, kThreads = 32 * kWarps;
constexpr int kDeclared = 24 * 1024;  // shared memory that the kernel declares, at most
constexpr int kMean = 96;  // tokens of a sequence that has its own blocks, on average at least
template <typename T, int CH>
using LanesOf = Lanes<CH, sizeof(T) == 2 ? 16 : 8>;  // tokens of a strip
template <typename T, int CH>
constexpr int kTileOf = kWarps * LanesOf<T, CH>::kTokens;
// x, r, i and z of every warp's strip.  The next strip's x, r and i are asked for when the first walk is done with this one's, z before it.
template <typename T, int CH, bool kRows>
constexpr int kSmem = (kRows ? 4 : 3) * kWarps * LanesOf<T, CH>::kPart * (int)sizeof(T);

// kPacked: sequences by offsets, else a stream for each batch row.  kRows: y and the final states, else only the states that the
// backward pass starts from.  VEC: elements of a piece of x, r, i and z; with more than one, pairs of channels of y are whole and aligned.
template <typename E, int CH, int VEC, bool kPacked, bool kRows>
__global__ void __launch_bounds__(kThreads, 2) gated_fwd_kernel(GatedParams p, int cluster, int blocks, int longest) {
    using L = LanesOf<E, CH>;
    constexpr int STRIP = sizeof(E) == 2 ? 16 : 8, TT = kTileOf<E, CH>, PART = L::kPart;
    extern __shared__ __align__(128) char shared[];
    __shared__ Affine maps[2][kWarps][L::kPairs];
    __shared__ Affine peers[2][kMostCluster][L::kPairs];
    __shared__ f2 ends[2][L::kPairs];
    __shared__ Marks<kPacked ? L::kTokens : 1> all_marks[kWarps];
    __shared__ int32_t offsets[kPacked ? kCachedOffsets : 1];
    static_assert(sizeof(maps) + sizeof(peers) + sizeof(ends) + sizeof(all_marks) + sizeof(offsets) <= kDeclared, "what a launch allows for");

    if constexpr (kPacked) {
        const bool needed = longest >= p.T || any_longer(p, longest);
        tc::grid_dep_wait();
        if (!needed) return;
    } else {
        tc::grid_dep_launch();
    }
    const int pair = L::pair(), strip = L::strip(), w = __shfl_sync(0xffffffffu, threadIdx.x / 32, 0);
    const int rank = cluster > 1 ? (int)cluster_rank() : 0;
    const int group = blockIdx.x / cluster, b = group / blocks, c0 = group % blocks * CH;
    const int c = c0 + 2 * pair, has = p.C - c0, n2 = min(2, p.C - c);  // channels of this lane: 2, 1 or none (<= 0)
    const Offsets m(kPacked ? p.cu : nullptr, p.N, p.T, offsets);
    const Stretch mine_of = kPacked ? Stretch{0, p.T, m.first(), m.last()} : p.cu ? sequence_rows<false>(p, b) : Stretch{(int64_t)b * p.T, p.T, 0, p.T};
    const int T = mine_of.T, first = mine_of.first, last = mine_of.last;
    if (!kPacked && last - first > longest) return;  // the stream's kernel does it all
    const int64_t row0 = mine_of.row0;
    const int stride = TT * cluster;  // tokens between a block's tiles
    const int steps = (int)(((int64_t)T + stride - 1) / stride);
    int w0 = rank * TT + w * L::kTokens, s0 = w0 + strip * STRIP;  // this warp's first token, this strip's

    // this warp's rows: x, r, i and z
    E* const mine = reinterpret_cast<E*>(shared) + w * (kRows ? 4 : 3) * PART;
    using F = Feed<E, CH, STRIP, VEC>;
    F fx(p.x, p.ldx, row0 + w0, c0, stride), fr(p.r, p.ldr, row0 + w0, c0, stride), fi(p.i, p.ldi, row0 + w0, c0, stride);
    F fz(p.z, p.ldz, row0 + w0, c0, stride);
    auto request = [&](int rows) {
        if (rows >= L::kTokens && has >= CH) {
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
    request(T - w0);

    const f2 rate = pack(n2 > 0 ? gated_rate(__ldg(p.lam + c), p.decay) : 0.f, n2 > 1 ? gated_rate(__ldg(p.lam + c + 1), p.decay) : 0.f);
    const bool small = __all_sync(0xffffffffu, small_rate(rate)) != 0;
    // sequences without tokens hand their states on
    if (kRows && p.final_state) {
        if constexpr (kPacked) {
            for (int n0 = (w * cluster + rank) * 32; n0 < p.N; n0 += kWarps * cluster * 32) {
                const int n = n0 + (int)threadIdx.x % 32;
                unsigned empty = __ballot_sync(0xffffffffu, n < p.N && m.end(n) <= m.begin(n));
                for (; empty; empty &= empty - 1) {
                    const int64_t at = (int64_t)(n0 + __ffs(empty) - 1) * p.C + c;
                    store_state(p.final_state, at, state_pair(p.initial, at, n2), n2);
                }
            }
        } else if (T == 0 && rank == 0 && w == 0) {
            const int64_t at = (int64_t)b * p.C + c;
            store_state(p.final_state, at, state_pair(p.initial, at, n2), n2);
        }
    }
    f2 carry = kPacked ? 0ull : state_pair(p.initial, (int64_t)b * p.C + c, n2);
    if (w == 0) ends[0][pair] = carry;
    if (cluster > 1) {  // everyone's shared memory is there
        cluster_arrive<false>();
        cluster_wait();
    }

    Walk<kPacked ? L::kTokens : 1> walk;
    const int* const starts = all_marks[w].start + (kPacked ? strip * STRIP : 0);
    const int* const lasts = all_marks[w].end + (kPacked ? strip * STRIP : 0);
    const int64_t block0 = p.cu ? row0 / kGatedBlock : (int64_t)b * ((p.T + kGatedBlock - 1) / kGatedBlock);
    E* to = static_cast<E*>(p.y) + (row0 + s0) * p.C + c;
    for (int it = 0; it < steps; ++it, w0 += stride, s0 += stride, to += (int64_t)stride * p.C) {
        const int buf = it & 1;
        if (kRows && p.z) {
            if (T - w0 >= L::kTokens && has >= CH) fz.request(mine + 3 * PART);
            else fz.request(mine + 3 * PART, T - w0, has);
        }
        copies_commit();
        if constexpr (kPacked) walk.look(m, w0, it * stride, (it + 1) * stride, all_marks[w]);
        const bool wide = walk.wide, clear = walk.clear;
        // the first walk: decays and inputs, and the strip's map
        copies_wait<1>();
        __syncwarp();
        const E* const in = mine + L::place();
        f2 a[STRIP], u[STRIP];
        auto first_walk = [&](auto small_rates) {
#pragma unroll
            for (int j = 0; j < STRIP; ++j) {
                const f2 x = pair_at(in + j * CH), r = pair_at(in + PART + j * CH), i = pair_at(in + 2 * PART + j * CH);
                const Decay d = Decay::of<decltype(small_rates)::value>(gate2(r), rate);
                a[j] = d.a;
                u[j] = mul2(mul2(root2(d.m2), gate2(i)), x);
            }
        };
        if (small) first_walk(std::true_type{});
        else first_walk(std::false_type{});
        __syncwarp();
        request(T - w0 - stride);
        if (w0 < first || w0 + L::kTokens > last) {
#pragma unroll
            for (int j = 0; j < STRIP; ++j)
                if (s0 + j < first || s0 + j >= last) a[j] = both(1.f), u[j] = 0ull;
        }
        Affine map{a[0], u[0]};
        if (!kPacked || clear) {
#pragma unroll
            for (int j = 1; j < STRIP; ++j) map = follow<false>(map, Affine{a[j], u[j]});
        } else {
#pragma unroll
            for (int j = 0; j < STRIP; ++j) {
                const int n = starts[j];
                if (n >= 0) {
                    if (p.initial) u[j] = fma2(a[j], state_pair(p.initial, (int64_t)n * p.C + c, n2), u[j]);
                    a[j] = both(-1.f);
                }
                map = j ? follow<true>(map, Affine{a[j], u[j]}) : Affine{a[j], u[j]};
            }
        }
        Affine total, before;
        if (!kPacked || clear) join_strips<L, false, true>(map, total, before);
        else join_strips<L, true, true>(map, total, before);
        if (strip == 0) maps[buf][w][pair] = total;
        __syncthreads();
        // the state before the strip: between the blocks by their tiles' maps, then by the strips before
        auto fold = [&](auto cuts) {
            constexpr bool kCuts = decltype(cuts)::value;
            f2 h;
            if (cluster > 1) {
                if (w == 0) {
                    Affine all = total;
#pragma unroll
                    for (int k = 1; k < kWarps; ++k) all = follow<kCuts>(all, maps[buf][k][pair]);
                    if (strip == 0)
                        for (int k = 0; k < cluster; ++k) store_at(k, &peers[buf][rank][pair], all);
                    __syncwarp();
                    cluster_arrive<true>();
                } else {
                    cluster_arrive<false>();
                }
                cluster_wait();
#pragma unroll
                for (int k = 0; k < kMostCluster; ++k)
                    if (k < cluster) {
                        if (k == rank) h = carry;
                        const Affine e = peers[buf][k][pair];
                        carry = apply<kCuts>(e.A, e.H, carry);
                    }
            } else {
                h = ends[buf][pair];
            }
#pragma unroll
            for (int k = 0; k < kWarps - 1; ++k)
                if (k < w) {
                    const Affine e = maps[buf][k][pair];
                    h = apply<kCuts>(e.A, e.H, h);
                }
            if constexpr (L::kStrips > 1) h = apply<kCuts>(before.A, before.H, h);
            return h;
        };
        f2 h = !kPacked || wide ? fold(std::false_type{}) : fold(std::true_type{});
        static_assert(kGatedBlock % STRIP == 0, "blocks begin at strips");
        if (p.states && s0 % kGatedBlock == 0 && s0 >= first && s0 < last) {
            const bool begins = s0 == first || (kPacked && !clear && starts[0] >= 0);
            const int64_t block = block0 + s0 / kGatedBlock;
            store_state(p.states, block * p.C + c, begins ? 0ull : h, n2);
        }
        if constexpr (kRows) {
            copies_wait<1>();  // z
            __syncwarp();
            const E* const zin = in + 3 * PART;
            if (VEC > 1 && (!kPacked || clear) && w0 >= first && w0 + L::kTokens <= last) {
                // all of the warp's tokens are of one sequence
                E* at = to;
                auto second_walk = [&](auto gated) {
#pragma unroll
                    for (int j = 0; j < STRIP; ++j, at += p.C) {
                        h = fma2(a[j], h, u[j]);
                        f2 y = h;
                        if constexpr (decltype(gated)::value) {
                            const f2 z = pair_at(zin + j * CH);
                            y = mul2(h, mul2(z, gate2(z)));
                        }
                        store_pair<E, true>(at, y, n2);
                    }
                };
                if (p.z) second_walk(std::true_type{});
                else second_walk(std::false_type{});
                if (!kPacked && p.final_state && s0 + STRIP == T) store_state(p.final_state, (int64_t)b * p.C + c, h, n2);
            } else {
#pragma unroll
                for (int j = 0; j < STRIP; ++j) {
                    h = apply<kPacked>(a[j], u[j], h);
                    const int t = s0 + j;
                    if (t >= first && t < last) {
                        const f2 z = pair_at(zin + j * CH);
                        store_pair<E, false>(to + (int64_t)j * p.C, p.z ? mul2(h, mul2(z, gate2(z))) : h, n2);
                    }
                    if (p.final_state) {
                        const int n = kPacked ? (clear ? -1 : lasts[j]) : (t == T - 1 ? b : -1);
                        if (n >= 0) store_state(p.final_state, (int64_t)n * p.C + c, h, n2);
                    }
                }
            }
            __syncwarp();
        } else {
#pragma unroll
            for (int j = 0; j < STRIP; ++j) h = apply<kPacked>(a[j], u[j], h);
        }
        if (cluster == 1 && w == kWarps - 1 && strip == L::kStrips - 1) ends[buf ^ 1][pair] = h;
    }
}

// One kernel's launch.  cluster: blocks of a sequence; error: the kernel cannot be set up.
template <typename T, int CH, int VEC, bool kPacked, bool kRows>
struct Launch {
    static constexpr int kBytes = kSmem<T, CH, kRows>;
    const GatedParams& p;
    const int64_t blocks, groups;
    cudaError_t error;
    int cluster = 1;
    Launch(const GatedParams& p, int streams) : p(p), blocks((p.C + CH - 1) / CH), groups(blocks * streams) {
        static ClusterRoom room;
        static std::atomic<uint64_t> allowed;
        const auto kern = gated_fwd_kernel<T, CH, VEC, kPacked, kRows>;
        error = allow_shared(kern, kDeclared, kBytes, allowed);
        if (error == cudaSuccess) error = gated_cluster(room, kern, groups, p.T, kTileOf<T, CH>, kThreads, kBytes, cluster);
    }
    int pace() const { return kTileOf<T, CH> * cluster; }  // tokens of a sequence at a time
    cudaError_t operator()(int longest, bool dependent, cudaStream_t st) const {
        if (error != cudaSuccess) return error;
        return launch_clusters(gated_fwd_kernel<T, CH, VEC, kPacked, kRows>, groups * cluster, cluster, kThreads, kBytes, dependent, st, p, cluster, (int)blocks, longest);
    }
};
// Calls f with the launch of the width that fits (32 channels of smaller pieces gain nothing forwards: 7 sequences of 1 to 700 x 1530 fp32 24 and 25 us).
template <typename T, int VEC, bool kPacked, bool kRows, typename F>
cudaError_t with_launch(const GatedParams& p, int streams, F f) {
    const int ch = gated_channels(p, streams);
    if (VEC * sizeof(T) == 16 && ch == 32) return f(Launch<T, VEC * sizeof(T) == 16 ? 32 : 64, VEC, kPacked, kRows>(p, streams));
    return ch == 16 ? f(Launch<T, 16, VEC, kPacked, kRows>(p, streams)) : f(Launch<T, 64, VEC, kPacked, kRows>(p, streams));
}
template <typename T, int VEC, bool kRows>
cudaError_t launch_streams(const GatedParams& p, cudaStream_t st) {
    if (!p.cu || (gated_each(p, kMean) && p.N == 1))
        return with_launch<T, VEC, false, kRows>(p, p.cu ? 1 : p.B, [&](const auto& each) { return each(p.T, false, st); });
    return with_launch<T, VEC, true, kRows>(p, 1, [&](const auto& stream) {
        if (!gated_each(p, kMean) || stream.error != cudaSuccess) return stream(p.T, false, st);
        return with_launch<T, VEC, false, kRows>(p, p.N, [&](const auto& each) {
            const int longest = longest_of(p, each.pace(), stream.pace());
            const cudaError_t e = each(longest, false, st);
            return e != cudaSuccess || longest == p.T ? e : stream(longest, true, st);
        });
    });
}
template <typename T, int VEC>
cudaError_t launch_rows(const GatedParams& p, cudaStream_t st) {
    return p.y || p.final_state ? launch_streams<T, VEC, true>(p, st) : launch_streams<T, VEC, false>(p, st);
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
