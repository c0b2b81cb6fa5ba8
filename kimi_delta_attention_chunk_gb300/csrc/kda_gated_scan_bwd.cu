// Gated linear recurrence over prompts: backward.
//
// With the forward's s, a, m, si = sigmoid(i), sr = sigmoid(r), u, h and yb = dy silu(z), per sequence and channel:
//     dh_t = yb_t + a_{t+1} dh_{t+1}   (behind the last token: the final state's gradient)
//     dx = dh m si,  di = dh u (1 - si),  dz = dy h silu'(z),  dinitial = a_0 dh_0
//     ds = dh (si x a^2 / m - a h_{t-1})      (dm / ds = e^-2s / m)
//     dr = ds rate sr (1 - sr),  dlam = decay sigmoid(lam) sum_t ds sr
// The forward pass leaves the state before every 32nd token, and tiles are multiples of those, so that every tile can form its own
// states; dh is carried from tile to tile backwards as the forward pass carries h (kda_gated_scan.cu): strips of four tokens a lane, their
// maps folded by shuffles and through shared memory, clusters where sequences and channels do not fill the machine.  What an
// element needs (a, u, m si, si x a^2 / m, sr, 1 - si, yb, dy silu'(z)) stays in registers between the two walks: 128 a thread, two blocks an
// SM, whose 16 warps issue 2.2 instructions a cycle: that and their latencies bound it.  Without the states a first pass of the forward kernel makes them (x, r and i are then
// read twice).  dlam's sums over tokens: one partial sum a block, added in a fixed order.
// bf16 with gates, 4096 channels: 4 x 2048 tokens in 138 us (66% of the bytes at the copy rate), 2 x 2048 in 74 (62%; rates above 1/4: 77), whose
// 256 blocks for 304 places leave 48 SMs with one: active for 96,000 to 146,000 cycles, 129,000 on average.  4 x 2048 with fp32 gradients
// 157 (90%), in fp32 206 (88%), with nothing kept 188 (bf16) and 258 (fp32).
// Slower when built: a tile's map sent before the rest is computed (92 for 89 then), the maps' lengths tested instead of padded with identities (100).
#include <algorithm>
#include <type_traits>

#include "kda_gated.cuh"
#include "kda_tc.cuh"

namespace kda {

namespace {

constexpr int kWarps = 8, kThreads = 32 * kWarps;
constexpr int kDeclared = 40 * 1024;  // shared memory that the kernel declares, at most
constexpr int kMean = 32;   // tokens of a sequence that has its own blocks, on average at least
constexpr int kStrip = 4;
template <int CH>
constexpr int kTile = kWarps * Lanes<CH, kStrip>::kTokens;
static_assert(kTile<64> % kGatedBlock == 0 && kTile<32> % kGatedBlock == 0 && kTile<16> % kGatedBlock == 0, "tiles begin at states that are left to them");

// x, r, i, z and dy of every warp's strip, in two stages.
constexpr int kStages = 2;
template <typename T, typename TG, int CH>
constexpr int kStageBytes = kWarps * Lanes<CH, kStrip>::kPart * (4 * (int)sizeof(T) + (int)sizeof(TG));

// VEC, GVEC: elements of a piece of x, r, i and z, and of dy; with VEC > 1, pairs of channels of the outputs are whole and aligned.
template <typename T, typename TG, int CH, int VEC, int GVEC, bool kPacked>
__global__ void __launch_bounds__(kThreads, 2) gated_bwd_kernel(GatedParams p, float* partial, int cluster, int blocks, int longest) {
    using L = Lanes<CH, kStrip>;
    constexpr int PART = L::kPart, TT = kTile<CH>, kStage = kStageBytes<T, TG, CH>;
    extern __shared__ __align__(128) char shared[];
    // The strips' maps, backwards [0, kWarps) and forwards [kAhead, kAhead + kWarps), with maps between them that change nothing: every
    // warp folds kWarps - 1 maps, those behind its own backwards and those before it forwards.
    constexpr int kAhead = 2 * kWarps - 1;
    __shared__ Affine maps[2][kAhead + kWarps][L::kPairs];
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
    const Stretch rows_of = kPacked ? Stretch{0, p.T, m.first(), m.last()} : p.cu ? sequence_rows<true>(p, b) : Stretch{(int64_t)b * p.T, p.T, 0, p.T};
    const int S = rows_of.T, first = rows_of.first, last = rows_of.last;
    if (!kPacked && last - first > longest) return;  // the stream's kernel does it all
    const int from = kPacked || !p.cu || b == 0 ? 0 : first;  // the first row that is this block's to write
    const int64_t row0 = rows_of.row0;
    const int stride = TT * cluster;  // tokens between a block's tiles
    const int steps = (int)(((int64_t)S + stride - 1) / stride);
    // this warp's first token and this strip's: tiles are taken from the stream's end
    int w0 = (steps - 1) * stride + rank * TT + w * L::kTokens, s0 = w0 + strip * kStrip;

    // this warp's rows: a stage holds x, r, i, z and dy
    char* const mine = shared + w * (kStage / kWarps);
    using F = Feed<T, CH, kStrip, VEC>;
    F fx(p.x, p.ldx, row0 + w0, c0, -stride), fr(p.r, p.ldr, row0 + w0, c0, -stride), fi(p.i, p.ldi, row0 + w0, c0, -stride);
    F fz(p.z, p.ldz, row0 + w0, c0, -stride);
    Feed<TG, CH, kStrip, GVEC> fy(p.dy, p.C, row0 + w0, c0, -stride);
    auto request = [&](int it) {
        const int rows = S - (w0 - stride);
        T* const in = reinterpret_cast<T*>(mine + (it & 1) * kStage);
        if (it < steps) {
            TG* const dys = reinterpret_cast<TG*>(in + 4 * PART);
            if (rows >= L::kTokens && has >= CH) {
                fx.request(in);
                fr.request(in + PART);
                fi.request(in + 2 * PART);
                fy.request(dys);
                if (p.z) fz.request(in + 3 * PART);
            } else {
                fx.request(in, rows, has);
                fr.request(in + PART, rows, has);
                fi.request(in + 2 * PART, rows, has);
                fy.request(dys, rows, has);
                if (p.z) fz.request(in + 3 * PART, rows, has);
            }
        }
        copies_commit();
    };
    w0 += stride;
    request(0);
    w0 -= stride;

    const f2 rate = pack(n2 > 0 ? gated_rate(__ldg(p.lam + c), p.decay) : 0.f, n2 > 1 ? gated_rate(__ldg(p.lam + c + 1), p.decay) : 0.f);
    const f2 down = neg2(rate);
    const bool small = __all_sync(0xffffffffu, small_rate(rate)) != 0;
    // through sequences without tokens the gradient goes as it comes
    if (p.dinitial) {
        if constexpr (kPacked) {
            for (int n0 = (w * cluster + rank) * 32; n0 < p.N; n0 += kWarps * cluster * 32) {
                const int n = n0 + (int)threadIdx.x % 32;
                unsigned empty = __ballot_sync(0xffffffffu, n < p.N && m.end(n) <= m.begin(n));
                for (; empty; empty &= empty - 1) {
                    const int64_t at = (int64_t)(n0 + __ffs(empty) - 1) * p.C + c;
                    store_state(p.dinitial, at, state_pair(p.dfinal, at, n2), n2);
                }
            }
        } else if (S == 0 && rank == 0 && w == 0) {
            const int64_t at = (int64_t)b * p.C + c;
            store_state(p.dinitial, at, state_pair(p.dfinal, at, n2), n2);
        }
    }
    f2 carry = kPacked ? 0ull : state_pair(p.dfinal, (int64_t)b * p.C + c, n2), dlam = 0ull;
    if (w == 0) ends[0][pair] = carry;
    if (w < kWarps - 1) maps[0][kWarps + w][pair] = maps[1][kWarps + w][pair] = identity();
    if (cluster > 1) {
        cluster_arrive<false>();
        cluster_wait();
    }

    // where this warp's first row of an output and the tile's state are; all move up by a stride of rows a step
    int64_t off = (row0 + s0) * p.C + c;
    const float* left = p.states + ((p.cu ? row0 / kGatedBlock : (int64_t)b * ((p.T + kGatedBlock - 1) / kGatedBlock)) + (w0 - w * L::kTokens) / kGatedBlock) * p.C + c;
    Walk<kPacked ? L::kTokens : 1> walk;
    const int* const starts = all_marks[w].start + (kPacked ? strip * kStrip : 0);
    const int* const lasts = all_marks[w].end + (kPacked ? strip * kStrip : 0);
    for (int it = 0; it < steps; ++it, w0 -= stride, s0 -= stride, off -= (int64_t)stride * p.C, left -= (int64_t)(stride / kGatedBlock) * p.C) {
        const int t0 = w0 - w * L::kTokens, buf = it & 1;
        f2 h = 0ull;
        if (t0 < S) {
            if (!kPacked && t0 <= first) h = state_pair(p.initial, (int64_t)b * p.C + c, n2);
            else if (VEC > 1) h = n2 > 0 ? *reinterpret_cast<const f2*>(left) : 0ull;
            else h = pack(n2 > 0 ? left[0] : 0.f, n2 > 1 ? left[1] : 0.f);
        }
        if constexpr (kPacked) walk.look(m, w0, t0 - rank * TT, t0 - rank * TT + stride, all_marks[w]);
        const bool wide = walk.wide, clear = walk.clear;
        copies_wait<0>();
        __syncwarp();  // the strip's rows are there, and every lane is past the strip before
        request(it + 1);
        const T* const in = reinterpret_cast<const T*>(mine + buf * kStage) + L::place();
        const TG* const dys = reinterpret_cast<const TG*>(in - L::place() + 4 * PART) + L::place();
        f2 a[kStrip], u[kStrip], wx[kStrip], wm[kStrip], sr[kStrip], ui[kStrip], yb[kStrip], gz[kStrip];
        auto gates = [&](auto small_rates) {
#pragma unroll
            for (int j = 0; j < kStrip; ++j) {
                const f2 x = pair_at(in + j * CH), r = pair_at(in + PART + j * CH), i = pair_at(in + 2 * PART + j * CH);
                sr[j] = gate2(r);
                const f2 si = gate2(i);
                const Decay d = Decay::of<decltype(small_rates)::value>(sr[j], rate);
                const f2 inv = inverse_root(d.m2), gx = mul2(si, x), m1 = mul2(d.m2, inv);
                a[j] = d.a;
                wx[j] = mul2(m1, si);
                u[j] = mul2(m1, gx);
                ui[j] = mul2(u[j], rest2(si));
                wm[j] = mul2(mul2(gx, inv), mul2(d.a, d.a));
                yb[j] = pair_at(dys + j * CH);
            }
        };
        // in a sequence's first and last tile some warps have nothing to do (skipped at this width only: 4 x 4096 x 4096 304 -> 286 us,
        // but with 32 channels 2 x 2048 x 4096 76 -> 81, by what the compiler keeps in registers)
        const bool idle = !kPacked && CH == 64 && (w0 + L::kTokens <= from || w0 >= S);
        if (!idle) {
            if (small) gates(std::true_type{});
            else gates(std::false_type{});
        }
        if (p.z && !idle) {
#pragma unroll
            for (int j = 0; j < kStrip; ++j) {
                const f2 z = pair_at(in + 3 * PART + j * CH), s = gate2(z), silu = mul2(z, s);
                gz[j] = mul2(yb[j], fma2(silu, rest2(s), s));  // silu' = s + z s (1 - s)
                yb[j] = mul2(yb[j], silu);
            }
        }
        if (w0 < first || w0 + L::kTokens > last) {
#pragma unroll
            for (int j = 0; j < kStrip; ++j)
                if (s0 + j < first || s0 + j >= last) a[j] = both(1.f), u[j] = yb[j] = 0ull;
        }
        // the strip's maps forwards (cut where a sequence begins) and backwards (cut where one ends)
        Affine fore, rear;
        if (!kPacked || clear) {
            fore = Affine{a[0], u[0]};
#pragma unroll
            for (int j = 1; j < kStrip; ++j) fore = follow<false>(fore, Affine{a[j], u[j]});
            rear.A = fore.A;
            rear.H = mul2(a[kStrip - 1], yb[kStrip - 1]);
#pragma unroll
            for (int j = kStrip - 2; j >= 0; --j) rear.H = mul2(a[j], add2(yb[j], rear.H));
        } else {
            fore = rear = identity();
#pragma unroll
            for (int j = 0; j < kStrip; ++j) {
                const int n = starts[j];
                if (n >= 0) fore = Affine{both(-1.f), fma2(a[j], state_pair(p.initial, (int64_t)n * p.C + c, n2), u[j])};
                else fore = follow<true>(fore, Affine{a[j], u[j]});
            }
#pragma unroll
            for (int j = kStrip - 1; j >= 0; --j) {
                const int n = lasts[j];
                if (n >= 0) {
                    yb[j] = add2(yb[j], state_pair(p.dfinal, (int64_t)n * p.C + c, n2));
                    rear = Affine{both(-1.f), mul2(a[j], yb[j])};
                } else {
                    rear = follow<true>(rear, Affine{a[j], mul2(a[j], yb[j])});
                }
            }
        }
        Affine fores, ahead, rears, behind;  // the warp's maps, and those of its strips in front of this one, and behind
        if (!kPacked || clear) {
            join_strips<L, false, true>(fore, fores, ahead);
            join_strips<L, false, false>(rear, rears, behind);
        } else {
            join_strips<L, true, true>(fore, fores, ahead);
            join_strips<L, true, false>(rear, rears, behind);
        }
        if (strip == 0) {
            maps[buf][w][pair] = rears;
            maps[buf][kAhead + w][pair] = fores;
        }
        __syncthreads();
        f2 g;
        auto publish = [&](auto cuts) {
            if (w == kWarps - 1) {
                Affine total = rears;
#pragma unroll
                for (int k = kWarps - 2; k >= 0; --k) total = follow<decltype(cuts)::value>(total, maps[buf][k][pair]);
                if (strip == 0)
                    for (int k = 0; k < cluster; ++k) store_at(k, &peers[buf][rank][pair], total);
                __syncwarp();
                cluster_arrive<true>();
            } else {
                cluster_arrive<false>();
            }
        };
        auto fold = [&](auto cuts) {
            constexpr bool kCuts = decltype(cuts)::value;
            if (cluster > 1) {
                cluster_wait();
                for (int k = cluster - 1; k > rank; --k) carry = apply<kCuts>(peers[buf][k][pair].A, peers[buf][k][pair].H, carry);
                g = carry;
                for (int k = rank; k >= 0; --k) carry = apply<kCuts>(peers[buf][k][pair].A, peers[buf][k][pair].H, carry);
            } else {
                g = ends[buf][pair];
            }
#pragma unroll
            for (int k = kWarps - 1; k > 0; --k) g = apply<kCuts>(maps[buf][w + k][pair].A, maps[buf][w + k][pair].H, g);
            if constexpr (L::kStrips > 1) g = apply<kCuts>(behind.A, behind.H, g);
        };
        if (!kPacked || wide) {
            if (cluster > 1) publish(std::false_type{});
#pragma unroll
            for (int k = 0; k < kWarps - 1; ++k) h = fma2(maps[buf][kWarps + w + k][pair].A, h, maps[buf][kWarps + w + k][pair].H);
            if constexpr (L::kStrips > 1) h = fma2(ahead.A, h, ahead.H);
        } else {
            if (cluster > 1) publish(std::true_type{});
#pragma unroll
            for (int k = 0; k < kWarps - 1; ++k) h = apply<true>(maps[buf][kWarps + w + k][pair].A, maps[buf][kWarps + w + k][pair].H, h);
            if constexpr (L::kStrips > 1) h = apply<true>(ahead.A, ahead.H, h);
        }
        const bool lean = VEC > 1 && (!kPacked || clear) && w0 >= first && w0 + L::kTokens <= last;  // the warp's tokens are of one sequence
        // the state before each token, and with it what dh is multiplied by: wm = si x a^2 / m - a h_{t-1}; dz is done
#pragma unroll
        for (int j = 0; j < kStrip; ++j) {
            if (kPacked && !clear) {
                const int n = starts[j];
                if (n >= 0) h = state_pair(p.initial, (int64_t)n * p.C + c, n2);
            }
            const f2 ah = mul2(a[j], h);
            wm[j] = fma2(ah, both(-1.f), wm[j]);
            h = add2(ah, u[j]);
            if (p.z) gz[j] = mul2(gz[j], h);
        }
        if (p.z && lean) {
            TG* to = static_cast<TG*>(p.dz) + off;
#pragma unroll
            for (int j = 0; j < kStrip; ++j, to += p.C) store_pair<TG, true>(to, gz[j], n2);
        }
        if (!kPacked || wide) fold(std::false_type{});
        else fold(std::true_type{});
        if (lean) {
            const int64_t up = (int64_t)(kStrip - 1) * p.C;
            TG *dx = static_cast<TG*>(p.dx) + off + up, *dr = static_cast<TG*>(p.dr) + off + up, *di = static_cast<TG*>(p.di) + off + up;
#pragma unroll
            for (int j = kStrip - 1; j >= 0; --j, dx -= p.C, dr -= p.C, di -= p.C) {
                const f2 dh = add2(yb[j], g), part = mul2(mul2(dh, wm[j]), sr[j]);
                g = mul2(a[j], dh);
                dlam = add2(dlam, part);
                store_pair<TG, true>(dx, mul2(dh, wx[j]), n2);
                store_pair<TG, true>(dr, mul2(part, fma2(sr[j], down, rate)), n2);
                store_pair<TG, true>(di, mul2(dh, ui[j]), n2);
            }
            if (!kPacked && s0 == from && p.dinitial) store_state(p.dinitial, (int64_t)b * p.C + c, g, n2);
        } else if (!idle) {
#pragma unroll
            for (int j = kStrip - 1; j >= 0; --j) {
                const int t = s0 + j;
                if (t < from || t >= S) continue;
                if (kPacked && !clear && lasts[j] >= 0) g = 0ull;
                const f2 dh = add2(yb[j], g);
                f2 part = mul2(mul2(dh, wm[j]), sr[j]), dx = mul2(dh, wx[j]), dr = mul2(part, fma2(sr[j], down, rate)), di = mul2(dh, ui[j]);
                g = mul2(a[j], dh);
                if (t >= first && t < last) dlam = add2(dlam, part);
                else dx = di = dr = gz[j] = 0ull;
                const int64_t o = off + (int64_t)j * p.C;
                store_pair<TG, false>(static_cast<TG*>(p.dx) + o, dx, n2);
                store_pair<TG, false>(static_cast<TG*>(p.dr) + o, dr, n2);
                store_pair<TG, false>(static_cast<TG*>(p.di) + o, di, n2);
                if (p.z) store_pair<TG, false>(static_cast<TG*>(p.dz) + o, gz[j], n2);
                if (p.dinitial) {
                    const int n = kPacked ? (clear ? -1 : starts[j]) : (t == from ? b : -1);
                    if (n >= 0) store_state(p.dinitial, (int64_t)n * p.C + c, g, n2);
                }
            }
        }
        if (cluster == 1 && w == 0 && strip == 0) ends[buf ^ 1][pair] = g;
    }
    tc::grid_dep_launch();
    __syncthreads();
    f2* const parts = reinterpret_cast<f2*>(maps);
    static_assert(sizeof(maps) >= kThreads * sizeof(f2), "a part each thread");
    parts[w * 32 + threadIdx.x % 32] = dlam;
    __syncthreads();
    if (w == 0 && strip == 0 && p.T > 0) {
        f2 sum = 0ull;
        for (int k = 0; k < kWarps * L::kStrips; ++k) sum = add2(sum, parts[k * L::kPairs + pair]);
        store_state(partial + ((int64_t)b * cluster + rank) * p.C, c, sum, n2);
    }
}

// dlam from the blocks' partial sums: `parts` of them, or `packed` where a sequence is longer than `longest`.  A block has 32 channels.
constexpr int kSummers = 8;
__global__ void __launch_bounds__(32 * kSummers) gated_dlam_kernel(GatedParams p, const float* partial, int parts, int packed, int longest) {
    __shared__ float sums[kSummers][32];
    const int c = blockIdx.x * 32 + threadIdx.x % 32, w = threadIdx.x / 32;
    if (p.cu && longest < p.T && any_longer(p, longest)) parts = packed;
    tc::grid_dep_wait();
    float sum = 0.f;
    if (c < p.C) {
#pragma unroll 4
        for (int k = w; k < parts; k += kSummers) sum += partial[(int64_t)k * p.C + c];
    }
    sums[w][threadIdx.x % 32] = sum;
    __syncthreads();
    if (w || c >= p.C) return;
    for (int k = 1; k < kSummers; ++k) sum += sums[k][threadIdx.x];
    const float l = __ldg(p.lam + c), e = expf(-fabsf(l));
    p.dlam[c] = p.decay * (l >= 0.f ? 1.f : e) / (1.f + e) * sum;
}

// (one partial sum a block)
size_t partial_bytes(const GatedParams& p) {
    const int64_t streams = gated_each(p, kMean) ? p.N : p.B;
    const int64_t blocks = streams * ((p.C + 63) / 64) > kSms ? 1 : most_blocks(p.T, kTile<64>);  // of a stream (narrower ones are more)
    const int64_t packed = p.cu ? most_blocks(p.T, kTile<64>) : 0;
    return ((size_t)(p.T > 0 ? std::max(streams * blocks, packed) : 0) * p.C * 4 + 255) / 256 * 256;
}

// One kernel's launch.  cluster: blocks of a sequence; error: the kernel cannot be set up.
template <typename T, typename TG, int CH, int VEC, int GVEC, bool kPacked>
struct Launch {
    static constexpr int kBytes = kStages * kStageBytes<T, TG, CH>;
    const GatedParams& p;
    const int64_t blocks, groups;
    cudaError_t error;
    int cluster = 1, parts;
    Launch(const GatedParams& p, int streams) : p(p), blocks((p.C + CH - 1) / CH), groups(blocks * streams) {
        static ClusterRoom room;
        static std::atomic<uint64_t> allowed;
        const auto kern = gated_bwd_kernel<T, TG, CH, VEC, GVEC, kPacked>;
        error = allow_shared(kern, kDeclared, kBytes, allowed);
        if (error == cudaSuccess) error = gated_cluster(room, kern, groups, p.T, kTile<CH>, kThreads, kBytes, cluster);
        parts = p.T > 0 ? streams * cluster : 0;  // partial sums of dlam
    }
    int pace() const { return kTile<CH> * cluster; }  // tokens of a sequence at a time
    cudaError_t operator()(int longest, bool dependent, cudaStream_t st) const {
        if (error != cudaSuccess || groups == 0) return error;
        return launch_clusters(gated_bwd_kernel<T, TG, CH, VEC, GVEC, kPacked>, groups * cluster, cluster, kThreads, kBytes, dependent, st, p, static_cast<float*>(p.ws), cluster,
                               (int)blocks, longest);
    }
};
// Calls f with the launch of the width that fits.
template <typename T, typename TG, int VEC, int GVEC, bool kPacked, typename F>
cudaError_t with_launch(const GatedParams& p, int streams, F f) {
    const int ch = gated_channels(p, streams);
    if (ch == 32) return f(Launch<T, TG, 32, VEC, GVEC, kPacked>(p, streams));
    return ch == 16 ? f(Launch<T, TG, 16, VEC, GVEC, kPacked>(p, streams)) : f(Launch<T, TG, 64, VEC, GVEC, kPacked>(p, streams));
}
template <typename T, typename TG, int VEC, int GVEC>
cudaError_t launch_streams(const GatedParams& p, cudaStream_t st) {
    auto sums = [&](int parts, int packed, int longest) {
        return tc::launch_dependent(gated_dlam_kernel, (unsigned)((p.C + 31) / 32), 32 * kSummers, 0, st, p, static_cast<const float*>(p.ws), parts, packed, longest);
    };
    if (!p.cu || (gated_each(p, kMean) && p.N == 1))
        return with_launch<T, TG, VEC, GVEC, false>(p, p.cu ? 1 : p.B, [&](const auto& each) {
            const cudaError_t e = each(p.T, false, st);
            return e != cudaSuccess ? e : sums(each.parts, 0, p.T);
        });
    return with_launch<T, TG, VEC, GVEC, true>(p, 1, [&](const auto& stream) {
        if (!gated_each(p, kMean) || stream.error != cudaSuccess) {
            const cudaError_t e = stream(p.T, false, st);
            return e != cudaSuccess ? e : sums(stream.parts, 0, p.T);
        }
        return with_launch<T, TG, VEC, GVEC, false>(p, p.N, [&](const auto& each) {
            const int longest = longest_of(p, each.pace(), stream.pace());
            cudaError_t e = each(longest, false, st);
            if (e == cudaSuccess && longest < p.T) e = stream(longest, true, st);
            return e != cudaSuccess ? e : sums(each.parts, stream.parts, longest);
        });
    });
}

}  // namespace

size_t gated_scan_bwd_workspace(const GatedParams& p) {
    const int64_t states = p.states ? 0 : (int64_t)p.B * ((p.T + kGatedBlock - 1) / kGatedBlock) * p.C;
    return partial_bytes(p) + (size_t)states * 4;
}

cudaError_t gated_scan_bwd(kda_dtype dt, kda_dtype gdt, const GatedParams& given, cudaStream_t st) {
    GatedParams p = given;
    if (!p.states && p.T > 0) {
        p.states = reinterpret_cast<float*>(static_cast<char*>(p.ws) + partial_bytes(p));
        GatedParams f = p;
        f.y = nullptr;
        f.final_state = nullptr;
        const cudaError_t e = gated_scan_fwd(dt, f, st);
        if (e != cudaSuccess) return e;
    }
    const int es = dt == KDA_BF16 ? 2 : 4, gs = gdt == KDA_BF16 ? 2 : 4;
    bool pairs = p.C % 2 == 0 && (uintptr_t)p.states % 8 == 0;
    for (const void* q : {(const void*)p.dx, (const void*)p.dr, (const void*)p.di, (const void*)p.dz}) pairs = pairs && (uintptr_t)q % (2 * gs) == 0;
    const bool wide = pairs && gated_pieces(p, es, 16) && (int64_t)p.C * gs % 16 == 0 && kda_host::aligned16(p.dy);
    const bool narrow = pairs && gated_pieces(p, es, 2 * es) && (uintptr_t)p.dy % (2 * gs) == 0;
    if (dt == KDA_F32) {
        if (wide) return launch_streams<float, float, 4, 4>(p, st);
        return narrow ? launch_streams<float, float, 2, 2>(p, st) : launch_streams<float, float, 1, 1>(p, st);
    }
    if (gdt == KDA_F32) {
        if (wide) return launch_streams<__nv_bfloat16, float, 8, 4>(p, st);
        return narrow ? launch_streams<__nv_bfloat16, float, 2, 2>(p, st) : launch_streams<__nv_bfloat16, float, 1, 1>(p, st);
    }
    if (wide) return launch_streams<__nv_bfloat16, __nv_bfloat16, 8, 8>(p, st);
    return narrow ? launch_streams<__nv_bfloat16, __nv_bfloat16, 2, 2>(p, st) : launch_streams<__nv_bfloat16, __nv_bfloat16, 1, 1>(p, st);
}

}  // namespace kda
