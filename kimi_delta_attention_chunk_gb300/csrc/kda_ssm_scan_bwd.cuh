// Selective state space scan over prompts: backward.
//
// With the forward's d, a = exp(d A), h (per sequence, channel and state) and yb = dout silu(z):
//     dh_t = C_t yb_t + a_{t+1} dh_{t+1}   (behind the last token: the final state's gradient)
//     q1 = sum_s dh B,  q2 = sum_s dh a h_{t-1} A
//     du = d q1 + D yb,  dd = q2 + u q1,  ddelta = dd softplus'(delta + bias),  dbias = sum_t ddelta
//     dA += d dh a h_{t-1},  dB_t = sum_c d u dh,  dC_t = sum_c yb h,  dD = sum_t yb u
//     dz = dout (sum_s C h + D u) silu'(z),  dh0 = a_0 dh_0
// Both recurrences are cut at every 64th token of the stream (or 32nd or 16th where there are few):
//   1. one walk forwards over each chunk gives its end state from a zero start, the sum of its step
//      sizes, and what the chunk hands to the left (sum over its tokens of the decay since the chunk's
//      start times C yb), so both directions cost one exponential per token and state; the state at the
//      chunk's middle is kept too;
//   2. a prefix in each direction turns them into the state before and the gradient behind each chunk;
//   3. each chunk's halves of 32 tokens, the later one first, are walked forwards once more, keeping the state of every
//      fourth token in shared memory, then backwards four tokens at a time with their states and decays
//      recomputed into registers.
// A lane has eight states of a channel in step 3: fewer lanes share a channel's scalars and shuffles, and
// twelve warps an SM fit with their states in 168 registers.  (Four states a lane, chunks not halved, and
// the sums over channels by shuffles took 640 us where step 3 takes 374 for 2 x 2048 x 4096 x 16.)
// Sums over channels (dB, dC) go through shared memory, 16 additions a lane and token, then the block's
// warps, and partial sums of the channel blocks; sums over tokens through partial sums of the chunks.
// Every sum has an order fixed by the sizes.  Instruction issue bounds steps 1 and 3 (2.3 and 2.1 a cycle and SM):
// 2 x 2048 x 4096 x 16 bf16 with every gradient takes 526 us, 119 + 19 + 374 in the steps and 21 in the last sums.
#pragma once

#include <stddef.h>

#include <type_traits>

#include "kda_layer.h"
#include "kda_ssm.cuh"
#include "kda_tc.cuh"

namespace kda {

namespace {

constexpr int kChunk = 64;  // tokens of a chunk at most
constexpr int kHalf = 32;

// Device scratch: per chunk and channel and state the end states (then start states, then dA's
// partial sums), the gradients handed left (then those coming from the right) and the states at the
// middle; per chunk and channel the sums of d to the end and to the middle, and the partial sums of dD
// and dbias; per channel block, token and state the partial sums of dB and dC; per chunk what begins and
// runs through.
constexpr int kStarts = 1;     // a sequence begins in the chunk: its start state does not reach its end
constexpr int kThrough = 2;    // the sequence at its first token is the one behind its last
constexpr int kMidStarts = 4;  // a sequence begins in its first half
constexpr int kPlain = 8;      // one sequence runs through all of its tokens and on
struct Scratch {
    float *state, *grad, *mid, *sum_d, *sum_mid, *dD, *dbias, *dBC;
    int* flags;
};
size_t carve(Scratch& s, void* ws, int64_t chunks, int blocks, const SsmScanParams& p) {
    size_t n = 0;
    auto take = [&](int64_t count) {
        float* at = ws ? reinterpret_cast<float*>(static_cast<char*>(ws) + n) : nullptr;
        n += (size_t)((count * 4 + 255) / 256) * 256;
        return at;
    };
    s.state = take(chunks * p.C * p.S);
    s.grad = take(chunks * p.C * p.S);
    s.mid = take(chunks * p.C * p.S);
    s.sum_d = take(chunks * p.C);
    s.sum_mid = take(chunks * p.C);
    s.dD = take(chunks * p.C);
    s.dbias = take(chunks * p.C);
    s.dBC = take((int64_t)blocks * p.total * 2 * p.S);
    s.flags = reinterpret_cast<int*>(take(chunks));
    return n;
}

// ---- 1. what each chunk does on its own -------------------------------------------------------

constexpr int kSumThreads = 128;

// Tokens whose rows are in shared memory at a time; tokens of a batch whose scalars are worked out together.
template <typename T, typename TG, int S>
struct SumShape {
    static constexpr int SPT = S < 16 ? S : 16, LPC = S / SPT, CH = kSumThreads / LPC, CHW = 32 / LPC, H2 = SPT / 2;
    static constexpr int TILE = sizeof(T) == 2 || S > 16 ? 16 : 8;
    static constexpr int BATCH = LPC == 4 ? 8 : 4, OWN = BATCH / LPC;
};
template <typename T, typename TG, int S>
struct SumShared {
    using Sh = SumShape<T, TG, S>;
    alignas(16) T rows[2][kSumThreads / 32][3][Sh::TILE][Sh::CHW];  // u, delta, z
    alignas(16) TG grads[2][kSumThreads / 32][Sh::TILE][Sh::CHW];
    alignas(16) T raw[2][2][Sh::TILE][S];                           // B, C
    alignas(16) float vec[2][Sh::TILE][S];
    TokenTile<kChunk> tile;
};

template <typename T, typename TG, int S>
__global__ void __launch_bounds__(kSumThreads, 4) scan_bwd_sum_kernel(SsmScanParams p, SeqMap m, Scratch w, int chunk, bool wide_vecs,
                                                                      bool wide_rows) {
    using Sh = SumShape<T, TG, S>;
    constexpr int LPC = Sh::LPC, CH = Sh::CH, CHW = Sh::CHW, H2 = Sh::H2, TILE = Sh::TILE, BATCH = Sh::BATCH, OWN = Sh::OWN;
    constexpr int PIECE = 16 / (int)sizeof(T), GPIECE = 16 / (int)sizeof(TG);
    extern __shared__ __align__(16) char raw_smem[];
    SumShared<T, TG, S>& sh = *reinterpret_cast<SumShared<T, TG, S>*>(raw_smem);
    const ChannelBlocks cb(p.C, p.G, CH);
    const int tid = threadIdx.x, lane = tid % LPC, warp = tid / 32, wlane = tid % 32, wch = wlane / LPC;
    const int g = cb.group(blockIdx.x), in_group = cb.in_group(blockIdx.x, CH) + tid / LPC;
    const bool on = in_group < cb.group_size;
    const int c = g * cb.group_size + (on ? in_group : 0);
    const int64_t cs = (int64_t)c * S + lane * 4;  // states 4 (q LPC + lane) ... + 3
    const int t0 = blockIdx.y * chunk, t1 = min(m.total, t0 + chunk);
    const int warp_first = cb.in_group(blockIdx.x, CH) + warp * CHW;
    const int warp_has = max(0, min(CHW, cb.group_size - warp_first));
    const int warp_c = g * cb.group_size + min(warp_first, cb.group_size - 1);

    auto request = [&](int ta, int buf) {
        const int n = min(TILE, t1 - ta);
#pragma unroll
        for (int v = 0; v < 2; ++v) {
            const int64_t ld = v ? p.ldc : p.ldb;
            const T* from = static_cast<const T*>(v ? p.Cm : p.Bm) + ta * ld + g * S;
            if (wide_vecs) {
                constexpr int PR = S / PIECE;
                for (int e = tid; e < n * PR; e += kSumThreads)
                    Row<T, PIECE>::copy_async(&sh.raw[buf][v][e / PR][e % PR * PIECE], from + e / PR * ld + e % PR * PIECE);
            } else {
                for (int e = tid; e < n * S; e += kSumThreads) sh.raw[buf][v][e / S][e % S] = __ldg(from + e / S * ld + e % S);
            }
        }
#pragma unroll
        for (int v = 0; v < 3; ++v) {
            const int64_t ld = v == 0 ? p.ldu : v == 1 ? p.ldd : p.ldz;
            const void* base = v == 0 ? p.u : v == 1 ? p.delta : p.z;
            if (!base) continue;
            const T* from = static_cast<const T*>(base) + ta * ld + warp_c;
            if (wide_rows) {
                constexpr int PR = CHW / PIECE;
                for (int e = wlane; e < n * PR; e += 32) {
                    const int r = e / PR, ch = e % PR * PIECE;
                    if (ch < warp_has) Row<T, PIECE>::copy_async(&sh.rows[buf][warp][v][r][ch], from + r * ld + ch);
                }
            } else if (wch < warp_has) {
                for (int r = lane; r < n; r += LPC) Row<T, 1>::copy_async(&sh.rows[buf][warp][v][r][wch], from + r * ld + wch);
            }
        }
        const TG* from = static_cast<const TG*>(p.dy) + (int64_t)ta * p.C + warp_c;
        if (wide_rows) {
            constexpr int PR = CHW / GPIECE > 0 ? CHW / GPIECE : 1;
            for (int e = wlane; e < n * PR; e += 32) {
                const int r = e / PR, ch = e % PR * GPIECE;
                if (ch < warp_has) Row<TG, GPIECE>::copy_async(&sh.grads[buf][warp][r][ch], from + (int64_t)r * p.C + ch);
            }
        } else if (wch < warp_has) {
            for (int r = lane; r < n; r += LPC) Row<TG, 1>::copy_async(&sh.grads[buf][warp][r][wch], from + (int64_t)r * p.C + wch);
        }
        copies_commit();
    };
    if (t0 < t1) request(t0, 0);

    f2 A2[H2], h[H2], P[H2], G[H2];
#pragma unroll
    for (int i = 0; i < H2; i += 2) {
        const float4 v = __ldg(reinterpret_cast<const float4*>(p.A + cs + 2 * i * LPC));
        A2[i] = pack(kLog2e * v.x, kLog2e * v.y);
        A2[i + 1] = pack(kLog2e * v.z, kLog2e * v.w);
    }
#pragma unroll
    for (int i = 0; i < H2; ++i) {
        h[i] = G[i] = 0ull;
        P[i] = pack(1.f, 1.f);
    }
    auto load_into = [&](f2 (&v)[H2], const float* from) {
#pragma unroll
        for (int i = 0; i < H2; i += 2) {
            const float4 x = *reinterpret_cast<const float4*>(from + 2 * i * LPC);
            v[i] = pack(x.x, x.y);
            v[i + 1] = pack(x.z, x.w);
        }
    };
    auto store_from = [&](const f2 (&v)[H2], float* to) {
#pragma unroll
        for (int i = 0; i < H2; i += 2) {
            float4 x;
            unpack(v[i], x.x, x.y);
            unpack(v[i + 1], x.z, x.w);
            *reinterpret_cast<float4*>(to + 2 * i * LPC) = x;
        }
    };
    const float bias = p.bias ? __ldg(p.bias + c) : 0.f;
    sh.tile.template build<kSumThreads>(m, t0);
    const int first = m.first(), last = m.last();
    const bool plain = sh.tile.plain && t0 >= first && t1 - t0 == chunk;
    bool carries = sh.tile.carry >= 0, starts = false, mid_starts = false;
    float sum_d = 0.f;
    const int64_t slot = (int64_t)blockIdx.y * p.C;
    int buf = 1;
    for (int t = t0; t < t1; t += BATCH) {
        const int k0 = (t - t0) % TILE;
        if (k0 == 0) {
            buf ^= 1;
            copies_wait<0>();
            __syncthreads();
            if (t + TILE < t1) request(t + TILE, buf ^ 1);
            for (int e = tid; e < 2 * TILE * S; e += kSumThreads) (&sh.vec[0][0][0])[e] = to_f32<T>((&sh.raw[buf][0][0][0])[e]);
            __syncthreads();
        }
        if (t == t0 + kHalf) {  // the state at the middle
            mid_starts = starts;
            if (on) {
                store_from(h, w.mid + slot * S + cs);
                if (lane == 0) w.sum_mid[slot + c] = sum_d;
            }
        }
        float d[OWN], du[OWN], yb[OWN];
#pragma unroll
        for (int j = 0; j < OWN; j += 2) {
            const int a = k0 + lane + j * LPC, b = a + LPC;
            const auto& rows = sh.rows[buf][warp];
            f2 dd = pack(to_f32<T>(rows[1][a][wch]) + bias, to_f32<T>(rows[1][b][wch]) + bias);
            if (p.softplus) dd = softplus2(dd);
            unpack(dd, d[j], d[j + 1]);
            unpack(mul2(dd, pack(to_f32<T>(rows[0][a][wch]), to_f32<T>(rows[0][b][wch]))), du[j], du[j + 1]);
            f2 y2 = pack(to_f32<TG>(sh.grads[buf][warp][a][wch]), to_f32<TG>(sh.grads[buf][warp][b][wch]));
            if (p.z) {
                const f2 zv = pack(to_f32<T>(rows[2][a][wch]), to_f32<T>(rows[2][b][wch]));
                y2 = mul2(y2, mul2(zv, sigmoid2(zv)));
            }
            unpack(y2, yb[j], yb[j + 1]);
        }
        // the batch's tokens; kAll: they lie inside one sequence, kCarries: the one at the chunk's first token
        auto tokens = [&](auto all, auto carry) {
            constexpr bool kAll = decltype(all)::value, kCarries = decltype(carry)::value;
#pragma unroll
            for (int i = 0; i < BATCH; ++i) {
                const int k = t - t0 + i;
                if (!kAll) {
                    if (t + i < first || t + i >= t1 || t + i >= last) continue;
                    const int s = sh.tile.start[k];
                    if (s >= 0) {
                        starts = true;
                        if (p.initial) load_into(h, p.initial + (int64_t)s * p.C * S + cs);
                        else
#pragma unroll
                            for (int j = 0; j < H2; ++j) h[j] = 0ull;
                    }
                }
                float di = d[i / LPC], dui = du[i / LPC], ybi = yb[i / LPC];
                if (LPC > 1) {
                    di = __shfl_sync(0xffffffffu, di, i % LPC, LPC);
                    dui = __shfl_sync(0xffffffffu, dui, i % LPC, LPC);
                    ybi = __shfl_sync(0xffffffffu, ybi, i % LPC, LPC);
                }
                sum_d += di;
                const f2 dd = pack(di, di), du2 = pack(dui, dui), yb2 = pack(ybi, ybi);
                const ulonglong2* Bv = reinterpret_cast<const ulonglong2*>(&sh.vec[0][k0 + i][lane * 4]);
                const ulonglong2* Cv = reinterpret_cast<const ulonglong2*>(&sh.vec[1][k0 + i][lane * 4]);
#pragma unroll
                for (int j = 0; j < H2; ++j) {
                    const f2 b = (j & 1) ? Bv[j / 2 * LPC].y : Bv[j / 2 * LPC].x;
                    const f2 a = ex2_2(mul2(dd, A2[j]));
                    h[j] = fma2(a, h[j], mul2(du2, b));
                    if (kAll ? kCarries : carries) {
                        const f2 q = (j & 1) ? Cv[j / 2 * LPC].y : Cv[j / 2 * LPC].x;
                        P[j] = mul2(P[j], a);
                        G[j] = fma2(P[j], mul2(yb2, q), G[j]);
                    }
                }
                if (!kAll && carries && sh.tile.end[k] >= 0) {
                    carries = false;
                    if (p.dfinal) {
                        f2 f[H2];
                        load_into(f, p.dfinal + (int64_t)sh.tile.end[k] * p.C * S + cs);
#pragma unroll
                        for (int j = 0; j < H2; ++j) G[j] = fma2(P[j], f[j], G[j]);
                    }
                }
            }
        };
        const bool fast = plain || (t >= first && t + BATCH <= min(t1, last) && sh.tile.template clear<BATCH>(t - t0));
        if (!fast) tokens(std::false_type{}, std::false_type{});
        else if (carries) tokens(std::true_type{}, std::true_type{});
        else tokens(std::true_type{}, std::false_type{});
    }
    tc::grid_dep_launch();
    if (on) {
        store_from(h, w.state + slot * S + cs);
        store_from(G, w.grad + slot * S + cs);
        if (lane == 0) w.sum_d[slot + c] = sum_d;
    }
    if (blockIdx.x == 0 && tid == 0)
        w.flags[blockIdx.y] = (starts ? kStarts : 0) | (carries ? kThrough : 0) | (mid_starts ? kMidStarts : 0) | (plain ? kPlain : 0);
}

// ---- 2. the state before and the gradient behind each chunk -------------------------------------

// One thread carries one state along; blockIdx.y 0: forwards, 1: backwards.  It is bound by the latency of
// its loads, so sixteen chunks' are requested together.
__global__ void __launch_bounds__(128) scan_bwd_prefix_kernel(const float* A, Scratch w, int chunks, int C, int S) {
    const int64_t i = blockIdx.x * 128ll + threadIdx.x, n = (int64_t)C * S;
    const int c = (int)(min(i, n - 1) / S);
    const float a = kLog2e * __ldg(A + min(i, n - 1));
    tc::grid_dep_wait();
    if (i >= n) return;
    const bool back = blockIdx.y == 1;
    float* io = (back ? w.grad : w.state) + i;
    const int stop = back ? kThrough : kStarts;
    float h = 0.f;
    constexpr int kAhead = 16;
    for (int j0 = 0; j0 < chunks; j0 += kAhead) {
        float e[kAhead], d[kAhead];
        bool on[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int x = min(j0 + k, chunks - 1), j = back ? chunks - 1 - x : x;
            e[k] = io[j * n];
            d[k] = w.sum_d[(int64_t)j * C + c];
            on[k] = ((w.flags[j] & stop) != 0) == back;
        }
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            if (j0 + k >= chunks) break;
            const int j = back ? chunks - 1 - (j0 + k) : j0 + k;
            io[j * n] = h;
            h = on[k] ? fmaf(ex2(d[k] * a), h, e[k]) : e[k];
        }
    }
    tc::grid_dep_launch();
}

// ---- 3. the gradients --------------------------------------------------------------------------

constexpr int kThreads = 128, kWarps = kThreads / 32;
constexpr int kBatch = 4, kBatches = kHalf / kBatch;
constexpr float kLn2 = 0.6931471805599453f;

template <int S>
struct BwdShape {
    static constexpr int LP = S / 8;           // lanes of a channel, eight states each
    static constexpr int CH = kThreads / LP;   // channels of a block
    static constexpr int NCH = 32 / LP;        // channels of a warp
    // a warp's terms of dB and dC: a row per channel, 2 S floats and so much more that the eight lanes of a
    // 16-byte access fall into eight different bank groups
    static constexpr int ROW = 2 * S + (LP * 4) % 32;
    // each lane adds up pairs of the 2 S sums, over eight channels (S = 64: two pairs over four)
    static constexpr int PAIRS = S == 64 ? 2 : 1, OVER = S == 64 ? 4 : 8;
};
template <int S>
struct BwdShared {
    using Sh = BwdShape<S>;
    float4 kept[kBatches][2][kThreads];
    alignas(16) float vec[2][kHalf][S];   // B, C, read four at a time
    alignas(16) float terms[kWarps][Sh::NCH * Sh::ROW];
    alignas(16) float d[kHalf][Sh::CH];   // step sizes, then dd
    alignas(16) float u[kHalf][Sh::CH];   // inputs, then du
    alignas(16) float yb[kHalf][Sh::CH];  // output gradients behind the gate, then sum_s C h
    alignas(16) float red[2][kWarps][kBatch][2 * S];
    TokenTile<kHalf> tile;
};

// Two neighbouring elements as they lie in memory, in one access where they are one (kPairs).
template <typename T, bool kPairs>
struct Two {
    Row<T, 2> r;
    T v[2];
    // b: there is a second
    __device__ __forceinline__ void load(const T* p, bool b) {
        if constexpr (kPairs) {
            r.load(p);
        } else {
            v[0] = __ldg(p);
            v[1] = __ldg(b ? p + 1 : p);
        }
    }
    __device__ __forceinline__ f2 get(bool b) const {
        if constexpr (kPairs) {
            f2 x[1];
            r.to(x);
            return x[0];
        } else {
            return pack(to_f32<T>(v[0]), b ? to_f32<T>(v[1]) : 0.f);
        }
    }
};
template <bool kPairs, typename T>
__device__ __forceinline__ void store_two(T* p, f2 x, bool b) {
    if constexpr (kPairs) {
        Row<T, 2> r;
        const f2 v[1] = {x};
        r.from(v);
        r.store(p);
    } else {
        float lo, hi;
        unpack(x, lo, hi);
        p[0] = from_f32<T>(lo);
        if (b) p[1] = from_f32<T>(hi);
    }
}

template <typename T, typename TG, int S, bool kPairs>
__global__ void __launch_bounds__(kThreads, S == 8 ? 2 : 3) scan_bwd_kernel(SsmScanParams p, SeqMap m, Scratch w, int chunk) {
    using Sh = BwdShape<S>;
    constexpr int LP = Sh::LP, CH = Sh::CH;
    extern __shared__ __align__(16) char raw_smem[];
    BwdShared<S>& sh = *reinterpret_cast<BwdShared<S>*>(raw_smem);
    const ChannelBlocks cb(p.C, p.G, CH);
    const int tid = threadIdx.x, lane = tid % LP, ch = tid / LP, warp = tid / 32, wlane = tid % 32;
    const int g = cb.group(blockIdx.x), base = cb.in_group(blockIdx.x, CH);
    const bool on = base + ch < cb.group_size;
    const int c = g * cb.group_size + (on ? base + ch : 0);
    const int64_t cs = (int64_t)c * S + lane * 4;  // states 4 (q LP + lane) ... + 3, q = 0, 1
    const int64_t slot = (int64_t)blockIdx.y * p.C;
    const int t0 = blockIdx.y * chunk, t1 = min(m.total, t0 + chunk);
    tc::grid_dep_wait();
    const int flags = w.flags[blockIdx.y];

    // rows come and go by channel pairs: this thread has one pair, in every kRows-th token, kAtOnce of
    // them requested together
    constexpr int kAcross = CH / 2, kRows = kThreads / kAcross, kMine = kHalf / kRows, kAtOnce = kMine < 8 ? kMine : 8;
    const int ech = tid % kAcross * 2, erow = tid / kAcross;
    const bool e0 = base + ech < cb.group_size, e1 = base + ech + 1 < cb.group_size;
    const int ec = g * cb.group_size + (e0 ? base + ech : 0);
    const f2 ebias = p.bias && e0 ? pack(__ldg(p.bias + ec), e1 ? __ldg(p.bias + ec + 1) : 0.f) : 0ull;
    const f2 eD = p.D && e0 ? pack(__ldg(p.D + ec), e1 ? __ldg(p.D + ec + 1) : 0.f) : 0ull;
    f2 dD = 0ull, dbias = 0ull;

    auto load8 = [&](const float* from, f2 (&v)[4]) {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const float4 x = *reinterpret_cast<const float4*>(from + q * LP * 4);
            v[2 * q] = pack(x.x, x.y);
            v[2 * q + 1] = pack(x.z, x.w);
        }
    };
    auto store8 = [&](const f2 (&v)[4], float* to) {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            float4 x;
            unpack(v[2 * q], x.x, x.y);
            unpack(v[2 * q + 1], x.z, x.w);
            *reinterpret_cast<float4*>(to + q * LP * 4) = x;
        }
    };
    auto zero8 = [&](f2 (&v)[4]) {
#pragma unroll
        for (int q = 0; q < 4; ++q) v[q] = 0ull;
    };
    auto initial_of = [&](int n, f2 (&v)[4]) {
        if (p.initial) load8(p.initial + (int64_t)n * p.C * S + cs, v);
        else zero8(v);
    };
    f2 A2[4], dA[4], carry[4];  // carry: gradient of the state behind the token at hand
    load8(p.A + cs, A2);
#pragma unroll
    for (int q = 0; q < 4; ++q) A2[q] = mul2(A2[q], pack(kLog2e, kLog2e));
    zero8(dA);
    // (a lane without a channel carries zeros: its products join the sums over channels)
    if (on) load8(w.grad + slot * S + cs, carry);
    else zero8(carry);
    const float Dc = p.D && on ? __ldg(p.D + c) : 0.f;
    // a chunk inside one sequence needs no look at the boundaries
    const int first = flags & kPlain ? 0 : m.first(), last = flags & kPlain ? m.total : m.last();
    Two<T, kPairs> ru[kAtOnce], rd[kAtOnce], rz[kAtOnce];
    Two<TG, kPairs> rg[kAtOnce];
    // rows r0 + j kRows of the half at th (behind the tokens: the last one)
    auto rows_of = [&](int th, int r0) {
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) {
            const int64_t t = min(th + r0 + j * kRows, t1 - 1);
            ru[j].load(static_cast<const T*>(p.u) + t * p.ldu + ec, e1);
            rd[j].load(static_cast<const T*>(p.delta) + t * p.ldd + ec, e1);
            rg[j].load(static_cast<const TG*>(p.dy) + t * p.C + ec, e1);
            if (p.z) rz[j].load(static_cast<const T*>(p.z) + t * p.ldz + ec, e1);
        }
    };

    for (int half = chunk > kHalf ? 1 : 0; half >= 0; --half) {
        const int th = t0 + half * kHalf;
        if (th >= t1) continue;
        const int lo = max(th, first), hi = min(min(t1, th + kHalf), last);
        __syncthreads();  // past the half before
#pragma unroll 1
        for (int r0 = erow; r0 < kHalf; r0 += kAtOnce * kRows) {
            rows_of(th, r0);
#pragma unroll
            for (int j = 0; j < kAtOnce; ++j) {
                const int r = r0 + j * kRows, t = th + r;
                f2 u = ru[j].get(e1), d = add2(rd[j].get(e1), ebias), yb = rg[j].get(e1);
                if (p.softplus) d = softplus2(d);
                if (p.z) {
                    const f2 zv = rz[j].get(e1);
                    yb = mul2(yb, mul2(zv, sigmoid2(zv)));
                }
                if (!e0 || t < lo || t >= hi) {
                    d = u = yb = 0ull;
                } else if (!e1) {  // no second channel: zeros
                    float x, y;
                    unpack(d, x, y);
                    d = pack(x, 0.f);
                }
                dD = fma2(yb, u, dD);
                *reinterpret_cast<f2*>(&sh.d[r][ech]) = d;
                *reinterpret_cast<f2*>(&sh.u[r][ech]) = u;
                *reinterpret_cast<f2*>(&sh.yb[r][ech]) = yb;
            }
        }
        {
            const T* Bm = static_cast<const T*>(p.Bm) + g * S;
            const T* Cm = static_cast<const T*>(p.Cm) + g * S;
            for (int e = tid; e < (min(t1, th + kHalf) - th) * S; e += kThreads) {
                const int k = e / S, s = e % S;
                sh.vec[0][k][s] = ld(Bm, (int64_t)(th + k) * p.ldb + s);
                sh.vec[1][k][s] = ld(Cm, (int64_t)(th + k) * p.ldc + s);
            }
        }
        const bool plain = flags & kPlain;
        if (plain) __syncthreads();
        else sh.tile.template build<kThreads>(m, th);

        // the state before the half
        f2 h[4];
        zero8(h);
        if (on && (plain || sh.tile.carry >= 0)) {
            if (half == 0 || !(flags & kMidStarts)) load8(w.state + slot * S + cs, h);
            if (half == 1) {
                f2 mid[4];
                load8(w.mid + slot * S + cs, mid);
                const float sd = w.sum_mid[slot + c];
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    h[q] = flags & kMidStarts ? mid[q] : fma2(ex2_2(mul2(A2[q], pack(sd, sd))), h[q], mid[q]);
            }
        }

        {
            // token k forwards: h, and its decays in `a`
            auto forward = [&](int k, f2 (&a)[4]) {
                const float d = sh.d[k][ch], du = d * sh.u[k][ch];
                const f2 dd = pack(d, d), du2 = pack(du, du);
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const ulonglong2 B = *reinterpret_cast<const ulonglong2*>(&sh.vec[0][k][(q * LP + lane) * 4]);
                    a[2 * q] = ex2_2(mul2(dd, A2[2 * q]));
                    a[2 * q + 1] = ex2_2(mul2(dd, A2[2 * q + 1]));
                    h[2 * q] = fma2(a[2 * q], h[2 * q], mul2(du2, B.x));
                    h[2 * q + 1] = fma2(a[2 * q + 1], h[2 * q + 1], mul2(du2, B.y));
                }
            };
            // a batch inside one sequence needs no look at its tokens
            auto fast = [&](int b) {
                return plain || (th + b * kBatch >= lo && th + (b + 1) * kBatch <= hi && sh.tile.template clear<kBatch>(b * kBatch));
            };
            auto inside = [&](int k) { return th + k >= lo && th + k < hi; };
            // forwards: the state before every batch
            auto sweep = [&](int b, auto all) {
                constexpr bool kAll = decltype(all)::value;
#pragma unroll
                for (int i = 0; i < kBatch; ++i) {
                    const int k = b * kBatch + i;
                    if (!kAll && !inside(k)) continue;
                    if (!kAll && sh.tile.start[k] >= 0) initial_of(sh.tile.start[k], h);
                    f2 a[4];
                    forward(k, a);
                }
            };
#pragma unroll 1
            for (int b = 0; b < kBatches; ++b) {
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    float4 x;
                    unpack(h[2 * q], x.x, x.y);
                    unpack(h[2 * q + 1], x.z, x.w);
                    sh.kept[b][q][tid] = x;
                }
                if (b + 1 == kBatches) break;
                if (fast(b)) sweep(b, std::true_type{});
                else sweep(b, std::false_type{});
            }
            // backwards
            auto back = [&](int b, auto all) {
                constexpr bool kAll = decltype(all)::value;
                f2 hs[kBatch][4], as[kBatch][4], before[4];
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const float4 x = sh.kept[b][q][tid];
                    before[2 * q] = h[2 * q] = pack(x.x, x.y);
                    before[2 * q + 1] = h[2 * q + 1] = pack(x.z, x.w);
                }
#pragma unroll
                for (int i = 0; i < kBatch; ++i) {
                    const int k = b * kBatch + i;
                    zero8(as[i]);
                    if (kAll || inside(k)) {
                        if (!kAll && sh.tile.start[k] >= 0) initial_of(sh.tile.start[k], h);
                        forward(k, as[i]);
                    }
#pragma unroll
                    for (int q = 0; q < 4; ++q) hs[i][q] = h[q];
                }
#pragma unroll
                for (int i = kBatch - 1; i >= 0; --i) {
                    const int k = b * kBatch + i;
                    if (!kAll && !inside(k)) continue;
                    const int start = kAll ? -1 : sh.tile.start[k], end = kAll ? -1 : sh.tile.end[k];
                    if (end >= 0) {
                        if (p.dfinal) load8(p.dfinal + (int64_t)end * p.C * S + cs, carry);
                        else zero8(carry);
                    }
                    const float d = sh.d[k][ch], u = sh.u[k][ch], yb = sh.yb[k][ch];
                    const float du = d * u;  // (zeros, as yb, in a lane without a channel)
                    const f2 yb2 = pack(yb, yb), dd = pack(d, d), du2 = pack(du, du);
                    f2 prev[4];
#pragma unroll
                    for (int q = 0; q < 4; ++q) prev[q] = i > 0 ? hs[i > 0 ? i - 1 : 0][q] : before[q];
                    if (start >= 0) initial_of(start, prev);
                    f2 q1 = 0ull, q2 = 0ull, yv = 0ull;
                    float* terms = &sh.terms[warp][wlane / LP * Sh::ROW + lane * 4];
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        const ulonglong2 B = *reinterpret_cast<const ulonglong2*>(&sh.vec[0][k][(q * LP + lane) * 4]);
                        const ulonglong2 C = *reinterpret_cast<const ulonglong2*>(&sh.vec[1][k][(q * LP + lane) * 4]);
                        ulonglong2 tb, tc;
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int x = 2 * q + e;
                            const f2 bv = e ? B.y : B.x, cv = e ? C.y : C.x;
                            const f2 dh = fma2(yb2, cv, carry[x]);
                            carry[x] = mul2(as[i][x], dh);
                            const f2 ah = mul2(carry[x], prev[x]);
                            dA[x] = fma2(ah, dd, dA[x]);
                            q1 = fma2(dh, bv, q1);
                            q2 = fma2(ah, A2[x], q2);
                            yv = fma2(hs[i][x], cv, yv);
                            (e ? tb.y : tb.x) = mul2(dh, du2);
                            (e ? tc.y : tc.x) = mul2(hs[i][x], yb2);
                        }
                        *reinterpret_cast<ulonglong2*>(terms + q * LP * 4) = tb;
                        *reinterpret_cast<ulonglong2*>(terms + S + q * LP * 4) = tc;
                    }
                    if (start >= 0 && p.dinitial && on) store8(carry, p.dinitial + (int64_t)start * p.C * S + cs);
                    float s1 = sum2(q1), s2 = kLn2 * sum2(q2), sy = sum2(yv);
#pragma unroll
                    for (int x = LP / 2; x > 0; x >>= 1) {
                        s1 += __shfl_xor_sync(0xffffffffu, s1, x);
                        s2 += __shfl_xor_sync(0xffffffffu, s2, x);
                        sy += __shfl_xor_sync(0xffffffffu, sy, x);
                    }
                    __syncwarp();  // the terms are there, and the channel's lanes past their reads of this token
                    if (lane == 0) {
                        sh.u[k][ch] = fmaf(d, s1, Dc * yb);
                        sh.d[k][ch] = fmaf(u, s1, s2);
                        sh.yb[k][ch] = sy;
                    }
                    // dB and dC over the warp's channels
#pragma unroll
                    for (int x = 0; x < Sh::PAIRS; ++x) {
                        const int pair = S < 32 ? wlane % S : wlane + 32 * x, part = S < 32 ? wlane / S : 0;
                        const float* from = &sh.terms[warp][part * Sh::OVER * Sh::ROW + pair * 2];
                        f2 a = *reinterpret_cast<const f2*>(from);
#pragma unroll
                        for (int y = 1; y < Sh::OVER; ++y) a = add2(a, *reinterpret_cast<const f2*>(from + y * Sh::ROW));
                        if (S < 32) {
                            float a0, a1;
                            unpack(a, a0, a1);
#pragma unroll
                            for (int y = S; y < 32; y <<= 1) {
                                a0 += __shfl_xor_sync(0xffffffffu, a0, y);
                                a1 += __shfl_xor_sync(0xffffffffu, a1, y);
                            }
                            a = pack(a0, a1);
                        }
                        if (part == 0) *reinterpret_cast<f2*>(&sh.red[b & 1][warp][i][pair * 2]) = a;
                    }
                    __syncwarp();
                }
            };
#pragma unroll 1
            for (int b = kBatches - 1; b >= 0; --b) {
                if (th + b * kBatch >= hi || th + (b + 1) * kBatch <= lo) continue;
                if (fast(b)) back(b, std::true_type{});
                else back(b, std::false_type{});
                __syncthreads();  // (the other half of `red` takes the next batch meanwhile)
                for (int e = tid; e < kBatch * 2 * S; e += kThreads) {
                    const int i = e / (2 * S), x = e % (2 * S), t = th + b * kBatch + i;
                    if (!inside(b * kBatch + i)) continue;
                    float a = 0.f;
#pragma unroll
                    for (int y = 0; y < kWarps; ++y) a += sh.red[b & 1][y][i][x];
                    w.dBC[((int64_t)blockIdx.x * m.total + t) * 2 * S + x] = a;
                }
            }
        }

        // outputs of the half, as the inputs came
#pragma unroll 1
        for (int r0 = erow; r0 < kHalf; r0 += kAtOnce * kRows) {
            rows_of(th, r0);
            if (r0 == erow) __syncthreads();
#pragma unroll
            for (int j = 0; j < kAtOnce; ++j) {
                const int r = r0 + j * kRows;
                const int64_t t = th + r;
                if (!e0 || t >= t1) continue;
                if (t < lo || t >= hi) {  // of no sequence: nothing depends on it
                    store_two<kPairs>(static_cast<TG*>(p.du) + t * p.C + ec, 0ull, e1);
                    store_two<kPairs>(static_cast<TG*>(p.ddelta) + t * p.C + ec, 0ull, e1);
                    if (p.z) store_two<kPairs>(static_cast<TG*>(p.dz) + t * p.C + ec, 0ull, e1);
                    continue;
                }
                f2 dd = *reinterpret_cast<const f2*>(&sh.d[r][ech]);
                if (p.softplus) dd = mul2(dd, sigmoid2(add2(rd[j].get(e1), ebias)));
                dbias = add2(dbias, dd);
                store_two<kPairs>(static_cast<TG*>(p.du) + t * p.C + ec, *reinterpret_cast<const f2*>(&sh.u[r][ech]), e1);
                store_two<kPairs>(static_cast<TG*>(p.ddelta) + t * p.C + ec, dd, e1);
                if (p.z) {
                    const f2 zv = rz[j].get(e1), sg = sigmoid2(zv), one = pack(1.f, 1.f), minus = pack(-1.f, -1.f);
                    const f2 y = fma2(eD, ru[j].get(e1), *reinterpret_cast<const f2*>(&sh.yb[r][ech]));
                    store_two<kPairs>(static_cast<TG*>(p.dz) + t * p.C + ec,
                                      mul2(mul2(rg[j].get(e1), y), mul2(sg, fma2(zv, fma2(minus, sg, one), one))), e1);
                }
            }
        }
    }
    tc::grid_dep_launch();
    if (on) store8(dA, w.state + slot * S + cs);

    // dD and dbias over the chunk: the kRows threads of a channel pair
    __syncthreads();
    f2* part = reinterpret_cast<f2*>(&sh.kept[0][0][0]);
    part[tid] = dD;
    part[kThreads + tid] = dbias;
    __syncthreads();
    if (tid < kAcross && e0) {
        f2 a = part[tid], b = part[kThreads + tid];
#pragma unroll
        for (int r = 1; r < kRows; ++r) {
            a = add2(a, part[r * kAcross + tid]);
            b = add2(b, part[kThreads + r * kAcross + tid]);
        }
        store_two<false>(w.dD + slot + ec, a, e1);
        store_two<false>(w.dbias + slot + ec, b, e1);
    }
    // a sequence without tokens hands the gradient of its state back
    if (p.dinitial && on)
        for (int n = blockIdx.y; n < m.N; n += gridDim.y)
            if (m.end(n) <= m.begin(n)) {
                f2 v[4];
                if (p.dfinal) load8(p.dfinal + (int64_t)n * p.C * S + cs, v);
                else zero8(v);
                store8(v, p.dinitial + (int64_t)n * p.C * S + cs);
            }
}

// ---- 4. the partial sums ------------------------------------------------------------------------

// dA, dD and dbias: sums over the chunks.  A block has 32 elements (of the three outputs one after the
// other) in eight threads each; a thread adds up every eighth chunk, and the eight sums are added in order.
struct ChunkSums {
    const float* in[3];
    float* out[3];
    int64_t n[3];
};
__device__ __forceinline__ void chunk_sums(const ChunkSums& s, int chunks, int block) {
    __shared__ float part[8][32];
    const int x = threadIdx.x % 32, y = threadIdx.x / 32;
    int64_t i = block * 32ll + x;
    int v = 0;
    while (v < 2 && i >= s.n[v]) i -= s.n[v++];
    const bool on = i < s.n[v] && s.out[v];
    float a = 0.f;
    if (on) {
#pragma unroll 8
        for (int j = y; j < chunks; j += 8) a += s.in[v][j * s.n[v] + i];
    }
    part[y][x] = a;
    __syncthreads();
    if (y == 0 && on) {
#pragma unroll
        for (int k = 1; k < 8; ++k) a += part[k][x];
        s.out[v][i] = a;
    }
}

// dB and dC from the channel blocks of each group.
template <typename TG, int S>
__device__ __forceinline__ void vec_sums(const float* in, const SeqMap& m, int G, int per_group, TG* dB, TG* dC, int block) {
    const int64_t i = block * 256ll + threadIdx.x;
    if (i >= (int64_t)m.total * G * 2 * S) return;
    const int j = (int)(i % (2 * S));
    const int64_t tg = i / (2 * S);
    const int g = (int)(tg % G), t = (int)(tg / G);
    float a = 0.f;
    if (t >= m.first() && t < m.last()) {  // (rows of no sequence: zeros)
#pragma unroll 16
        for (int b = 0; b < per_group; ++b) a += in[((int64_t)(g * per_group + b) * m.total + t) * 2 * S + j];
    }
    TG* out = j < S ? dB : dC;
    out[tg * S + j % S] = from_f32<TG>(a);
}

// Both, by blocks of one launch: the first `chunk_blocks` for the sums over the chunks.
template <typename TG, int S>
__global__ void __launch_bounds__(256) scan_bwd_partial_kernel(ChunkSums s, int chunks, int chunk_blocks, const float* in, SeqMap m, int G,
                                                               int per_group, TG* dB, TG* dC) {
    tc::grid_dep_wait();
    if ((int)blockIdx.x < chunk_blocks) chunk_sums(s, chunks, blockIdx.x);
    else vec_sums<TG, S>(in, m, G, per_group, dB, dC, blockIdx.x - chunk_blocks);
}

int bwd_blocks(const SsmScanParams& p) {
    const int ch = kThreads * 8 / p.S;
    return p.G * ((p.C / p.G + ch - 1) / ch);
}
// Tokens of a chunk: 64, less where blocks are few and a chunk's length is what the call takes.  64 tokens of 512
// channels, S = 16, take 59 us in one chunk and 30 in four of 16; up to two blocks an SM the shorter chunks are
// faster (512 tokens 32 us by 16, 39 by 32), with four they are not (1024 tokens 47 us by 16, 43 by 32, 60 by
// 64).  32 against 64: 1024 tokens of 2048 channels (1024 blocks) 91 us and 105, 4096 of them 280 and 276.
int chunk_of(const SsmScanParams& p) {
    constexpr int kSms = 152;
    const int64_t blocks = bwd_blocks(p);
    if (blocks * ((p.total + 15) / 16) <= 2 * kSms) return 16;
    return blocks * ((p.total + 31) / 32) <= 15 * kSms ? 32 : kChunk;
}
int chunk_count(int total, int chunk) { return total > 0 ? (total + chunk - 1) / chunk : 1; }

template <typename T, typename TG, int S>
cudaError_t launch(const SsmScanParams& p, cudaStream_t st) {
    const SeqMap m{p.cu, p.N, p.T, p.total};
    const int chunk = chunk_of(p), chunks = chunk_count(p.total, chunk), blocks = bwd_blocks(p);
    Scratch w;
    carve(w, p.ws, chunks, blocks, p);
    constexpr int kSumChannels = SumShape<T, TG, S>::CH;
    const int sum_blocks = p.G * ((p.C / p.G + kSumChannels - 1) / kSumChannels);
    using kda_host::rows_aligned;
    const int piece = 16 / (int)sizeof(T), gpiece = 16 / (int)sizeof(TG);
    const bool wide_vecs = rows_aligned(p.Bm, p.ldb, piece) && rows_aligned(p.Cm, p.ldc, piece);
    const bool wide_rows = rows_aligned(p.u, p.ldu, piece) && rows_aligned(p.delta, p.ldd, piece) && rows_aligned(p.z, p.ldz, piece) &&
                           rows_aligned(p.dy, p.C, gpiece) && p.C / p.G % piece == 0;
    const auto two = [](const void* q, int64_t ld, size_t es) { return (uintptr_t)q % (2 * es) == 0 && ld % 2 == 0; };
    bool pairs = p.C / p.G % 2 == 0 && two(p.u, p.ldu, sizeof(T)) && two(p.delta, p.ldd, sizeof(T)) && two(p.z, p.ldz, sizeof(T));
    for (const void* q : {p.dy, (const void*)p.du, (const void*)p.ddelta, (const void*)p.dz}) pairs = pairs && two(q, 0, sizeof(TG));
    cudaError_t e = cudaFuncSetAttribute(scan_bwd_sum_kernel<T, TG, S>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)sizeof(SumShared<T, TG, S>));
    if (e != cudaSuccess) return e;
    scan_bwd_sum_kernel<T, TG, S><<<dim3(sum_blocks, chunks), kSumThreads, sizeof(SumShared<T, TG, S>), st>>>(p, m, w, chunk, wide_vecs, wide_rows);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const int64_t states = (int64_t)p.C * S;
    // Each of the others may start while the one before it ends, as in the forward scan (2 x 2048 x 4096 x 16 takes 8 us
    // less so; 64 tokens of 512 channels 26 us, 28 without).
    e = tc::launch_dependent(scan_bwd_prefix_kernel, dim3((unsigned)((states + 127) / 128), 2), 128, 0, st, p.A, w, chunks, p.C, S);
    if (e != cudaSuccess) return e;
    constexpr int smem = sizeof(BwdShared<S>);
    const auto kern = pairs ? scan_bwd_kernel<T, TG, S, true> : scan_bwd_kernel<T, TG, S, false>;
    if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) != cudaSuccess) return e;
    if ((e = tc::launch_dependent(kern, dim3(blocks, chunks), kThreads, smem, st, p, m, w, chunk)) != cudaSuccess) return e;
    const ChunkSums sums{{w.state, w.dD, w.dbias}, {p.dA, p.dD, p.dbias}, {(int64_t)p.C * S, p.C, p.C}};
    const int chunk_blocks = (int)(((int64_t)p.C * (S + 2) + 31) / 32);
    const int64_t vec_blocks = ((int64_t)p.total * p.G * 2 * S + 255) / 256;
    return tc::launch_dependent(scan_bwd_partial_kernel<TG, S>, (unsigned)(chunk_blocks + vec_blocks), 256, 0, st, sums, chunks,
                                chunk_blocks, w.dBC, m, p.G, blocks / p.G, static_cast<TG*>(p.dB), static_cast<TG*>(p.dC));
}

template <typename T, typename TG>
cudaError_t dispatch(const SsmScanParams& p, cudaStream_t st) {
    if (p.S == 8) return launch<T, TG, 8>(p, st);
    if (p.S == 16) return launch<T, TG, 16>(p, st);
    if (p.S == 32) return launch<T, TG, 32>(p, st);
    return launch<T, TG, 64>(p, st);
}

}  // namespace

}  // namespace kda
