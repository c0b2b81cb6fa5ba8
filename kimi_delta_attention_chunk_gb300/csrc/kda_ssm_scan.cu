// Selective state space scan over prompts: forward.
//
// Per sequence, channel c (group g) and state s, over the tokens:
//     d = softplus(delta + bias),  h_s <- exp(d A_s) h_s + d u B_s,  y = (sum_s C_s h_s + D u) silu(z)
// A channel's row is four elements (u, delta, z, y), 8 bytes in bf16, against S exponentials and 4 S
// multiply-adds, so at S = 16 instruction issue bounds it before HBM does.  A thread owns a channel and 16
// of its states (S = 32, 64: two or four lanes a channel) with the state and A in registers, in pairs of
// packed fp32.  What a token costs per channel and not per state (softplus, the gate, D u) is done for
// several tokens at once, packed in pairs, each lane of a channel for tokens of its own.  B and C of a tile
// of tokens are turned to fp32 once per block and read from shared memory by everyone.  u, delta and z come
// to shared memory a tile ahead, and y leaves through it, each warp for its own channels: a load or store of
// one element from global memory costs ten instructions of address arithmetic, a tenth of a token.
//
// The recurrence leaves C threads' worth of parallelism (times the sequences); where that does not fill
// the machine the stream is cut into runs: every run's end state from a zero start and the sum of its step
// sizes (its decay is exp(A sum d)), a short prefix over the runs, and the runs again from their true
// starts.  Cuts fall at fixed places of the flat token stream; sequences begin and end inside runs.
//
// 16384 x 4096 x 16 bf16 with gate and states: 532 us in 19 runs of 864 tokens, the two walks at 2.4
// instructions a cycle and SM, 74 and 112 per token and 32 channels; 2450 x 1530 x 64 fp32, ragged: 137 us.
#include <type_traits>

#include "kda_layer.h"
#include "kda_ssm.cuh"
#include "kda_tc.cuh"

namespace kda {

namespace {

constexpr int kThreads = 128;
constexpr int kSms = 152;
constexpr int kRunStep = 16;  // runs are whole tiles

// Tokens whose rows are in shared memory at a time: 16 bf16 rows of a warp's 32 channels (32 rows leave fewer
// blocks an SM: 16384 x 4096 x 16 in 600 us against 547).
template <typename T, int S>
constexpr int kTileOf = sizeof(T) == 2 || S > 16 ? 16 : 8;

template <int S>
struct Shape {
    static constexpr int SPT = S < 16 ? S : 16;   // states of a thread
    static constexpr int LPC = S / SPT;           // lanes of a channel
    static constexpr int CH = kThreads / LPC;     // channels of a block
    static constexpr int BATCH = LPC == 4 ? 8 : 4;
    static constexpr int OWN = BATCH / LPC;       // tokens of a batch whose scalars a lane works out
};

// The runs' scratch: end states (then start states) [runs][C][S], sums of d [runs][C], and whether a
// sequence begins inside the run (the run's start then does not reach its end) [runs].
struct Runs {
    float* state;
    float* sum_d;
    int* cut;
};
size_t runs_bytes(int64_t runs, int C, int S) {
    return (size_t)((runs * C * S + runs * C) * 4 + ((runs * 4 + 15) / 16) * 16);
}
Runs runs_at(void* ws, int64_t runs, int C, int S) {
    float* f = static_cast<float*>(ws);
    return Runs{f, f + runs * C * S, reinterpret_cast<int*>(f + runs * C * S + runs * C)};
}

// kOutputs: from the true start states, with y and the final states; else the runs' end states.
// wide_vecs: B's and C's rows are 16-byte pieces; wide_rows: u's, delta's, z's and y's are.
template <typename T, int S, bool kOutputs, bool wide_rows>
__global__ void __launch_bounds__(kThreads, 4) scan_kernel(SsmScanParams p, SeqMap m, int run, Runs runs, bool split,
                                                           bool wide_vecs) {
    using Sh = Shape<S>;
    constexpr int SPT = Sh::SPT, LPC = Sh::LPC, CH = Sh::CH, H2 = SPT / 2, BATCH = Sh::BATCH, OWN = Sh::OWN;
    constexpr int VECS = kOutputs ? 2 : 1;  // B, and C
    constexpr bool kTurn = sizeof(T) == 2;  // fp32 vectors are read as they come
    constexpr int kTile = kTileOf<T, S>, PIECE = 16 / (int)sizeof(T);
    constexpr int CHW = 32 / LPC, ROWS = kOutputs ? 3 : 2;  // channels of a warp; u, delta, and z
    __shared__ __align__(16) float vec[kTurn ? VECS : 1][kTurn ? kTile : 1][S];
    __shared__ __align__(16) T raw[2][VECS][kTile][S];
    __shared__ __align__(16) T rows[2][kThreads / 32][ROWS][kTile][CHW];
    __shared__ TokenTile<kTile> tile;

    const ChannelBlocks cb(p.C, p.G, CH);
    const int tid = threadIdx.x, lane = tid % LPC, warp = tid / 32, wlane = tid % 32, wch = wlane / LPC;
    const int g = cb.group(blockIdx.x), in_group = cb.in_group(blockIdx.x, CH) + tid / LPC;
    const bool on = in_group < cb.group_size;
    const unsigned c = g * cb.group_size + (on ? in_group : 0);
    // lane l has states 4 (q LPC + l) ... + 3, q < SPT / 4: the lanes of a channel read 16-byte pieces side by side
    const int64_t cs = (int64_t)c * S + lane * 4;
    const int first = m.first(), last = m.last();
    const int r0 = blockIdx.y * run, r1 = (int)min((int64_t)m.total, (int64_t)r0 + run);

    // the first channel of the warp in its group, and how many it has
    const int warp_first = cb.in_group(blockIdx.x, CH) + warp * CHW;
    const int warp_has = max(0, min(CHW, cb.group_size - warp_first));
    const int warp_c = g * cb.group_size + min(warp_first, cb.group_size - 1);

    // the rows of the tile at t0, on their way: B and C by the block, u, delta and z by each warp
    auto request = [&](int t0, int buf) {
        const int n = min(kTile, r1 - t0);
#pragma unroll
        for (int v = 0; v < VECS; ++v) {
            const int64_t ld = v ? p.ldc : p.ldb;
            const T* from = static_cast<const T*>(v ? p.Cm : p.Bm) + t0 * ld + g * S;
            if (wide_vecs) {
                constexpr int PR = S / PIECE;
                for (int e = tid; e < n * PR; e += kThreads)
                    Row<T, PIECE>::copy_async(&raw[buf][v][e / PR][e % PR * PIECE], from + e / PR * ld + e % PR * PIECE);
            } else {
                for (int e = tid; e < n * S; e += kThreads) raw[buf][v][e / S][e % S] = __ldg(from + e / S * ld + e % S);
            }
        }
#pragma unroll
        for (int v = 0; v < ROWS; ++v) {
            const int64_t ld = v == 0 ? p.ldu : v == 1 ? p.ldd : p.ldz;
            const void* base = v == 0 ? p.u : v == 1 ? p.delta : p.z;
            if (v == 2 && !base) continue;
            const T* from = static_cast<const T*>(base) + t0 * ld + warp_c;
            if constexpr (wide_rows) {
                constexpr int PR = CHW / PIECE;
#pragma unroll
                for (int k = 0; k < kTile * PR; k += 32) {
                    const int e = k + wlane, r = e / PR, ch = e % PR * PIECE;
                    if (r < n && ch < warp_has) Row<T, PIECE>::copy_async(&rows[buf][warp][v][r][ch], from + r * ld + ch);
                }
            } else if (wch < warp_has) {
                from += lane * ld + wch;
                if constexpr (sizeof(T) == 4) {
#pragma unroll 1
                    for (int r = lane; r < n; r += LPC, from += LPC * ld) Row<T, 1>::copy_async(&rows[buf][warp][v][r][wch], from);
                } else {  // two bytes have no asynchronous copy: all loads first
                    T x[kTile / LPC];
#pragma unroll
                    for (int j = 0; j < kTile / LPC; ++j, from += LPC * ld)
                        if (lane + j * LPC < n) x[j] = __ldg(from);
#pragma unroll
                    for (int j = 0; j < kTile / LPC; ++j)
                        if (lane + j * LPC < n) rows[buf][warp][v][lane + j * LPC][wch] = x[j];
                }
            }
        }
        copies_commit();
    };
    if (r0 < r1) request(r0, 0);

    f2 A2[H2], h[H2];
#pragma unroll
    for (int i = 0; i < H2; i += 2) {
        const float4 v = __ldg(reinterpret_cast<const float4*>(p.A + cs + 2 * i * LPC));
        A2[i] = pack(kLog2e * v.x, kLog2e * v.y);
        A2[i + 1] = pack(kLog2e * v.z, kLog2e * v.w);
    }
    const float bias = p.bias ? __ldg(p.bias + c) : 0.f;
    const float Dc = kOutputs && p.D ? __ldg(p.D + c) : 0.f;

    auto load_state = [&](const float* from) {
#pragma unroll
        for (int i = 0; i < H2; i += 2) {
            const float4 v = *reinterpret_cast<const float4*>(from + 2 * i * LPC);
            h[i] = pack(v.x, v.y);
            h[i + 1] = pack(v.z, v.w);
        }
    };
    auto store_state = [&](float* to) {
#pragma unroll
        for (int i = 0; i < H2; i += 2) {
            float4 v;
            unpack(h[i], v.x, v.y);
            unpack(h[i + 1], v.z, v.w);
            *reinterpret_cast<float4*>(to + 2 * i * LPC) = v;
        }
    };
    auto clear_state = [&]() {
#pragma unroll
        for (int i = 0; i < H2; ++i) h[i] = 0ull;
    };
    auto begin_at = [&](int n) {
        if (p.initial) load_state(p.initial + (int64_t)n * p.C * S + cs);
        else clear_state();
    };

    if (kOutputs) tc::grid_dep_wait();  // the runs' starts
    // a sequence without tokens hands its state on
    if (kOutputs && p.final_state && on)
        for (int n = blockIdx.y; n < m.N; n += gridDim.y)
            if (m.end(n) <= m.begin(n)) {
                begin_at(n);
                store_state(p.final_state + (int64_t)n * p.C * S + cs);
            }
    clear_state();

    float sum_d = 0.f;
    bool cut = false, plain = false;
    int until = r0;  // no boundary before this token
    int buf = 1;
    for (int t = r0; t < r1; t += BATCH) {
        const int k0 = (t - r0) % kTile;
        if (k0 == 0) {
            buf ^= 1;
            copies_wait<0>();
            __syncthreads();  // the tile's rows are there, and everyone is past the one before (y's included)
            if (t + kTile < r1) request(t + kTile, buf ^ 1);
            if constexpr (kTurn) {
#pragma unroll
                for (int v = 0; v < VECS; ++v)
#pragma unroll
                    for (int e = tid; e < kTile * S; e += kThreads) vec[v][e / S][e % S] = to_f32<T>(raw[buf][v][e / S][e % S]);
            }
            plain = t > r0 && t + kTile < until;
            if (plain) {
                if constexpr (kTurn) __syncthreads();
            } else {
                tile.template build<kThreads>(m, t);
                until = tile.until;
                plain = tile.plain;
                if (t == r0 && tile.carry >= 0 && kOutputs && split) load_state(runs.state + (int64_t)blockIdx.y * p.C * S + cs);
            }
        }
        T(&mine)[ROWS][kTile][CHW] = rows[buf][warp];
        // what depends on the channel alone, in pairs of tokens
        float d[OWN], du[OWN], u[OWN], gate[OWN], y[OWN];
#pragma unroll
        for (int j = 0; j < OWN; j += 2) {
            const int at = k0 + lane + j * LPC;  // tokens behind the stream: whatever is there
            f2 dd = pack(to_f32<T>(mine[1][at][wch]) + bias, to_f32<T>(mine[1][at + LPC][wch]) + bias);
            if (p.softplus) dd = softplus2(dd);
            unpack(dd, d[j], d[j + 1]);
            u[j] = to_f32<T>(mine[0][at][wch]);
            u[j + 1] = to_f32<T>(mine[0][at + LPC][wch]);
            unpack(mul2(dd, pack(u[j], u[j + 1])), du[j], du[j + 1]);
            if (kOutputs && p.z) {
                const f2 zv = pack(to_f32<T>(mine[ROWS - 1][at][wch]), to_f32<T>(mine[ROWS - 1][at + LPC][wch]));
                unpack(mul2(zv, sigmoid2(zv)), gate[j], gate[j + 1]);
            }
            y[j] = y[j + 1] = 0.f;
        }
        // the batch's tokens; kAll: all of them belong to one sequence
        auto tokens = [&](auto all) {
            constexpr bool kAll = decltype(all)::value;
#pragma unroll
            for (int i = 0; i < BATCH; ++i) {
                if (!kAll) {
                    if (t + i < first || t + i >= r1 || t + i >= last) continue;
                    const int s = plain ? -1 : tile.start[k0 + i];
                    if (s >= 0) {
                        begin_at(s);
                        cut = true;
                    }
                }
                float di = d[i / LPC], dui = du[i / LPC];
                if (LPC > 1) {
                    di = __shfl_sync(0xffffffffu, di, i % LPC, LPC);
                    dui = __shfl_sync(0xffffffffu, dui, i % LPC, LPC);
                }
                if (!kOutputs) sum_d += di;
                const f2 dd = pack(di, di), du2 = pack(dui, dui);
                f2 y2 = 0ull;
                const ulonglong2 *Bv, *Cv;
                if constexpr (kTurn) {
                    Bv = reinterpret_cast<const ulonglong2*>(&vec[0][k0 + i][lane * 4]);
                    Cv = reinterpret_cast<const ulonglong2*>(&vec[VECS - 1][k0 + i][lane * 4]);
                } else {
                    Bv = reinterpret_cast<const ulonglong2*>(&raw[buf][0][k0 + i][lane * 4]);
                    Cv = reinterpret_cast<const ulonglong2*>(&raw[buf][VECS - 1][k0 + i][lane * 4]);
                }
#pragma unroll
                for (int j = 0; j < H2 / 2; ++j) {
                    const ulonglong2 b = Bv[j * LPC];
                    h[2 * j] = fma2(ex2_2(mul2(dd, A2[2 * j])), h[2 * j], mul2(du2, b.x));
                    h[2 * j + 1] = fma2(ex2_2(mul2(dd, A2[2 * j + 1])), h[2 * j + 1], mul2(du2, b.y));
                    if (kOutputs) {
                        const ulonglong2 q = Cv[j * LPC];
                        y2 = fma2(h[2 * j], q.x, y2);
                        y2 = fma2(h[2 * j + 1], q.y, y2);
                    }
                }
                if (kOutputs) {
                    float o = sum2(y2);
#pragma unroll
                    for (int x = LPC / 2; x > 0; x >>= 1) o += __shfl_xor_sync(0xffffffffu, o, x);
                    if (LPC == 1 || lane == i % LPC) y[i / LPC] = o;
                    if (!kAll && p.final_state) {
                        const int e = plain ? -1 : tile.end[k0 + i];
                        if (e >= 0 && on) store_state(p.final_state + (int64_t)e * p.C * S + cs);
                    }
                }
            }
        };
        const bool fast = t + BATCH <= r1 && (plain || (t >= first && t + BATCH <= last && tile.template clear<BATCH>(k0)));
        if (fast) tokens(std::true_type{});
        else tokens(std::false_type{});
        if (kOutputs) {
            // y takes u's place, and leaves with the tile's last batch
#pragma unroll
            for (int j = 0; j < OWN; ++j) {
                float o = fmaf(Dc, u[j], y[j]);
                if (p.z) o *= gate[j];
                mine[0][k0 + lane + j * LPC][wch] = from_f32<T>(o);
            }
            if (k0 + BATCH == kTile || t + BATCH >= r1) {
                __syncwarp();
                const int t0 = t - k0, n = min(kTile, r1 - t0);
                T* to = static_cast<T*>(p.y) + (int64_t)t0 * p.C + warp_c;
                if constexpr (wide_rows) {
                    constexpr int PR = CHW / PIECE;
#pragma unroll
                    for (int k = 0; k < kTile * PR; k += 32) {
                        const int e = k + wlane, r = e / PR, ch = e % PR * PIECE;
                        if (r < n && ch < warp_has && t0 + r >= first && t0 + r < last) {
                            Row<T, PIECE> out;
                            out.from_shared(&mine[0][r][ch]);
                            out.store(to + (int64_t)r * p.C + ch);
                        }
                    }
                } else if (wch < warp_has) {
                    for (int r = lane; r < n; r += LPC)
                        if (t0 + r >= first && t0 + r < last) to[(int64_t)r * p.C + wch] = mine[0][r][wch];
                }
            }
        }
    }
    if (!kOutputs) tc::grid_dep_launch();
    if (!kOutputs && on) {
        store_state(runs.state + (int64_t)blockIdx.y * p.C * S + cs);
        if (lane == 0) runs.sum_d[(int64_t)blockIdx.y * p.C + c] = sum_d;
        if (blockIdx.x == 0 && tid == 0) runs.cut[blockIdx.y] = cut;
    }
}

// Start states of the runs from their end states, in place: one thread carries one state along, with
// eight runs requested together.
__global__ void __launch_bounds__(128) scan_prefix_kernel(const float* A, Runs r, int runs, int C, int S) {
    const int64_t i = blockIdx.x * 128ll + threadIdx.x, n = (int64_t)C * S;
    const int c = (int)(min(i, n - 1) / S);
    const float a = kLog2e * __ldg(A + min(i, n - 1));
    tc::grid_dep_wait();
    if (i >= n) return;
    float h = 0.f;
    constexpr int kAhead = 8;
    for (int j0 = 0; j0 < runs; j0 += kAhead) {
        float e[kAhead], d[kAhead];
        int cut[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int j = min(j0 + k, runs - 2);  // nobody starts from the last run's end
            e[k] = r.state[j * n + i];
            d[k] = r.sum_d[(int64_t)j * C + c];
            cut[k] = r.cut[j];
        }
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            if (j0 + k >= runs) break;
            r.state[(j0 + k) * n + i] = h;
            h = cut[k] ? e[k] : fmaf(ex2(d[k] * a), h, e[k]);
        }
    }
    tc::grid_dep_launch();
}

// Tokens of a run, and whether runs depend on one another.
struct Plan {
    int run, runs, blocks;
    bool split;
};
Plan plan(const SsmScanParams& p) {
    const int ch = p.S <= 16 ? kThreads : kThreads * 16 / p.S;
    Plan q{};
    q.blocks = p.G * ((p.C / p.G + ch - 1) / ch);
    if (!p.cu && p.T > 0 && (int64_t)p.N * q.blocks >= 2 * kSms && p.N <= 65535) {
        q.run = p.T;  // the sequences alone fill the machine
        q.runs = p.N;
        return q;
    }
    // as many runs as one filling of the machine holds: four blocks an SM
    const int want = 4 * kSms / q.blocks > 0 ? 4 * kSms / q.blocks : 1;
    int run = (p.total + want - 1) / want;
    run = (run + kRunStep - 1) / kRunStep * kRunStep;
    // The prefix takes longer the more runs there are: 4096 tokens of 128 channels, S = 16, 29 us with 96 runs, 32
    // with 64 and 37 with 256.  Where a run has more blocks the cap costs something: 16384 of 512 channels take 101, 107 and 90.
    constexpr int kMostRuns = 96;
    const int least = (p.total + kMostRuns - 1) / kMostRuns;
    if (run < least) run = (least + kRunStep - 1) / kRunStep * kRunStep;
    // A token takes 0.2 us where a block has its SM to itself, and two more launches cost 6: 64 tokens take 15 us uncut
    // and 13 to 20 cut, 96 of 512 channels 21 and 13.  With more blocks the runs get in one another's way: 96
    // tokens of 4096 channels, S = 64, 22 us and 26.
    if (p.total <= 64 || p.total <= 40 + q.blocks / 2) run = (p.total + kRunStep - 1) / kRunStep * kRunStep;
    q.run = run;
    q.runs = p.total > 0 ? p.total / run + (p.total % run != 0) : 1;  // (total + run may pass 2^31)
    q.split = q.runs > 1;
    return q;
}

template <typename T, int S, bool wide_rows>
cudaError_t launch_rows(const SsmScanParams& p, cudaStream_t st) {
    const Plan q = plan(p);
    const SeqMap m{p.cu, p.N, p.T, p.total};
    const dim3 grid(q.blocks, q.runs);
    const int piece = 16 / (int)sizeof(T);
    const bool wide_vecs = kda_host::rows_aligned(p.Bm, p.ldb, piece) && kda_host::rows_aligned(p.Cm, p.ldc, piece);
    Runs r{};
    if (q.split) {
        r = runs_at(p.ws, q.runs, p.C, S);
        scan_kernel<T, S, false, wide_rows><<<dim3(q.blocks, q.runs - 1), kThreads, 0, st>>>(p, m, q.run, r, true, wide_vecs);
        cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
        const int64_t states = (int64_t)p.C * S;
        // Each of the next two may start while the one before it ends (16384 x 4096 x 16 in 532 us, 536 without).  A block asks
        // for that with its last stores only: blocks that start earlier are spread unevenly over the SMs (16384 x 512 x 16
        // in 112 us with the prefix asking at its start, 98 at its end, 101 without).
        if ((e = tc::launch_dependent(scan_prefix_kernel, (unsigned)((states + 127) / 128), 128, 0, st, p.A, r, q.runs, p.C, S)) != cudaSuccess)
            return e;
        return tc::launch_dependent(scan_kernel<T, S, true, wide_rows>, grid, kThreads, 0, st, p, m, q.run, r, true, wide_vecs);
    }
    scan_kernel<T, S, true, wide_rows><<<grid, kThreads, 0, st>>>(p, m, q.run, r, false, wide_vecs);
    return cudaGetLastError();
}

template <typename T, int S>
cudaError_t launch(const SsmScanParams& p, cudaStream_t st) {
    const int piece = 16 / (int)sizeof(T);
    const bool wide_rows = kda_host::rows_aligned(p.u, p.ldu, piece) && kda_host::rows_aligned(p.delta, p.ldd, piece) &&
                           kda_host::rows_aligned(p.z, p.ldz, piece) && kda_host::rows_aligned(p.y, p.C, piece) &&
                           p.C / p.G % piece == 0;
    return wide_rows ? launch_rows<T, S, true>(p, st) : launch_rows<T, S, false>(p, st);
}

template <typename T>
cudaError_t dispatch(const SsmScanParams& p, cudaStream_t st) {
    if (p.S == 8) return launch<T, 8>(p, st);
    if (p.S == 16) return launch<T, 16>(p, st);
    if (p.S == 32) return launch<T, 32>(p, st);
    return launch<T, 64>(p, st);
}

}  // namespace

size_t ssm_scan_workspace(const SsmScanParams& p) {
    const Plan q = plan(p);
    return q.split ? runs_bytes(q.runs, p.C, p.S) : 0;
}

cudaError_t ssm_scan_fwd(kda_dtype dt, const SsmScanParams& p, cudaStream_t st) {
    return dt == KDA_BF16 ? dispatch<__nv_bfloat16>(p, st) : dispatch<float>(p, st);
}

}  // namespace kda
