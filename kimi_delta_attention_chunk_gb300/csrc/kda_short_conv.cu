// The short causal convolution on its own: forward with the history carried in and out, backward,
// and the single-token form ("kimi-k3-mlx" review, section "Attention is 93 layers ...": a short
// convolution of kernel size 4 on q, k and v, ahead of the recurrence).
//
// Depthwise over C channels, W taps, sequence by sequence; line = [history | inputs]:
//     p_t = bias + sum_j w[c][j] line_{t-(W-1)+j},   y = p or p sigmoid(p)
// and backwards, with dp = dy act'(p):
//     dline_i = sum_j w[c][j] dp_{i+(W-1)-j} (+ the final history's gradient),
//     dw[c][j] = sum_t dp_t line_{t-(W-1)+j},   dbias = sum_t dp_t.
// Each direction reads and writes its rows once, so HBM bounds it.  A thread owns 16 bytes of channels
// (8 backwards, where it holds more per channel; one channel where the rows are not such pieces) and
// walks a run of tokens with the last W - 1 inputs (and, backwards, the W - 1 unfinished input
// gradients) in registers; runs meet at W - 1 rows that both read.  Rows arrive by asynchronous copies
// into shared memory, batches ahead of their use; a thread reads back only what it copied itself, so
// nothing in the walk waits for another thread.
//
// 70k x 12288 bf16 forwards with histories: 554 us, 6.2 TB/s, 91% of a copy's rate.  4096 x 12288 backwards: 65.5 us, 4.6
// TB/s, bound by issue (2.05 instructions a cycle and SM) and by one filling's start and end; 32,768 tokens 5.6 TB/s.
// One token of 256 sequences: 12.3 us, 4.1 TB/s: 768 blocks in 456 places (142 registers a thread leave three blocks an SM),
// each a chain of slot, history and store.
//
// Rows that are no whole pieces go one channel a thread: 16384 x 12290 forwards in 419 us where 12288 take 139, 4096 x 12290
// backwards in 186 where 12288 take 63, 256 rows of one token in 16.6 where they take 9.8 (graph replays).  Two bytes have no
// asynchronous copy, so nothing is on its way while a batch is worked on, and one channel does the work of a pair.
#include "kda_layer.h"
#include "kda_segments.cuh"
#include "kda_slots.cuh"
#include "kda_tc.cuh"

namespace kda {

namespace {

constexpr int kThreads = 128;
constexpr int kSms = 152;
// Blocks of an SM that the kernels are built for.  Five forwards (70k x 12288 in 565 us, 600 with four, although the
// instance of eight bf16 channels and four taps then spills 62 bytes, the only one that does);
// three backwards, with 168 registers a thread (4096 x 12288 in 68 us, 72 with four, 82 with five, which spill).
constexpr int kFwdResident = 5, kBwdResident = 3;
constexpr int kTile = 64;     // tokens of one look at the sequence boundaries
// Asynchronous groups of a thread: one in use, one on its way.  (Three groups of eight rows measured 17%
// slower backwards, two of four and two of sixteen as well.)
constexpr int kStages = 2;

// Rows of one group: 33 KB of shared memory a block.
constexpr int batch_of(int bytes) { return bytes <= 16 ? 8 : 4; }

template <typename T, int VEC>
struct FwdShared {
    static constexpr int kBatch = batch_of(Row<T, VEC>::kBytes);
    typename Row<T, VEC>::Raw ring[kStages][kBatch][kThreads];
    TokenTile<kTile> tile;
};
template <typename T, typename TG, int VEC>
struct BwdShared {
    static constexpr int kBatch = batch_of(Row<T, VEC>::kBytes + Row<TG, VEC>::kBytes);
    typename Row<T, VEC>::Raw ring[kStages][kBatch][kThreads];
    typename Row<TG, VEC>::Raw gring[kStages][kBatch][kThreads];
    TokenTile<kTile> tile;
};

template <typename T, int VEC, int W>
__device__ __forceinline__ void load_history(const T* hist, int64_t n, int C, int c0, f2 (&win)[W - 1][Row<T, VEC>::N2]) {
#pragma unroll
    for (int k = 0; k < W - 1; ++k) {
        Row<T, VEC> r;
        r.zero();
        if (hist) r.load(hist + (n * (W - 1) + k) * C + c0);
        r.to(win[k]);
    }
}

// The W - 1 line entries before token t of sequence n, which began at s <= t.
template <typename T, int VEC, int W>
__device__ __forceinline__ void load_window(const T* x, int64_t ldx, const T* hist, int n, int s, int t, int C, int c0,
                                            f2 (&win)[W - 1][Row<T, VEC>::N2]) {
#pragma unroll
    for (int k = 0; k < W - 1; ++k) {
        const int pos = t - (W - 1) + k;
        Row<T, VEC> r;
        r.zero();
        if (pos >= s) r.load(x + pos * ldx + c0);
        else if (hist) r.load(hist + ((int64_t)n * (W - 1) + (W - 1) + pos - s) * C + c0);
        r.to(win[k]);
    }
}

template <typename T, int VEC, int W>
__device__ __forceinline__ void store_history(T* hist, int64_t n, int C, int c0, const f2 (&win)[W - 1][Row<T, VEC>::N2]) {
#pragma unroll
    for (int k = 0; k < W - 1; ++k) {
        Row<T, VEC> r;
        r.from(win[k]);
        r.store(hist + (n * (W - 1) + k) * C + c0);
    }
}

// The taps and biases of VEC channels, which lie side by side; 16-byte pieces for VEC > 1.
template <int VEC, int W>
__device__ __forceinline__ void load_taps(const float* weight, const float* bias, int c0, f2 (&w)[W][(VEC + 1) / 2],
                                          f2 (&b)[(VEC + 1) / 2]) {
    if constexpr (VEC == 1) {
#pragma unroll
        for (int j = 0; j < W; ++j) w[j][0] = pack(__ldg(weight + (int64_t)c0 * W + j), 0.f);
        b[0] = bias ? pack(__ldg(bias + c0), 0.f) : 0ull;
    } else {
        float raw[VEC * W], rb[VEC] = {};
        const float4* at = reinterpret_cast<const float4*>(weight + (int64_t)c0 * W);
        auto put = [](float* to, float4 x) { to[0] = x.x; to[1] = x.y; to[2] = x.z; to[3] = x.w; };
#pragma unroll
        for (int i = 0; i < VEC * W / 4; ++i) put(raw + 4 * i, __ldg(at + i));
        if (bias)
#pragma unroll
            for (int i = 0; i < VEC / 4; ++i) put(rb + 4 * i, __ldg(reinterpret_cast<const float4*>(bias + c0) + i));
#pragma unroll
        for (int i = 0; i < VEC / 2; ++i) {
#pragma unroll
            for (int j = 0; j < W; ++j) w[j][i] = pack(raw[2 * i * W + j], raw[(2 * i + 1) * W + j]);
            b[i] = pack(rb[2 * i], rb[2 * i + 1]);
        }
    }
}

template <int N2, int W>
__device__ __forceinline__ void preact(const f2 (&w)[W][N2], const f2 (&b)[N2], const f2 (&win)[W - 1][N2], const f2 (&v)[N2],
                                       f2 (&p)[N2]) {
#pragma unroll
    for (int k = 0; k < N2; ++k) {
        p[k] = b[k];
#pragma unroll
        for (int j = 0; j < W - 1; ++j) p[k] = fma2(w[j][k], win[j][k], p[k]);
        p[k] = fma2(w[W - 1][k], v[k], p[k]);
    }
}
template <int N2, int R>
__device__ __forceinline__ void shift(f2 (&win)[R][N2], const f2 (&v)[N2]) {
#pragma unroll
    for (int k = 0; k < N2; ++k) {
#pragma unroll
        for (int j = 0; j + 1 < R; ++j) win[j][k] = win[j + 1][k];
        win[R - 1][k] = v[k];
    }
}

template <typename T, int VEC, int W>
__global__ void __launch_bounds__(kThreads, kFwdResident) conv_fwd_kernel(ConvParams p, SeqMap m, int run) {
    typedef Row<T, VEC> R;
    constexpr int N2 = R::N2;
    typedef FwdShared<T, VEC> Sh;
    constexpr int kBatch = Sh::kBatch;
    extern __shared__ __align__(16) char smem[];
    Sh& sh = *reinterpret_cast<Sh*>(smem);
    auto& tile = sh.tile;
    auto& ring = sh.ring;
    const int tid = threadIdx.x;
    const int c0 = (blockIdx.x * kThreads + tid) * VEC;
    const bool on = c0 < p.C;
    const T* x = static_cast<const T*>(p.x) + (on ? c0 : 0);
    const T* hist = static_cast<const T*>(p.initial);
    T* y = static_cast<T*>(p.y) + c0;
    T* fin = static_cast<T*>(p.final_hist);
    const int r0 = blockIdx.y * run, r1 = (int)min((int64_t)m.total, (int64_t)r0 + run);
    auto request = [&](int t) {
        if (t < r1) {
            const int s = (t - r0) / kBatch % kStages, more = r1 - 1 - t;
            const T* from = x + t * p.ldx;
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                R::copy_async(&ring[s][i][tid], from);
                if (i < more) from += p.ldx;  // the last row again behind the run
            }
        }
        copies_commit();
    };
#pragma unroll
    for (int s = 0; s < kStages - 1; ++s) request(r0 + s * kBatch);
    f2 w[W][N2], b[N2], win[W - 1][N2];
#pragma unroll
    for (int k = 0; k < N2; ++k) {
        b[k] = 0ull;
#pragma unroll
        for (int j = 0; j < W - 1; ++j) win[j][k] = 0ull;
    }
    if (on) load_taps<VEC, W>(p.weight, p.bias, c0, w, b);
    // a sequence without tokens hands its history on
    if (fin && on)
        for (int n = blockIdx.y; n < m.N; n += gridDim.y)
            if (m.end(n) <= m.begin(n)) {
                f2 h[W - 1][N2];
                load_history<T, VEC, W>(hist, n, p.C, c0, h);
                store_history<T, VEC, W>(fin, n, p.C, c0, h);
            }
    const int first = m.first(), last = m.last();
    auto row = [&](int t, const R& in) {
        f2 v[N2], o[N2];
        in.to(v);
        preact<N2, W>(w, b, win, v, o);
        if (p.act) {
#pragma unroll
            for (int k = 0; k < N2; ++k) o[k] = mul2(o[k], sigmoid2(o[k]));
        }
        shift<N2, W - 1>(win, v);
        R out;
        out.from(o);
        out.store(y + (int64_t)t * p.C);
    };
    int until = r0;  // no boundary before this token
    bool plain = false;
    for (int t = r0; t < r1; t += kBatch) {
        if ((t - r0) % kTile == 0) {
            plain = t > r0 && t + kTile < until && t >= first;
            if (!plain) {
                __syncthreads();
                tile.template build<kThreads>(m, t);
                until = tile.until;
                plain = tile.plain && t >= first;
                if (t == r0 && tile.carry >= 0 && on)
                    load_window<T, VEC, W>(x - c0, p.ldx, hist, tile.carry, tile.carry_start, t, p.C, c0, win);
            }
        }
        request(t + (kStages - 1) * kBatch);
        copies_wait<kStages - 1>();
        if (!on) continue;
        const auto& rows = ring[(t - r0) / kBatch % kStages];
        const int k0 = (t - r0) % kTile;
        if (t + kBatch <= r1 && (plain || (t >= first && t + kBatch <= last && tile.template clear<kBatch>(k0)))) {
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                R in;
                in.from_shared(&rows[i][tid]);
                row(t + i, in);
            }
        } else {
#pragma unroll 1
            for (int i = 0; i < kBatch; ++i) {
                if (t + i >= r1 || t + i >= last) break;
                if (t + i < first) continue;
                const int s = plain ? -1 : tile.start[k0 + i], e = plain ? -1 : tile.end[k0 + i];
                if (s >= 0) load_history<T, VEC, W>(hist, s, p.C, c0, win);
                R in;
                in.from_shared(&rows[i][tid]);
                row(t + i, in);
                if (e >= 0 && fin) store_history<T, VEC, W>(fin, e, p.C, c0, win);
            }
        }
    }
}

// Backward over tokens [r0, r1) of a run and the W - 1 behind it, whose dp the run's last inputs
// need.  acc[k] is the unfinished gradient of line entry t - (W - 1) + k.
template <typename T, typename TG, int VEC, int W>
__global__ void __launch_bounds__(kThreads, kBwdResident) conv_bwd_kernel(ConvParams p, SeqMap m, int run) {
    typedef Row<T, VEC> R;
    typedef Row<TG, VEC> RG;
    constexpr int N2 = R::N2;
    typedef BwdShared<T, TG, VEC> Sh;
    constexpr int kBatch = Sh::kBatch;
    extern __shared__ __align__(16) char smem[];
    Sh& sh = *reinterpret_cast<Sh*>(smem);
    auto& tile = sh.tile;
    auto& ring = sh.ring;
    auto& gring = sh.gring;
    const int tid = threadIdx.x;
    const int c0 = (blockIdx.x * kThreads + tid) * VEC;
    const bool on = c0 < p.C;
    const T* x = static_cast<const T*>(p.x) + (on ? c0 : 0);
    const T* hist = static_cast<const T*>(p.initial);
    const TG* dy = static_cast<const TG*>(p.dy) + (on ? c0 : 0);
    const TG* dfin = static_cast<const TG*>(p.dfinal);
    TG* dx = static_cast<TG*>(p.dx) + c0;
    TG* dinit = static_cast<TG*>(p.dinitial);
    const int r0 = blockIdx.y * run, r1 = (int)min((int64_t)m.total, (int64_t)r0 + run), stop = min(m.total, r1 + W - 1);
    auto request = [&](int t) {
        if (t < stop) {
            const int s = (t - r0) / kBatch % kStages, more = stop - 1 - t;
            const T* from = x + t * p.ldx;
            const TG* gfrom = dy + (int64_t)t * p.C;
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                R::copy_async(&ring[s][i][tid], from);
                RG::copy_async(&gring[s][i][tid], gfrom);
                if (i < more) {  // the last row again behind the tokens
                    from += p.ldx;
                    gfrom += p.C;
                }
            }
        }
        copies_commit();
    };
#pragma unroll
    for (int s = 0; s < kStages - 1; ++s) request(r0 + s * kBatch);
    f2 w[W][N2], b[N2], win[W - 1][N2], acc[W][N2], dw[W][N2], db[N2];
#pragma unroll
    for (int k = 0; k < N2; ++k) {
        b[k] = db[k] = 0ull;
#pragma unroll
        for (int j = 0; j < W; ++j) acc[j][k] = dw[j][k] = 0ull;
#pragma unroll
        for (int j = 0; j < W - 1; ++j) win[j][k] = 0ull;
    }
    if (on) load_taps<VEC, W>(p.weight, p.bias, c0, w, b);
    // a sequence without tokens hands its history's gradient back
    if (dinit && on)
        for (int n = blockIdx.y; n < m.N; n += gridDim.y)
            if (m.end(n) <= m.begin(n)) {
                f2 h[W - 1][N2];
                load_history<TG, VEC, W>(dfin, n, p.C, c0, h);
                store_history<TG, VEC, W>(dinit, n, p.C, c0, h);
            }
    const int first = m.first(), last = m.last();
    int seq = -1, begin = r0;  // the sequence of the token at hand and its first token
    // line entry `pos` of the sequence at hand is finished
    auto finish = [&](int pos, const f2 (&g)[N2]) {
        RG r;
        r.from(g);
        if (pos >= begin) {
            if (pos >= r0 && pos < r1) r.store(dx + (int64_t)pos * p.C);
        } else if (dinit && seq >= 0 && begin >= r0 && begin < r1) {
            r.store(dinit + ((int64_t)seq * (W - 1) + (W - 1) + pos - begin) * p.C + c0);
        }
    };
    // token t; `mine`: it lies in the run, so its share of dw and dbias is this run's
    auto row = [&](const R& in, const RG& gr, bool mine) {
        f2 v[N2], d[N2];
        in.to(v);
        gr.to(d);
        if (p.act) {
            f2 a[N2];
            preact<N2, W>(w, b, win, v, a);
            const f2 one = pack(1.f, 1.f), minus = pack(-1.f, -1.f);
#pragma unroll
            for (int k = 0; k < N2; ++k) {
                const f2 sg = sigmoid2(a[k]);
                d[k] = mul2(d[k], mul2(sg, fma2(a[k], fma2(minus, sg, one), one)));
            }
        }
#pragma unroll
        for (int k = 0; k < N2; ++k) {
#pragma unroll
            for (int j = 0; j < W; ++j) acc[j][k] = fma2(w[j][k], d[k], acc[j][k]);
            if (mine) {
#pragma unroll
                for (int j = 0; j < W - 1; ++j) dw[j][k] = fma2(d[k], win[j][k], dw[j][k]);
                dw[W - 1][k] = fma2(d[k], v[k], dw[W - 1][k]);
                db[k] = add2(db[k], d[k]);
            }
        }
        shift<N2, W - 1>(win, v);
    };
    const f2 zero[N2] = {};
    int until = r0;
    bool plain = false, done = false;
    for (int t = r0; t < stop; t += kBatch) {
        if ((t - r0) % kTile == 0) {
            plain = t > r0 && t + kTile < until && t >= first;
            if (!plain) {
                __syncthreads();
                tile.template build<kThreads>(m, t);
                until = tile.until;
                plain = tile.plain && t >= first;
                if (t == r0 && tile.carry >= 0 && on) {
                    seq = tile.carry;
                    begin = tile.carry_start;
                    load_window<T, VEC, W>(x - c0, p.ldx, hist, seq, begin, t, p.C, c0, win);
                }
            }
        }
        request(t + (kStages - 1) * kBatch);
        copies_wait<kStages - 1>();
        if (!on || done) continue;
        const int s = (t - r0) / kBatch % kStages;
        const int k0 = (t - r0) % kTile;
        if (t + kBatch <= r1 && t - (W - 1) >= max(begin, r0) &&
            (plain || (seq >= 0 && t + kBatch <= last && tile.template clear<kBatch>(k0)))) {
            // every entry finished here is a token of the run
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                R in;
                RG gr, out;
                in.from_shared(&ring[s][i][tid]);
                gr.from_shared(&gring[s][i][tid]);
                row(in, gr, true);
                out.from(acc[0]);
                out.store(dx + (int64_t)(t + i - (W - 1)) * p.C);
                shift<N2, W>(acc, zero);
            }
        } else {
#pragma unroll 1
            for (int i = 0; i < kBatch; ++i) {
                const int at = t + i;
                if (at >= stop || at >= last) break;
                if (at < first) continue;
                const int sb = plain ? -1 : tile.start[k0 + i], se = plain ? -1 : tile.end[k0 + i];
                if (sb >= 0) {
                    if (at >= r1) {
                        done = true;  // the run's entries are finished
                        break;
                    }
                    seq = sb;
                    begin = at;
                    load_history<T, VEC, W>(hist, sb, p.C, c0, win);
#pragma unroll
                    for (int j = 0; j < W; ++j)
#pragma unroll
                        for (int k = 0; k < N2; ++k) acc[j][k] = 0ull;
                }
                R in;
                RG gr;
                in.from_shared(&ring[s][i][tid]);
                gr.from_shared(&gring[s][i][tid]);
                row(in, gr, at < r1);
                finish(at - (W - 1), acc[0]);
                shift<N2, W>(acc, zero);
                if (se >= 0) {
                    // the sequence's last W - 1 entries: no more dp, but the final history's gradient
#pragma unroll
                    for (int j = 0; j < W - 1; ++j) {
                        if (dfin) {
                            f2 f[N2];
                            RG r;
                            r.load(dfin + ((int64_t)se * (W - 1) + j) * p.C + c0);
                            r.to(f);
#pragma unroll
                            for (int k = 0; k < N2; ++k) acc[j][k] = add2(acc[j][k], f[k]);
                        }
                        finish(at - (W - 2) + j, acc[j]);
                    }
                    if (at >= r1) {
                        done = true;
                        break;
                    }
                }
            }
        }
    }
    if (on) {
        // the run's rows of no sequence, on which nothing depends
        RG none;
        none.zero();
        for (int t = r0; t < min(r1, first); ++t) none.store(dx + (int64_t)t * p.C);
        for (int t = max(r0, last); t < r1; ++t) none.store(dx + (int64_t)t * p.C);
    }
    tc::grid_dep_launch();
    if (on) {
        // [run][tap, and the bias][C]
        float* out = p.partial + (int64_t)blockIdx.y * (W + 1) * p.C + c0;
#pragma unroll
        for (int j = 0; j <= W; ++j)
#pragma unroll
            for (int k = 0; k < N2; ++k) {
                float a, c;
                unpack(j < W ? dw[j < W ? j : 0][k] : db[k], a, c);
                out[(int64_t)j * p.C + 2 * k] = a;
                if (2 * k + 1 < VEC) out[(int64_t)j * p.C + 2 * k + 1] = c;
            }
    }
}

// dw and dbias from the runs' partial sums, in the order of the runs.
__global__ void __launch_bounds__(128) conv_bwd_sum_kernel(const float* partial, int runs, int C, int W, float* dw,
                                                           float* db) {
    const int64_t i = (int64_t)blockIdx.x * 128 + threadIdx.x, n = (int64_t)C * (W + 1);
    tc::grid_dep_wait();
    if (i >= n) return;
    float a = 0.f;
#pragma unroll 16
    for (int r = 0; r < runs; ++r) a += partial[r * n + i];
    const int64_t c = i % C;
    const int j = (int)(i / C);
    if (j < W) dw[c * W + j] = a;
    else if (db) db[c] = a;
}

// kRows rows of the batch a block, so that the taps are fetched once for them: they are as many
// bytes as two rows' histories.
template <typename T, int VEC, int W, int kRows>
__global__ void __launch_bounds__(kThreads) conv_step_kernel(ConvStepParams p) {
    typedef Row<T, VEC> R;
    constexpr int N2 = R::N2;
    const int row0 = blockIdx.x * kRows;
    const int c0 = (blockIdx.y * kThreads + threadIdx.x) * VEC;
    const bool on = c0 < p.C;
    T* hist = static_cast<T*>(p.history);
    int page[kRows];
    R in[kRows], past[kRows][W - 1];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        page[i] = row0 + i < p.N ? page_of_row(p.slots, row0 + i, p.P) : -1;
        if (!on || page[i] < 0) continue;
        in[i].load(static_cast<const T*>(p.x) + (row0 + i) * p.ldx + c0);
#pragma unroll
        for (int k = 0; k < W - 1; ++k) past[i][k].load_rw(hist + ((int64_t)page[i] * (W - 1) + k) * p.C + c0);
    }
    f2 w[W][N2], b[N2];
    if (on) load_taps<VEC, W>(p.weight, p.bias, c0, w, b);
    const unsigned refused = rows_refused<kRows>(p.slots, row0, p.N, page, p.status);
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        if (row0 + i >= p.N || (refused >> i & 1) || !on) continue;
        f2 win[W - 1][N2], v[N2], o[N2];
        in[i].to(v);
#pragma unroll
        for (int k = 0; k < W - 1; ++k) past[i][k].to(win[k]);
        preact<N2, W>(w, b, win, v, o);
        if (p.act) {
#pragma unroll
            for (int k = 0; k < N2; ++k) o[k] = mul2(o[k], sigmoid2(o[k]));
        }
        R out;
        out.from(o);
        out.store(static_cast<T*>(p.y) + (int64_t)(row0 + i) * p.C + c0);
#pragma unroll
        for (int k = 0; k + 1 < W - 1; ++k) past[i][k + 1].store(hist + ((int64_t)page[i] * (W - 1) + k) * p.C + c0);
        in[i].store(hist + ((int64_t)page[i] * (W - 1) + W - 2) * p.C + c0);
    }
}

// Tokens of one run: as many runs as one filling of the machine holds, at least 32 tokens each so
// that the W - 1 rows read twice stay below a tenth; three fillings where the runs then still have 128
// tokens, which evens out what blocks finish early (70k x 12288 forwards: 554 us against 566).
int run_tokens(int total, int C, int vec, int resident) {
    const int blocks = (C + kThreads * vec - 1) / (kThreads * vec);
    const int runs = kSms * resident / blocks > 0 ? kSms * resident / blocks : 1;
    int run = total / runs + (total % runs != 0);
    if (run >= 3 * 128) run = (run + 2) / 3;
    run = (run + 7) / 8 * 8;
    return run < 32 ? 32 : run;
}
// (total + run may pass 2^31)
int run_count(int total, int run) { return total > 0 ? total / run + (total % run != 0) : 1; }

SeqMap seq_map(const ConvParams& p) { return SeqMap{p.cu, p.N, p.T, p.total}; }

template <typename K>
cudaError_t launch_runs(K kern, const ConvParams& p, int vec, int resident, int smem, cudaStream_t st) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    const int run = run_tokens(p.total, p.C, vec, resident);
    const dim3 grid((p.C + kThreads * vec - 1) / (kThreads * vec), run_count(p.total, run));
    kern<<<grid, kThreads, smem, st>>>(p, seq_map(p), run);
    return cudaGetLastError();
}

template <typename T, int VEC>
cudaError_t launch_fwd(const ConvParams& p, cudaStream_t st) {
    constexpr int smem = sizeof(FwdShared<T, VEC>);
    if (p.W == 4) return launch_runs(conv_fwd_kernel<T, VEC, 4>, p, VEC, kFwdResident, smem, st);
    if (p.W == 3) return launch_runs(conv_fwd_kernel<T, VEC, 3>, p, VEC, kFwdResident, smem, st);
    return launch_runs(conv_fwd_kernel<T, VEC, 2>, p, VEC, kFwdResident, smem, st);
}

template <typename T, typename TG, int VEC>
cudaError_t launch_bwd(const ConvParams& p, cudaStream_t st) {
    constexpr int smem = sizeof(BwdShared<T, TG, VEC>);
    cudaError_t e = p.W == 4   ? launch_runs(conv_bwd_kernel<T, TG, VEC, 4>, p, VEC, kBwdResident, smem, st)
                    : p.W == 3 ? launch_runs(conv_bwd_kernel<T, TG, VEC, 3>, p, VEC, kBwdResident, smem, st)
                               : launch_runs(conv_bwd_kernel<T, TG, VEC, 2>, p, VEC, kBwdResident, smem, st);
    if (e != cudaSuccess) return e;
    const int runs = run_count(p.total, run_tokens(p.total, p.C, VEC, kBwdResident));
    const int64_t n = (int64_t)p.C * (p.W + 1);
    // (it may start while the runs end: 4096 x 12288 in 65.5 us, 67.7 without)
    return tc::launch_dependent(conv_bwd_sum_kernel, (unsigned)((n + 127) / 128), 128, 0, st, p.partial, runs, p.C, p.W, p.dweight,
                                p.dbias);
}

template <typename T, int VEC, int W>
cudaError_t launch_step_rows(const ConvStepParams& p, cudaStream_t st) {
    const int blocks = (p.C + kThreads * VEC - 1) / (kThreads * VEC);
    // four rows a block once that leaves two blocks an SM, else one
    if ((int64_t)(p.N + 3) / 4 * blocks >= 2 * kSms) conv_step_kernel<T, VEC, W, 4><<<dim3((p.N + 3) / 4, blocks), kThreads, 0, st>>>(p);
    else conv_step_kernel<T, VEC, W, 1><<<dim3(p.N, blocks), kThreads, 0, st>>>(p);
    return cudaGetLastError();
}
template <typename T, int VEC>
cudaError_t launch_step(const ConvStepParams& p, cudaStream_t st) {
    if (p.W == 4) return launch_step_rows<T, VEC, 4>(p, st);
    if (p.W == 3) return launch_step_rows<T, VEC, 3>(p, st);
    return launch_step_rows<T, VEC, 2>(p, st);
}

// Backwards a thread has four channels: 8 bytes of bf16, 16 of fp32.
constexpr int kBwdVec = 4;

}  // namespace

cudaError_t short_conv_fwd(kda_dtype dt, const ConvParams& p, cudaStream_t st) {
    using kda_host::rows_aligned;
    const int vec = dt == KDA_BF16 ? 8 : 4;
    const bool wide = rows_aligned(p.x, p.ldx, vec) && rows_aligned(p.weight, 0, 4) && rows_aligned(p.bias, 0, 4) && rows_aligned(p.y, p.C, vec) && rows_aligned(p.initial, p.C, vec) &&
                      rows_aligned(p.final_hist, p.C, vec) && p.C % vec == 0;
    if (dt == KDA_BF16) return wide ? launch_fwd<__nv_bfloat16, 8>(p, st) : launch_fwd<__nv_bfloat16, 1>(p, st);
    return wide ? launch_fwd<float, 4>(p, st) : launch_fwd<float, 1>(p, st);
}

size_t short_conv_bwd_partial(int total, int C, int W) {
    // the runs of the wide and of the narrow variant: either may be the more
    const int wide = run_count(total, run_tokens(total, C, kBwdVec, kBwdResident));
    const int narrow = run_count(total, run_tokens(total, C, 1, kBwdResident));
    return (size_t)(wide > narrow ? wide : narrow) * C * (W + 1);
}

cudaError_t short_conv_bwd(kda_dtype dt, kda_dtype gdt, const ConvParams& p, cudaStream_t st) {
    using kda_host::rows_aligned;
    const void* rows[] = {p.initial, p.dy, p.dfinal, p.dx, p.dinitial};
    bool wide = rows_aligned(p.x, p.ldx, kBwdVec) && rows_aligned(p.weight, 0, 4) && rows_aligned(p.bias, 0, 4) && p.C % kBwdVec == 0;
    for (const void* r : rows) wide = wide && rows_aligned(r, p.C, kBwdVec);
    if (dt == KDA_F32) return wide ? launch_bwd<float, float, kBwdVec>(p, st) : launch_bwd<float, float, 1>(p, st);
    if (gdt == KDA_F32)
        return wide ? launch_bwd<__nv_bfloat16, float, kBwdVec>(p, st) : launch_bwd<__nv_bfloat16, float, 1>(p, st);
    return wide ? launch_bwd<__nv_bfloat16, __nv_bfloat16, kBwdVec>(p, st) : launch_bwd<__nv_bfloat16, __nv_bfloat16, 1>(p, st);
}

cudaError_t short_conv_step(kda_dtype dt, const ConvStepParams& p, cudaStream_t st) {
    using kda_host::rows_aligned;
    const int vec = dt == KDA_BF16 ? 8 : 4;
    const bool wide = rows_aligned(p.x, p.ldx, vec) && rows_aligned(p.weight, 0, 4) && rows_aligned(p.bias, 0, 4) && rows_aligned(p.y, p.C, vec) && rows_aligned(p.history, p.C, vec) &&
                      p.C % vec == 0;
    if (dt == KDA_BF16) return wide ? launch_step<__nv_bfloat16, 8>(p, st) : launch_step<__nv_bfloat16, 1>(p, st);
    return wide ? launch_step<float, 4>(p, st) : launch_step<float, 1>(p, st);
}

}  // namespace kda
