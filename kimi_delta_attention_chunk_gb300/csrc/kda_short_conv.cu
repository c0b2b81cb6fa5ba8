// The short causal convolution on its own: forward with the history carried in and out, backward,
// and the single-token form ("kimi-k3-mlx" review, section "Attention is 93 layers ...": a short
// convolution of kernel size 4 on q, k and v, ahead of the recurrence).
//
// Depthwise over C channels, W taps, sequence by sequence; line = [history | inputs]:
//     p_t = bias + sum_j w[c][j] line_{t-(W-1)+j},   y = p or p sigmoid(p)
// and backwards, with dp = dy act'(p):
//     dline_i = sum_j w[c][j] dp_{i+(W-1)-j} (+ the final history's gradient),
//     dw[c][j] = sum_t dp_t line_{t-(W-1)+j},   dbias = sum_t dp_t.
// Everything moves W rows through registers, so each direction reads and writes its rows once and
// HBM bounds it.  A thread owns 16 bytes of channels (or one channel where the rows are not 16-byte
// pieces) and walks a run of tokens with the last W - 1 inputs (and, backwards, the W - 1 unfinished
// input gradients) in registers; runs meet at W - 1 rows that both read.  Eight rows are requested
// before the first is used.
#include "kda_layer.h"
#include "kda_segments.cuh"
#include "kda_slots.cuh"

namespace kda {

namespace {

constexpr int kThreads = 128;
constexpr int kTile = 64;   // tokens of one look at the sequence boundaries
constexpr int kBatch = 8;   // rows in flight per thread

template <typename T, int VEC, int W>
__device__ __forceinline__ void load_history(const T* hist, int64_t n, int C, int c0, float (&win)[W - 1][VEC]) {
#pragma unroll
    for (int k = 0; k < W - 1; ++k) {
        if (hist) {
            Row<T, VEC> r;
            r.load(hist + (n * (W - 1) + k) * C + c0);
            r.to(win[k]);
        } else {
#pragma unroll
            for (int i = 0; i < VEC; ++i) win[k][i] = 0.f;
        }
    }
}

// The W - 1 line entries before token t of sequence n, which began at s <= t.
template <typename T, int VEC, int W>
__device__ __forceinline__ void load_window(const T* x, int64_t ldx, const T* hist, int n, int s, int t, int C, int c0,
                                            float (&win)[W - 1][VEC]) {
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
__device__ __forceinline__ void store_history(T* hist, int64_t n, int C, int c0, const float (&win)[W - 1][VEC]) {
#pragma unroll
    for (int k = 0; k < W - 1; ++k) {
        Row<T, VEC> r;
        r.from(win[k]);
        r.store(hist + (n * (W - 1) + k) * C + c0);
    }
}

template <int VEC, int W>
__device__ __forceinline__ void load_taps(const float* weight, const float* bias, int c0, float (&w)[W][VEC],
                                          float (&b)[VEC]) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
#pragma unroll
        for (int j = 0; j < W; ++j) w[j][i] = __ldg(weight + (int64_t)(c0 + i) * W + j);
        b[i] = bias ? __ldg(bias + c0 + i) : 0.f;
    }
}

template <typename T, int VEC, int W>
__global__ void __launch_bounds__(kThreads, VEC > 1 ? 4 : 8) conv_fwd_kernel(ConvParams p, SeqMap m, int run) {
    __shared__ TokenTile<kTile> tile;
    const int c0 = (blockIdx.x * kThreads + threadIdx.x) * VEC;
    const bool on = c0 < p.C;
    const T* x = static_cast<const T*>(p.x);
    const T* hist = static_cast<const T*>(p.initial);
    T* y = static_cast<T*>(p.y);
    T* fin = static_cast<T*>(p.final_hist);
    float w[W][VEC], b[VEC], win[W - 1][VEC] = {};
    if (on) load_taps<VEC, W>(p.weight, p.bias, c0, w, b);
    // a sequence without tokens hands its history on
    if (fin && on)
        for (int n = blockIdx.y; n < m.N; n += gridDim.y)
            if (m.end(n) <= m.begin(n)) {
                float h[W - 1][VEC];
                load_history<T, VEC, W>(hist, n, p.C, c0, h);
                store_history<T, VEC, W>(fin, n, p.C, c0, h);
            }
    const int r0 = blockIdx.y * run, r1 = min(m.total, r0 + run);
    for (int t0 = r0; t0 < r1; t0 += kTile) {
        __syncthreads();
        tile.build<kThreads>(m, t0);
        if (!on) continue;
        if (t0 == r0 && tile.carry >= 0)
            load_window<T, VEC, W>(x, p.ldx, hist, tile.carry, tile.carry_start, t0, p.C, c0, win);
        const int lo = max(t0, m.first()), hi = min(min(t0 + kTile, r1), m.last());
        for (int t = lo; t < hi; t += kBatch) {
            Row<T, VEC> in[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i)
                if (t + i < hi) in[i].load(x + (int64_t)(t + i) * p.ldx + c0);
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                if (t + i >= hi) break;
                const int s = tile.start[t + i - t0], e = tile.end[t + i - t0];
                if (s >= 0) load_history<T, VEC, W>(hist, s, p.C, c0, win);
                float v[VEC], o[VEC];
                in[i].to(v);
#pragma unroll
                for (int k = 0; k < VEC; ++k) {
                    float a = b[k];
#pragma unroll
                    for (int j = 0; j < W - 1; ++j) a = fmaf(w[j][k], win[j][k], a);
                    a = fmaf(w[W - 1][k], v[k], a);
                    o[k] = p.act ? a * sigmoid(a) : a;
#pragma unroll
                    for (int j = 0; j < W - 2; ++j) win[j][k] = win[j + 1][k];
                    win[W - 2][k] = v[k];
                }
                Row<T, VEC> out;
                out.from(o);
                out.store(y + (int64_t)(t + i) * p.C + c0);
                if (e >= 0 && fin) store_history<T, VEC, W>(fin, e, p.C, c0, win);
            }
        }
    }
}

// Backward over tokens [r0, r1) of a run and the W - 1 behind it, whose dp the run's last inputs
// need.  ring[k] is the unfinished gradient of line entry t - (W - 1) + k.
template <typename T, typename TG, int VEC, int W>
__global__ void __launch_bounds__(kThreads, VEC > 1 ? 3 : 8) conv_bwd_kernel(ConvParams p, SeqMap m, int run) {
    __shared__ TokenTile<kTile> tile;
    const int c0 = (blockIdx.x * kThreads + threadIdx.x) * VEC;
    const bool on = c0 < p.C;
    const T* x = static_cast<const T*>(p.x);
    const T* hist = static_cast<const T*>(p.initial);
    const TG* dy = static_cast<const TG*>(p.dy);
    const TG* dfin = static_cast<const TG*>(p.dfinal);
    TG* dx = static_cast<TG*>(p.dx);
    TG* dinit = static_cast<TG*>(p.dinitial);
    float w[W][VEC], b[VEC], win[W - 1][VEC] = {}, ring[W][VEC] = {};
    float dw[W][VEC] = {}, db[VEC] = {};
    if (on) load_taps<VEC, W>(p.weight, p.bias, c0, w, b);
    // a sequence without tokens hands its history's gradient back
    if (dinit && on)
        for (int n = blockIdx.y; n < m.N; n += gridDim.y)
            if (m.end(n) <= m.begin(n)) {
                float h[W - 1][VEC];
                load_history<TG, VEC, W>(dfin, n, p.C, c0, h);
                store_history<TG, VEC, W>(dinit, n, p.C, c0, h);
            }
    const int r0 = blockIdx.y * run, r1 = min(m.total, r0 + run);
    const int last = m.last();
    int seq = -1, begin = r0;   // the sequence of the token at hand and its first token
    bool done = false;          // behind the run: the run's entries are finished
    // line entry `pos` of the sequence at hand is finished
    auto finish = [&](int pos, const float* g) {
        if (pos >= begin) {
            if (pos < r0 || pos >= r1) return;
            Row<TG, VEC> r;
            r.from(g);
            r.store(dx + (int64_t)pos * p.C + c0);
        } else if (dinit && seq >= 0 && begin >= r0 && begin < r1) {
            Row<TG, VEC> r;
            r.from(g);
            r.store(dinit + ((int64_t)seq * (W - 1) + (W - 1) + pos - begin) * p.C + c0);
        }
    };
    for (int t0 = r0; t0 < min(last, r1 + W - 1); t0 += kTile) {
        __syncthreads();
        tile.build<kThreads>(m, t0);
        if (!on) continue;
        if (t0 == r0 && tile.carry >= 0) {
            seq = tile.carry;
            begin = tile.carry_start;
            load_window<T, VEC, W>(x, p.ldx, hist, seq, begin, t0, p.C, c0, win);
        }
        const int lo = max(t0, m.first()), hi = min(min(t0 + kTile, r1 + W - 1), last);
        for (int t = lo; t < hi && !done; t += kBatch) {
            Row<T, VEC> in[kBatch];
            Row<TG, VEC> gr[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i)
                if (t + i < hi) {
                    in[i].load(x + (int64_t)(t + i) * p.ldx + c0);
                    gr[i].load(dy + (int64_t)(t + i) * p.C + c0);
                }
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                if (t + i >= hi || done) break;
                const int s = tile.start[t + i - t0], e = tile.end[t + i - t0];
                if (s >= 0) {
                    if (t + i >= r1) {
                        done = true;
                        break;
                    }
                    seq = s;
                    begin = t + i;
                    load_history<T, VEC, W>(hist, s, p.C, c0, win);
#pragma unroll
                    for (int j = 0; j < W; ++j)
#pragma unroll
                        for (int k = 0; k < VEC; ++k) ring[j][k] = 0.f;
                }
                const bool mine = t + i < r1;
                float v[VEC], d[VEC];
                in[i].to(v);
                gr[i].to(d);
#pragma unroll
                for (int k = 0; k < VEC; ++k) {
                    if (p.act) {
                        float a = b[k];
#pragma unroll
                        for (int j = 0; j < W - 1; ++j) a = fmaf(w[j][k], win[j][k], a);
                        a = fmaf(w[W - 1][k], v[k], a);
                        const float sg = sigmoid(a);
                        d[k] *= sg * fmaf(a, 1.f - sg, 1.f);
                    }
#pragma unroll
                    for (int j = 0; j < W; ++j) ring[j][k] = fmaf(w[j][k], d[k], ring[j][k]);
                    if (mine) {
#pragma unroll
                        for (int j = 0; j < W - 1; ++j) dw[j][k] = fmaf(d[k], win[j][k], dw[j][k]);
                        dw[W - 1][k] = fmaf(d[k], v[k], dw[W - 1][k]);
                        db[k] += d[k];
                    }
#pragma unroll
                    for (int j = 0; j < W - 2; ++j) win[j][k] = win[j + 1][k];
                    win[W - 2][k] = v[k];
                }
                finish(t + i - (W - 1), ring[0]);
#pragma unroll
                for (int j = 0; j < W - 1; ++j)
#pragma unroll
                    for (int k = 0; k < VEC; ++k) ring[j][k] = ring[j + 1][k];
#pragma unroll
                for (int k = 0; k < VEC; ++k) ring[W - 1][k] = 0.f;
                if (e >= 0) {
                    // the sequence's last W - 1 entries: no more dp, but the final history's gradient
#pragma unroll
                    for (int j = 0; j < W - 1; ++j) {
                        if (dfin) {
                            float f[VEC];
                            Row<TG, VEC> r;
                            r.load(dfin + ((int64_t)e * (W - 1) + j) * p.C + c0);
                            r.to(f);
#pragma unroll
                            for (int k = 0; k < VEC; ++k) ring[j][k] += f[k];
                        }
                        finish(t + i - (W - 2) + j, ring[j]);
                    }
                    if (!mine) done = true;
                }
            }
        }
    }
    if (on) {
        float* out = p.partial + ((int64_t)blockIdx.y * p.C + c0) * (W + 1);
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
#pragma unroll
            for (int j = 0; j < W; ++j) out[k * (W + 1) + j] = dw[j][k];
            out[k * (W + 1) + W] = db[k];
        }
    }
}

// dw and dbias from the runs' partial sums, in the order of the runs.
__global__ void __launch_bounds__(256) conv_bwd_sum_kernel(const float* partial, int runs, int C, int W, float* dw,
                                                           float* db) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, n = (int64_t)C * (W + 1);
    if (i >= n) return;
    float a = 0.f;
    for (int r = 0; r < runs; ++r) a += partial[r * n + i];
    const int64_t c = i / (W + 1);
    const int j = (int)(i % (W + 1));
    if (j < W) dw[c * W + j] = a;
    else if (db) db[c] = a;
}

template <typename T, int VEC, int W>
__global__ void __launch_bounds__(kThreads) conv_step_kernel(ConvStepParams p) {
    const int row = blockIdx.x;
    const int page = page_of_row(p.slots, row, p.P);
    if (row_refused(p.slots, row, page, p.status)) return;
    const int c0 = (blockIdx.y * kThreads + threadIdx.x) * VEC;
    if (c0 >= p.C) return;
    T* hist = static_cast<T*>(p.history);
    Row<T, VEC> in;
    in.load(static_cast<const T*>(p.x) + row * p.ldx + c0);
    Row<T, VEC> past[W - 1];
#pragma unroll
    for (int k = 0; k < W - 1; ++k) past[k].load_rw(hist + ((int64_t)page * (W - 1) + k) * p.C + c0);
    float w[W][VEC], b[VEC], v[VEC], o[VEC];
    load_taps<VEC, W>(p.weight, p.bias, c0, w, b);
    in.to(v);
#pragma unroll
    for (int k = 0; k < VEC; ++k) o[k] = fmaf(w[W - 1][k], v[k], b[k]);
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
        float h[VEC];
        past[j].to(h);
#pragma unroll
        for (int k = 0; k < VEC; ++k) o[k] = fmaf(w[j][k], h[k], o[k]);
    }
    if (p.act) {
#pragma unroll
        for (int k = 0; k < VEC; ++k) o[k] *= sigmoid(o[k]);
    }
    Row<T, VEC> out;
    out.from(o);
    out.store(static_cast<T*>(p.y) + (int64_t)row * p.C + c0);
#pragma unroll
    for (int k = 0; k + 1 < W - 1; ++k) past[k + 1].store(hist + ((int64_t)page * (W - 1) + k) * p.C + c0);
    in.store(hist + ((int64_t)page * (W - 1) + W - 2) * p.C + c0);
}

// Tokens of one run: enough runs to fill the machine about twice over, at least 32 tokens each
// so that the W - 1 rows read twice stay below a tenth.
int run_tokens(int total, int C, int vec) {
    const int blocks = (C + kThreads * vec - 1) / (kThreads * vec);
    const int runs = (152 * 8 + blocks - 1) / blocks;
    int run = (total + runs - 1) / runs;
    run = (run + kBatch - 1) / kBatch * kBatch;
    return run < 32 ? 32 : run;
}
int run_count(int total, int run) { return total > 0 ? (total + run - 1) / run : 1; }

SeqMap seq_map(const ConvParams& p) { return SeqMap{p.cu, p.N, p.T, p.total}; }

template <typename T, int VEC>
cudaError_t launch_fwd(const ConvParams& p, cudaStream_t st) {
    const int run = run_tokens(p.total, p.C, VEC);
    const dim3 grid((p.C + kThreads * VEC - 1) / (kThreads * VEC), run_count(p.total, run));
    if (p.W == 4) conv_fwd_kernel<T, VEC, 4><<<grid, kThreads, 0, st>>>(p, seq_map(p), run);
    else if (p.W == 3) conv_fwd_kernel<T, VEC, 3><<<grid, kThreads, 0, st>>>(p, seq_map(p), run);
    else conv_fwd_kernel<T, VEC, 2><<<grid, kThreads, 0, st>>>(p, seq_map(p), run);
    return cudaGetLastError();
}

template <typename T, typename TG, int VEC>
cudaError_t launch_bwd(const ConvParams& p, cudaStream_t st) {
    const int run = run_tokens(p.total, p.C, VEC), runs = run_count(p.total, run);
    const dim3 grid((p.C + kThreads * VEC - 1) / (kThreads * VEC), runs);
    if (p.W == 4) conv_bwd_kernel<T, TG, VEC, 4><<<grid, kThreads, 0, st>>>(p, seq_map(p), run);
    else if (p.W == 3) conv_bwd_kernel<T, TG, VEC, 3><<<grid, kThreads, 0, st>>>(p, seq_map(p), run);
    else conv_bwd_kernel<T, TG, VEC, 2><<<grid, kThreads, 0, st>>>(p, seq_map(p), run);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const int64_t n = (int64_t)p.C * (p.W + 1);
    conv_bwd_sum_kernel<<<(unsigned)((n + 255) / 256), 256, 0, st>>>(p.partial, runs, p.C, p.W, p.dweight, p.dbias);
    return cudaGetLastError();
}

template <typename T, int VEC>
cudaError_t launch_step(const ConvStepParams& p, cudaStream_t st) {
    const dim3 grid(p.N, (p.C + kThreads * VEC - 1) / (kThreads * VEC));
    if (p.W == 4) conv_step_kernel<T, VEC, 4><<<grid, kThreads, 0, st>>>(p);
    else if (p.W == 3) conv_step_kernel<T, VEC, 3><<<grid, kThreads, 0, st>>>(p);
    else conv_step_kernel<T, VEC, 2><<<grid, kThreads, 0, st>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t short_conv_fwd(kda_dtype dt, const ConvParams& p, cudaStream_t st) {
    using kda_host::rows_aligned;
    const int vec = dt == KDA_BF16 ? 8 : 4;
    const bool wide = rows_aligned(p.x, p.ldx, vec) && rows_aligned(p.y, p.C, vec) && rows_aligned(p.initial, p.C, vec) &&
                      rows_aligned(p.final_hist, p.C, vec) && p.C % vec == 0;
    if (dt == KDA_BF16) return wide ? launch_fwd<__nv_bfloat16, 8>(p, st) : launch_fwd<__nv_bfloat16, 1>(p, st);
    return wide ? launch_fwd<float, 4>(p, st) : launch_fwd<float, 1>(p, st);
}

size_t short_conv_bwd_partial(int total, int C, int W) {
    // the narrow variant has the fewer runs: more blocks along the channels
    return (size_t)run_count(total, run_tokens(total, C, 8)) * C * (W + 1);
}

cudaError_t short_conv_bwd(kda_dtype dt, kda_dtype gdt, const ConvParams& p, cudaStream_t st) {
    using kda_host::rows_aligned;
    const int vec = dt == KDA_BF16 ? 8 : 4;
    const void* rows[] = {p.initial, p.dy, p.dfinal, p.dx, p.dinitial};
    bool wide = rows_aligned(p.x, p.ldx, vec) && p.C % vec == 0;
    for (const void* r : rows) wide = wide && rows_aligned(r, p.C, vec);
    if (dt == KDA_F32) return wide ? launch_bwd<float, float, 4>(p, st) : launch_bwd<float, float, 1>(p, st);
    if (gdt == KDA_F32)
        return wide ? launch_bwd<__nv_bfloat16, float, 8>(p, st) : launch_bwd<__nv_bfloat16, float, 1>(p, st);
    return wide ? launch_bwd<__nv_bfloat16, __nv_bfloat16, 8>(p, st) : launch_bwd<__nv_bfloat16, __nv_bfloat16, 1>(p, st);
}

cudaError_t short_conv_step(kda_dtype dt, const ConvStepParams& p, cudaStream_t st) {
    using kda_host::rows_aligned;
    const int vec = dt == KDA_BF16 ? 8 : 4;
    const bool wide = rows_aligned(p.x, p.ldx, vec) && rows_aligned(p.y, p.C, vec) && rows_aligned(p.history, p.C, vec) &&
                      p.C % vec == 0;
    if (dt == KDA_BF16) return wide ? launch_step<__nv_bfloat16, 8>(p, st) : launch_step<__nv_bfloat16, 1>(p, st);
    return wide ? launch_step<float, 4>(p, st) : launch_step<float, 1>(p, st);
}

}  // namespace kda
