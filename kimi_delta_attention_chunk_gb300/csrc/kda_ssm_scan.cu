// Selective state space scan over prompts: forward.
//
// Per sequence, channel c (group g) and state s, over the tokens:
//     d = softplus(delta + bias),  h_s <- exp(d A_s) h_s + d u B_s,  y = (sum_s C_s h_s + D u) silu(z)
// A channel's row is four elements (u, delta, z, y), 8 bytes in bf16, against S exponentials and 4 S
// multiply-adds, so at S = 16 the special-function and fp32 units bound it before HBM does.  A thread
// owns a channel and 16 of its states (S = 32, 64: two or four lanes a channel, y summed by shuffles)
// with the state and A in registers, in pairs of packed fp32; B and C of a tile of tokens are turned to
// fp32 once per block and read from shared memory by everyone; u, delta and z are requested eight tokens
// ahead.
//
// The recurrence leaves C threads' worth of parallelism (times the sequences); where that does not fill
// the machine the stream is cut into runs: every run's end state from a zero start and the sum of its step
// sizes (its decay is exp(A sum d)), a short prefix over the runs, and the runs again from their true
// starts.  Cuts fall at fixed places of the flat token stream; sequences begin and end inside runs.
#include "kda_layer.h"
#include "kda_ssm.cuh"

namespace kda {

namespace {

constexpr int kThreads = 128;
constexpr int kTile = 32;   // tokens of B and C in shared memory
constexpr int kBatch = 8;   // tokens of u, delta and z in registers
constexpr int kSms = 152;

template <int S>
struct Shape {
    static constexpr int SPT = S < 16 ? S : 16;   // states of a thread
    static constexpr int LPC = S / SPT;           // lanes of a channel
    static constexpr int CH = kThreads / LPC;     // channels of a block
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
template <typename T, int S, bool kOutputs>
__global__ void __launch_bounds__(kThreads, 4) scan_kernel(SsmScanParams p, SeqMap m, int run, Runs runs, bool split) {
    using Sh = Shape<S>;
    constexpr int SPT = Sh::SPT, LPC = Sh::LPC, CH = Sh::CH, H2 = SPT / 2;
    constexpr int VECS = kOutputs ? 2 : 1;  // B, and C
    constexpr int PER = kTile * S / kThreads;
    __shared__ TokenTile<kTile> tile;
    __shared__ __align__(16) float vec[2][VECS][kTile][S];

    const ChannelBlocks cb(p.C, p.G, CH);
    const int tid = threadIdx.x, lane = tid % LPC;
    const int g = cb.group(blockIdx.x), in_group = cb.in_group(blockIdx.x, CH) + tid / LPC;
    const bool on = in_group < cb.group_size;
    const int c = g * cb.group_size + (on ? in_group : 0);
    const int64_t cs = (int64_t)c * S + lane * SPT;

    f2 A2[H2], h[H2];
#pragma unroll
    for (int i = 0; i < H2; ++i) {
        A2[i] = pack(kLog2e * __ldg(p.A + cs + 2 * i), kLog2e * __ldg(p.A + cs + 2 * i + 1));
        h[i] = 0ull;
    }
    const float bias = p.bias ? __ldg(p.bias + c) : 0.f;
    const float Dc = kOutputs && p.D ? __ldg(p.D + c) : 0.f;
    const T* u = static_cast<const T*>(p.u) + c;
    const T* dl = static_cast<const T*>(p.delta) + c;
    const T* z = static_cast<const T*>(p.z) + c;
    T* y = static_cast<T*>(p.y) + c;
    const T* Bm = static_cast<const T*>(p.Bm) + g * S;
    const T* Cm = static_cast<const T*>(p.Cm) + g * S;

    auto load_state = [&](const float* from) {
#pragma unroll
        for (int i = 0; i < H2; i += 2) {
            const float4 v = *reinterpret_cast<const float4*>(from + 2 * i);
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
            *reinterpret_cast<float4*>(to + 2 * i) = v;
        }
    };
    auto begin_at = [&](int n) {
        if (p.initial) load_state(p.initial + (int64_t)n * p.C * S + cs);
        else
#pragma unroll
            for (int i = 0; i < H2; ++i) h[i] = 0ull;
    };

    // a sequence without tokens hands its state on
    if (kOutputs && p.final_state && on)
        for (int n = blockIdx.y; n < m.N; n += gridDim.y)
            if (m.end(n) <= m.begin(n)) {
                begin_at(n);
                store_state(p.final_state + (int64_t)n * p.C * S + cs);
            }
#pragma unroll
    for (int i = 0; i < H2; ++i) h[i] = 0ull;

    const int first = m.first(), last = m.last();
    const int r0 = blockIdx.y * run, r1 = (int)min((int64_t)m.total, (int64_t)r0 + run);
    float sum_d = 0.f;
    bool cut = false;

    // B and C of the tile at t0, element tid + k * kThreads of [token][state]
    float next[VECS][PER];
    auto request = [&](int t0) {
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            const int e = tid + k * kThreads, t = t0 + e / S;
            const bool in = t < r1;
            next[0][k] = in ? ld(Bm, t * p.ldb + e % S) : 0.f;
            if constexpr (VECS == 2) next[1][k] = in ? ld(Cm, t * p.ldc + e % S) : 0.f;
        }
    };
    request(r0);
    int until = r0;  // no boundary before this token
    for (int t0 = r0, buf = 0; t0 < r1; t0 += kTile, buf ^= 1) {
        // two buffers: a thread fills one while the others may still read the one before
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            const int e = tid + k * kThreads;
#pragma unroll
            for (int v = 0; v < VECS; ++v) vec[buf][v][e / S][e % S] = next[v][k];
        }
        __syncthreads();
        if (t0 + kTile < r1) request(t0 + kTile);
        bool plain = t0 + kTile < until && t0 > r0;
        const bool looked = !plain;
        if (looked) {
            tile.template build<kThreads>(m, t0);
            until = tile.until;
            plain = tile.plain;
            if (t0 == r0 && tile.carry >= 0 && kOutputs && split) load_state(runs.state + (int64_t)blockIdx.y * p.C * S + cs);
        }
        const int lo = max(t0, first), hi = min(min(t0 + kTile, r1), last);
        for (int t = lo; t < hi; t += kBatch) {
            T ru[kBatch], rd[kBatch], rz[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const int64_t at = min(t + i, hi - 1);
                ru[i] = __ldg(u + at * p.ldu);
                rd[i] = __ldg(dl + at * p.ldd);
                if (kOutputs && p.z) rz[i] = __ldg(z + at * p.ldz);
            }
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                if (t + i >= hi) break;
                const int k = t + i - t0;
                if (!plain) {
                    const int s = tile.start[k];
                    if (s >= 0) {
                        begin_at(s);
                        cut = true;
                    }
                }
                float d = to_f32<T>(rd[i]) + bias;
                if (p.softplus) d = softplus(d);
                const float uv = to_f32<T>(ru[i]), du = d * uv;
                if (!kOutputs) sum_d += d;
                const f2 dd = pack(d, d), du2 = pack(du, du);
                f2 y2 = 0ull;
                const ulonglong2* Bv = reinterpret_cast<const ulonglong2*>(&vec[buf][0][k][lane * SPT]);
                const ulonglong2* Cv = reinterpret_cast<const ulonglong2*>(&vec[buf][VECS - 1][k][lane * SPT]);
#pragma unroll
                for (int j = 0; j < H2 / 2; ++j) {
                    const ulonglong2 b = Bv[j];
                    h[2 * j] = fma2(ex2_2(mul2(dd, A2[2 * j])), h[2 * j], mul2(du2, b.x));
                    h[2 * j + 1] = fma2(ex2_2(mul2(dd, A2[2 * j + 1])), h[2 * j + 1], mul2(du2, b.y));
                    if (kOutputs) {
                        const ulonglong2 q = Cv[j];
                        y2 = fma2(h[2 * j], q.x, y2);
                        y2 = fma2(h[2 * j + 1], q.y, y2);
                    }
                }
                if (kOutputs) {
                    float o = sum2(y2);
#pragma unroll
                    for (int x = LPC / 2; x > 0; x >>= 1) o += __shfl_xor_sync(0xffffffffu, o, x);
                    o = fmaf(Dc, uv, o);
                    if (p.z) {
                        const float zv = to_f32<T>(rz[i]);
                        o *= zv * sigmoid(zv);
                    }
                    if (on && lane == 0) y[(int64_t)(t + i) * p.C] = from_f32<T>(o);
                    if (!plain && p.final_state) {
                        const int e = tile.end[k];
                        if (e >= 0 && on) store_state(p.final_state + (int64_t)e * p.C * S + cs);
                    }
                }
            }
        }
        if (looked) __syncthreads();  // the tile's boundaries may be looked up anew
    }
    if (!kOutputs && on) {
        store_state(runs.state + (int64_t)blockIdx.y * p.C * S + cs);
        if (lane == 0) runs.sum_d[(int64_t)blockIdx.y * p.C + c] = sum_d;
        if (blockIdx.x == 0 && tid == 0) runs.cut[blockIdx.y] = cut;
    }
}

// Start states of the runs from their end states, in place: one thread carries four states along.
__global__ void __launch_bounds__(128) scan_prefix_kernel(const float* A, Runs r, int runs, int C, int S) {
    const int64_t q = blockIdx.x * 128ll + threadIdx.x, quads = (int64_t)C * S / 4;
    if (q >= quads) return;
    const int c = (int)(q * 4 / S);
    float4 a = reinterpret_cast<const float4*>(A)[q];
    a.x *= kLog2e; a.y *= kLog2e; a.z *= kLog2e; a.w *= kLog2e;
    float4 h = make_float4(0.f, 0.f, 0.f, 0.f);
    float4* st = reinterpret_cast<float4*>(r.state) + q;
    constexpr int kAhead = 8;
    for (int j0 = 0; j0 < runs; j0 += kAhead) {
        float4 e[kAhead];
        float d[kAhead];
        int cut[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int j = min(j0 + k, runs - 1);
            e[k] = st[j * quads];
            d[k] = r.sum_d[(int64_t)j * C + c];
            cut[k] = r.cut[j];
        }
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            if (j0 + k >= runs) break;
            st[(j0 + k) * quads] = h;
            if (cut[k]) {
                h = e[k];
            } else {
                h.x = fmaf(ex2(d[k] * a.x), h.x, e[k].x);
                h.y = fmaf(ex2(d[k] * a.y), h.y, e[k].y);
                h.z = fmaf(ex2(d[k] * a.z), h.z, e[k].z);
                h.w = fmaf(ex2(d[k] * a.w), h.w, e[k].w);
            }
        }
    }
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
    const int want = (4 * kSms + q.blocks - 1) / q.blocks;
    int run = (p.total + want - 1) / want;
    run = (run + kTile - 1) / kTile * kTile;
    if (run < 64) run = 64;
    q.run = run;
    q.runs = p.total > 0 ? (p.total + run - 1) / run : 1;
    q.split = q.runs > 1;
    return q;
}

template <typename T, int S>
cudaError_t launch(const SsmScanParams& p, cudaStream_t st) {
    const Plan q = plan(p);
    const SeqMap m{p.cu, p.N, p.T, p.total};
    const dim3 grid(q.blocks, q.runs);
    Runs r{};
    if (q.split) {
        r = runs_at(p.ws, q.runs, p.C, S);
        scan_kernel<T, S, false><<<grid, kThreads, 0, st>>>(p, m, q.run, r, true);
        cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
        const int64_t quads = (int64_t)p.C * S / 4;
        scan_prefix_kernel<<<(unsigned)((quads + 127) / 128), 128, 0, st>>>(p.A, r, q.runs, p.C, S);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
    scan_kernel<T, S, true><<<grid, kThreads, 0, st>>>(p, m, q.run, r, q.split);
    return cudaGetLastError();
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
