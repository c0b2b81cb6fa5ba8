// Group norm with an activation, channels last, over the tokens of a sequence and a group's channels (the formulas stand in
// kda_group_norm.cuh).
//
// The statistics of a whole sequence come before its first output, so x (and dy) are read twice: by a pass over runs of tokens that
// leaves partial sums a channel, and by the pass that writes.  Runs are cut at fixed places of the token stream; a run and a sequence that meet
// make a piece, and piece (run + sequence) has a place of its own in the scratch.  Sums are joined in a fixed order.  Variances:
// the mean of a batch of 4 to 16 rows and the squares around it, joined with those of the rows before (and so on up), so that neither a mean far from zero nor a
// first token far from the others costs digits.
// 8 x 4096 x 512 bf16 in 32 groups: 23 us forwards (44% of the bytes at the copy rate: x is read a second time, most of it from L2, and three
// kernels follow one another), 2 x 2048 x 4096 in 32 groups 40 us backwards (38%).
#include "kda_group_norm.cuh"

namespace kda {

namespace {

constexpr int kThreads = 256;
constexpr int kPieces = 32;                   // row pieces of a block, side by side
constexpr int kSubs = kThreads / kPieces;     // rows of a block at a time
constexpr int kDeclared = 16 * 1024;          // shared memory that a kernel declares, at most
constexpr int kBatches = 3;                   // batches of a thread's rows under way, the one at hand among them

struct Cut {
    int run, runs;
};
// Runs of tokens, whole batches: one filling of the machine by `resident` blocks an SM, 64 tokens at least.  Where channels alone are a
// third of it or more, up to eight runs in the number of fillings that leaves the least idle (4478 x 4979 backwards, 156 blocks: seven runs in four
// fillings, one in one).
Cut cut_of(const NormParams& p, int blocks, int resident) {
    Cut q;
    const int places = kSms * resident;
    int want = places / blocks;
    if (want < 1) want = 1;
    if (want < 3) {
        auto fillings = [&](int n) { return ((int64_t)blocks * n + places - 1) / places; };
        for (int n = want + 1; n <= 8; ++n)
            if (fillings(n) * want < fillings(want) * n) want = n;
    }
    q.run = p.total / want + (p.total % want != 0);
    q.run = (q.run + 31) / 32 * 32;
    if (q.run < 64) q.run = 64;
    q.runs = p.total / q.run + (p.total % q.run != 0);
    if (q.runs < 1) q.runs = 1;
    return q;
}

// The sequences that meet tokens [r0, r1) one after another: f(n, first token, one behind the last).  Whole warps call it.
template <typename F>
__device__ __forceinline__ void each_piece(const SeqMap& m, int r0, int r1, F f) {
    int n = max(m.begun_before(r0 + 1) - 1, 0);
    for (; n < m.N; ++n) {
        const int s = m.begin(n);
        if (s >= r1) break;
        const int b = max(s, r0), e = min(m.end(n), r1);
        if (b < e) f(n, b, e);
    }
}

template <int VEC>
struct ChannelSums {
    static constexpr int N2 = (VEC + 1) / 2;
    f2 a[N2], b[N2];
};
// Adds the block's rows of sums together (in the order of the rows) and stores them, [2][C] at `to`.
template <int VEC>
__device__ __forceinline__ void store_sums(const ChannelSums<VEC>& s, f2 (*join)[kThreads], float* to, int C, int c, bool on) {
    constexpr int N2 = ChannelSums<VEC>::N2;
#pragma unroll
    for (int v = 0; v < 2; ++v) {
        __syncthreads();
#pragma unroll
        for (int e = 0; e < N2; ++e) join[e][threadIdx.x] = v ? s.b[e] : s.a[e];
        __syncthreads();
        if (threadIdx.x < kPieces && on) {
#pragma unroll
            for (int e = 0; e < N2; ++e) {
                f2 t = join[e][threadIdx.x];
                for (int r = 1; r < kSubs; ++r) t = add2(t, join[e][threadIdx.x + r * kPieces]);
                float x, y;
                unpack(t, x, y);
                to[(int64_t)v * C + c + 2 * e] = x;
                if (2 * e + 1 < VEC) to[(int64_t)v * C + c + 2 * e + 1] = y;
            }
        }
    }
}

__device__ __forceinline__ f2 low_halves(f2 x, f2 y) {
    float a, b, none;
    unpack(x, a, none);
    unpack(y, b, none);
    return pack(a, b);
}
// Rows of a thread's batch: more where pieces are small.
template <int VEC>
constexpr int kFwdRows = VEC == 1 ? 16 : VEC == 2 ? 8 : 4;
template <int VEC>
constexpr int kBwdRows = VEC == 1 ? 16 : VEC == 2 ? 8 : 2;

// A thread's own pieces of batches of ROWS rows (every kSubs-th token), on their way through shared memory: what a thread asks for it
// alone reads, so that no thread waits for another.  (Two-byte pieces have no asynchronous copy: a batch is loaded when asked for, all of it
// at once and none of it conditionally.)
template <typename T, int VEC, int ROWS>
struct Ring {
    static constexpr int kBytes = kBatches * ROWS * kThreads * VEC * (int)sizeof(T);
    T* mine;
    __device__ __forceinline__ explicit Ring(void* shared) : mine(static_cast<T*>(shared) + threadIdx.x * VEC) {}
    __device__ __forceinline__ T* at(int batch, int j) const { return mine + ((batch % kBatches) * ROWS + j) * kThreads * VEC; }
    // `left` rows are there from `from` on, ld apart.
    __device__ __forceinline__ void request(int batch, int left, const T* from, int64_t ld) const {
        if constexpr (VEC * sizeof(T) < 4) {
            T v[ROWS];
#pragma unroll
            for (int j = 0; j < ROWS; ++j) v[j] = from[min(j, (left - 1) / kSubs) * kSubs * ld];
#pragma unroll
            for (int j = 0; j < ROWS; ++j) *at(batch, j) = v[j];
            return;
        }
#pragma unroll
        for (int j = 0; j < ROWS; ++j, from += kSubs * ld)
            if (j * kSubs < left) Row<T, VEC>::copy_async(at(batch, j), from);
    }
    __device__ __forceinline__ void take(int batch, int j, f2 (&v)[(VEC + 1) / 2]) const {
        Row<T, VEC> r;
        r.from_shared(at(batch, j));
        r.to(v);
    }
    // Row j in pairs of channels, or (VEC = 1) rows j and j + 1 of one channel as a pair, zero where there is no second (two).
    static constexpr int PER = VEC == 1 ? 2 : 1;
    __device__ __forceinline__ void take_rows(int batch, int j, bool two, f2 (&v)[(VEC + 1) / 2]) const {
        take(batch, j, v);
        if constexpr (VEC == 1) {
            f2 more[1] = {0ull};
            if (two) take(batch, j + 1, more);
            v[0] = low_halves(v[0], more[0]);
        }
    }
};
// Stores what take_rows' pairs became, the second row `next` elements behind the first.
template <int VEC, typename T>
__device__ __forceinline__ void store_rows(T* to, int64_t next, bool two, const f2 (&v)[(VEC + 1) / 2]) {
    if constexpr (VEC == 1) {
        float a, b;
        unpack(v[0], a, b);
        to[0] = from_f32<T>(a);
        if (two) to[next] = from_f32<T>(b);
    } else {
        Row<T, VEC> out;
        out.from(v);
        out.store(to);
    }
}
// One of the weights of a thread's channels for take_rows' pairs.
template <int VEC>
__device__ __forceinline__ void weights_of(const float* p, float none, f2 (&v)[(VEC + 1) / 2]) {
    vec_pairs<VEC>(p, none, v);
    if constexpr (VEC == 1) v[0] = low_halves(v[0], v[0]);
}
// Walks a thread's rows b + sub, + kSubs ... before e: request(batch, first token of it) asks for a batch, f(batch, first token) has it.
template <int ROWS, typename Q, typename F>
__device__ __forceinline__ void each_batch(int b, int e, Q request, F f) {
    constexpr int STEP = ROWS * kSubs;
#pragma unroll
    for (int i = 0; i < kBatches - 1; ++i) {
        if (b + i * STEP < e) request(i, b + i * STEP);
        copies_commit();
    }
    int i = 0;
    for (int t = b; t < e; t += STEP, ++i) {
        copies_wait<kBatches - 2>();
        f(i, t);
        if (t + (kBatches - 1) * STEP < e) request(i + kBatches - 1, t + (kBatches - 1) * STEP);
        copies_commit();
    }
}

// n, mean and sum of squares around it, joined with those of nb more values (the same counts in both halves).
struct Moments {
    f2 mean, m2;
    __device__ __forceinline__ void join(float n, float nb, const Moments& b) {
        const float share = nb * rcp(n + nb);
        const f2 d = add2(b.mean, neg2(mean));
        mean = fma2(d, both(share), mean);
        m2 = fma2(mul2(d, d), both(n * share), add2(m2, b.m2));
    }
};

// Per piece and channel the mean and the sum of squares around it: pieces[run + n][2][C].
template <typename T, int VEC>
__global__ void __launch_bounds__(kThreads, 3) seq_moments_kernel(NormParams p, SeqMap m, int run, float* pieces) {
    constexpr int N2 = (VEC + 1) / 2;
    constexpr int ROWS = kFwdRows<VEC>;
    extern __shared__ __align__(16) char shared[];
    __shared__ Moments join[N2][kThreads];
    static_assert(sizeof(join) <= kDeclared, "what a launch allows for");
    const Ring<T, VEC, ROWS> ring(shared);
    const int piece = threadIdx.x % kPieces, sub = threadIdx.x / kPieces, c = (blockIdx.x * kPieces + piece) * VEC;
    const bool on = c < p.C;
    const int r0 = blockIdx.y * run, r1 = (int)min((int64_t)m.total, (int64_t)r0 + run);
    const T* const x = static_cast<const T*>(p.x) + (on ? c : 0);
    each_piece(m, r0, r1, [&](int n, int b, int e) {
        Moments mine[N2];
#pragma unroll
        for (int i = 0; i < N2; ++i) mine[i] = Moments{0ull, 0ull};
        float seen = 0.f;
        each_batch<ROWS>(b + sub, e, [&](int batch, int t) { ring.request(batch, e - t, x + t * p.ldx, p.ldx); }, [&](int batch, int t) {
            const int have = min(ROWS, (e - t + kSubs - 1) / kSubs);
            const float inv = have == ROWS ? 1.f / ROWS : 1.f / (float)have;
            f2 v[ROWS][N2];
#pragma unroll
            for (int j = 0; j < ROWS; ++j) ring.take(batch, j < have ? j : 0, v[j]);
#pragma unroll
            for (int i = 0; i < N2; ++i) {
                Moments few{0ull, 0ull};
                if (have == ROWS) {
                    f2 sum[ROWS / 2];
#pragma unroll
                    for (int j = 0; j < ROWS / 2; ++j) sum[j] = add2(v[2 * j][i], v[2 * j + 1][i]);
#pragma unroll
                    for (int half = ROWS / 4; half > 0; half /= 2)
#pragma unroll
                        for (int j = 0; j < half; ++j) sum[j] = add2(sum[2 * j], sum[2 * j + 1]);
                    few.mean = mul2(sum[0], both(inv));
#pragma unroll
                    for (int j = 0; j < ROWS; ++j) {
                        const f2 d = add2(v[j][i], neg2(few.mean));
                        few.m2 = fma2(d, d, few.m2);
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < ROWS; ++j)
                        if (j < have) few.mean = add2(few.mean, v[j][i]);
                    few.mean = mul2(few.mean, both(inv));
#pragma unroll
                    for (int j = 0; j < ROWS; ++j) {
                        const f2 d = add2(v[j][i], neg2(few.mean));
                        if (j < have) few.m2 = fma2(d, d, few.m2);
                    }
                }
                mine[i].join(seen, (float)have, few);
            }
            seen += (float)have;
        });
        __syncthreads();
#pragma unroll
        for (int i = 0; i < N2; ++i) join[i][threadIdx.x] = mine[i];
        __syncthreads();
        // a thread joins the rows of a pair of channels
        float* const to = pieces + (int64_t)(blockIdx.y + n) * 2 * p.C + blockIdx.x * kPieces * VEC;
        for (int k = threadIdx.x; k < kPieces * N2; k += kThreads) {
            const int i = k / kPieces, pc = k % kPieces, at = pc * VEC + 2 * i;
            if (blockIdx.x * kPieces * VEC + pc * VEC >= p.C) continue;
            Moments all = join[i][pc];
            float count = (float)((e - b + kSubs - 1) / kSubs);
            for (int r = 1; r < kSubs && b + r < e; ++r) {
                const float more = (float)((e - b - r + kSubs - 1) / kSubs);
                all.join(count, more, join[i][pc + r * kPieces]);
                count += more;
            }
            float x0, x1, q0, q1;
            unpack(all.mean, x0, x1);
            unpack(all.m2, q0, q1);
            to[at] = x0;
            to[p.C + at] = q0;
            if (2 * i + 1 < VEC) {
                to[at + 1] = x1;
                to[p.C + at + 1] = q1;
            }
        }
    });
}

// Sums of `v` over the block's threads, in a fixed order; everyone gets it.
__device__ __forceinline__ float block_sum(float v, float* buf) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    __syncthreads();
    if (threadIdx.x % 32 == 0) buf[threadIdx.x / 32] = v;
    __syncthreads();
    v = 0.f;
    for (int k = 0; k < (int)blockDim.x / 32; ++k) v += buf[k];
    return v;
}

// The pieces of a sequence: those of the runs from its first token's to its last one's.
struct PieceRange {
    int n, b, e, run, first, count;
    __device__ __forceinline__ PieceRange(const SeqMap& m, int n, int run) : n(n), b(m.begin(n)), e(m.end(n)), run(run) {
        first = b / run;
        count = e > b ? (e - 1) / run - first + 1 : 0;
    }
    __device__ __forceinline__ int64_t place(int k) const { return (int64_t)(first + k) + n; }
    __device__ __forceinline__ int tokens(int k) const {
        const int64_t r0 = (int64_t)(first + k) * run;
        return (int)(min((int64_t)e, r0 + run) - max((int64_t)b, r0));
    }
};

// mean and 1 / deviation of every sequence and group from the pieces: stats [N][G][2], a block each in turn.
template <int NTH>
__global__ void __launch_bounds__(NTH) seq_stats_kernel(NormParams p, SeqMap m, int run, const float* pieces, float* stats) {
    constexpr int kKept = 8;  // pairs of a piece's mean and squares that a thread keeps between the two sums
    __shared__ float buf[NTH / 32];
    const int cg = p.C / p.G;
    tc::grid_dep_wait();
    for (int64_t i = blockIdx.x; i < (int64_t)p.N * p.G; i += gridDim.x) {
        const int n = (int)(i / p.G), g = (int)(i - (int64_t)n * p.G);
        const PieceRange r(m, n, run);
        if (r.count == 0) {
            if (threadIdx.x == 0) stats[2 * i] = 0.f, stats[2 * i + 1] = rsqrtf(p.eps);
            continue;
        }
        const float* const at = pieces + g * cg;
        const int all = r.count * cg;
        const float inv = 1.f / ((float)(r.e - r.b) * (float)cg);
        auto entry = [&](int k, float& tokens, float& mean, float& m2) {
            const int piece = k / cg;
            const float* const x = at + r.place(piece) * 2 * p.C + (k - piece * cg);
            tokens = (float)r.tokens(piece);
            mean = x[0];
            m2 = x[p.C];
        };
        float tk[kKept], mk[kKept], qk[kKept], s = 0.f, q = 0.f;
#pragma unroll
        for (int j = 0; j < kKept; ++j) {
            const int k = threadIdx.x + j * NTH;
            if (k < all) entry(k, tk[j], mk[j], qk[j]);
            else tk[j] = mk[j] = qk[j] = 0.f;
        }
#pragma unroll
        for (int j = 0; j < kKept; ++j) s = fmaf(tk[j], mk[j], s);
#pragma unroll 4
        for (int k = threadIdx.x + kKept * NTH; k < all; k += NTH) {
            float t, x, m2;
            entry(k, t, x, m2);
            s = fmaf(t, x, s);
        }
        const float mean = block_sum(s, buf) * inv;
#pragma unroll
        for (int j = 0; j < kKept; ++j) {
            const float d = mk[j] - mean;
            q += fmaf(tk[j] * d, d, qk[j]);
        }
#pragma unroll 4
        for (int k = threadIdx.x + kKept * NTH; k < all; k += NTH) {
            float t, x, m2;
            entry(k, t, x, m2);
            q += fmaf(t * (x - mean), x - mean, m2);
        }
        const float var = block_sum(q, buf) * inv;
        if (threadIdx.x == 0) stats[2 * i] = mean, stats[2 * i + 1] = rsqrtf(var + p.eps);
    }
    tc::grid_dep_launch();
}

// Mean (negated) and 1 / deviation of a thread's channels in sequence n.
template <int VEC>
__device__ __forceinline__ void stats_of(const NormParams& p, const float* stats, int n, int c, f2 (&mean)[(VEC + 1) / 2], f2 (&rstd)[(VEC + 1) / 2]) {
    const int cg = p.C / p.G;
    const float2* const at = reinterpret_cast<const float2*>(stats) + (int64_t)n * p.G;
#pragma unroll
    for (int i = 0; i < (VEC + 1) / 2; ++i) {
        const float2 a = at[(c + 2 * i) / cg], b = VEC > 1 ? at[(c + 2 * i + 1) / cg] : a;
        mean[i] = pack(-a.x, -b.x);
        rstd[i] = pack(a.y, b.y);
    }
}

template <typename T, int VEC>
__global__ void __launch_bounds__(kThreads, 3) seq_apply_kernel(NormParams p, SeqMap m, int run, const float* stats) {
    constexpr int N2 = (VEC + 1) / 2, ROWS = kFwdRows<VEC>;
    extern __shared__ __align__(16) char shared[];
    const Ring<T, VEC, ROWS> ring(shared);
    const int piece = threadIdx.x % kPieces, sub = threadIdx.x / kPieces, c = (blockIdx.x * kPieces + piece) * VEC;
    const bool on = c < p.C;
    const int64_t next = (int64_t)kSubs * p.C;
    // the last runs first: they were read last
    const int r0 = (gridDim.y - 1 - blockIdx.y) * run, r1 = (int)min((int64_t)m.total, (int64_t)r0 + run);
    f2 w[N2], bias[N2];
    weights_of<VEC>(on && p.weight ? p.weight + c : nullptr, 1.f, w);
    weights_of<VEC>(on && p.bias ? p.bias + c : nullptr, 0.f, bias);
    tc::grid_dep_wait();
    each_piece(m, r0, r1, [&](int n, int b, int e) {
        if (!on) return;
        f2 mean[N2], scale[N2];
        stats_of<VEC>(p, stats, n, c, mean, scale);
#pragma unroll
        for (int i = 0; i < N2; ++i) scale[i] = mul2(scale[i], w[i]);
        const T* const x = static_cast<const T*>(p.x) + c;
        each_batch<ROWS>(b + sub, e, [&](int batch, int t) { ring.request(batch, e - t, x + t * p.ldx, p.ldx); }, [&](int batch, int t) {
            T* to = static_cast<T*>(p.y) + (int64_t)t * p.C + c;
#pragma unroll
            for (int j = 0; j < ROWS; j += ring.PER, to += ring.PER * next) {
                if (t + j * kSubs >= e) break;
                const bool two = t + (j + 1) * kSubs < e;
                f2 v[N2];
                ring.take_rows(batch, j, two, v);
#pragma unroll
                for (int i = 0; i < N2; ++i) v[i] = fma2(add2(v[i], mean[i]), scale[i], bias[i]);
                if (p.act) {
#pragma unroll
                    for (int i = 0; i < N2; ++i) v[i] = silu2(v[i]);
                }
                store_rows<VEC>(to, next, two, v);
            }
        });
    });
}

// Per piece and channel sum dp xh and sum dp, and the same per run: pieces[run + n][2][C], per_run[run][2][C].
template <typename T, typename TG, int VEC>
__global__ void __launch_bounds__(kThreads, 2) seq_grads_kernel(NormParams p, SeqMap m, int run, const float* stats, float* pieces, float* per_run) {
    constexpr int N2 = (VEC + 1) / 2, ROWS = kBwdRows<VEC>;
    extern __shared__ __align__(16) char shared[];
    const Ring<T, VEC, ROWS> ring(shared);
    const Ring<TG, VEC, ROWS> ring_dy(shared + ring.kBytes);
    __shared__ f2 join[N2][kThreads];
    static_assert(sizeof(join) <= kDeclared, "what a launch allows for");
    const int piece = threadIdx.x % kPieces, sub = threadIdx.x / kPieces, c = (blockIdx.x * kPieces + piece) * VEC;
    const bool on = c < p.C;
    const int cc = on ? c : 0;
    const int r0 = blockIdx.y * run, r1 = (int)min((int64_t)m.total, (int64_t)r0 + run);
    f2 w[N2], bias[N2];
    weights_of<VEC>(p.weight ? p.weight + cc : nullptr, 1.f, w);
    weights_of<VEC>(p.bias ? p.bias + cc : nullptr, 0.f, bias);
    ChannelSums<VEC> all;
#pragma unroll
    for (int i = 0; i < N2; ++i) all.a[i] = all.b[i] = 0ull;
    tc::grid_dep_wait();
    each_piece(m, r0, r1, [&](int n, int b, int e) {
        f2 mean[N2], rstd[N2];
        stats_of<VEC>(p, stats, n, cc, mean, rstd);
        ChannelSums<VEC> s;
#pragma unroll
        for (int i = 0; i < N2; ++i) s.a[i] = s.b[i] = 0ull;
        const T* const x = static_cast<const T*>(p.x) + cc;
        const TG* const dy = static_cast<const TG*>(p.dy) + cc;
        each_batch<ROWS>(b + sub, e, [&](int batch, int t) {
            ring.request(batch, e - t, x + t * p.ldx, p.ldx);
            ring_dy.request(batch, e - t, dy + (int64_t)t * p.C, p.C);
        }, [&](int batch, int t) {
#pragma unroll
            for (int j = 0; j < ROWS; j += ring.PER) {
                if (t + j * kSubs >= e) break;
                const bool two = t + (j + 1) * kSubs < e;
                f2 v[N2], g[N2];
                ring.take_rows(batch, j, two, v);
                ring_dy.take_rows(batch, j, two, g);
#pragma unroll
                for (int i = 0; i < N2; ++i) v[i] = mul2(add2(v[i], mean[i]), rstd[i]);
                if (p.act) {
#pragma unroll
                    for (int i = 0; i < N2; ++i) g[i] = mul2(g[i], silu_slope2(fma2(v[i], w[i], bias[i])));
                }
#pragma unroll
                for (int i = 0; i < N2; ++i) {
                    s.a[i] = fma2(g[i], v[i], s.a[i]);
                    s.b[i] = add2(s.b[i], g[i]);
                }
            }
        });
        if constexpr (VEC == 1) {
            s.a[0] = pack(sum2(s.a[0]), 0.f);
            s.b[0] = pack(sum2(s.b[0]), 0.f);
        }
#pragma unroll
        for (int i = 0; i < N2; ++i) {
            all.a[i] = add2(all.a[i], s.a[i]);
            all.b[i] = add2(all.b[i], s.b[i]);
        }
        store_sums<VEC>(s, join, pieces + (int64_t)(blockIdx.y + n) * 2 * p.C, p.C, c, on);
    });
    store_sums<VEC>(all, join, per_run + (int64_t)blockIdx.y * 2 * p.C, p.C, c, on);
    tc::grid_dep_launch();
}

// Blocks [0, weight_blocks): dweight and dbias.  The others: mean(q xh) and mean(q) of every sequence and group, means [N][G][2].
template <int NTH>
__global__ void __launch_bounds__(NTH) seq_means_kernel(NormParams p, SeqMap m, int run, int runs, const float* pieces, const float* per_run,
                                                        int weight_blocks, float* means) {
    __shared__ float buf[NTH / 32];
    tc::grid_dep_wait();
    if ((int)blockIdx.x < weight_blocks) {
        if (threadIdx.x < 256) norm_weight_sums(per_run, runs, p.C, p.dweight, p.dbias, blockIdx.x);
        tc::grid_dep_launch();
        return;
    }
    const int cg = p.C / p.G;
    for (int64_t i = blockIdx.x - weight_blocks; i < (int64_t)p.N * p.G; i += gridDim.x - weight_blocks) {
        const int n = (int)(i / p.G), g = (int)(i - (int64_t)n * p.G);
        const PieceRange r(m, n, run);
        const float* const at = pieces + g * cg;
        const int all = r.count * cg;
        float a = 0.f, b = 0.f;
#pragma unroll 4
        for (int k = threadIdx.x; k < all; k += NTH) {
            const int piece = k / cg, ch = k - piece * cg;
            const float* const x = at + r.place(piece) * 2 * p.C + ch;
            const float w = p.weight ? __ldg(p.weight + g * cg + ch) : 1.f;
            a = fmaf(w, x[0], a);
            b = fmaf(w, x[p.C], b);
        }
        a = block_sum(a, buf);
        b = block_sum(b, buf);
        const float inv = r.count > 0 ? 1.f / ((float)(r.e - r.b) * (float)cg) : 0.f;
        if (threadIdx.x == 0) means[2 * i] = a * inv, means[2 * i + 1] = b * inv;
    }
    tc::grid_dep_launch();
}

template <typename T, typename TG, int VEC>
__global__ void __launch_bounds__(kThreads, 2) seq_dx_kernel(NormParams p, SeqMap m, int run, const float* stats, const float* means) {
    constexpr int N2 = (VEC + 1) / 2, ROWS = kBwdRows<VEC>;
    extern __shared__ __align__(16) char shared[];
    const Ring<T, VEC, ROWS> ring(shared);
    const Ring<TG, VEC, ROWS> ring_dy(shared + ring.kBytes);
    const int piece = threadIdx.x % kPieces, sub = threadIdx.x / kPieces, c = (blockIdx.x * kPieces + piece) * VEC;
    const bool on = c < p.C;
    const int r0 = (gridDim.y - 1 - blockIdx.y) * run, r1 = (int)min((int64_t)m.total, (int64_t)r0 + run);
    const int64_t next = (int64_t)kSubs * p.C;
    f2 w[N2], bias[N2];
    weights_of<VEC>(on && p.weight ? p.weight + c : nullptr, 1.f, w);
    weights_of<VEC>(on && p.bias ? p.bias + c : nullptr, 0.f, bias);
    tc::grid_dep_wait();
    if (on) {  // rows of no sequence: zeros
        const int first = m.first(), last = m.last();
        Row<TG, VEC> zero;
        zero.zero();
        for (int t = r0 + sub; t < r1; t += kSubs)
            if (t < first || t >= last) zero.store(static_cast<TG*>(p.dx) + (int64_t)t * p.C + c);
    }
    each_piece(m, r0, r1, [&](int n, int b, int e) {
        if (!on) return;
        f2 mean[N2], rstd[N2], mqx[N2], mq[N2];
        stats_of<VEC>(p, stats, n, c, mean, rstd);
        stats_of<VEC>(p, means, n, c, mqx, mq);  // -mean(q xh), mean(q)
        const T* const x = static_cast<const T*>(p.x) + c;
        const TG* const dy = static_cast<const TG*>(p.dy) + c;
        each_batch<ROWS>(b + sub, e, [&](int batch, int t) {
            ring.request(batch, e - t, x + t * p.ldx, p.ldx);
            ring_dy.request(batch, e - t, dy + (int64_t)t * p.C, p.C);
        }, [&](int batch, int t) {
            TG* to = static_cast<TG*>(p.dx) + (int64_t)t * p.C + c;
#pragma unroll
            for (int j = 0; j < ROWS; j += ring.PER, to += ring.PER * next) {
                if (t + j * kSubs >= e) break;
                const bool two = t + (j + 1) * kSubs < e;
                f2 v[N2], g[N2];
                ring.take_rows(batch, j, two, v);
                ring_dy.take_rows(batch, j, two, g);
#pragma unroll
                for (int i = 0; i < N2; ++i) v[i] = mul2(add2(v[i], mean[i]), rstd[i]);
                if (p.act) {
#pragma unroll
                    for (int i = 0; i < N2; ++i) g[i] = mul2(g[i], silu_slope2(fma2(v[i], w[i], bias[i])));
                }
#pragma unroll
                for (int i = 0; i < N2; ++i) g[i] = mul2(rstd[i], fma2(v[i], mqx[i], fma2(g[i], w[i], neg2(mq[i]))));
                store_rows<VEC>(to, next, two, g);
            }
        });
    });
}

// ---- launches -------------------------------------------------------------------------------------------

constexpr int kFwdResident = 3, kBwdResident = 2;
int blocks_of(const NormParams& p, int vec) { return (p.C + kPieces * vec - 1) / (kPieces * vec); }
int64_t groups_grid(const NormParams& p) {
    const int64_t n = (int64_t)p.N * p.G;
    return n < 1 ? 1 : n < 8 * kSms ? n : 8 * kSms;
}
// Whether a sequence's pieces of a group are more than a small block keeps in registers (by the mean length of the sequences: one
// sequence, one group of 4096 channels in 19 runs takes 78,000 entries, and one block for it 130 us with 128 threads).
bool large_groups(const NormParams& p, const Cut& q) { return (int64_t)(q.runs / (p.N > 0 ? p.N : 1) + 1) * (p.C / p.G) > 1024; }
// Places of pieces at p's sizes, whichever variant runs.
int64_t most_runs(const NormParams& p) {
    int most = 0;
    for (const int vec : {1, 2, 4, 8})
        for (const int resident : {kFwdResident, kBwdResident}) {
            const int runs = cut_of(p, blocks_of(p, vec), resident).runs;
            if (runs > most) most = runs;
        }
    return most;
}
size_t pieces_bytes(const NormParams& p) { return (size_t)(((most_runs(p) + p.N) * 2 * p.C * 4 + 255) / 256 * 256); }
size_t per_run_bytes(const NormParams& p) { return (size_t)((most_runs(p) * 2 * p.C * 4 + 255) / 256 * 256); }
size_t stats_bytes(const NormParams& p) { return (size_t)(((int64_t)p.N * p.G * 8 + 255) / 256 * 256); }

template <typename T, int VEC>
cudaError_t launch_stats(const NormParams& p, const SeqMap& m, const Cut& q, float* pieces, float* stats, cudaStream_t st) {
    const auto kern = seq_moments_kernel<T, VEC>;
    constexpr int smem = Ring<T, VEC, kFwdRows<VEC>>::kBytes;
    static std::atomic<uint64_t> allowed;
    cudaError_t e = allow_shared(kern, kDeclared, smem, allowed);
    if (e != cudaSuccess) return e;
    kern<<<dim3(blocks_of(p, VEC), q.runs), kThreads, smem, st>>>(p, m, q.run, pieces);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    if (large_groups(p, q)) return tc::launch_dependent(seq_stats_kernel<1024>, (unsigned)groups_grid(p), 1024, 0, st, p, m, q.run, (const float*)pieces, stats);
    return tc::launch_dependent(seq_stats_kernel<128>, (unsigned)groups_grid(p), 128, 0, st, p, m, q.run, (const float*)pieces, stats);
}

template <typename T, int VEC>
cudaError_t launch_fwd(const NormParams& p, cudaStream_t st) {
    const SeqMap m{p.cu, p.N, p.T, p.total};
    const Cut q = cut_of(p, blocks_of(p, VEC), kFwdResident);
    char* const ws = static_cast<char*>(p.ws);
    float* const stats = p.stats ? p.stats : reinterpret_cast<float*>(ws + pieces_bytes(p));
    cudaError_t e = launch_stats<T, VEC>(p, m, q, reinterpret_cast<float*>(ws), stats, st);
    if (e != cudaSuccess) return e;
    const auto kern = seq_apply_kernel<T, VEC>;
    constexpr int smem = Ring<T, VEC, kFwdRows<VEC>>::kBytes;
    static std::atomic<uint64_t> allowed;
    if ((e = allow_shared(kern, 0, smem, allowed)) != cudaSuccess) return e;
    return tc::launch_dependent(kern, dim3(blocks_of(p, VEC), q.runs), kThreads, smem, st, p, m, q.run, (const float*)stats);
}

template <typename T, typename TG, int VEC>
cudaError_t launch_bwd(const NormParams& p, cudaStream_t st) {
    const SeqMap m{p.cu, p.N, p.T, p.total};
    const Cut q = cut_of(p, blocks_of(p, VEC), kBwdResident);
    char* at = static_cast<char*>(p.ws);
    float* const pieces = reinterpret_cast<float*>(at);
    float* const per_run = reinterpret_cast<float*>(at += pieces_bytes(p));
    float* const means = reinterpret_cast<float*>(at += per_run_bytes(p));
    float* stats = p.stats;
    if (!stats) {
        stats = reinterpret_cast<float*>(at + stats_bytes(p));
        const cudaError_t e = launch_stats<T, VEC>(p, m, q, pieces, stats, st);
        if (e != cudaSuccess) return e;
    }
    const dim3 grid(blocks_of(p, VEC), q.runs);
    const auto grads = seq_grads_kernel<T, TG, VEC>;
    const auto dx = seq_dx_kernel<T, TG, VEC>;
    constexpr int smem = Ring<T, VEC, kBwdRows<VEC>>::kBytes + Ring<TG, VEC, kBwdRows<VEC>>::kBytes;
    static std::atomic<uint64_t> grads_allowed, dx_allowed;
    cudaError_t e = allow_shared(grads, kDeclared, smem, grads_allowed);
    if (e == cudaSuccess) e = allow_shared(dx, 0, smem, dx_allowed);
    if (e != cudaSuccess) return e;
    if (p.stats) {  // the call's first kernel: it waits for whatever made its inputs
        grads<<<grid, kThreads, smem, st>>>(p, m, q.run, stats, pieces, per_run);
        e = cudaGetLastError();
    } else {
        e = tc::launch_dependent(grads, grid, kThreads, smem, st, p, m, q.run, (const float*)stats, pieces, per_run);
    }
    if (e != cudaSuccess) return e;
    const int weight_blocks = p.dweight || p.dbias ? (p.C + 31) / 32 : 0;
    const bool large = large_groups(p, q);
    e = tc::launch_dependent(large ? seq_means_kernel<1024> : seq_means_kernel<256>, (unsigned)(weight_blocks + groups_grid(p)), large ? 1024 : 256, 0, st, p, m,
                             q.run, q.runs, (const float*)pieces, (const float*)per_run, weight_blocks, means);
    if (e != cudaSuccess) return e;
    return tc::launch_dependent(dx, grid, kThreads, smem, st, p, m, q.run, (const float*)stats, (const float*)means);
}

}  // namespace

size_t group_norm_fwd_workspace(const NormParams& p) { return p.over_sequence ? pieces_bytes(p) + (p.stats ? 0 : stats_bytes(p)) : 0; }
size_t group_norm_bwd_workspace(const NormParams& p) {
    if (!p.over_sequence) return norm_token_bwd_workspace(p);
    return pieces_bytes(p) + per_run_bytes(p) + (p.stats ? 1 : 2) * stats_bytes(p);
}

cudaError_t group_norm_fwd(kda_dtype dt, const NormParams& p, cudaStream_t st) {
    if (!p.over_sequence) return norm_token_fwd(dt, p, st);
    using kda_host::rows_aligned;
    const int vec = dt == KDA_BF16 ? 8 : 4;
    const bool wide = p.C % vec == 0 && rows_aligned(p.x, p.ldx, vec) && rows_aligned(p.y, p.C, vec);
    const int es = dt == KDA_BF16 ? 2 : 4;
    const bool pairs = p.C % 2 == 0 && p.ldx % 2 == 0 && (uintptr_t)p.x % (2 * es) == 0 && (uintptr_t)p.y % (2 * es) == 0;
    if (dt == KDA_BF16) return wide ? launch_fwd<__nv_bfloat16, 8>(p, st) : pairs ? launch_fwd<__nv_bfloat16, 2>(p, st) : launch_fwd<__nv_bfloat16, 1>(p, st);
    return wide ? launch_fwd<float, 4>(p, st) : pairs ? launch_fwd<float, 2>(p, st) : launch_fwd<float, 1>(p, st);
}

cudaError_t group_norm_bwd(kda_dtype dt, kda_dtype gdt, const NormParams& p, cudaStream_t st) {
    if (!p.over_sequence) return norm_token_bwd(dt, gdt, p, st);
    using kda_host::rows_aligned;
    const int vec = dt == KDA_BF16 && gdt == KDA_BF16 ? 8 : 4;
    const bool wide = p.C % vec == 0 && rows_aligned(p.x, p.ldx, dt == KDA_BF16 ? 8 : 4) && rows_aligned(p.dy, p.C, vec) && rows_aligned(p.dx, p.C, vec);
    const int es = dt == KDA_BF16 ? 2 : 4, gs = gdt == KDA_BF16 ? 2 : 4;
    const bool pairs = p.C % 2 == 0 && p.ldx % 2 == 0 && (uintptr_t)p.x % (2 * es) == 0 && (uintptr_t)p.dy % (2 * gs) == 0 && (uintptr_t)p.dx % (2 * gs) == 0;
    if (dt == KDA_F32) return wide ? launch_bwd<float, float, 4>(p, st) : pairs ? launch_bwd<float, float, 2>(p, st) : launch_bwd<float, float, 1>(p, st);
    if (gdt == KDA_F32) {
        if (wide) return launch_bwd<__nv_bfloat16, float, 4>(p, st);
        return pairs ? launch_bwd<__nv_bfloat16, float, 2>(p, st) : launch_bwd<__nv_bfloat16, float, 1>(p, st);
    }
    if (wide) return launch_bwd<__nv_bfloat16, __nv_bfloat16, 8>(p, st);
    return pairs ? launch_bwd<__nv_bfloat16, __nv_bfloat16, 2>(p, st) : launch_bwd<__nv_bfloat16, __nv_bfloat16, 1>(p, st);
}

}  // namespace kda
