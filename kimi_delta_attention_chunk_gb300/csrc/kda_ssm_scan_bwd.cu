// Selective state space scan over prompts: backward.
//
// With the forward's d, a = exp(d A), h (per sequence, channel and state) and yb = dout silu(z):
//     dh_t = C_t yb_t + a_{t+1} dh_{t+1}   (behind the last token: the final state's gradient)
//     q1 = sum_s dh B,  q2 = sum_s dh a h_{t-1} A
//     du = d q1 + D yb,  dd = q2 + u q1,  ddelta = dd softplus'(delta + bias),  dbias = sum_t ddelta
//     dA += d dh a h_{t-1},  dB_t = sum_c d u dh,  dC_t = sum_c yb h,  dD = sum_t yb u
//     dz = dout (sum_s C h + D u) silu'(z),  dh0 = a_0 dh_0
// Both recurrences are cut at every 64th token of the stream:
//   1. one walk forwards over each chunk gives its end state from a zero start, the sum of its step
//      sizes, and what the chunk hands to the left (sum over its tokens of the decay since the chunk's
//      start times C yb), so both directions cost one exponential per token and state;
//   2. a prefix in each direction turns them into the state before and the gradient behind each chunk;
//   3. each chunk is walked forwards once more, keeping the state of every eighth token, then backwards
//      eight tokens at a time with their states and decays recomputed into registers.
// Sums over channels (dB, dC) go through a shuffle reduction that leaves one value a lane, the block's
// warps, and partial sums of the channel blocks; sums over tokens through partial sums of the chunks.
// Every sum has an order fixed by the sizes.  The fp32 units and shuffles bound step 3.
#include <stddef.h>

#include "kda_layer.h"
#include "kda_ssm.cuh"

namespace kda {

namespace {

constexpr int kChunk = 64;
constexpr int kBatch = 8;
constexpr int kBatches = kChunk / kBatch;

// Device scratch: per chunk and channel and state the end states (then start states, then dA's
// partial sums) and the gradients handed left (then those coming from the right); per chunk and
// channel the sums of d, and the partial sums of dD and dbias; per channel block, token and state the
// partial sums of dB and dC; per chunk kStarts and kThrough.
constexpr int kStarts = 1;   // a sequence begins in the chunk: its start state does not reach its end
constexpr int kThrough = 2;  // the sequence at its first token is the one behind its last
struct Scratch {
    float *state, *grad, *sum_d, *dD, *dbias, *dBC;
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
    s.sum_d = take(chunks * p.C);
    s.dD = take(chunks * p.C);
    s.dbias = take(chunks * p.C);
    s.dBC = take((int64_t)blocks * p.total * 2 * p.S);
    s.flags = reinterpret_cast<int*>(take(chunks));
    return n;
}

template <typename T>
__device__ __forceinline__ float step_size(const SsmScanParams& p, T raw, float bias) {
    const float d = to_f32<T>(raw) + bias;
    return p.softplus ? softplus(d) : d;
}

// ---- 1. what each chunk does on its own -------------------------------------------------------

constexpr int kSumThreads = 128;

template <typename T, typename TG, int S>
__global__ void __launch_bounds__(kSumThreads, 4) scan_bwd_sum_kernel(SsmScanParams p, SeqMap m, Scratch w) {
    constexpr int SPT = S < 16 ? S : 16, LPC = S / SPT, CH = kSumThreads / LPC, H2 = SPT / 2;
    __shared__ TokenTile<kChunk> tile;
    __shared__ __align__(16) float vec[2][kChunk][S];
    const ChannelBlocks cb(p.C, p.G, CH);
    const int tid = threadIdx.x, lane = tid % LPC;
    const int g = cb.group(blockIdx.x), in_group = cb.in_group(blockIdx.x, CH) + tid / LPC;
    const bool on = in_group < cb.group_size;
    const int c = g * cb.group_size + (on ? in_group : 0);
    const int64_t cs = (int64_t)c * S + lane * SPT;
    const int t0 = blockIdx.y * kChunk, t1 = min(m.total, t0 + kChunk);
    {
        const T* Bm = static_cast<const T*>(p.Bm) + g * S;
        const T* Cm = static_cast<const T*>(p.Cm) + g * S;
        for (int e = tid; e < (t1 - t0) * S; e += kSumThreads) {
            const int k = e / S, s = e % S;
            vec[0][k][s] = ld(Bm, (int64_t)(t0 + k) * p.ldb + s);
            vec[1][k][s] = ld(Cm, (int64_t)(t0 + k) * p.ldc + s);
        }
    }
    tile.template build<kSumThreads>(m, t0);
    const bool plain = tile.plain;
    f2 A2[H2], h[H2], P[H2], G[H2];
#pragma unroll
    for (int i = 0; i < H2; ++i) {
        A2[i] = pack(kLog2e * __ldg(p.A + cs + 2 * i), kLog2e * __ldg(p.A + cs + 2 * i + 1));
        h[i] = G[i] = 0ull;
        P[i] = pack(1.f, 1.f);
    }
    const float bias = p.bias ? __ldg(p.bias + c) : 0.f;
    const T* u = static_cast<const T*>(p.u) + c;
    const T* dl = static_cast<const T*>(p.delta) + c;
    const T* z = static_cast<const T*>(p.z) + c;
    const TG* dy = static_cast<const TG*>(p.dy) + c;
    bool carries = tile.carry >= 0, starts = false;
    float sum_d = 0.f;
    const int lo = max(t0, m.first()), hi = min(t1, m.last());
    for (int t = lo; t < hi; t += kBatch) {
        T ru[kBatch], rd[kBatch], rz[kBatch];
        TG rg[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int64_t at = min(t + i, hi - 1);
            ru[i] = __ldg(u + at * p.ldu);
            rd[i] = __ldg(dl + at * p.ldd);
            rg[i] = __ldg(dy + at * p.C);
            if (p.z) rz[i] = __ldg(z + at * p.ldz);
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            if (t + i >= hi) break;
            const int k = t + i - t0;
            if (!plain && tile.start[k] >= 0) {
                starts = true;
                const int64_t at = (int64_t)tile.start[k] * p.C * S + cs;
#pragma unroll
                for (int j = 0; j < H2; ++j)
                    h[j] = p.initial ? pack(__ldg(p.initial + at + 2 * j), __ldg(p.initial + at + 2 * j + 1)) : 0ull;
            }
            const float d = step_size<T>(p, rd[i], bias);
            sum_d += d;
            const float du = d * to_f32<T>(ru[i]);
            float yb = to_f32<TG>(rg[i]);
            if (p.z) {
                const float zv = to_f32<T>(rz[i]);
                yb *= zv * sigmoid(zv);
            }
            const f2 dd = pack(d, d), du2 = pack(du, du), yb2 = pack(yb, yb);
            const ulonglong2* Bv = reinterpret_cast<const ulonglong2*>(&vec[0][k][lane * SPT]);
            const ulonglong2* Cv = reinterpret_cast<const ulonglong2*>(&vec[1][k][lane * SPT]);
#pragma unroll
            for (int j = 0; j < H2; ++j) {
                const f2 b = (j & 1) ? Bv[j / 2].y : Bv[j / 2].x;
                const f2 a = ex2_2(mul2(dd, A2[j]));
                h[j] = fma2(a, h[j], mul2(du2, b));
                if (carries) {
                    const f2 q = (j & 1) ? Cv[j / 2].y : Cv[j / 2].x;
                    P[j] = mul2(P[j], a);
                    G[j] = fma2(P[j], mul2(yb2, q), G[j]);
                }
            }
            if (!plain && carries && tile.end[k] >= 0) {
                carries = false;
                if (p.dfinal) {
                    const int64_t at = (int64_t)tile.end[k] * p.C * S + cs;
#pragma unroll
                    for (int j = 0; j < H2; ++j)
                        G[j] = fma2(P[j], pack(__ldg(p.dfinal + at + 2 * j), __ldg(p.dfinal + at + 2 * j + 1)), G[j]);
                }
            }
        }
    }
    if (!on) return;
    const int64_t at = (int64_t)blockIdx.y * p.C * S + cs;
#pragma unroll
    for (int j = 0; j < H2; j += 2) {
        float4 v;
        unpack(h[j], v.x, v.y);
        unpack(h[j + 1], v.z, v.w);
        *reinterpret_cast<float4*>(w.state + at + 2 * j) = v;
        unpack(G[j], v.x, v.y);
        unpack(G[j + 1], v.z, v.w);
        *reinterpret_cast<float4*>(w.grad + at + 2 * j) = v;
    }
    if (lane == 0) w.sum_d[(int64_t)blockIdx.y * p.C + c] = sum_d;
    if (blockIdx.x == 0 && tid == 0) w.flags[blockIdx.y] = (starts ? kStarts : 0) | (carries ? kThrough : 0);
}

// ---- 2. the state before and the gradient behind each chunk -------------------------------------

__global__ void __launch_bounds__(128) scan_bwd_prefix_kernel(const float* A, Scratch w, int chunks, int C, int S) {
    const int64_t q = blockIdx.x * 128ll + threadIdx.x, quads = (int64_t)C * S / 4;
    if (q >= quads) return;
    const int c = (int)(q * 4 / S);
    float4 a = reinterpret_cast<const float4*>(A)[q];
    a.x *= kLog2e; a.y *= kLog2e; a.z *= kLog2e; a.w *= kLog2e;
    const bool back = blockIdx.y == 1;
    float4* io = reinterpret_cast<float4*>(back ? w.grad : w.state) + q;
    const int stop = back ? kThrough : kStarts;
    float4 h = make_float4(0.f, 0.f, 0.f, 0.f);
    constexpr int kAhead = 8;
    for (int j0 = 0; j0 < chunks; j0 += kAhead) {
        float4 e[kAhead];
        float d[kAhead];
        bool on[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int i = min(j0 + k, chunks - 1), j = back ? chunks - 1 - i : i;
            e[k] = io[j * quads];
            d[k] = w.sum_d[(int64_t)j * C + c];
            on[k] = ((w.flags[j] & stop) != 0) == back;
        }
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            if (j0 + k >= chunks) break;
            const int j = back ? chunks - 1 - (j0 + k) : j0 + k;
            io[j * quads] = h;
            if (on[k]) {
                h.x = fmaf(ex2(d[k] * a.x), h.x, e[k].x);
                h.y = fmaf(ex2(d[k] * a.y), h.y, e[k].y);
                h.z = fmaf(ex2(d[k] * a.z), h.z, e[k].z);
                h.w = fmaf(ex2(d[k] * a.w), h.w, e[k].w);
            } else {
                h = e[k];
            }
        }
    }
}

// ---- 3. the gradients --------------------------------------------------------------------------

// Four states a thread.  S = 8 takes half the threads so that its channels' rows still fit twice.
template <int S>
struct BwdShape {
    static constexpr int NT = S == 8 ? 128 : 256;
    static constexpr int LP = S / 4;           // lanes of a channel
    static constexpr int CH = NT / LP;         // channels of a block
    static constexpr int NCH = 32 / LP;        // channels of a warp
    static constexpr int NW = NT / 32;
    static constexpr int KEEP = NCH >= 8 ? 1 : 8 / NCH;  // sums of dB and dC that a lane is left with
};
template <int S>
struct BwdShared {
    using Sh = BwdShape<S>;
    float4 kept[kBatches][Sh::NT];
    alignas(16) float vec[2][kChunk][S];  // B, C, read four at a time
    float d[kChunk][Sh::CH];    // step sizes, then dd
    float u[kChunk][Sh::CH];    // inputs, then du
    float yb[kChunk][Sh::CH];   // output gradients behind the gate, then sum_s C h
    float red[Sh::NW][kBatch][2 * S];
    TokenTile<kChunk> tile;
};

static_assert(offsetof(BwdShared<8>, vec) % 16 == 0 && offsetof(BwdShared<16>, vec) % 16 == 0 &&
                  offsetof(BwdShared<32>, vec) % 16 == 0 && offsetof(BwdShared<64>, vec) % 16 == 0,
              "16-byte reads of B and C");

template <typename T, typename TG, int S>
__global__ void __launch_bounds__(BwdShape<S>::NT, 512 / BwdShape<S>::NT) scan_bwd_kernel(SsmScanParams p, SeqMap m, Scratch w) {
    using Sh = BwdShape<S>;
    constexpr int NT = Sh::NT, LP = Sh::LP, CH = Sh::CH;
    extern __shared__ __align__(16) char raw_smem[];
    BwdShared<S>& sh = *reinterpret_cast<BwdShared<S>*>(raw_smem);
    const ChannelBlocks cb(p.C, p.G, CH);
    const int tid = threadIdx.x, lane = tid % LP, ch = tid / LP;
    const int g = cb.group(blockIdx.x), base = cb.in_group(blockIdx.x, CH);
    const bool on = base + ch < cb.group_size;
    const int c = g * cb.group_size + (on ? base + ch : 0);
    const int64_t cs = (int64_t)c * S + lane * 4;
    const int t0 = blockIdx.y * kChunk, t1 = min(m.total, t0 + kChunk);
    const int first = m.first(), last = m.last();
    const int lo = max(t0, first), hi = min(t1, last);

    // inputs of the chunk: element tid + k * NT of [token][channel], so a thread keeps one channel
    const int ech = tid % CH;
    const bool eon = base + ech < cb.group_size;
    const int ec = g * cb.group_size + (eon ? base + ech : 0);
    const float ebias = p.bias ? __ldg(p.bias + ec) : 0.f;
    constexpr int ROWS = NT / CH, PER = kChunk / ROWS;
    const T* pu = static_cast<const T*>(p.u) + ec;
    const T* pd = static_cast<const T*>(p.delta) + ec;
    const T* pz = static_cast<const T*>(p.z) + ec;
    const TG* pg = static_cast<const TG*>(p.dy) + ec;
    float dD = 0.f;
#pragma unroll 8
    for (int k = 0; k < PER; ++k) {
        const int r = tid / CH + k * ROWS;
        const int64_t t = t0 + r;
        float d = 0.f, u = 0.f, yb = 0.f;
        if (eon && t >= lo && t < hi) {
            u = ld(pu, t * p.ldu);
            d = step_size<T>(p, __ldg(pd + t * p.ldd), ebias);
            yb = ld(pg, t * p.C);
            if (p.z) {
                const float zv = ld(pz, t * p.ldz);
                yb *= zv * sigmoid(zv);
            }
        }
        sh.d[r][ech] = d;
        sh.u[r][ech] = u;
        sh.yb[r][ech] = yb;
        dD = fmaf(yb, u, dD);
    }
    {
        const T* Bm = static_cast<const T*>(p.Bm) + g * S;
        const T* Cm = static_cast<const T*>(p.Cm) + g * S;
        for (int e = tid; e < (t1 - t0) * S; e += NT) {
            const int k = e / S, s = e % S;
            sh.vec[0][k][s] = ld(Bm, (int64_t)(t0 + k) * p.ldb + s);
            sh.vec[1][k][s] = ld(Cm, (int64_t)(t0 + k) * p.ldc + s);
        }
    }
    sh.tile.template build<NT>(m, t0);
    const bool plain = sh.tile.plain && hi - lo == kChunk;

    auto load4 = [&](const float* from, f2 (&v)[2]) {
        const float4 x = *reinterpret_cast<const float4*>(from);
        v[0] = pack(x.x, x.y);
        v[1] = pack(x.z, x.w);
    };
    auto as4 = [&](const f2 (&v)[2]) {
        float4 x;
        unpack(v[0], x.x, x.y);
        unpack(v[1], x.z, x.w);
        return x;
    };
    auto initial_of = [&](int n, f2 (&v)[2]) {
        if (p.initial) load4(p.initial + (int64_t)n * p.C * S + cs, v);
        else v[0] = v[1] = 0ull;
    };
    f2 A[2], A2[2], h[2];
    load4(p.A + cs, A);
    A2[0] = mul2(A[0], pack(kLog2e, kLog2e));
    A2[1] = mul2(A[1], pack(kLog2e, kLog2e));
    const int64_t slot = (int64_t)blockIdx.y * p.C * S + cs;
    // (a lane without a channel carries zeros: its products join the sums over channels)
    if (on && sh.tile.carry >= 0) load4(w.state + slot, h);
    else h[0] = h[1] = 0ull;

    // forwards: the state before every batch
    for (int b = 0; b < kBatches; ++b) {
        sh.kept[b][tid] = as4(h);
        if (b + 1 == kBatches) break;
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int k = b * kBatch + i;
            if (!plain) {
                if (t0 + k < lo || t0 + k >= hi) continue;
                if (sh.tile.start[k] >= 0) initial_of(sh.tile.start[k], h);
            }
            const float d = sh.d[k][ch], du = d * sh.u[k][ch];
            const f2 dd = pack(d, d), du2 = pack(du, du);
            const ulonglong2 B = *reinterpret_cast<const ulonglong2*>(&sh.vec[0][k][lane * 4]);
            h[0] = fma2(ex2_2(mul2(dd, A2[0])), h[0], mul2(du2, B.x));
            h[1] = fma2(ex2_2(mul2(dd, A2[1])), h[1], mul2(du2, B.y));
        }
    }

    // backwards
    f2 carry[2], dA[2] = {0ull, 0ull};  // gradient of the state behind the token at hand
    if (on) load4(w.grad + slot, carry);
    else carry[0] = carry[1] = 0ull;
    const float Dc = p.D ? __ldg(p.D + c) : 0.f;
    for (int b = kBatches - 1; b >= 0; --b) {
        if (t0 + b * kBatch >= hi || t0 + (b + 1) * kBatch <= lo) continue;
        f2 hs[kBatch][2], as[kBatch][2], before[2];
        {
            const float4 x = sh.kept[b][tid];
            before[0] = pack(x.x, x.y);
            before[1] = pack(x.z, x.w);
        }
        h[0] = before[0];
        h[1] = before[1];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int k = b * kBatch + i;
            as[i][0] = as[i][1] = 0ull;
            if (plain || (t0 + k >= lo && t0 + k < hi)) {
                if (!plain && sh.tile.start[k] >= 0) initial_of(sh.tile.start[k], h);
                const float d = sh.d[k][ch], du = d * sh.u[k][ch];
                const f2 dd = pack(d, d), du2 = pack(du, du);
                const ulonglong2 B = *reinterpret_cast<const ulonglong2*>(&sh.vec[0][k][lane * 4]);
                as[i][0] = ex2_2(mul2(dd, A2[0]));
                as[i][1] = ex2_2(mul2(dd, A2[1]));
                h[0] = fma2(as[i][0], h[0], mul2(du2, B.x));
                h[1] = fma2(as[i][1], h[1], mul2(du2, B.y));
            }
            hs[i][0] = h[0];
            hs[i][1] = h[1];
        }
#pragma unroll
        for (int i = kBatch - 1; i >= 0; --i) {
            const int k = b * kBatch + i;
            if (!plain && (t0 + k < lo || t0 + k >= hi)) continue;
            if (!plain && sh.tile.end[k] >= 0) {
                if (p.dfinal) load4(p.dfinal + (int64_t)sh.tile.end[k] * p.C * S + cs, carry);
                else carry[0] = carry[1] = 0ull;
            }
            const float d = sh.d[k][ch], u = sh.u[k][ch], yb = sh.yb[k][ch];
            const ulonglong2 B = *reinterpret_cast<const ulonglong2*>(&sh.vec[0][k][lane * 4]);
            const ulonglong2 C = *reinterpret_cast<const ulonglong2*>(&sh.vec[1][k][lane * 4]);
            const f2 yb2 = pack(yb, yb), dd = pack(d, d);
            const f2 dh[2] = {fma2(yb2, C.x, carry[0]), fma2(yb2, C.y, carry[1])};
            f2 prev[2] = {i > 0 ? hs[i > 0 ? i - 1 : 0][0] : before[0], i > 0 ? hs[i > 0 ? i - 1 : 0][1] : before[1]};
            if (!plain && sh.tile.start[k] >= 0) initial_of(sh.tile.start[k], prev);
            carry[0] = mul2(as[i][0], dh[0]);
            carry[1] = mul2(as[i][1], dh[1]);
            if (!plain && sh.tile.start[k] >= 0 && p.dinitial && on)
                *reinterpret_cast<float4*>(p.dinitial + (int64_t)sh.tile.start[k] * p.C * S + cs) = as4(carry);
            const f2 ah[2] = {mul2(carry[0], prev[0]), mul2(carry[1], prev[1])};
            dA[0] = fma2(ah[0], dd, dA[0]);
            dA[1] = fma2(ah[1], dd, dA[1]);
            float q1 = sum2(fma2(dh[1], B.y, mul2(dh[0], B.x)));
            float q2 = sum2(fma2(ah[1], A[1], mul2(ah[0], A[0])));
            float yv = sum2(fma2(hs[i][1], C.y, mul2(hs[i][0], C.x)));
#pragma unroll
            for (int x = LP / 2; x > 0; x >>= 1) {
                q1 += __shfl_xor_sync(0xffffffffu, q1, x);
                q2 += __shfl_xor_sync(0xffffffffu, q2, x);
                yv += __shfl_xor_sync(0xffffffffu, yv, x);
            }
            // dB and dC: what this channel adds, then the sum over the warp's channels, after which lane
            // `lane` of channel position `pos` holds KEEP of the eight sums of its four states
            const float du = on ? d * u : 0.f, ybo = on ? yb : 0.f;
            float v[8];
            unpack(mul2(dh[0], pack(du, du)), v[0], v[1]);
            unpack(mul2(dh[1], pack(du, du)), v[2], v[3]);
            unpack(mul2(hs[i][0], pack(ybo, ybo)), v[4], v[5]);
            unpack(mul2(hs[i][1], pack(ybo, ybo)), v[6], v[7]);
            int n = 8, which = 0;
#pragma unroll
            for (int x = LP; x < 32; x <<= 1) {
                if (n > 1) {
                    n >>= 1;
                    const bool up = (tid & x) != 0;
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (j < n) {
                            const float send = up ? v[j] : v[j + n];
                            const float keep = up ? v[j + n] : v[j];
                            v[j] = keep + __shfl_xor_sync(0xffffffffu, send, x);
                        }
                    which += up ? n : 0;
                } else {
                    v[0] += __shfl_xor_sync(0xffffffffu, v[0], x);
                }
            }
#pragma unroll
            for (int j = 0; j < Sh::KEEP; ++j)
                sh.red[tid / 32][i][(which + j) / 4 * S + lane * 4 + (which + j) % 4] = v[j];
            __syncwarp();  // the channel's lanes are past their reads of this token
            if (lane == 0) {
                sh.u[k][ch] = fmaf(d, q1, Dc * yb);
                sh.d[k][ch] = fmaf(u, q1, q2);
                sh.yb[k][ch] = yv;
            }
        }
        __syncthreads();
        for (int e = tid; e < kBatch * 2 * S; e += NT) {
            const int i = e / (2 * S), j = e % (2 * S), t = t0 + b * kBatch + i;
            if (t < lo || t >= hi) continue;
            float a = 0.f;
#pragma unroll
            for (int x = 0; x < Sh::NW; ++x) a += sh.red[x][i][j];
            w.dBC[((int64_t)blockIdx.x * m.total + t) * 2 * S + j] = a;
        }
        __syncthreads();
    }
    if (on) *reinterpret_cast<float4*>(w.state + slot) = as4(dA);
    __syncthreads();

    // outputs, element by element as the inputs came
    TG* du = static_cast<TG*>(p.du) + ec;
    TG* dl = static_cast<TG*>(p.ddelta) + ec;
    TG* dz = static_cast<TG*>(p.dz) + ec;
    const float De = p.D ? __ldg(p.D + ec) : 0.f;
    float dbias = 0.f;
#pragma unroll 8
    for (int k = 0; k < PER; ++k) {
        const int r = tid / CH + k * ROWS;
        const int64_t t = t0 + r;
        if (!eon || t < lo || t >= hi) continue;
        float dd = sh.d[r][ech];
        if (p.softplus) dd *= sigmoid(ld(pd, t * p.ldd) + ebias);
        dbias += dd;
        du[t * p.C] = from_f32<TG>(sh.u[r][ech]);
        dl[t * p.C] = from_f32<TG>(dd);
        if (p.z) {
            const float zv = ld(pz, t * p.ldz), sg = sigmoid(zv);
            const float y = fmaf(De, ld(pu, t * p.ldu), sh.yb[r][ech]);
            dz[t * p.C] = from_f32<TG>(ld(pg, t * p.C) * y * (sg * fmaf(zv, 1.f - sg, 1.f)));
        }
    }
    // dD and dbias over the chunk: the ROWS threads of a channel
    __syncthreads();
    float* part = &sh.yb[0][0];
    part[tid] = dD;
    part[NT + tid] = dbias;
    __syncthreads();
    if (tid < CH && eon) {
        float a = 0.f, b = 0.f;
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
            a += part[r * CH + tid];
            b += part[NT + r * CH + tid];
        }
        w.dD[(int64_t)blockIdx.y * p.C + ec] = a;
        w.dbias[(int64_t)blockIdx.y * p.C + ec] = b;
    }
    // a sequence without tokens hands the gradient of its state back
    if (p.dinitial && on)
        for (int n = blockIdx.y; n < m.N; n += gridDim.y)
            if (m.end(n) <= m.begin(n)) {
                float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
                if (p.dfinal) v = *reinterpret_cast<const float4*>(p.dfinal + (int64_t)n * p.C * S + cs);
                *reinterpret_cast<float4*>(p.dinitial + (int64_t)n * p.C * S + cs) = v;
            }
}

// ---- 4. the partial sums ------------------------------------------------------------------------

// out[i] = sum of the chunks' in[i], chunk by chunk.
__global__ void __launch_bounds__(128) scan_bwd_chunks_kernel(const float* in, int chunks, int64_t n, float* out) {
    const int64_t i = blockIdx.x * 128ll + threadIdx.x;
    if (i >= n) return;
    float a = 0.f;
#pragma unroll 8
    for (int j = 0; j < chunks; ++j) a += in[j * n + i];
    out[i] = a;
}

// dB and dC from the channel blocks of each group.
template <typename TG, int S>
__global__ void __launch_bounds__(256) scan_bwd_vec_kernel(const float* in, SeqMap m, int G, int per_group, TG* dB, TG* dC) {
    const int64_t i = blockIdx.x * 256ll + threadIdx.x;
    if (i >= (int64_t)m.total * G * 2 * S) return;
    const int j = (int)(i % (2 * S));
    const int64_t tg = i / (2 * S);
    const int g = (int)(tg % G), t = (int)(tg / G);
    if (t < m.first() || t >= m.last()) return;
    float a = 0.f;
#pragma unroll 8
    for (int b = 0; b < per_group; ++b) a += in[((int64_t)(g * per_group + b) * m.total + t) * 2 * S + j];
    TG* out = j < S ? dB : dC;
    out[tg * S + j % S] = from_f32<TG>(a);
}

int bwd_blocks(const SsmScanParams& p) {
    const int ch = p.S == 8 ? BwdShape<8>::CH : BwdShape<16>::NT * 4 / p.S;
    return p.G * ((p.C / p.G + ch - 1) / ch);
}
int chunk_count(int total) { return total > 0 ? (total + kChunk - 1) / kChunk : 1; }

template <typename T, typename TG, int S>
cudaError_t launch(const SsmScanParams& p, cudaStream_t st) {
    const SeqMap m{p.cu, p.N, p.T, p.total};
    const int chunks = chunk_count(p.total), blocks = bwd_blocks(p);
    Scratch w;
    carve(w, p.ws, chunks, blocks, p);
    constexpr int kSumChannels = S <= 16 ? kSumThreads : kSumThreads * 16 / S;
    const int sum_blocks = p.G * ((p.C / p.G + kSumChannels - 1) / kSumChannels);
    scan_bwd_sum_kernel<T, TG, S><<<dim3(sum_blocks, chunks), kSumThreads, 0, st>>>(p, m, w);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const int64_t quads = (int64_t)p.C * S / 4;
    scan_bwd_prefix_kernel<<<dim3((unsigned)((quads + 127) / 128), 2), 128, 0, st>>>(p.A, w, chunks, p.C, S);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    constexpr int smem = sizeof(BwdShared<S>);
    e = cudaFuncSetAttribute(scan_bwd_kernel<T, TG, S>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    scan_bwd_kernel<T, TG, S><<<dim3(blocks, chunks), BwdShape<S>::NT, smem, st>>>(p, m, w);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    auto over_chunks = [&](const float* in, int64_t n, float* out) {
        if (out) scan_bwd_chunks_kernel<<<(unsigned)((n + 127) / 128), 128, 0, st>>>(in, chunks, n, out);
    };
    over_chunks(w.state, (int64_t)p.C * S, p.dA);
    over_chunks(w.dD, p.C, p.dD);
    over_chunks(w.dbias, p.C, p.dbias);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    const int64_t n = (int64_t)p.total * p.G * 2 * S;
    if (n > 0)
        scan_bwd_vec_kernel<TG, S><<<(unsigned)((n + 255) / 256), 256, 0, st>>>(w.dBC, m, p.G, blocks / p.G, static_cast<TG*>(p.dB),
                                                                               static_cast<TG*>(p.dC));
    return cudaGetLastError();
}

template <typename T, typename TG>
cudaError_t dispatch(const SsmScanParams& p, cudaStream_t st) {
    if (p.S == 8) return launch<T, TG, 8>(p, st);
    if (p.S == 16) return launch<T, TG, 16>(p, st);
    if (p.S == 32) return launch<T, TG, 32>(p, st);
    return launch<T, TG, 64>(p, st);
}

}  // namespace

size_t ssm_scan_bwd_workspace(const SsmScanParams& p) {
    Scratch w;
    return carve(w, nullptr, chunk_count(p.total), bwd_blocks(p), p);
}

cudaError_t ssm_scan_bwd(kda_dtype dt, kda_dtype gdt, const SsmScanParams& p, cudaStream_t st) {
    if (dt == KDA_F32) return dispatch<float, float>(p, st);
    if (gdt == KDA_F32) return dispatch<__nv_bfloat16, float>(p, st);
    return dispatch<__nv_bfloat16, __nv_bfloat16>(p, st);
}

}  // namespace kda
