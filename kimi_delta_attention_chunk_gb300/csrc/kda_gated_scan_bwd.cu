// Gated linear recurrence over prompts: backward.
//
// With the forward's s, a, m, si = sigmoid(i), sr = sigmoid(r), u, h and yb = dy silu(z), per sequence and channel:
//     dh_t = yb_t + a_{t+1} dh_{t+1}   (behind the last token: the final state's gradient)
//     dx = dh m si,  di = dh u (1 - si),  dz = dy h silu'(z),  dinitial = a_0 dh_0
//     ds = dh (si x a^2 / m - a h_{t-1})      (dm / ds = e^-2s / m)
//     dr = ds rate sr (1 - sr),  dlam = decay sigmoid(lam) sum_t ds sr
// The forward pass leaves the state before every 32nd token, so that every tile of 32 tokens can form its own states;
// dh is carried from tile to tile backwards as the forward pass carries h (kda_gated_scan.cu): strips of four tokens a warp, their
// maps folded through shared memory, tiles side by side in a cluster.  What an element needs (a, u, m si, si x a^2 / m, sr, 1 - si, yb, dy
// silu'(z)) stays in registers between the two walks: 128 a thread, two blocks an SM.  Without those states a first pass of the forward
// kernel makes them (x, r and i are then read twice).  dlam's sums over tokens: one partial sum a block, added in a fixed order.
#include "kda_gated.cuh"
#include "kda_tc.cuh"

namespace kda {

namespace {

constexpr int kStrip = 4, kTile = kGatedWarps * kStrip;
static_assert(kTile == kGatedBlock, "a tile begins at a state that is left to it");

template <typename T>
constexpr int kStages = sizeof(T) == 2 ? 4 : 2;
template <typename T, typename TG>
constexpr int kStageBytes = kTile * kGatedCh * (4 * (int)sizeof(T) + (int)sizeof(TG));

template <typename T, typename TG, int VEC, int GVEC, bool kPacked>
__global__ void __launch_bounds__(kGatedThreads, 2) gated_bwd_kernel(GatedParams p, float* partial, int cluster, int blocks, bool whole_pairs) {
    constexpr int TILE = kTile * kGatedCh, STAGES = kStages<T>;
    extern __shared__ __align__(128) char shared[];
    __shared__ Affine ahead[kGatedWarps][32], back[kGatedWarps][32];
    __shared__ Affine peers[2][kMostCluster][32];
    __shared__ TokenTile<kPacked ? kTile : 1> tile;

    const int lane = threadIdx.x % 32, w = threadIdx.x / 32;
    const int rank = cluster > 1 ? (int)cluster_rank() : 0;
    const int group = blockIdx.x / cluster, b = group / blocks, c0 = group % blocks * kGatedCh;
    const int has = min(kGatedCh, p.C - c0), c = c0 + 2 * lane, n2 = min(2, p.C - c);
    const SeqMap m{p.cu, p.N, p.T, p.T};
    const int first = kPacked ? m.first() : 0, last = kPacked ? m.last() : p.T;
    const int steps = (int)(((int64_t)p.T + kTile * cluster - 1) / (kTile * cluster));
    const int64_t row0 = (int64_t)b * p.T, block0 = (int64_t)b * ((p.T + kTile - 1) / kTile);

    // step `it` counts from the stream's end
    auto tile_of = [&](int it) { return ((steps - 1 - it) * cluster + rank) * kTile; };
    auto request = [&](int it) {
        const int t0 = it < steps ? tile_of(it) : 0;
        const int rows = it < steps ? min(kTile, p.T - t0) : 0;
        char* const to = shared + it % STAGES * kStageBytes<T, TG>;
        if (rows > 0) {
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                const void* base = v == 0 ? p.x : v == 1 ? p.r : v == 2 ? p.i : p.z;
                const int64_t ld = v == 0 ? p.ldx : v == 1 ? p.ldr : v == 2 ? p.ldi : p.ldz;
                if (v == 3 && !base) continue;
                request_rows<T, kTile, VEC>(reinterpret_cast<T*>(to) + v * TILE, static_cast<const T*>(base) + (row0 + t0) * ld + c0, ld, rows, has);
            }
            request_rows<TG, kTile, GVEC>(reinterpret_cast<TG*>(to + 4 * TILE * sizeof(T)), static_cast<const TG*>(p.dy) + (row0 + t0) * p.C + c0, p.C,
                                          rows, has);
        }
        copies_commit();
    };
#pragma unroll
    for (int s = 0; s < STAGES - 1; ++s) request(s);

    const f2 rate = pack(n2 > 0 ? gated_rate(__ldg(p.lam + c), p.decay) : 0.f, n2 > 1 ? gated_rate(__ldg(p.lam + c + 1), p.decay) : 0.f);
    // through sequences without tokens the gradient goes as it comes
    if (p.dinitial) {
        const int warps = kGatedWarps * cluster;
        for (int n0 = (w * cluster + rank) * 32; n0 < p.N; n0 += warps * 32) {
            if (!kPacked && p.T > 0) break;
            const int n = n0 + lane;
            unsigned empty = __ballot_sync(0xffffffffu, n < p.N && (!kPacked || m.end(n) <= m.begin(n)));
            for (; empty; empty &= empty - 1) {
                const int64_t at = (int64_t)(n0 + __ffs(empty) - 1) * p.C + c;
                store_state(p.dinitial, at, state_pair(p.dfinal, at, n2), n2);
            }
        }
    }
    f2 carry = kPacked ? 0ull : state_pair(p.dfinal, (int64_t)b * p.C + c, n2), dlam = 0ull;
    if (cluster > 1) {
        cluster_arrive();
        cluster_wait();
    }

    int from = 0x7fffffff;  // behind this token, up to the tile before, no boundary
    for (int it = 0; it < steps; ++it) {
        const int t0 = tile_of(it), rows = min(kTile, p.T - t0);
        f2 start = 0ull;
        if (rows > 0) {
            if (!kPacked && t0 == 0) start = state_pair(p.initial, (int64_t)b * p.C + c, n2);
            else {
                const float* s = p.states + (block0 + t0 / kTile) * p.C + c;
                start = pack(n2 > 0 ? s[0] : 0.f, n2 > 1 ? s[1] : 0.f);
            }
        }
        copies_wait<STAGES - 2>();
        __syncthreads();  // the tile is there, and everyone is past the one before
        request(it + STAGES - 1);
        bool clear = true;
        if constexpr (kPacked) {
            if (t0 <= from && rows > 0) {
                tile.template build<kGatedThreads>(m, t0);
                from = tile.carry >= 0 ? tile.carry_start : 0x7fffffff;
                clear = tile.plain || tile.template clear<kStrip>(w * kStrip);
            }
        }
        const char* const at = shared + it % STAGES * kStageBytes<T, TG>;
        const T* const in = reinterpret_cast<const T*>(at) + w * kStrip * kGatedCh + 2 * lane;
        const TG* const dys = reinterpret_cast<const TG*>(at + 4 * TILE * sizeof(T)) + w * kStrip * kGatedCh + 2 * lane;
        f2 a[kStrip], u[kStrip], wx[kStrip], wm[kStrip], sr[kStrip], ci[kStrip], yb[kStrip], gz[kStrip];
#pragma unroll
        for (int j = 0; j < kStrip; ++j) {
            const f2 x = pair_at(in + j * kGatedCh), r = pair_at(in + TILE + j * kGatedCh), i = pair_at(in + 2 * TILE + j * kGatedCh);
            yb[j] = pair_at(dys + j * kGatedCh);
            sr[j] = rcp2(one_plus<false>(r));
            const Decay d(sr[j], rate);
            a[j] = d.a;
            f2 si;
            if (p.z) {
                const f2 z = pair_at(in + 3 * TILE + j * kGatedCh), di = one_plus<true>(i), dz = one_plus<true>(z);
                const f2 inv = rcp2(mul2(di, dz)), sz = mul2(inv, di), silu = mul2(z, sz);
                si = mul2(inv, dz);
                gz[j] = mul2(yb[j], fma2(silu, fma2(neg2(sz), both(1.f), both(1.f)), sz));  // silu' = s + z s (1 - s)
                yb[j] = mul2(yb[j], silu);
            } else {
                si = rcp2(one_plus<false>(i));
                gz[j] = 0ull;
            }
            const f2 inv = inverse_root(d.m2), gx = mul2(si, x);
            wx[j] = mul2(mul2(d.m2, inv), si);
            u[j] = mul2(wx[j], x);
            ci[j] = add2(both(1.f), neg2(si));
            wm[j] = mul2(mul2(gx, inv), mul2(a[j], a[j]));
        }
        if (rows < kTile) {
#pragma unroll
            for (int j = 0; j < kStrip; ++j)
                if (w * kStrip + j >= rows) a[j] = both(1.f), u[j] = yb[j] = 0ull;
        }
        // the strip's maps forwards (af, u: cut where a sequence begins) and backwards (cut where one ends)
        Affine fore = identity(), rear = identity();
        if (!kPacked || clear) {
#pragma unroll
            for (int j = 0; j < kStrip; ++j) fore = follow<false>(fore, Affine{a[j], u[j]});
            rear.A = fore.A;
#pragma unroll
            for (int j = kStrip - 1; j >= 0; --j) rear.H = mul2(a[j], add2(yb[j], rear.H));
        } else {
#pragma unroll
            for (int j = 0; j < kStrip; ++j) {
                const int n = tile.start[w * kStrip + j];
                if (n >= 0) fore = Affine{both(-1.f), fma2(a[j], state_pair(p.initial, (int64_t)n * p.C + c, n2), u[j])};
                else fore = follow<true>(fore, Affine{a[j], u[j]});
            }
#pragma unroll
            for (int j = kStrip - 1; j >= 0; --j) {
                const int n = tile.end[w * kStrip + j];
                if (n >= 0) {
                    yb[j] = add2(yb[j], state_pair(p.dfinal, (int64_t)n * p.C + c, n2));
                    rear = Affine{both(-1.f), mul2(a[j], yb[j])};
                } else {
                    rear = follow<true>(rear, Affine{a[j], mul2(a[j], yb[j])});
                }
            }
        }
        ahead[w][lane] = fore;
        back[w][lane] = rear;
        __syncthreads();
        f2 h = start;
        for (int k = 0; k < w; ++k) {
            const Affine e = ahead[k][lane];
            h = apply<kPacked>(e.A, e.H, h);
        }
        Affine behind = identity(), total = identity();
#pragma unroll
        for (int k = kGatedWarps - 1; k >= 0; --k) {
            if (k == w) behind = total;
            total = follow<kPacked>(total, back[k][lane]);
        }
        f2 g = carry;
        if (cluster > 1) {
            const int buf = it & 1;
            if (w < cluster) store_at(w, &peers[buf][rank][lane], total);
            cluster_arrive();
            cluster_wait();
            for (int k = cluster - 1; k >= 0; --k) {
                if (k == rank) g = carry;
                const Affine e = peers[buf][k][lane];
                carry = apply<kPacked>(e.A, e.H, carry);
            }
        } else {
            carry = apply<kPacked>(total.A, total.H, carry);
        }
        g = apply<kPacked>(behind.A, behind.H, g);
        // the state before each token
        f2 hp[kStrip];
        const int64_t row = (row0 + t0 + w * kStrip) * p.C + c;
#pragma unroll
        for (int j = 0; j < kStrip; ++j) {
            if (kPacked && !clear) {
                const int n = tile.start[w * kStrip + j];
                if (n >= 0) h = state_pair(p.initial, (int64_t)n * p.C + c, n2);
            }
            hp[j] = h;
            h = fma2(a[j], h, u[j]);
            gz[j] = mul2(gz[j], h);
        }
#pragma unroll
        for (int j = kStrip - 1; j >= 0; --j) {
            const int t = t0 + w * kStrip + j;
            if (w * kStrip + j >= rows) continue;
            const bool in_one = !kPacked || (t >= first && t < last);
            if (kPacked && !clear && tile.end[w * kStrip + j] >= 0) g = 0ull;
            const f2 dh = add2(yb[j], g);
            f2 dx = mul2(dh, wx[j]), di = mul2(mul2(dh, u[j]), ci[j]);
            const f2 ds = mul2(dh, fma2(neg2(a[j]), hp[j], wm[j])), part = mul2(ds, sr[j]);
            f2 dr = mul2(mul2(part, rate), fma2(neg2(sr[j]), both(1.f), both(1.f))), dz = gz[j];
            g = mul2(a[j], dh);
            if (in_one) dlam = add2(dlam, part);
            else dx = di = dr = dz = 0ull;
            const int64_t off = row + (int64_t)j * p.C;
            auto put = [&](void* to, f2 v) {
                if (whole_pairs) store_pair<TG, true>(static_cast<TG*>(to) + off, v, n2);
                else store_pair<TG, false>(static_cast<TG*>(to) + off, v, n2);
            };
            put(p.dx, dx);
            put(p.dr, dr);
            put(p.di, di);
            if (p.z) put(p.dz, dz);
            if (p.dinitial) {
                const int n = kPacked ? (clear ? -1 : tile.start[w * kStrip + j]) : (t == 0 ? b : -1);
                if (n >= 0) store_state(p.dinitial, (int64_t)n * p.C + c, g, n2);
            }
        }
    }
    tc::grid_dep_launch();
    __syncthreads();
    ahead[w][lane].A = dlam;
    __syncthreads();
    if (w == 0 && steps > 0) {
        f2 sum = 0ull;
#pragma unroll
        for (int k = 0; k < kGatedWarps; ++k) sum = add2(sum, ahead[k][lane].A);
        store_state(partial + ((int64_t)b * cluster + rank) * p.C, c, sum, n2);
    }
}

// dlam from the blocks' partial sums.
__global__ void __launch_bounds__(128) gated_dlam_kernel(const float* partial, int parts, const float* lam, float decay, int C, float* dlam) {
    const int c = blockIdx.x * 128 + threadIdx.x;
    tc::grid_dep_wait();
    if (c >= C) return;
    float sum = 0.f;
    for (int k = 0; k < parts; ++k) sum += partial[(int64_t)k * C + c];
    const float l = __ldg(lam + c), e = expf(-fabsf(l));
    dlam[c] = decay * (l >= 0.f ? 1.f : e) / (1.f + e) * sum;
}

int clusters_of(const GatedParams& p) {
    return cluster_size((int64_t)((p.C + kGatedCh - 1) / kGatedCh) * p.B, p.T, kTile);
}
size_t partial_bytes(const GatedParams& p) {
    return ((size_t)p.B * (p.T > 0 ? clusters_of(p) : 0) * p.C * 4 + 255) / 256 * 256;
}

template <typename T, typename TG, int VEC, int GVEC, bool kPacked>
cudaError_t launch(const GatedParams& p, bool whole_pairs, cudaStream_t st) {
    const int blocks = (p.C + kGatedCh - 1) / kGatedCh;
    const int64_t groups = (int64_t)blocks * p.B;
    const int cluster = clusters_of(p);
    float* const partial = static_cast<float*>(p.ws);
    int parts = 0;
    if (groups > 0) {
        const cudaError_t e = launch_clusters(gated_bwd_kernel<T, TG, VEC, GVEC, kPacked>, groups * cluster, cluster, kStages<T> * kStageBytes<T, TG>, st,
                                              p, partial, cluster, blocks, whole_pairs);
        if (e != cudaSuccess) return e;
        parts = p.T > 0 ? p.B * cluster : 0;
    }
    return tc::launch_dependent(gated_dlam_kernel, (unsigned)((p.C + 127) / 128), 128, 0, st, partial, parts, p.lam, p.decay, p.C, p.dlam);
}
template <typename T, typename TG, int VEC, int GVEC>
cudaError_t launch_packed(const GatedParams& p, bool whole_pairs, cudaStream_t st) {
    return p.cu ? launch<T, TG, VEC, GVEC, true>(p, whole_pairs, st) : launch<T, TG, VEC, GVEC, false>(p, whole_pairs, st);
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
    bool whole_pairs = p.C % 2 == 0, wide = gated_pieces(p, es, 16) && (int64_t)p.C * gs % 16 == 0 && kda_host::aligned16(p.dy);
    for (const void* q : {(const void*)p.dx, (const void*)p.dr, (const void*)p.di, (const void*)p.dz}) whole_pairs = whole_pairs && (uintptr_t)q % (2 * gs) == 0;
    const bool narrow = gated_pieces(p, es, 4) && (int64_t)p.C * gs % 4 == 0 && (uintptr_t)p.dy % 4 == 0;
    if (dt == KDA_F32)
        return wide ? launch_packed<float, float, 4, 4>(p, whole_pairs, st) : launch_packed<float, float, 1, 1>(p, whole_pairs, st);
    if (gdt == KDA_F32) {
        if (wide) return launch_packed<__nv_bfloat16, float, 8, 4>(p, whole_pairs, st);
        return narrow ? launch_packed<__nv_bfloat16, float, 2, 1>(p, whole_pairs, st) : launch_packed<__nv_bfloat16, float, 1, 1>(p, whole_pairs, st);
    }
    if (wide) return launch_packed<__nv_bfloat16, __nv_bfloat16, 8, 8>(p, whole_pairs, st);
    return narrow ? launch_packed<__nv_bfloat16, __nv_bfloat16, 2, 2>(p, whole_pairs, st) : launch_packed<__nv_bfloat16, __nv_bfloat16, 1, 1>(p, whole_pairs, st);
}

}  // namespace kda
