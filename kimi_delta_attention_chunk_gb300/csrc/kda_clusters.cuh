// What the kernels of the gated recurrence and the group norm share: packed fp32 helpers, offsets of packed sequences, clusters.
#pragma once

#include <atomic>

#include "kda_segments.cuh"

namespace kda {

constexpr int kSms = 152;

__device__ __forceinline__ f2 both(float v) { return pack(v, v); }
__device__ __forceinline__ f2 neg2(f2 x) { return x ^ 0x8000000080000000ull; }
// 1 / (1 + e^-x) of a pair, packed but for the special functions.
__device__ __forceinline__ f2 gate2(f2 x) {
    float a, b;
    unpack(add2(ex2_2(mul2(x, both(-kLog2e))), both(1.f)), a, b);
    return pack(rcp(a), rcp(b));
}

// ---- packed sequences --------------------------------------------------------------------------------------

// N sequences in a stream of T tokens by their offsets, in shared memory where there are few.
constexpr int kCachedOffsets = 256;
struct Offsets {
    const int32_t* cu;  // (global or shared)
    int N, T;
    // Every thread of the block calls it.
    __device__ __forceinline__ Offsets(const int32_t* cu, int N, int T, int32_t* cache) : cu(cu), N(N), T(T) {
        if (!cu || N >= kCachedOffsets) return;
        for (int k = threadIdx.x; k <= N; k += blockDim.x) cache[k] = __ldg(cu + k);
        __syncthreads();
        this->cu = cache;
    }
    __device__ __forceinline__ int begin(int n) const { return min(max(cu[n], 0), T); }
    __device__ __forceinline__ int end(int n) const { return begin(n + 1); }
    // Tokens outside [first, last) belong to no sequence.
    __device__ __forceinline__ int first() const { return N > 0 ? begin(0) : 0; }
    __device__ __forceinline__ int last() const { return N > 0 ? begin(N) : 0; }
    // How many sequences begin before token `key` (a whole warp calls it with one key), by 32 probes a round.  On offsets that are not
    // sorted it still ends and stays within [0, N].
    __device__ __forceinline__ int begun_before(int key) const {
        const int lane = threadIdx.x & 31;
        int lo = 0, hi = N;
        while (hi > lo) {
            const int step = (hi - lo + 31) / 32, at = lo + (lane + 1) * step - 1;
            const int cnt = __popc(__ballot_sync(0xffffffffu, at < hi && begin(at) < key));
            const int next = min(hi, lo + (cnt + 1) * step - 1);
            lo = min(hi, lo + cnt * step);
            hi = max(lo, next);
            if (step == 1) break;
        }
        return lo;
    }
};

// ---- clusters ----------------------------------------------------------------------------------------------

constexpr int kMostCluster = 8;

__device__ __forceinline__ unsigned cluster_rank() {
    unsigned r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
// kStores: this thread has stored into another block's shared memory (the fence waits for its stores to global memory too, and
// is left to the warps that need it).
template <bool kStores>
__device__ __forceinline__ void cluster_arrive() {
    if constexpr (kStores) asm volatile("barrier.cluster.arrive.release;" ::: "memory");
    else asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }
// The address of `mine` (in this block's shared memory) in block `rank` of the cluster.
__device__ __forceinline__ uint32_t address_at(unsigned rank, const void* mine) {
    uint32_t to;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(to) : "r"((uint32_t)__cvta_generic_to_shared(mine)), "r"(rank));
    return to;
}

// Devices for which a launch remembers something; on others it asks every time.
constexpr int kMostDevices = 64;

// Lets a kernel that declares up to `declared` bytes of shared memory have `bytes` more, once a device.  48 KB in all need no leave.
template <typename K>
cudaError_t allow_shared(K kern, int declared, int bytes, std::atomic<uint64_t>& done) {
    if (declared + bytes < 48 * 1024) return cudaSuccess;
    int dev = kMostDevices;
    cudaError_t e = cudaGetDevice(&dev);
    const uint64_t mark = dev < kMostDevices ? 1ull << dev : 0;
    if (e != cudaSuccess || (done.load(std::memory_order_relaxed) & mark)) return e;
    if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes)) == cudaSuccess) done.fetch_or(mark, std::memory_order_relaxed);
    return e;
}

// Launches a kernel (its shared memory set) in clusters of `cluster` blocks.  dependent: it may begin while the one before it on the
// stream still runs.
template <typename... KArgs, typename... Args>
cudaError_t launch_clusters(void (*kern)(KArgs...), int64_t grid, int cluster, int threads, int smem, bool dependent, cudaStream_t st, Args... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = threads;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = cluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = dependent ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, static_cast<KArgs>(args)...);
}

inline int most_blocks(int T, int tile) {
    const int tiles = T / tile + (T % tile != 0);
    return tiles < 1 ? 1 : tiles < kMostCluster ? tiles : kMostCluster;
}

// The launch of one kernel in clusters: how many of each size a device holds at once, asked for once a device.  What fails is not
// remembered: the call has the error.
struct ClusterRoom {
    std::atomic<int> known[kMostDevices][kMostCluster + 1];  // one more than the answer, 0: not asked yet
    template <typename K>
    cudaError_t of(K kern, int dev, int size, int threads, int smem, int& n) {
        n = dev < kMostDevices ? known[dev][size].load(std::memory_order_relaxed) - 1 : -1;
        if (n >= 0) return cudaSuccess;
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3(size * 1024);
        cfg.blockDim = threads;
        cfg.dynamicSmemBytes = smem;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = size;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        const cudaError_t e = cudaOccupancyMaxActiveClusters(&n, kern, &cfg);
        if (e != cudaSuccess) return e;
        n = n > 0 ? n : 0;
        if (dev < kMostDevices) known[dev][size].store(n + 1, std::memory_order_relaxed);
        return cudaSuccess;
    }
    // Blocks of a cluster for `groups` clusters of streams of T tokens: as many as run at once, no more than there are tiles.
    template <typename K>
    cudaError_t size_for(K kern, int64_t groups, int T, int tile, int threads, int smem, int& size) {
        int dev = 0, n = 0;
        cudaError_t e = cudaGetDevice(&dev);
        for (size = most_blocks(T, tile); e == cudaSuccess && size > 1; --size) {
            e = of(kern, dev, size, threads, smem, n);
            if (e == cudaSuccess && groups <= n) break;
        }
        return e;
    }
};

}  // namespace kda
