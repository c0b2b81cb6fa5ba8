// Rows of a batch that read and write pages of a pool by slot.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/kda.h"

namespace kda {

// The page of batch row i: slots[i] if it is in [0, P), -1 for padding (slot -1), -2 for any
// other slot.  Null slots: page i.
__device__ __forceinline__ int page_of_row(const int32_t* slots, int i, int P) {
    if (!slots) return i;
    const int s = __ldg(slots + i);
    return s >= -1 && s < P ? s : -2;
}

// Which of the rows row0 + i < N, whose page_of_row is page[i], are to be left alone (bit i): padded
// rows, slots out of range, and slots that an earlier row of the batch has (no two rows may write one
// page); the last two set *status to KDA_ERR_RANGE.  Every thread of the block calls it, once a
// kernel.  The repeats are found by reading the slots before the rows, row0 / blockDim loads a thread
// and one meeting of the block, in all blocks of the row.  That is little next to a page's bytes for some thousand
// rows and grows with their square: a convolution of 768 channels takes 26 us with slots and 20 without for 4096 rows, 104
// and 44 for 16384, 1426 and 132 for 65536; 29 ms for the most rows, KDA_MOST_SLOTS, so that every call ends soon.
template <int kRows>
__device__ __forceinline__ unsigned rows_refused(const int32_t* slots, int row0, int N, const int (&page)[kRows],
                                                 int32_t* status) {
    if (!slots) return 0;
    if constexpr (kRows == 1) {
        if (page[0] == -1) return 1;
        bool again = page[0] < 0;
        for (int j = threadIdx.x; j < row0; j += blockDim.x) again |= __ldg(slots + j) == page[0];
        if (!__syncthreads_or(again)) return 0;
        if (status && threadIdx.x == 0) *status = KDA_ERR_RANGE;
        return 1;
    }
    __shared__ unsigned part[32];
    unsigned bad = 0, pad = 0;
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        if (row0 + i >= N) continue;
        if (page[i] == -2) bad |= 1u << i;
        if (page[i] == -1) pad |= 1u << i;
    }
    const int before = min(row0 + kRows - 1, N);
    for (int j = threadIdx.x; j < before; j += blockDim.x) {
        const int s = __ldg(slots + j);
#pragma unroll
        for (int i = 0; i < kRows; ++i)
            if (s == page[i] && s >= 0 && j < row0 + i && row0 + i < N) bad |= 1u << i;
    }
    bad = __reduce_or_sync(0xffffffffu, bad);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = bad;
    __syncthreads();
    bad = 0;
    for (int w = 0; w < (int)blockDim.x / 32; ++w) bad |= part[w];
    if (bad && status && threadIdx.x == 0) *status = KDA_ERR_RANGE;
    return bad | pad;
}

}  // namespace kda
