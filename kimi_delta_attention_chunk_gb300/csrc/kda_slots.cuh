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

// Whether row i, whose page_of_row is `page`, is to be left alone: a padded row, a slot out of
// range, or a slot that an earlier row of the batch has (no two rows may write one page); the
// last two set *status to KDA_ERR_RANGE.  Every thread of the block calls it with the same row.
// The repeats are found by reading the slots before i, i / blockDim loads a thread: the blocks of
// one row all do it, but next to a page's bytes it is little.
__device__ __forceinline__ bool row_refused(const int32_t* slots, int i, int page, int32_t* status) {
    if (!slots) return false;
    if (page == -1) return true;
    bool bad = page < 0;
    for (int j = threadIdx.x; j < i; j += blockDim.x) bad |= __ldg(slots + j) == page;
    if (!__syncthreads_or(bad)) return false;
    if (status && threadIdx.x == 0) *status = KDA_ERR_RANGE;
    return true;
}

}  // namespace kda
