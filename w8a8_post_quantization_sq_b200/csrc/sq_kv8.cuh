// The paged int8 K/V cache: K and V codes [num_blocks, Hkv, block, D], one
// scale per block and head in kqs, vqs [num_blocks, Hkv] (value = code / qs),
// and for each sequence a row of block numbers, its length, and its range of
// the flattened new tokens (cu_q).
#pragma once

#include <stdint.h>

namespace sq {

// The sequence that holds flattened token t: the last b < B with cu[b] <= t.
// All 32 lanes search together (32 probes a round).
__device__ __forceinline__ int kv8_sequence_of(const int32_t* cu, int B, int64_t t, int lane) {
    int lo = 0, hi = B;
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) >> 5;
        const int i = lo + lane * step;
        const unsigned at = __ballot_sync(0xffffffffu, i < hi && (lane == 0 || (int64_t)__ldg(cu + i) <= t));
        lo += (31 - __clz(at)) * step;
        hi = min(hi, lo + step);
    }
    return lo;
}

}  // namespace sq
