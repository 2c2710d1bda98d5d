// relative_bias.cuh -- a relative position bias inside an attention tile.
//
// The bias of a 32 x 32 piece of a tile depends on j - i alone: 63 offsets.
// Lane l of the warp that holds the piece's 32 rows keeps the buckets of two of
// them, (first diagonal - 32 + l) and (first diagonal + l); element (row lane r,
// column i) is on diagonal i - r, whose value is in lane (i - r) mod 32 and
// takes one shuffle.  Buckets widen with distance, so most pieces have a single
// bucket and one value for all 1024 elements.
//
// The bucket of every offset is one byte in global memory (relative_bias.cu);
// a tile's bytes are asked for one tile ahead, while the warp would wait for
// the MMAs anyway (asked for where they are used, their latency was 1.5 times
// the rest of the tile).  The head's values by bucket are in shared memory.
#pragma once

#include <stdint.h>

namespace vsa {

constexpr int kMaxBuckets = 256;

// bm points at offset 0; offsets beyond R share the bucket of R on their side.
__device__ __forceinline__ int bias_bucket(const uint8_t *bm, int R, int o) {
    return __ldg(bm + min(max(o, -R), R));
}

struct BiasPiece {
    int lo, hi;      // this lane's two buckets
    bool uniform;    // one bucket for the whole piece: hi, in every lane
};
__device__ __forceinline__ BiasPiece bias_piece(int lo, int hi) {
    const int b0 = __shfl_sync(0xffffffffu, hi, 0);
    return BiasPiece{lo, hi, __all_sync(0xffffffffu, lo == b0 && hi == b0) != 0};
}
// Element (row lane, column i)'s value from the values of this lane's buckets.
__device__ __forceinline__ float bias_at(float lo, float hi, int i, int lane) {
    return __shfl_sync(0xffffffffu, lane <= i ? hi : lo, (i - lane) & 31);
}

// The head's values by bucket (log2e already in them) to shared memory.
__device__ __forceinline__ void bias_table(float *smem, const float *tab, int head, int buckets, int thread, int threads) {
    for (int b = thread; b < buckets; b += threads) smem[b] = __ldg(tab + static_cast<size_t>(head) * buckets + b);
}

}  // namespace vsa
