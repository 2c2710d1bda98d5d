// relative_bias.cuh -- a relative position bias inside an attention tile: its
// value at an offset j - i, fetched for whole pieces of the tile at a time
// (the values by offset and the buckets come from relative_bias.cu).
#pragma once

#include <stdint.h>

namespace vsa {

// The bias of a 32 x 32 piece of a tile depends on j - i alone, so a warp
// needs 63 values of it: lane l loads values l - 32 and l (relative to the
// piece's first diagonal), and element (row lane r, column i) takes value
// i - r from lane (i - r) mod 32 with one shuffle.  `dir` is +1 where columns
// are keys and -1 where rows are.
struct BiasPiece {
    float lo, hi;
};
__device__ __forceinline__ BiasPiece bias_piece(const float *E, int R, int dir, int o0, int lane) {
    const int a = dir * (o0 - 32 + lane), b = dir * (o0 + lane);
    return BiasPiece{__ldg(E + min(max(a, -R), R)), __ldg(E + min(max(b, -R), R))};
}
__device__ __forceinline__ float bias_at(const BiasPiece &p, int i, int lane) {
    return __shfl_sync(0xffffffffu, lane <= i ? p.hi : p.lo, (i - lane) & 31);
}
// Whether every offset of a 128 x 128 tile around `d` (first key - first
// query) falls into one bucket; E is constant over it then.
__device__ __forceinline__ bool bias_uniform(const uint8_t *bm, int R, int d, int &bucket) {
    const int lo = d - 127, hi = d + 127;
    bucket = __ldg(bm + min(max(lo, -R), R));
    return (lo > 0 || hi <= 0) && bucket == __ldg(bm + min(max(hi, -R), R));
}

}  // namespace vsa
