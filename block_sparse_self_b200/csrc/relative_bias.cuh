// relative_bias.cuh -- a relative position bias inside an attention tile.
//
// The bias of a 32 x 32 piece of a tile depends on j - i alone: 63 diagonals.
// Lane l of the warp that holds the piece's 32 rows keeps the buckets of two of
// them, l - 32 and l (element (row lane r, column i) is on diagonal i - r).
// Buckets widen with distance, so a piece is one of three kinds:
//   one bucket: one value for all 1024 elements;
//   two, with one border: columns below r + border take the first value;
//   more (close to the main diagonal): diagonal m's value is in lane m mod 32
//   and takes one shuffle per element.
// The second kind is half of all pieces where 64 buckets reach 2048 positions.
// Selects in place of shuffles took the forward kernel from 2.74 to 2.32 ms and
// the dK/dV pass from 3.69 to 3.60 (S = 30720, 24 heads); the dQ pass, which has
// half the columns per thread, is faster with shuffles alone.
//
// The bucket of every offset is one byte in global memory (relative_bias.cu);
// a tile's bytes are asked for one tile ahead, while the warp would wait for
// the MMAs anyway (asked for where they are used, their latency was 1.5 times
// the rest of the tile).  The head's values by bucket are in shared memory.
#pragma once

#include <stdint.h>

#include "chain.cuh"
#include "common.cuh"

namespace vsa {

constexpr int kMaxBuckets = 256;

// bm points at offset 0; offsets beyond R share the bucket of R on their side.
__device__ __forceinline__ int bias_bucket(const uint8_t *bm, int R, int o) {
    return chain_load(bm + min(max(o, -R), R));
}

enum : int { BIAS_ONE = 0, BIAS_TWO = 1, BIAS_MORE = 2 };
struct BiasPiece {
    int lo, hi;         // this lane's two buckets
    int kind;           // the rest is the same in every lane
    int first, second;  // buckets of the first and the last diagonal
    int border;         // BIAS_TWO: the first diagonal of `second`
};
__device__ __forceinline__ BiasPiece bias_piece(int lo, int hi) {
    BiasPiece p{lo, hi, BIAS_MORE, __shfl_sync(0xffffffffu, lo, 1), __shfl_sync(0xffffffffu, hi, 31), 0};
    // lane 0's diagonal -32 is outside the piece
    const uint32_t a0 = __ballot_sync(0xffffffffu, lo == p.first) | 1u, a1 = __ballot_sync(0xffffffffu, hi == p.first);
    const uint32_t b0 = __ballot_sync(0xffffffffu, lo == p.second) & ~1u, b1 = __ballot_sync(0xffffffffu, hi == p.second);
    const uint64_t a = static_cast<uint64_t>(a1) << 32 | a0, b = static_cast<uint64_t>(b1) << 32 | b0;
    if (a == ~0ull) p.kind = BIAS_ONE;
    else if (a == ~b && (a & (a + 1)) == 0) {
        p.kind = BIAS_TWO;
        p.border = __popcll(a) - 32;
    }
    return p;
}
// BIAS_TWO: the row's columns that take the second value, as bits.
__device__ __forceinline__ uint32_t bias_second(const BiasPiece &p, int lane) { return span_bits(0, lane + p.border, 32); }
// Element (row lane, column i)'s value from the values of this lane's buckets.
__device__ __forceinline__ float bias_at(float lo, float hi, int i, int lane) {
    return __shfl_sync(0xffffffffu, lane <= i ? hi : lo, (i - lane) & 31);
}

// The head's values by bucket (log2e already in them) to shared memory.
__device__ __forceinline__ void bias_table(float *smem, const float *tab, int head, int buckets, int thread, int threads) {
    for (int b = thread; b < buckets; b += threads) smem[b] = chain_load(tab + static_cast<size_t>(head) * buckets + b);
}

}  // namespace vsa
