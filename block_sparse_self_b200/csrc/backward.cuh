// backward.cuh -- what the two passes of the attention's backward pass share:
// arguments, the tiles they walk, the masks inside a tile and the relative
// position bias.
//
// With x_ij = scale q_i.k_j (+ bias), P_ij = exp(x_ij - lse_i) (lse saved by
// the forward pass), g = dL/dO and delta_i = g_i.o_i:
//   dV_j = sum_i P_ij g_i
//   dX_ij = P_ij (g_i.v_j - delta_i)
//   dQ_i = scale sum_j dX_ij k_j,  dK_j = scale sum_i dX_ij q_i
//   dbias[b] = sum over the pairs (i, j) whose offset j - i is in bucket b of dX_ij
// P is recomputed, never stored.  One pass owns a query block and walks the
// key blocks of its list (dQ); the other owns a key block and walks the
// query blocks that list it (dK, dV, dbias).  Each sum has one owner and one order,
// so results repeat bit for bit and nothing is accumulated in memory; the
// price is that S and dP are computed in both passes (7 products instead of
// 5 per pair of blocks).
//
// delta carries the forward pass's roundings of P and o, and one error in
// delta_i shifts a whole row of dX.  Exactly, sum_j dX_ij = 0; so the dQ pass,
// which walks whole rows, sums each row of its dX (from delta as it is) and
// adds the sum to delta_i, and the dK/dV pass, which runs after it, works with
// the corrected delta.  dbias is summed there for that reason: it adds up many
// dX of one sign of error.
//
// The sum is that of delta's error only where o and lse belong to the keys that the
// row walks.  With those of a softmax over more keys (partial results joined) it is a
// part of the gradient.  delta's error is mostly that of o, half a step of bf16 for its
// terms, so a sum beyond kSlack sum_d |g_d o_d| is no error: such a row keeps its delta.
#pragma once

#include <math.h>

#include "chain.cuh"
#include "common.cuh"
#include "internal.h"
#include "relative_bias.cuh"

namespace vsa {

constexpr float kSlack = 0x1p-7f;  // two half steps of bf16, and in size alone: the errors of D terms differ in sign

struct BwdArgs {
    int P;           // positions per head (tiled mode: of the padded grid)
    int Pw;          // P rounded up to 128: row length of nlse and ndelta
    int S_out;       // rows per head of q, k, v, o and the gradients
    int BH, H;       // (batch, head) rows; heads
    int nt;          // row tiles per head (blocks of BS positions)
    int lead;        // dK/dV pass: leading key blocks of every head that are taken first
    // dQ pass: the forward lists; dK/dV pass: transposed lists (offsets [lists, nb+1], rows [lists, nb*cap])
    const int32_t *idx, *cnt;
    int cap, list_per_head, nb;
    const int32_t *t_off, *t_rows;
    int group, gstride;
    int half, sink, dense;
    float scale, scale_log2;
    const float *nlse, *ndelta;  // [BH, Pw]: -lse log2e (-inf: the row has no gradient) and -delta
    float *ndelta_out;           // dQ pass: ndelta with the row sums of dX taken off (see below)
    const float *slack;          // [BH, Pw]: the most that a row's sum of dX can be of delta's error (see above)
    const float *none;           // 128 values of -inf, then 128 of 0: the statistics of columns past a list's end
    const float *kmean;          // mean key of each block (window mode: tile of 128), [BH, nt, D] (see backward_dq.cu)
    const uint32_t *valid;       // [BH, Pw/32] bits: which positions hold a token; nullptr when all do
    void *d0, *d1;               // dQ pass: dq; dK/dV pass: dk, dv
    int out_f32;
    int *status;
    // window mode with a bias: tab[h][b] = log2e bias of bucket b, bm[o] = bucket of offset o (key - query), |o| <= R
    const float *tab;
    const uint8_t *bm;
    int R, buckets;
    float *dbias_part;  // dK/dV pass: [BH, nt, buckets]
    // tiled mode
    int H2, W2;  // the padded grid's frame
    RealGrid real;
    TileSet tiles;
    const int32_t *choice;
    struct BoxGeom {
        FastDiv m, nthw, ntw;  // m = volume / BS, tiles per frame, tiles per tile row
        int bt;                // frames of one block's box
    } geom[kMaxTiles];
};

// Tensor maps of q, k, v and g, one per candidate tiling; a kernel that has no
// tilings takes one of each (a tenth of the parameters that a launch copies).
template <int N>
struct BwdMapsOf {
    CUtensorMap q[N], k[N], v[N], g[N];
};
using BwdMaps = BwdMapsOf<kMaxTiles>;
static_assert(sizeof(BwdMaps) + sizeof(BwdArgs) <= 32764, "kernel parameters");

template <bool TILED>
auto bwd_maps(const BwdMaps &m) {
    if constexpr (TILED) return m;
    else return BwdMapsOf<1>{{m.q[0]}, {m.k[0]}, {m.v[0]}, {m.g[0]}};
}

constexpr int kBwdThreads = 320;  // warps 0-7 element-wise work, 8 TMA producer, 9 MMA issuer and TMEM owner

__device__ __forceinline__ uint64_t mul_f32x2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// Untiled bulk copy global -> shared (16-byte aligned, a multiple of 16 bytes).
__device__ __forceinline__ void bulk_load(void *dst, const void *src, uint32_t bytes, uint64_t *bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                     smem_u32(dst)),
                 "l"(src), "r"(bytes), "r"(smem_u32(bar))
                 : "memory");
}

// One block of BS rows of a [BH, S, D] tensor (permuted order: 3-D map; T-major: its 5-D box).
template <int D, int BS, bool TILED>
__device__ __forceinline__ void bwd_load_block(uint8_t *dst, const CUtensorMap *map, uint64_t *bar, int b, int bh,
                                               const BwdArgs &a, int tc) {
    constexpr int SLAB = 128 * 128;
    if constexpr (TILED) {
        const BwdArgs::BoxGeom &g = a.geom[tc];
        const uint32_t tile = fdiv(static_cast<uint32_t>(b), g.m), part = b - tile * g.m.d;
        const uint32_t ct = fdiv(tile, g.nthw), rem = tile - ct * g.nthw.d;
        const uint32_t ch = fdiv(rem, g.ntw), cw = rem - ch * g.ntw.d;
        const int w = static_cast<int>(cw) * a.tiles.w[tc], h = static_cast<int>(ch) * a.tiles.h[tc];
        const int t = static_cast<int>(ct * g.m.d + part) * g.bt;
        #pragma unroll
        for (int s = 0; s < D / 64; ++s) tma_load_5d(dst + s * SLAB, map, bar, s * 64, w, h, t, bh);
    } else {
        #pragma unroll
        for (int s = 0; s < D / 64; ++s) tma_load_3d(dst + s * SLAB, map, bar, s * 64, b * BS, bh);
    }
}

// Row of a head's tensor that holds position p, or -1 (padding, past the end).
template <bool TILED>
__device__ __forceinline__ int bwd_row_of(int p, const BwdArgs &a, int tc) {
    if (p >= a.P) return -1;
    if constexpr (TILED) {
        int t, h, w;
        tile_coords(p, a.H2, a.W2, a.tiles.t[tc], a.tiles.h[tc], a.tiles.w[tc], t, h, w);
        return real_token(t, h, w, a.real);
    }
    return p;
}

// Columns base .. base + 31 that share row position p's group (both kinds of
// groups are symmetric, so the same bits serve queries and keys as rows).
__device__ __forceinline__ uint32_t group_bits(const BwdArgs &a, int p, int base) {
    if (a.group > 0) {
        const int g0 = (p / a.group) * a.group;
        return span_bits(base, g0, g0 + a.group);
    }
    const int s = a.gstride, o = (p - base) & (s - 1);
    if (o >= 32) return 0u;
    uint32_t bits = 1u << o;
    for (int e = s; e < 32; e <<= 1) bits |= bits << e;
    return bits;
}

// One row of gradients: 32 columns from tensor memory, times `f`, to out.
__device__ __forceinline__ void bwd_store32(const uint32_t (&x)[32], float f, void *out, int out_f32, size_t at) {
    if (out_f32) {
        float4 *dst = reinterpret_cast<float4 *>(static_cast<float *>(out) + at);
        #pragma unroll
        for (int e = 0; e < 8; ++e)
            dst[e] = make_float4(__uint_as_float(x[4 * e]) * f, __uint_as_float(x[4 * e + 1]) * f,
                                 __uint_as_float(x[4 * e + 2]) * f, __uint_as_float(x[4 * e + 3]) * f);
    } else {
        uint4 *dst = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(out) + at);
        #pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint32_t *u = &x[8 * e];
            dst[e] = make_uint4(pack_bf16x2(__uint_as_float(u[0]) * f, __uint_as_float(u[1]) * f),
                                pack_bf16x2(__uint_as_float(u[2]) * f, __uint_as_float(u[3]) * f),
                                pack_bf16x2(__uint_as_float(u[4]) * f, __uint_as_float(u[5]) * f),
                                pack_bf16x2(__uint_as_float(u[6]) * f, __uint_as_float(u[7]) * f));
        }
    }
}

__device__ __forceinline__ void bwd_zero_row(void *out, int out_f32, size_t at, int D) {
    uint4 *dst = out_f32 ? reinterpret_cast<uint4 *>(static_cast<float *>(out) + at)
                         : reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(out) + at);
    const int n = D * (out_f32 ? 4 : 2) / 16;
    for (int e = 0; e < n; ++e) dst[e] = make_uint4(0u, 0u, 0u, 0u);
}

// dQ of every query block; dK, dV and the bias's partial sums of every key block.  `kind`
// of kernel: block is 32, 64 or 128; window and bias need 128.
vsa_status launch_bwd_dq(const BwdMaps &maps, const BwdArgs &a, int D, int block, bool window, bool tiled, bool bias,
                         cudaStream_t st);
vsa_status launch_bwd_dkv(const BwdMaps &maps, const BwdArgs &a, int D, int block, bool window, bool tiled, bool bias,
                          cudaStream_t st);

}  // namespace vsa
