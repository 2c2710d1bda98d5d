// backward.cu -- the steps around the backward pass's two tensor-core passes:
// per-row statistics, workspace, tensor maps and launches.
//
// Row statistics: delta_i = g_i.o_i and the size of its error, one pass over g and o (bandwidth bound:
// 2 x 2 S D bytes per head in bf16), written in position order beside -lse so
// that both passes read 128 consecutive values per tile whatever the tiling.
// Positions that hold no token and rows whose forward pass saw no key get
// -lse = -inf, i.e. P = 0 everywhere: they reach no gradient.
#include "backward.cuh"

namespace vsa {

namespace {

struct StatArgs {
    const void *o, *g, *o_lo;
    const float *lse;
    int P, Pw, S_out;
    TileDivs divs[kMaxTiles];
    RealGrid real;
    int tiled, n_tiles;
    const int32_t *choice;
    float *nlse, *ndelta, *slack, *none;
    uint32_t *valid;  // nullptr when every position holds a token
};

// A warp takes 32 consecutive positions of one head, 32 / LPR rows at a time
// (LPR lanes of 16 bytes of g per row).
template <int D, bool O_F32>
__global__ void __launch_bounds__(256) row_stats_kernel(const __grid_constant__ StatArgs a) {
    constexpr int LPR = D / 8, ROWS = 32 / LPR;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, bh = blockIdx.y;
    grid_release();
    if (blockIdx.x == 0 && bh == 0) a.none[threadIdx.x] = threadIdx.x < 128 ? -INFINITY : 0.f;
    const int p0 = (blockIdx.x * 8 + warp) * 32;
    if (p0 >= a.Pw) {
        grid_wait();
        return;
    }
    const int p = p0 + lane;
    int tok = p < a.P ? p : -1;
    if (a.tiled && tok >= 0) {
        int tc = a.choice ? __ldg(a.choice + bh) : 0;
        if (tc < 0 || tc >= a.n_tiles) tc = 0;  // the head is not computed
        uint32_t t, h, w;
        tile_coords_fast(p, a.divs[tc], t, h, w);
        tok = real_token(t, h, w, a.real);
    }
    const uint32_t bits = __ballot_sync(0xffffffffu, tok >= 0);
    if (a.valid && lane == 0) a.valid[static_cast<size_t>(bh) * (a.Pw / 32) + p0 / 32] = bits;
    const int sub = lane / LPR, at = lane % LPR;
    float delta = 0.f, size = 0.f;  // sums of g o and |g o|
    // eight groups of rows at a time: all their loads first (rows without a
    // token load the head's first row and count as zero)
    constexpr int U = 8;
    static_assert(32 % (U * ROWS) == 0, "groups of rows");
    #pragma unroll 1
    for (int r0 = 0; r0 < 32; r0 += U * ROWS) {
        uint4 gv[U], ov[U], lv[U];
        [[maybe_unused]] uint4 ow[U];  // fp32 o: the second four of a lane's eight values
        #pragma unroll
        for (int u = 0; u < U; ++u) {
            const int rt = max(__shfl_sync(0xffffffffu, tok, r0 + u * ROWS + sub), 0);
            const size_t e = (static_cast<size_t>(bh) * a.S_out + rt) * D + at * 8;
            gv[u] = __ldg(reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(a.g) + e));
            if constexpr (O_F32) {
                ov[u] = __ldg(reinterpret_cast<const uint4 *>(static_cast<const float *>(a.o) + e));
                ow[u] = __ldg(reinterpret_cast<const uint4 *>(static_cast<const float *>(a.o) + e + 4));
            } else {
                ov[u] = __ldg(reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(a.o) + e));
                lv[u] = make_uint4(0u, 0u, 0u, 0u);
                if (a.o_lo) lv[u] = __ldg(reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(a.o_lo) + e));
            }
        }
        #pragma unroll
        for (int u = 0; u < U; ++u) {
            const uint32_t gw[4] = {gv[u].x, gv[u].y, gv[u].z, gv[u].w};
            const uint32_t x[4] = {ov[u].x, ov[u].y, ov[u].z, ov[u].w};
            float o[8];
            if constexpr (O_F32) {
                const uint32_t y[4] = {ow[u].x, ow[u].y, ow[u].z, ow[u].w};
                #pragma unroll
                for (int c = 0; c < 4; ++c) {
                    o[c] = __uint_as_float(x[c]);
                    o[c + 4] = __uint_as_float(y[c]);
                }
            } else {
                const uint32_t y[4] = {lv[u].x, lv[u].y, lv[u].z, lv[u].w};
                #pragma unroll
                for (int c = 0; c < 4; ++c) {
                    o[2 * c] = __uint_as_float(x[c] << 16) + __uint_as_float(y[c] << 16);
                    o[2 * c + 1] = __uint_as_float(x[c] & 0xffff0000u) + __uint_as_float(y[c] & 0xffff0000u);
                }
            }
            float s = 0.f, n = 0.f;
            #pragma unroll
            for (int c = 0; c < 4; ++c) {
                const float g0 = __uint_as_float(gw[c] << 16), g1 = __uint_as_float(gw[c] & 0xffff0000u);
                s = fmaf(g0, o[2 * c], s);
                s = fmaf(g1, o[2 * c + 1], s);
                n = fmaf(fabsf(g0), fabsf(o[2 * c]), n);
                n = fmaf(fabsf(g1), fabsf(o[2 * c + 1]), n);
            }
            #pragma unroll
            for (int m = LPR / 2; m > 0; m >>= 1) {
                s += __shfl_xor_sync(0xffffffffu, s, m);
                n += __shfl_xor_sync(0xffffffffu, n, m);
            }
            // lane r0 + u ROWS + v keeps that row's sum, held by the lanes of group v
            #pragma unroll
            for (int v = 0; v < ROWS; ++v) {
                const float t = __shfl_sync(0xffffffffu, s, v * LPR), z = __shfl_sync(0xffffffffu, n, v * LPR);
                if (lane == r0 + u * ROWS + v) {
                    delta = t;
                    size = z;
                }
            }
        }
    }
    float nl = -INFINITY;
    if (tok >= 0) {
        const float l = __ldg(a.lse + static_cast<size_t>(bh) * a.S_out + tok);
        // -inf: no key was seen, no gradient.  +inf and NaN have no finite
        // softmax to differentiate; NaN lets the gradients show it.
        nl = l == -INFINITY ? -INFINITY : l == INFINITY ? NAN : -l * 1.4426950408889634f;
    }
    if (nl == -INFINITY) delta = 0.f;  // also a row that holds no token
    const size_t out = static_cast<size_t>(bh) * a.Pw + p;
    a.nlse[out] = nl;
    a.ndelta[out] = -delta;
    a.slack[out] = kSlack * size;
    grid_wait();
}

// kmean[bh][t][d]: the mean of the keys of block t (of its rows that hold one; 0
// if none does).  One CTA per block: thread (g, c) sums 8 columns of every (2048 / D)-th
// row; the rows' sums are joined in a fixed order.  Bandwidth bound: K read once.
template <int D, int BS>
__global__ void __launch_bounds__(256) block_means_kernel(const __grid_constant__ StatArgs a,
                                                          const __nv_bfloat16 *__restrict__ k, int nt,
                                                          float *__restrict__ kmean) {
    constexpr int CH = D / 8, GROUPS = 256 / CH;
    __shared__ float part[GROUPS][D + 8];
    const int t = blockIdx.x, bh = blockIdx.y, c = threadIdx.x % CH, g = threadIdx.x / CH;
    grid_release();
    int tc = a.tiled && a.choice ? __ldg(a.choice + bh) : 0;
    if (tc < 0 || tc >= a.n_tiles) tc = 0;  // the head is not computed
    float s[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    int rows = 0;
    #pragma unroll
    for (int i = 0; i < BS / GROUPS; ++i) {
        const int p = t * BS + i * GROUPS + g;
        int tok = p < a.P ? p : -1;
        if (a.tiled && tok >= 0) {
            uint32_t ft, fh, fw;
            tile_coords_fast(p, a.divs[tc], ft, fh, fw);
            tok = real_token(ft, fh, fw, a.real);
        }
        if (tok >= 0) {
            ++rows;
            const uint4 x = __ldg(reinterpret_cast<const uint4 *>(k + (static_cast<size_t>(bh) * a.S_out + tok) * D + c * 8));
            const uint32_t w[4] = {x.x, x.y, x.z, x.w};
            #pragma unroll
            for (int e = 0; e < 4; ++e) {
                s[2 * e] += __uint_as_float(w[e] << 16);
                s[2 * e + 1] += __uint_as_float(w[e] & 0xffff0000u);
            }
        }
    }
    #pragma unroll
    for (int e = 0; e < 8; ++e) part[g][c * 8 + e] = s[e];
    if (c == 0) part[g][D] = static_cast<float>(rows);
    __syncthreads();
    for (int d = threadIdx.x; d < D; d += 256) {
        float x = 0.f, n = 0.f;
        for (int y = 0; y < GROUPS; ++y) {
            x += part[y][d];
            n += part[y][D];
        }
        kmean[(static_cast<size_t>(bh) * nt + t) * D + d] = n > 0.f ? x / n : 0.f;
    }
    grid_wait();
}

size_t up256(size_t x) { return (x + 255) & ~size_t(255); }

struct Layout {
    size_t nlse, ndelta, slack, none, valid, kmean, t_off, t_rows, bits, part, bias, total;
};

Layout layout(int BH, int H, int positions, int S, int lists, int nb, int cap, int buckets, int far) {
    const size_t Pw = (static_cast<size_t>(positions) + 127) / 128 * 128;
    Layout L{};
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t o = at;
        at += up256(bytes);
        return o;
    };
    L.nlse = take(BH * Pw * 4);
    L.ndelta = take(BH * Pw * 4);
    L.slack = take(BH * Pw * 4);
    L.none = take(256 * 4);
    L.valid = take(BH * (Pw / 32) * 4);
    L.kmean = take(BH * (lists > 0 ? nb : Pw / 128) * 128 * 4);  // D <= 128
    if (lists > 0) {
        L.t_off = take(static_cast<size_t>(lists) * (nb + 1) * 4);
        L.t_rows = take(static_cast<size_t>(lists) * nb * cap * 4);
        L.bits = take(transpose_lists_workspace_bytes(lists, nb));
    }
    if (buckets > 0) {
        L.part = take(BH * (Pw / 128) * static_cast<size_t>(buckets) * 4);
        L.bias = take(bias_workspace_bytes(H, S, buckets, far));
    }
    L.total = at;
    return L;
}

}  // namespace

size_t backward_workspace_bytes(int BH, int H, int positions, int S, int lists, int nb, int cap, int buckets, int far) {
    return layout(BH, H, positions, S, lists, nb, cap, buckets, far).total;
}

vsa_status launch_backward(const BackwardLaunch &B, void *workspace, int *status, cudaStream_t st) {
    const AttnLaunch &L = B.a;
    const int positions = L.tiled ? L.Tp * L.Hp * L.Wp : L.S;
    const int lists = L.window ? 0 : L.list_per_head ? L.BH : 1;
    const int buckets = B.bias ? B.buckets : 0;
    const Layout lay = layout(L.BH, B.H, positions, L.S, lists, L.nb, L.cap, buckets, B.far);
    char *ws = static_cast<char *>(workspace);
    auto f32_at = [&](size_t o) { return reinterpret_cast<float *>(ws + o); };

    BwdArgs a{};
    a.P = positions;
    a.Pw = (positions + 127) / 128 * 128;
    a.S_out = L.S;
    a.BH = L.BH;
    a.H = B.H;
    a.nt = (positions + L.block - 1) / L.block;
    a.idx = L.idx;
    a.cnt = L.cnt;
    a.cap = L.cap;
    a.list_per_head = L.list_per_head;
    a.nb = L.nb;
    a.group = L.group;
    a.gstride = L.gstride;
    a.half = L.half;
    a.sink = L.sink;
    a.dense = L.dense;
    a.scale = L.scale;
    a.scale_log2 = L.scale * 1.4426950408889634f;
    a.nlse = f32_at(lay.nlse);
    a.ndelta = f32_at(lay.ndelta);
    a.ndelta_out = f32_at(lay.ndelta);
    a.slack = f32_at(lay.slack);
    a.none = f32_at(lay.none);
    a.out_f32 = B.grad_f32;
    a.status = status;
    a.real = RealGrid{L.T, L.Hg, L.Wg};
    a.tiles = L.tiles;
    a.choice = L.choice;
    a.H2 = L.Hp;
    a.W2 = L.Wp;
    const bool padded = L.tiled && positions != L.S;
    if (padded) a.valid = reinterpret_cast<const uint32_t *>(ws + lay.valid);

    StatArgs s{};
    s.o = B.o;
    s.o_lo = B.o_lo;
    s.g = B.g;
    s.lse = B.lse;
    s.P = a.P;
    s.Pw = a.Pw;
    s.S_out = L.S;
    s.real = a.real;
    s.tiled = L.tiled;
    s.n_tiles = L.tiles.n;
    s.choice = L.choice;
    s.nlse = f32_at(lay.nlse);
    s.ndelta = f32_at(lay.ndelta);
    s.slack = f32_at(lay.slack);
    s.none = f32_at(lay.none);
    s.valid = padded ? reinterpret_cast<uint32_t *>(ws + lay.valid) : nullptr;

    BwdMaps maps = {};
    bool ok = true;
    if (L.tiled) {
        for (int c = 0; c < L.tiles.n; ++c) {
            const int tt = L.tiles.t[c], th = L.tiles.h[c], tw = L.tiles.w[c], m = tt * th * tw / L.block;
            s.divs[c] = make_tile_divs(L.Hp, L.Wp, tt, th, tw);
            auto &g = a.geom[c];
            g.m = make_fastdiv(m);
            g.nthw = make_fastdiv((L.Hp / th) * (L.Wp / tw));
            g.ntw = make_fastdiv(L.Wp / tw);
            g.bt = tt / m;
            // the real tensors: boxes reaching past them read zeros
            const struct { CUtensorMap *m; const void *x; } four[4] = {
                {&maps.q[c], L.q}, {&maps.k[c], L.k}, {&maps.v[c], L.v}, {&maps.g[c], B.g}};
            for (auto &f : four) ok = ok && make_box_map(f.m, f.x, L.D, L.T, L.Hg, L.Wg, L.BH, g.bt, th, tw);
        }
    } else {
        ok = make_tile_map(&maps.q[0], L.q, L.D, L.S, L.BH, L.block) &&
             make_tile_map(&maps.k[0], L.k, L.D, L.S, L.BH, L.block) &&
             make_tile_map(&maps.v[0], L.v, L.D, L.S, L.BH, L.block) &&
             make_tile_map(&maps.g[0], B.g, L.D, L.S, L.BH, L.block);
    }
    if (!ok) return fail(VSA_ERR_CUDA, "cuTensorMapEncodeTiled failed (driver entry point or arguments)");

    // one chain of launches (see chain.cuh): bias values, mean keys, row statistics, transposed lists, dQ, dK and dV, the bias's gradient
    if (buckets > 0) {
        const vsa_status r = check_cuda(launch_bias_expand(B.bias, B.bias_f32, B.H, L.S, buckets, B.far, ws + lay.bias,
                                                           &a.tab, &a.bm, st),
                                        "relative bias launch");
        if (r != VSA_OK) return r;
        a.R = bias_reach(L.S, B.far);
        a.buckets = buckets;
        a.dbias_part = B.dbias ? f32_at(lay.part) : nullptr;
    }
    {
        float *kmean = f32_at(lay.kmean);
        auto means = L.D == 128 ? (L.block == 128 ? block_means_kernel<128, 128> : L.block == 64 ? block_means_kernel<128, 64> : block_means_kernel<128, 32>)
                                : (L.block == 128 ? block_means_kernel<64, 128> : L.block == 64 ? block_means_kernel<64, 64> : block_means_kernel<64, 32>);
        const vsa_status r = check_cuda(launch_kernel(buckets > 0, means, dim3(a.nt, L.BH), dim3(256), 0, st, s,
                                                      static_cast<const __nv_bfloat16 *>(L.k), a.nt, kmean),
                                        "attention backward launch (mean keys)");
        if (r != VSA_OK) return r;
        a.kmean = kmean;
    }
    const dim3 grid((a.Pw / 32 + 7) / 8, L.BH);
    auto row_stats = L.D == 128 ? (B.o_f32 ? row_stats_kernel<128, true> : row_stats_kernel<128, false>)
                                : (B.o_f32 ? row_stats_kernel<64, true> : row_stats_kernel<64, false>);
    vsa_status r = check_cuda(launch_kernel(true, row_stats, grid, dim3(256), 0, st, s),
                              "attention backward launch (row statistics)");
    if (r != VSA_OK) return r;
    if (lists > 0) {
        int32_t *off = reinterpret_cast<int32_t *>(ws + lay.t_off), *rows = reinterpret_cast<int32_t *>(ws + lay.t_rows);
        r = check_cuda(launch_transpose_lists(L.idx, L.cnt, lists, L.nb, L.cap, off, rows, false, ws + lay.bits, status, true, st),
                       "attention backward launch (transposed lists)");
        if (r != VSA_OK) return r;
        a.t_off = off;
        a.t_rows = rows;
    }
    // the key blocks that the sinks are in are listed by every query block
    a.lead = L.window ? (L.dense ? 0 : (L.sink + 127) / 128) : 1;
    if (a.lead > a.nt) a.lead = a.nt;
    a.d0 = B.dq;
    r = launch_bwd_dq(maps, a, L.D, L.block, L.window, L.tiled, buckets > 0, st);
    if (r != VSA_OK) return r;
    a.d0 = B.dk;
    a.d1 = B.dv;
    r = launch_bwd_dkv(maps, a, L.D, L.block, L.window, L.tiled, buckets > 0, st);
    if (r != VSA_OK) return r;
    if (a.dbias_part)
        r = check_cuda(launch_dbias(a.dbias_part, L.BH / B.H, B.H, a.nt, buckets, B.dbias, B.bias_f32, st),
                       "relative bias gradient launch");
    return r;
}

}  // namespace vsa
