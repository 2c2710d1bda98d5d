// backward_dkv.cu -- dK and dV of block-sparse and sliding-window attention on
// tcgen05 tensor cores: one CTA per (key block, batch x head), walking the
// query blocks that list it (see backward.cuh for the mathematics).
//
// Everything is kept transposed, keys along the rows: per tile of 128 queries
//   S^T = K Q^T, dP^T = V g^T            (shared-memory operands)
//   P^T = 2^(scale_log2 S^T - lse), dX^T = P^T (dP^T - delta)   (registers)
//   dV += P^T g, dK += dX^T Q            (P^T and dX^T are tensor-memory operands)
// so that P and dX never leave the SM's tensor memory, K and V stay in shared
// memory, and only Q and g are streamed.  Tensor memory at D = 128 is full:
// S^T, dP^T, dV and dK, 128 columns each; P^T (bf16) is written over S^T and
// dX^T over dP^T, each half of the columns by the warps that read it.
//
// Blocks of 32 and 64 tokens: the rows past the block hold stale values that
// only reach their own (unwritten) rows; 4 or 2 listed query blocks fill the
// 128 columns of a tile, and the columns past the list's end repeat its last
// block with lse = +inf, i.e. P = 0.
//
// dbias: dX summed by the bucket of j - i, in fp32 from unrounded values.  A
// 32 x 32 piece whose offsets share one bucket (most do: buckets widen with
// distance) adds its row sums to a register, written out when the bucket
// changes; in the others each warp sums the diagonals by shuffles and then
// runs of equal buckets.  Every warp has its own partial sums, and all sums
// have one order.
#include "backward.cuh"

namespace vsa {

namespace {

template <int D>
struct DkvCfg {
    static constexpr int TILE = 128 * D * 2;
    static constexpr int NQ = D == 128 ? 2 : 3;  // ring of Q tiles with their lse and delta
    static constexpr int NG = D == 128 ? 2 : 3;  // ring of g tiles
    static constexpr int STAT = 2 * 128 * 4;
    static constexpr int N_BARS = 1 + 2 * NQ + 2 * NG + 7;
    static constexpr int SMEM = 1024 + (2 + NQ + NG) * TILE + NQ * STAT + N_BARS * 8 + 16;
    static_assert(SMEM <= 232448, "shared memory");
    static constexpr int S_COL = 0, DP_COL = 128, DV_COL = 256, DK_COL = 256 + D;
};

template <int D, int BS, bool WINDOW, bool TILED, bool BIAS>
__global__ void __launch_bounds__(kBwdThreads, 1)
bwd_dkv_kernel(const __grid_constant__ BwdMapsOf<TILED ? kMaxTiles : 1> maps, const __grid_constant__ BwdArgs a) {
    using C = DkvCfg<D>;
    constexpr int SLAB = 128 * 128, NSUB = 128 / BS;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *base = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *sK = base, *sV = sK + C::TILE;
    uint8_t *sQ = sV + C::TILE;
    uint8_t *sG = sQ + C::NQ * C::TILE;
    float *sStat = reinterpret_cast<float *>(sG + C::NG * C::TILE);  // [NQ][2][128]: -lse log2e, -delta
    uint64_t *kv_full = reinterpret_cast<uint64_t *>(sStat + C::NQ * 256);
    uint64_t *q_full = kv_full + 1, *q_empty = q_full + C::NQ;
    uint64_t *g_full = q_empty + C::NQ, *g_empty = g_full + C::NG;
    uint64_t *s_full = g_empty + C::NG, *p_full = s_full + 1, *dp_full = p_full + 1, *ds_full = dp_full + 1;
    uint64_t *dv_done = ds_full + 1, *dk_done = dv_done + 1, *mma_done = dk_done + 1;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(mma_done + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    float *sPart = reinterpret_cast<float *>(tmem_slot + 4);  // BIAS: [8 warps][kMaxBuckets]
    float *sTab = sPart + 8 * kMaxBuckets;                     // BIAS: [kMaxBuckets]

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // the leading key blocks of every head first (a sink block is listed by
    // every query block: the longest work goes first), then head by head
    int bh, kb;
    {
        const int id = blockIdx.x, first = a.lead * a.BH;
        if (id < first) {
            bh = id / a.lead;
            kb = id - bh * a.lead;
        } else {
            const int per = a.nt - a.lead;
            bh = (id - first) / per;
            kb = a.lead + (id - first) - bh * per;
        }
    }
    if (threadIdx.x == 0) {
        mbar_init(kv_full, 1);
        for (int s = 0; s < C::NQ; ++s) {
            mbar_init(&q_full[s], 1);
            mbar_init(&q_empty[s], 1);
        }
        for (int s = 0; s < C::NG; ++s) {
            mbar_init(&g_full[s], 1);
            mbar_init(&g_empty[s], 1);
        }
        mbar_init(s_full, 1);
        mbar_init(p_full, 8);
        mbar_init(dp_full, 1);
        mbar_init(ds_full, 8);
        mbar_init(dv_done, 1);
        mbar_init(dk_done, 1);
        mbar_init(mma_done, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 9) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    grid_wait();  // the lists, statistics and bias values below are the earlier kernels'
    if constexpr (BIAS) bias_table(sTab, a.tab, bh % a.H, a.buckets, threadIdx.x, kBwdThreads);
    int tc = 0;
    bool head_ok = true;
    if constexpr (TILED) {
        if (a.choice) tc = __ldg(a.choice + bh);
        if (tc < 0 || tc >= a.tiles.n) {  // the head is left unwritten (reported by the dQ pass)
            head_ok = false;
            tc = 0;
        }
    }
    // the query blocks to walk: a list, or a range of tiles in window mode
    const int32_t *list = nullptr;
    int count = 0, q_lo = 0;
    if constexpr (WINDOW) {
        const int ks = kb * 128;
        if (a.dense || ks < a.sink) {
            count = a.nt;
        } else {
            q_lo = max(0, ks - a.half) / 128;
            count = min(a.P - 1, ks + 127 + a.half) / 128 - q_lo + 1;
        }
    } else {
        const size_t ls = a.list_per_head ? bh : 0;
        const int32_t *off = a.t_off + ls * (a.nb + 1);
        const int o0 = chain_load(off + kb);
        count = chain_load(off + kb + 1) - o0;
        list = a.t_rows + ls * a.nb * a.cap + o0;
    }
    if (!head_ok) count = 0;
    if constexpr (TILED) {
        // a key block wholly in the padding has no row to write
        if (a.valid) {
            bool any = false;
            for (int u = 0; u < BS / 32; ++u)
                any = any || chain_load(a.valid + static_cast<size_t>(bh) * (a.Pw / 32) + kb * (BS / 32) + u) != 0;
            if (!any) count = 0;
        }
    }
    const int n = (count + NSUB - 1) / NSUB;
    auto qblock = [&](int x) { return WINDOW ? q_lo + x : chain_load(list + x); };
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // this CTA has its tensor memory: without a bias's gradient the next kernel is the
    // caller's, and may allocate some
    grid_release();
    const uint32_t tmem = *tmem_slot;

    if (warp == 8) {
        // ================= TMA producer =================
        if (lane == 0 && n > 0) {
            const CUtensorMap *mQ = &maps.q[tc], *mG = &maps.g[tc];
            tma_prefetch_desc(mQ);
            tma_prefetch_desc(mG);
            mbar_arrive_expect_tx(kv_full, 2 * BS * D * 2);
            bwd_load_block<D, BS, TILED>(sK, &maps.k[tc], kv_full, kb, bh, a, tc);
            bwd_load_block<D, BS, TILED>(sV, &maps.v[tc], kv_full, kb, bh, a, tc);
            bool ok = true;
            int jq = 0, jg = 0;
            for (int j = 0; j < n; ++j) {
                const int qs = j % C::NQ, gs = j % C::NG;
                if (j >= C::NQ && !mbar_wait(&q_empty[qs], ((j / C::NQ) - 1) & 1, abort_flag)) { ok = false; break; }
                mbar_arrive_expect_tx(&q_full[qs], C::TILE + C::STAT);
                #pragma unroll
                for (int u = 0; u < NSUB; ++u) {
                    const int x = j * NSUB + u;
                    const int b = qblock(min(x, count - 1));
                    bwd_load_block<D, BS, TILED>(sQ + qs * C::TILE + u * BS * 128, mQ, &q_full[qs], b, bh, a, tc);
                    const size_t at = static_cast<size_t>(bh) * a.Pw + static_cast<size_t>(b) * BS;
                    float *st = sStat + qs * 256 + u * BS;
                    bulk_load(st, x < count ? a.nlse + at : a.none, BS * 4, &q_full[qs]);
                    bulk_load(st + 128, x < count ? a.ndelta + at : a.none + 128, BS * 4, &q_full[qs]);
                }
                ++jq;
                if (j >= C::NG && !mbar_wait(&g_empty[gs], ((j / C::NG) - 1) & 1, abort_flag)) { ok = false; break; }
                mbar_arrive_expect_tx(&g_full[gs], C::TILE);
                #pragma unroll
                for (int u = 0; u < NSUB; ++u)
                    bwd_load_block<D, BS, TILED>(sG + gs * C::TILE + u * BS * 128, mG, &g_full[gs],
                                                 qblock(min(j * NSUB + u, count - 1)), bh, a, tc);
                ++jg;
            }
            if (!ok) {
                if (!*abort_flag) { report(a.status, DEV_TIMEOUT); *abort_flag = 1; }
                // let the loads already issued land before the CTA exits
                mbar_wait(kv_full, 0, nullptr);
                for (int c = max(0, jq - C::NQ); c < jq; ++c) mbar_wait(&q_full[c % C::NQ], (c / C::NQ) & 1, nullptr);
                for (int c = max(0, jg - C::NG); c < jg; ++c) mbar_wait(&g_full[c % C::NG], (c / C::NG) & 1, nullptr);
            }
        }
        __syncwarp();
    } else if (warp == 9) {
        // ================= MMA issuer =================
        //   S(0) dP(0) | per tile j: dV(j) S(j+1) dK(j) dP(j+1)
        // S(j+1) overwrites the P(j) that dV(j) reads and dP(j+1) the dX(j)
        // that dK(j) reads; an MMA only orders behind an earlier one with the
        // same accumulator, so each waits for the reader to complete.
        if (elect_one()) {
            constexpr uint32_t idesc_s = idesc_bf16_f32(128, 128, false);
            constexpr uint32_t idesc_d = idesc_bf16_f32(128, D, true);
            // the CTA holds all of tensor memory, so it starts at column 0
            constexpr uint32_t tm = 0;
            const uint64_t dK = sdesc_sw128(smem_u32(sK), 16, 1024), dV = sdesc_sw128(smem_u32(sV), 16, 1024);
            const uint64_t dQ = sdesc_sw128(smem_u32(sQ), 16, 1024), dG = sdesc_sw128(smem_u32(sG), 16, 1024);
            const uint64_t dQt = sdesc_sw128(smem_u32(sQ), SLAB, 1024), dGt = sdesc_sw128(smem_u32(sG), SLAB, 1024);
            constexpr uint64_t kT = C::TILE >> 4;
            bool ok = true;
            auto wait = [&](uint64_t *bar, uint32_t parity) { return mbar_wait(bar, parity, abort_flag); };
            auto score = [&](uint64_t A, uint64_t B, uint32_t d, uint64_t *bar) {
                #pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint64_t off = static_cast<uint64_t>(((kk >> 2) * SLAB + (kk & 3) * 32) >> 4);
                    umma_bf16(tm + d, A + off, B + off, idesc_s, kk > 0 ? 1u : 0u);
                }
                umma_commit(bar);
            };
            auto accum = [&](uint32_t A, uint64_t B, uint32_t d, bool first) {
                #pragma unroll
                for (int kk = 0; kk < 8; ++kk)
                    umma_bf16_ts(tm + d, tm + A + (kk >> 2) * 64 + (kk & 3) * 8,
                                 B + static_cast<uint64_t>((kk * 2048) >> 4), idesc_d, (kk > 0 || !first) ? 1u : 0u);
            };
            if (n > 0) {
                ok = wait(kv_full, 0) && wait(&q_full[0], 0);
                if (ok) {
                    tc_fence_after();
                    score(dK, dQ, C::S_COL, s_full);
                    ok = wait(&g_full[0], 0);
                }
                if (ok) {
                    tc_fence_after();
                    score(dV, dG, C::DP_COL, dp_full);
                }
                // ring positions of tiles j (qs, gs) and j + 1 (qn, gn, with their parities)
                int qs = 0, gs = 0, qn = 1, gn = 1, qp = 0, gp = 0;
                for (int j = 0; ok && j < n; ++j) {
                    if (!(ok = wait(p_full, j & 1))) break;
                    tc_fence_after();
                    accum(C::S_COL, dGt + gs * kT, C::DV_COL, j == 0);
                    umma_commit(dv_done);
                    umma_commit(&g_empty[gs]);
                    if (j + 1 < n) {
                        if (!(ok = wait(&q_full[qn], qp) && wait(dv_done, j & 1))) break;
                        tc_fence_after();
                        score(dK, dQ + qn * kT, C::S_COL, s_full);
                    }
                    if (!(ok = wait(ds_full, j & 1))) break;
                    tc_fence_after();
                    accum(C::DP_COL, dQt + qs * kT, C::DK_COL, j == 0);
                    umma_commit(dk_done);
                    umma_commit(&q_empty[qs]);
                    if (j + 1 < n) {
                        if (!(ok = wait(&g_full[gn], gp) && wait(dk_done, j & 1))) break;
                        tc_fence_after();
                        score(dV, dG + gn * kT, C::DP_COL, dp_full);
                    }
                    qs = qn;
                    gs = gn;
                    if (++qn == C::NQ) { qn = 0; qp ^= 1; }
                    if (++gn == C::NG) { gn = 0; gp ^= 1; }
                }
                if (!ok && !*abort_flag) { report(a.status, DEV_TIMEOUT); *abort_flag = 1; }
            }
            umma_commit(mma_done);
            mbar_wait(mma_done, 0, nullptr);
        }
        __syncwarp();
    } else {
        // ================= element-wise work (warps 0-7) =================
        // warp w: TMEM lanes (key rows) 32 (w % 4) .., columns (queries) 64 (w / 4) ..
        const int wq = warp & 3, hf = warp >> 2;
        const int row = wq * 32 + lane;
        const int p = kb * BS + row;                  // this row's key position
        const bool rows_live = wq * 32 < BS;          // warp-uniform
        const uint32_t t_lane = tmem + (static_cast<uint32_t>(wq * 32) << 16);
        const float sl2 = a.scale_log2;
        // the bias's gradient: per warp a partial sum for each bucket, and in
        // registers the sum of the bucket that the last uniform pieces were in
        [[maybe_unused]] float *part = sPart + warp * kMaxBuckets;
        [[maybe_unused]] float run_sum[2] = {0.f, 0.f};
        [[maybe_unused]] int run_bucket[2] = {-1, -1};
        auto flush = [&](int u) {
            float t = run_sum[u];
            #pragma unroll
            for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
            if (lane == 0 && run_bucket[u] >= 0) part[run_bucket[u]] += t;
            __syncwarp();
            run_sum[u] = 0.f;
        };
        // buckets of a query tile's three runs of 32 offsets (this lane's of each)
        [[maybe_unused]] int bk[3] = {0, 0, 0};
        [[maybe_unused]] auto fetch_buckets = [&](int j) {
            const int o0 = (kb - qblock(j)) * 128 - 64 * hf + wq * 32 + 32 - lane;
            #pragma unroll
            for (int u = 0; u < 3; ++u) bk[u] = bias_bucket(a.bm, a.R, o0 - 32 * u);
        };
        if constexpr (BIAS) {
            for (int b = lane; b < kMaxBuckets; b += 32) part[b] = 0.f;
            __syncwarp();
            if (n > 0) fetch_buckets(0);
        }
        bool ok = true;
        for (int j = 0; j < n; ++j) {
            if (BS < 128 && !rows_live) {  // rows past the block: keep the barriers' phases
                if (!__all_sync(0xffffffffu, mbar_wait(s_full, j & 1, abort_flag))) { ok = false; break; }
                if (lane == 0) mbar_arrive(p_full);
                if (!__all_sync(0xffffffffu, mbar_wait(dp_full, j & 1, abort_flag))) { ok = false; break; }
                if (lane == 0) mbar_arrive(ds_full);
                continue;
            }
            const int qs = j % C::NQ;
            // the statistics arrive with Q, before S is computed: -lse is in registers
            // by the time S is
            bool got = mbar_wait(&q_full[qs], (j / C::NQ) & 1, abort_flag);
            float nlr[64];
            {
                const float4 *nl = reinterpret_cast<const float4 *>(sStat + qs * 256 + 64 * hf);
                #pragma unroll
                for (int c4 = 0; c4 < 16; ++c4) {
                    const float4 l4 = nl[c4];
                    nlr[4 * c4] = l4.x;
                    nlr[4 * c4 + 1] = l4.y;
                    nlr[4 * c4 + 2] = l4.z;
                    nlr[4 * c4 + 3] = l4.w;
                }
            }
            got = got && mbar_wait(s_full, j & 1, abort_flag);
            if (!__all_sync(0xffffffffu, got)) {
                ok = false;
                break;
            }
            tc_fence_after();
            float pr[64];
            [[maybe_unused]] BiasPiece piece[2];
            {
                uint32_t x[64];
                tmem_ld32(t_lane + C::S_COL + 64 * hf, *reinterpret_cast<uint32_t(*)[32]>(&x[0]));
                tmem_ld32(t_lane + C::S_COL + 64 * hf + 32, *reinterpret_cast<uint32_t(*)[32]>(&x[32]));
                // which of the 64 columns this row's key is seen from
                uint32_t see[2] = {~0u, ~0u};
                bool masked = false;
                if constexpr (WINDOW) {
                    const int q0 = qblock(j) * 128, ks = kb * 128;
                    masked = ks + 128 > a.P || !(a.dense || ks + 128 <= a.sink ||
                                                 max(q0 + 127 - ks, ks + 127 - q0) <= a.half);
                    if (p >= a.P) {  // no such key: it must not reach dbias
                        see[0] = see[1] = 0u;
                    } else if (masked && !a.dense && p >= a.sink) {
                        #pragma unroll
                        for (int u = 0; u < 2; ++u)
                            see[u] = span_bits(q0 + 64 * hf + 32 * u, p - a.half, p + a.half + 1);
                    }
                    if constexpr (BIAS) {
                        // rows past the last have lse = +inf, which a NaN entry of the bias would turn into NaN
                        if (q0 + 128 > a.P) {
                            masked = true;
                            #pragma unroll
                            for (int u = 0; u < 2; ++u) see[u] &= span_bits(q0 + 64 * hf + 32 * u, 0, a.P);
                        }
                    }
                } else if (a.group > 0 || a.gstride > 1) {
                    masked = true;
                    #pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const int c = 64 * hf + 32 * u;
                        see[u] = group_bits(a, p, qblock(min(j * NSUB + c / BS, count - 1)) * BS + c % BS);
                    }
                }
                [[maybe_unused]] float flat[2] = {0.f, 0.f};
                if constexpr (BIAS) {
                    #pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        piece[u] = bias_piece(bk[u], bk[u + 1]);
                        if (piece[u].kind == BIAS_ONE) flat[u] = sTab[piece[u].first];
                    }
                }
                tmem_ld_wait();
                // the exponents, in place; the mask is one branch after all of them, so
                // that the exponentials below are one straight run
                const uint64_t sl2x2 = f32x2(sl2, sl2);
                #pragma unroll
                for (int c = 0; c < 64; c += 2) {
                    float y0, y1;
                    uint64_t b = f32x2(nlr[c], nlr[c + 1]);
                    if constexpr (BIAS) b = add_f32x2(b, f32x2(flat[c >> 5], flat[c >> 5]));
                    f32x2_split(fma_f32x2(f32x2(__uint_as_float(x[c]), __uint_as_float(x[c + 1])), sl2x2, b), y0, y1);
                    x[c] = __float_as_uint(y0);
                    x[c + 1] = __float_as_uint(y1);
                }
                if constexpr (BIAS) {
                    #pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        if (piece[u].kind == BIAS_TWO) {
                            const float b0 = sTab[piece[u].first], b1 = sTab[piece[u].second];
                            const uint32_t second = bias_second(piece[u], lane);
                            #pragma unroll
                            for (int c = 32 * u; c < 32 * u + 32; ++c)
                                x[c] = __float_as_uint(__uint_as_float(x[c]) + ((second >> (c & 31)) & 1u ? b1 : b0));
                        } else if (piece[u].kind == BIAS_MORE) {
                            const float lo = sTab[piece[u].lo], hi = sTab[piece[u].hi];
                            #pragma unroll
                            for (int c = 32 * u; c < 32 * u + 32; ++c)
                                x[c] = __float_as_uint(__uint_as_float(x[c]) + bias_at(lo, hi, c & 31, lane));
                        }
                    }
                }
                if (masked) {
                    #pragma unroll
                    for (int c = 0; c < 64; ++c)
                        if (!((see[c >> 5] >> (c & 31)) & 1u)) x[c] = 0xff800000u;  // -inf
                }
                #pragma unroll
                for (int c = 0; c < 64; ++c) pr[c] = ex2_approx(__uint_as_float(x[c]));
                // P enters dV rounded to bf16 (the MMA's operand type); dX below
                // uses it unrounded, so it is rounded once on its way to dK
                uint32_t pk[32];
                #pragma unroll
                for (int c = 0; c < 32; ++c) pk[c] = pack_bf16x2(pr[2 * c], pr[2 * c + 1]);
                tmem_st32(t_lane + C::S_COL + 64 * hf, pk);
                tmem_st_wait();
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(p_full);
            if (!__all_sync(0xffffffffu, mbar_wait(dp_full, j & 1, abort_flag))) { ok = false; break; }
            tc_fence_after();
            {
                const float4 *nd = reinterpret_cast<const float4 *>(sStat + qs * 256 + 128 + 64 * hf);
                uint32_t dsk[32];
                #pragma unroll
                for (int u = 0; u < 2; ++u) {
                    uint32_t x[32];
                    tmem_ld32(t_lane + C::DP_COL + 64 * hf + 32 * u, x);
                    tmem_ld_wait();
                    #pragma unroll
                    for (int c4 = 0; c4 < 8; ++c4) {
                        const float4 d4 = nd[8 * u + c4];
                        const float *q = &pr[32 * u + 4 * c4];
                        float y0, y1, y2, y3;
                        f32x2_split(mul_f32x2(f32x2(q[0], q[1]),
                                              add_f32x2(f32x2(__uint_as_float(x[4 * c4]), __uint_as_float(x[4 * c4 + 1])),
                                                        f32x2(d4.x, d4.y))),
                                    y0, y1);
                        f32x2_split(mul_f32x2(f32x2(q[2], q[3]),
                                              add_f32x2(f32x2(__uint_as_float(x[4 * c4 + 2]), __uint_as_float(x[4 * c4 + 3])),
                                                        f32x2(d4.z, d4.w))),
                                    y2, y3);
                        dsk[16 * u + 2 * c4] = pack_bf16x2(y0, y1);
                        dsk[16 * u + 2 * c4 + 1] = pack_bf16x2(y2, y3);
                        if constexpr (BIAS) {
                            float *q2 = &pr[32 * u + 4 * c4];
                            q2[0] = y0;
                            q2[1] = y1;
                            q2[2] = y2;
                            q2[3] = y3;
                        }
                    }
                }
                tmem_st32(t_lane + C::DP_COL + 64 * hf, dsk);
                tmem_st_wait();
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(ds_full);
            if constexpr (BIAS) {
                // the unrounded dX (in pr) by bucket, after the MMA has its operand
                #pragma unroll
                for (int u = 0; u < 2; ++u) {
                    if (!a.dbias_part) break;
                    if (piece[u].kind == BIAS_ONE) {
                        if (piece[u].first != run_bucket[u]) {
                            flush(u);
                            run_bucket[u] = piece[u].first;
                        }
                        uint64_t t0 = 0, t1 = 0;  // two pairs of fp32 zeros
                        #pragma unroll
                        for (int c = 32 * u; c < 32 * u + 32; c += 4) {
                            t0 = add_f32x2(t0, f32x2(pr[c], pr[c + 1]));
                            t1 = add_f32x2(t1, f32x2(pr[c + 2], pr[c + 3]));
                        }
                        float a0, a1;
                        f32x2_split(add_f32x2(t0, t1), a0, a1);
                        run_sum[u] += a0 + a1;
                    } else if (piece[u].kind == BIAS_TWO) {
                        const uint32_t second = bias_second(piece[u], lane);
                        float t0 = 0.f, t1 = 0.f;
                        #pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            if ((second >> i) & 1u) t1 += pr[32 * u + i];
                            else t0 += pr[32 * u + i];
                        }
                        #pragma unroll
                        for (int o = 16; o > 0; o >>= 1) {
                            t0 += __shfl_xor_sync(0xffffffffu, t0, o);
                            t1 += __shfl_xor_sync(0xffffffffu, t1, o);
                        }
                        if (lane == 0) {
                            part[piece[u].first] += t0;
                            part[piece[u].second] += t1;
                        }
                        __syncwarp();
                    } else {
                        // sums of the piece's diagonals: element (r, i) goes to lane (i - r) mod 32
                        float diag[2] = {0.f, 0.f};  // i - r = lane - 32 and lane
                        #pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            const float v = __shfl_sync(0xffffffffu, pr[32 * u + i], (i - lane) & 31);
                            if (i >= lane) diag[1] += v;
                            else diag[0] += v;
                        }
                        #pragma unroll
                        for (int m = 0; m < 2; ++m) {
                            // offsets fall with the lane, so equal buckets are neighbours:
                            // sum each run, its last lane adds to the warp's partial
                            const int b = m == 0 ? piece[u].lo : piece[u].hi;
                            float v = diag[m];
                            #pragma unroll
                            for (int x = 1; x < 32; x <<= 1) {
                                const float t = __shfl_up_sync(0xffffffffu, v, x);
                                const int tb = __shfl_up_sync(0xffffffffu, b, x);
                                if (lane >= x && tb == b) v += t;
                            }
                            const int next = __shfl_down_sync(0xffffffffu, b, 1);
                            if (lane == 31 || next != b) part[b] += v;
                            __syncwarp();
                        }
                    }
                }
                if (j + 1 < n) fetch_buckets(j + 1);
            }
        }
        if (!ok && !*abort_flag) { report(a.status, DEV_TIMEOUT); *abort_flag = 1; }
        if constexpr (BIAS) {
            if (a.dbias_part) {
                flush(0);
                flush(1);
            }
            named_barrier(1, 256);
            if (a.dbias_part && static_cast<int>(threadIdx.x) < a.buckets) {
                float t = 0.f;
                for (int x = 0; x < 8; ++x) t += sPart[x * kMaxBuckets + threadIdx.x];
                a.dbias_part[(static_cast<size_t>(bh) * a.nt + kb) * a.buckets + threadIdx.x] = t;
            }
        }

        // ---- epilogue: warps 0-3 write dV, warps 4-7 dK ----
        const int r = rows_live && row < BS && head_ok ? bwd_row_of<TILED>(p, a, tc) : -1;
        const size_t at = (static_cast<size_t>(bh) * a.S_out + max(r, 0)) * D;
        void *out = hf == 0 ? a.d1 : a.d0;
        if (ok && n > 0) {
            if (!__all_sync(0xffffffffu, mbar_wait(dk_done, (n - 1) & 1, abort_flag) &&
                                             mbar_wait(dv_done, (n - 1) & 1, abort_flag))) {
                if (!*abort_flag) { report(a.status, DEV_TIMEOUT); *abort_flag = 1; }
            } else if (rows_live) {
                tc_fence_after();
                const uint32_t col = hf == 0 ? C::DV_COL : C::DK_COL;
                const float f = hf == 0 ? 1.f : a.scale;
                #pragma unroll
                for (int c = 0; c < D / 32; ++c) {
                    uint32_t x[32];
                    tmem_ld32(t_lane + col + 32 * c, x);
                    tmem_ld_wait();
                    if (r >= 0) bwd_store32(x, f, out, a.out_f32, at + 32 * c);
                }
            }
        } else if (n == 0 && r >= 0) {
            bwd_zero_row(out, a.out_f32, at, D);  // no query block lists these keys
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

template <int D, int BS, bool WINDOW, bool TILED, bool BIAS>
vsa_status run(const BwdMaps &maps, const BwdArgs &a, cudaStream_t st) {
    using C = DkvCfg<D>;
    auto kern = bwd_dkv_kernel<D, BS, WINDOW, TILED, BIAS>;
    constexpr int smem = C::SMEM + (BIAS ? 9 * kMaxBuckets * 4 : 0);
    static_assert(smem <= 232448, "shared memory");
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return check_cuda(e, "cudaFuncSetAttribute(attention backward, dK and dV)");
    return check_cuda(launch_kernel(true, kern, dim3(static_cast<unsigned>(a.nt) * a.BH), dim3(kBwdThreads), smem, st,
                                    bwd_maps<TILED>(maps), a),
                      "attention backward launch (dK and dV)");
}

template <int D>
vsa_status pick(const BwdMaps &maps, const BwdArgs &a, int block, bool window, bool tiled, bool bias, cudaStream_t st) {
    if (window) return bias ? run<D, 128, true, false, true>(maps, a, st) : run<D, 128, true, false, false>(maps, a, st);
    if (tiled) {
        if (block == 128) return run<D, 128, false, true, false>(maps, a, st);
        return block == 64 ? run<D, 64, false, true, false>(maps, a, st) : run<D, 32, false, true, false>(maps, a, st);
    }
    if (block == 128) return run<D, 128, false, false, false>(maps, a, st);
    return block == 64 ? run<D, 64, false, false, false>(maps, a, st) : run<D, 32, false, false, false>(maps, a, st);
}

}  // namespace

vsa_status launch_bwd_dkv(const BwdMaps &maps, const BwdArgs &a, int D, int block, bool window, bool tiled, bool bias,
                          cudaStream_t st) {
    return D == 128 ? pick<128>(maps, a, block, window, tiled, bias, st) : pick<64>(maps, a, block, window, tiled, bias, st);
}

}  // namespace vsa
