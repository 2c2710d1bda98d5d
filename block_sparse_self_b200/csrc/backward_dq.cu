// backward_dq.cu -- dQ of block-sparse and sliding-window attention on tcgen05
// tensor cores: one CTA per (query block, batch x head), walking the key blocks
// of its list (see backward.cuh for the mathematics).  It also corrects delta
// by the row sums of dX for the dK/dV pass.
//
// Queries along the rows: per tile of 128 keys
//   S = Q K^T, dP = g V^T                  (shared-memory operands)
//   P = 2^(scale_log2 S - lse), dX = P (dP - delta)    (registers)
//   dQ += dX K                             (dX is a tensor-memory operand)
// Q and g stay in shared memory, K and V are streamed.  Tensor memory at
// D = 128: two S buffers, dP and dQ.  dX (bf16) is written over the S it came
// from, so the next tile's S is computed while this one is worked on, and dP
// is refilled as soon as it has been read.
//
// Centering: the keys that a row sees often have a mean far larger than their spread
// (neighbouring positions are alike, a projection has a bias), and then dQ, which only
// depends on the spread since sum_j dX_ij = 0, drowns in that mean times the errors of
// dX.  So the row's sum of dX as the MMA got it, times a vector close to its mean key,
// is taken off again at the end:
//   dQ_i = scale (sum_j dX_ij k_j - (sum_j dX_ij) c),
// an identity for any c.
//  - Lists: c is the mean of the listed blocks' mean keys.  Keys with a mean of 0, 1, 4 and
//    16 times their spread, lists of 12 of 40 blocks of 128: dQ's error against 64 bits is
//    2.4e-3 of its norm for each, without it 2.4, 3.5, 10.5 and 39e-3 (1.7e-3 is the rounding
//    to bf16).  The one sum also corrects delta; a sum of unrounded dX beside it would leave
//    dK at 2.34e-3 in place of 2.45e-3 and take another 2 % of the training step.  With
//    the blocks weighted by their mass of P, as for windows, dQ's error was 3.5 against
//    3.6e-3 for lists of 3 of 1080 blocks of 32, and equal from 5 blocks of 64 on.
//  - Windows: c is, per 32 rows, the mean key of every tile of 128 weighted with the mass
//    of P in it (from a quarter of the columns): a wide window's plain mean is far from
//    the keys at its middle.  4.1e-3 -> 2.6e-3 (window 4096, S = 16384), 4.6e-3 -> 2.6e-3
//    (window 159, S = 2048).
#include "backward.cuh"

namespace vsa {

namespace {

template <int D>
struct DqCfg {
    static constexpr int TILE = 128 * D * 2;
    static constexpr int NK = D == 128 ? 3 : 4;  // ring of K tiles
    static constexpr int NV = D == 128 ? 2 : 4;  // ring of V tiles
    static constexpr int N_BARS = 1 + 2 * NK + 2 * NV + 2 + 4;
    static constexpr int SMEM = 1024 + (2 + NK + NV) * TILE + N_BARS * 8 + 16 + 128 * 4;
    static_assert(SMEM <= 232448, "shared memory");
    static constexpr int DP_COL = 256, DQ_COL = 384;  // S buffers at 0 and 128
};

template <bool WINDOW>
struct KeyWalk {
    int n, r0_len, r1_start;  // window: key tiles [0, r0_len), then from r1_start on
    const int32_t *list;
    int count;
    __device__ __forceinline__ int at(int x) const {
        if constexpr (WINDOW) return x < r0_len ? x : r1_start + (x - r0_len);
        else return __ldg(list + x);
    }
};

template <int D, int BS, bool WINDOW, bool TILED, bool BIAS>
__global__ void __launch_bounds__(kBwdThreads, 1)
bwd_dq_kernel(const __grid_constant__ BwdMapsOf<TILED ? kMaxTiles : 1> maps, const __grid_constant__ BwdArgs a) {
    using C = DqCfg<D>;
    constexpr int SLAB = 128 * 128, NSUB = 128 / BS;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *base = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *sQ = base, *sG = sQ + C::TILE;
    uint8_t *sK = sG + C::TILE;
    uint8_t *sV = sK + C::NK * C::TILE;
    uint64_t *q_full = reinterpret_cast<uint64_t *>(sV + C::NV * C::TILE);
    uint64_t *k_full = q_full + 1, *k_empty = k_full + C::NK;
    uint64_t *v_full = k_empty + C::NK, *v_empty = v_full + C::NV;
    uint64_t *s_full = v_empty + C::NV;  // [2]
    uint64_t *dp_full = s_full + 2, *ds_full = dp_full + 1, *dq_done = ds_full + 1, *mma_done = dq_done + 1;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(mma_done + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    int *list_ok = reinterpret_cast<int *>(tmem_slot + 2);
    float *sSum = reinterpret_cast<float *>(tmem_slot + 4);  // [128]: row sums of the second half of the columns
    float *sTab = sSum + 128;                                // BIAS: [kMaxBuckets]

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int qb = blockIdx.x, bh = blockIdx.y;
    KeyWalk<WINDOW> w{};
    if constexpr (WINDOW) {
        const int q0 = qb * 128;
        if (a.dense) {
            w.r0_len = w.n = a.nt;
        } else {
            const int lo = max(0, q0 - a.half), hi = min(a.P, min(q0 + 128, a.P) + a.half);
            const int lb0 = lo / 128, lb1 = (hi + 127) / 128, sb = (a.sink + 127) / 128;
            if (sb == 0) {
                w.r1_start = lb0;
                w.n = lb1 - lb0;
            } else if (lb0 <= sb) {
                w.n = w.r0_len = max(lb1, sb);
            } else {
                w.r0_len = sb;
                w.r1_start = lb0;
                w.n = sb + (lb1 - lb0);
            }
        }
        w.count = w.n;
    } else {
        const size_t lrow = (a.list_per_head ? static_cast<size_t>(bh) * a.nb : 0) + qb;
        w.list = a.idx + lrow * a.cap;
        w.count = __ldg(a.cnt + lrow);
    }
    if (threadIdx.x == 0) {
        mbar_init(q_full, 1);
        for (int s = 0; s < C::NK; ++s) {
            mbar_init(&k_full[s], 1);
            mbar_init(&k_empty[s], 1);
        }
        for (int s = 0; s < C::NV; ++s) {
            mbar_init(&v_full[s], 1);
            mbar_init(&v_empty[s], 1);
        }
        mbar_init(&s_full[0], 1);
        mbar_init(&s_full[1], 1);
        mbar_init(dp_full, 1);
        mbar_init(ds_full, 8);
        mbar_init(dq_done, 1);
        mbar_init(mma_done, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if constexpr (!WINDOW) {
        if (warp == 0) {
            bool ok = w.count >= 1 && w.count <= a.cap;
            if (ok) {
                for (int j = lane; j < w.count; j += 32) {
                    const int v = __ldg(w.list + j);
                    ok = ok && v >= 0 && v < a.nb && (j == 0 || __ldg(w.list + j - 1) < v);
                }
            }
            ok = __all_sync(0xffffffffu, ok);
            if (lane == 0) *list_ok = ok ? 1 : 0;
        }
    }
    if (warp == 9) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    grid_wait();  // what comes before reads the caller's lists only
    if constexpr (BIAS) bias_table(sTab, a.tab, bh % a.H, a.buckets, threadIdx.x, kBwdThreads);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // only now that this CTA has its tensor memory: a CTA of the dK/dV pass on this SM
    // could take it first and would then wait for this one
    grid_release();
    const uint32_t tmem = *tmem_slot;
    bool head_ok = true;
    int tc = 0;
    if constexpr (!WINDOW) {
        if (!*list_ok) {  // the rows get zeros
            w.count = 0;
            if (threadIdx.x == 0) report(a.status, DEV_RUNTIME);
        }
    }
    if constexpr (TILED) {
        if (a.choice) tc = __ldg(a.choice + bh);
        if (tc < 0 || tc >= a.tiles.n) {  // the head is left unwritten
            if (threadIdx.x == 0) report(a.status, DEV_RUNTIME);
            head_ok = false;
            w.count = 0;
            tc = 0;
        }
        if (a.valid) {
            bool any = false;  // a query block wholly in the padding has no row to write
            for (int u = 0; u < BS / 32; ++u)
                any = any || chain_load(a.valid + static_cast<size_t>(bh) * (a.Pw / 32) + qb * (BS / 32) + u) != 0;
            if (!any) w.count = 0;
        }
    }
    if constexpr (!WINDOW) w.n = (w.count + NSUB - 1) / NSUB;
    const int n = w.n;

    if (warp == 8) {
        // ================= TMA producer =================
        if (lane == 0 && n > 0) {
            const CUtensorMap *mK = &maps.k[tc], *mV = &maps.v[tc];
            tma_prefetch_desc(mK);
            tma_prefetch_desc(mV);
            mbar_arrive_expect_tx(q_full, 2 * BS * D * 2);
            bwd_load_block<D, BS, TILED>(sQ, &maps.q[tc], q_full, qb, bh, a, tc);
            bwd_load_block<D, BS, TILED>(sG, &maps.g[tc], q_full, qb, bh, a, tc);
            bool ok = true;
            int jk = 0, jv = 0;
            for (int j = 0; j < n; ++j) {
                const int ks = j % C::NK, vs = j % C::NV;
                if (j >= C::NK && !mbar_wait(&k_empty[ks], ((j / C::NK) - 1) & 1, abort_flag)) { ok = false; break; }
                mbar_arrive_expect_tx(&k_full[ks], C::TILE);
                #pragma unroll
                for (int u = 0; u < NSUB; ++u)
                    bwd_load_block<D, BS, TILED>(sK + ks * C::TILE + u * BS * 128, mK, &k_full[ks],
                                                 w.at(min(j * NSUB + u, w.count - 1)), bh, a, tc);
                ++jk;
                if (j >= C::NV && !mbar_wait(&v_empty[vs], ((j / C::NV) - 1) & 1, abort_flag)) { ok = false; break; }
                mbar_arrive_expect_tx(&v_full[vs], C::TILE);
                #pragma unroll
                for (int u = 0; u < NSUB; ++u)
                    bwd_load_block<D, BS, TILED>(sV + vs * C::TILE + u * BS * 128, mV, &v_full[vs],
                                                 w.at(min(j * NSUB + u, w.count - 1)), bh, a, tc);
                ++jv;
            }
            if (!ok) {
                if (!*abort_flag) { report(a.status, DEV_TIMEOUT); *abort_flag = 1; }
                // let the loads already issued land before the CTA exits
                mbar_wait(q_full, 0, nullptr);
                for (int c = max(0, jk - C::NK); c < jk; ++c) mbar_wait(&k_full[c % C::NK], (c / C::NK) & 1, nullptr);
                for (int c = max(0, jv - C::NV); c < jv; ++c) mbar_wait(&v_full[c % C::NV], (c / C::NV) & 1, nullptr);
            }
        }
        __syncwarp();
    } else if (warp == 9) {
        // ================= MMA issuer =================
        //   S(0) dP(0) S(1) | per tile j, once dX(j) is written: dQ(j) dP(j+1) S(j+2)
        // S(j+2) overwrites the dX(j) that dQ(j) reads and waits for it to
        // complete, with dP(j+1) in the pipe meanwhile.
        if (elect_one()) {
            constexpr uint32_t idesc_s = idesc_bf16_f32(128, 128, false);
            constexpr uint32_t idesc_d = idesc_bf16_f32(128, D, true);
            // the CTA holds all of tensor memory, so it starts at column 0
            constexpr uint32_t tm = 0;
            const uint64_t dQ = sdesc_sw128(smem_u32(sQ), 16, 1024), dG = sdesc_sw128(smem_u32(sG), 16, 1024);
            const uint64_t dK = sdesc_sw128(smem_u32(sK), 16, 1024), dV = sdesc_sw128(smem_u32(sV), 16, 1024);
            const uint64_t dKt = sdesc_sw128(smem_u32(sK), SLAB, 1024);
            constexpr uint64_t kT = C::TILE >> 4;
            bool ok = true;
            auto wait = [&](uint64_t *bar, uint32_t parity) { return mbar_wait(bar, parity, abort_flag); };
            auto score = [&](uint64_t A, uint64_t B, uint32_t d) {
                #pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint64_t off = static_cast<uint64_t>(((kk >> 2) * SLAB + (kk & 3) * 32) >> 4);
                    umma_bf16(tm + d, A + off, B + off, idesc_s, kk > 0 ? 1u : 0u);
                }
            };
            // ring positions, advanced without divisions
            int ks = 0, kp = 0, vs = 0, vp = 0, kd = 0;
            auto s_tile = [&](int j) -> bool {
                if (!wait(&k_full[ks], kp)) return false;
                if (j >= 2 && !wait(dq_done, (j - 2) & 1)) return false;
                tc_fence_after();
                score(dQ, dK + ks * kT, (j & 1) * 128);
                umma_commit(&s_full[j & 1]);
                if (++ks == C::NK) { ks = 0; kp ^= 1; }
                return true;
            };
            auto dp_tile = [&]() -> bool {
                if (!wait(&v_full[vs], vp)) return false;
                tc_fence_after();
                score(dG, dV + vs * kT, C::DP_COL);
                umma_commit(dp_full);
                umma_commit(&v_empty[vs]);
                if (++vs == C::NV) { vs = 0; vp ^= 1; }
                return true;
            };
            if (n > 0) {
                ok = wait(q_full, 0) && s_tile(0) && dp_tile() && (n < 2 || s_tile(1));
                for (int j = 0; ok && j < n; ++j) {
                    if (!(ok = wait(ds_full, j & 1))) break;
                    tc_fence_after();
                    const uint32_t A = tm + (j & 1) * 128;
                    #pragma unroll
                    for (int kk = 0; kk < 8; ++kk)
                        umma_bf16_ts(tm + C::DQ_COL, A + (kk >> 2) * 64 + (kk & 3) * 8,
                                     dKt + kd * kT + static_cast<uint64_t>((kk * 2048) >> 4), idesc_d,
                                     (kk > 0 || j > 0) ? 1u : 0u);
                    umma_commit(dq_done);
                    umma_commit(&k_empty[kd]);
                    if (++kd == C::NK) kd = 0;
                    if (j + 1 < n) ok = dp_tile();
                    if (ok && j + 2 < n) ok = s_tile(j + 2);
                }
                if (!ok && !*abort_flag) { report(a.status, DEV_TIMEOUT); *abort_flag = 1; }
            }
            umma_commit(mma_done);
            mbar_wait(mma_done, 0, nullptr);
        }
        __syncwarp();
    } else {
        // ================= element-wise work (warps 0-7) =================
        // warp w: TMEM lanes (query rows) 32 (w % 4) .., columns (keys) 64 (w / 4) ..
        const int wq = warp & 3, hf = warp >> 2;
        const int row = wq * 32 + lane;
        const int p = qb * BS + row;          // this row's query position
        const bool rows_live = wq * 32 < BS;  // warp-uniform
        const uint32_t t_lane = tmem + (static_cast<uint32_t>(wq * 32) << 16);
        const float sl2 = a.scale_log2;
        float nl = -INFINITY, nd = 0.f;
        if (row < BS && p < a.Pw) {
            nl = chain_load(a.nlse + static_cast<size_t>(bh) * a.Pw + p);
            nd = chain_load(a.ndelta + static_cast<size_t>(bh) * a.Pw + p);
        }
        // the row's sum of dX, unrounded and as rounded; windows: the mass of P in this
        // warp's columns; sum of mean keys, in windows times their mass (columns CPL lane ..)
        constexpr int CPL = D / 32;
        [[maybe_unused]] float row_sum[2] = {0.f, 0.f}, mass = 0.f;
        float used_sum[2] = {0.f, 0.f}, center[CPL];
        #pragma unroll
        for (int e = 0; e < CPL; ++e) center[e] = 0.f;
        // += f times the mean key of the x-th listed block
        auto add_mean = [&](int x, float f, float (&to)[CPL]) {
            const float *km = a.kmean + (static_cast<size_t>(bh) * a.nt + w.at(x)) * D + CPL * lane;
            #pragma unroll
            for (int e = 0; e < CPL; ++e) to[e] = fmaf(f, chain_load(km + e), to[e]);
        };
        // buckets of a key tile's three runs of 32 offsets (this lane's of each)
        [[maybe_unused]] int bk[3] = {0, 0, 0};
        [[maybe_unused]] auto fetch_buckets = [&](int j) {
            const int o0 = (w.at(j) - qb) * 128 + 64 * hf - wq * 32 - 32 + lane;
            #pragma unroll
            for (int u = 0; u < 3; ++u) bk[u] = bias_bucket(a.bm, a.R, o0 + 32 * u);
        };
        if constexpr (BIAS) {
            if (n > 0) fetch_buckets(0);
        }
        if constexpr (!WINDOW) {
            // every eighth listed block per warp, before the first scores are there
            #pragma unroll 4
            for (int x = warp; x < w.count; x += 8) add_mean(x, 1.f, center);
        }
        bool ok = true;
        for (int j = 0; j < n; ++j) {
            if (BS < 128 && !rows_live) {  // rows past the block: keep the barriers' phases
                if (!__all_sync(0xffffffffu, mbar_wait(&s_full[j & 1], (j >> 1) & 1, abort_flag))) { ok = false; break; }
                if (!__all_sync(0xffffffffu, mbar_wait(dp_full, j & 1, abort_flag))) { ok = false; break; }
                if (lane == 0) mbar_arrive(ds_full);
                continue;
            }
            // which of the 64 columns this row sees
            uint32_t see[2] = {~0u, ~0u};
            bool masked = false;
            {
                if constexpr (WINDOW) {
                    const int q0 = qb * 128, ks = w.at(j) * 128;
                    masked = !((ks + 128 <= a.P) && (a.dense || ks + 128 <= a.sink ||
                                                     max(min(q0 + 128, a.P) - 1 - ks, ks + 127 - q0) <= a.half));
                    if (masked) {
                        #pragma unroll
                        for (int u = 0; u < 2; ++u) {
                            const int c = ks + 64 * hf + 32 * u;
                            see[u] = a.dense ? ~0u : span_bits(c, p - a.half, p + a.half + 1) | span_bits(c, 0, a.sink);
                            see[u] &= span_bits(c, 0, a.P);
                        }
                    }
                } else {
                    if (a.group > 0 || a.gstride > 1 || a.valid || w.count % NSUB != 0) {
                        masked = true;
                        #pragma unroll
                        for (int u = 0; u < 2; ++u) {
                            const int c = 64 * hf + 32 * u, x = j * NSUB + c / BS;
                            const int kc = w.at(min(x, w.count - 1)) * BS + c % BS;
                            if (a.group > 0 || a.gstride > 1) see[u] = group_bits(a, p, kc);
                            if (a.valid) see[u] &= chain_load(a.valid + static_cast<size_t>(bh) * (a.Pw / 32) + kc / 32);
                            if (x >= w.count) see[u] = 0u;  // past the list's end: its last block again
                        }
                    }
                }
            }
            [[maybe_unused]] float mean[CPL] = {};
            if constexpr (WINDOW) add_mean(j, 1.f, mean);
            if (!__all_sync(0xffffffffu, mbar_wait(&s_full[j & 1], (j >> 1) & 1, abort_flag))) { ok = false; break; }
            tc_fence_after();
            float pr[64];
            {
                uint32_t x[64];
                tmem_ld32(t_lane + (j & 1) * 128 + 64 * hf, *reinterpret_cast<uint32_t(*)[32]>(&x[0]));
                tmem_ld32(t_lane + (j & 1) * 128 + 64 * hf + 32, *reinterpret_cast<uint32_t(*)[32]>(&x[32]));
                [[maybe_unused]] float flat[2] = {0.f, 0.f};
                [[maybe_unused]] BiasPiece piece[2];
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
                    const float y0 = BIAS ? nl + flat[c >> 5] : nl;
                    float y[2];
                    f32x2_split(fma_f32x2(f32x2(__uint_as_float(x[c]), __uint_as_float(x[c + 1])), sl2x2, f32x2(y0, y0)),
                                y[0], y[1]);
                    x[c] = __float_as_uint(y[0]);
                    x[c + 1] = __float_as_uint(y[1]);
                }
                if constexpr (BIAS) {
                    #pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        // shuffles for both other kinds: here a path of selects for one border
                        // measured 2.25 ms against 2.17 (S = 30720, 24 heads, 64 buckets to 2048)
                        if (piece[u].kind != BIAS_ONE) {
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
            }
            if constexpr (WINDOW) {
                float m = 0.f;
                #pragma unroll
                for (int c = 0; c < 64; c += 4) m += pr[c];
                m = m < 1e30f ? m : 0.f;  // a row that is not finite must not reach its neighbours
                #pragma unroll
                for (int o = 16; o > 0; o >>= 1) m += __shfl_xor_sync(0xffffffffu, m, o);
                mass += m;
                #pragma unroll
                for (int e = 0; e < CPL; ++e) center[e] = fmaf(m, mean[e], center[e]);
            }
            if (!__all_sync(0xffffffffu, mbar_wait(dp_full, j & 1, abort_flag))) { ok = false; break; }
            tc_fence_after();
            {
                uint32_t dsk[32];
                const uint64_t ndx2 = f32x2(nd, nd);
                #pragma unroll
                for (int u = 0; u < 2; ++u) {
                    uint32_t x[32];
                    tmem_ld32(t_lane + C::DP_COL + 64 * hf + 32 * u, x);
                    tmem_ld_wait();
                    #pragma unroll
                    for (int c = 0; c < 32; c += 2) {
                        float &d0 = pr[32 * u + c], &d1 = pr[32 * u + c + 1];
                        f32x2_split(mul_f32x2(f32x2(d0, d1),
                                              add_f32x2(f32x2(__uint_as_float(x[c]), __uint_as_float(x[c + 1])), ndx2)),
                                    d0, d1);
                        if constexpr (WINDOW) {
                            row_sum[0] += d0;
                            row_sum[1] += d1;
                        }
                        const uint32_t pk = pack_bf16x2(d0, d1);  // bf16: the type of the MMA's operand
                        add_bf16x2_f32(pk, used_sum[0], used_sum[1]);
                        dsk[16 * u + (c >> 1)] = pk;
                    }
                }
                tmem_st32(t_lane + (j & 1) * 128 + 64 * hf, dsk);
                tmem_st_wait();
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(ds_full);
            if constexpr (BIAS) {
                if (j + 1 < n) fetch_buckets(j + 1);
            }
        }
        if (!ok && !*abort_flag) { report(a.status, DEV_TIMEOUT); *abort_flag = 1; }
        // delta + the row's sum of dX, for the dK/dV pass (see backward.cuh)
        const float mine = WINDOW ? row_sum[0] + row_sum[1] : used_sum[0] + used_sum[1];
        if (hf == 1) sSum[row] = mine;
        named_barrier(1, 256);
        if (hf == 0 && ok && n > 0 && row < BS && nl != -INFINITY) {
            const float sum = mine + sSum[row];
            if (fabsf(sum) <= chain_load(a.slack + static_cast<size_t>(bh) * a.Pw + p))
                a.ndelta_out[static_cast<size_t>(bh) * a.Pw + p] = nd - sum;
        }

        // ---- epilogue: warps 0-3 write the first half of the columns, 4-7 the second ----
        const int r = rows_live && row < BS && head_ok ? bwd_row_of<TILED>(p, a, tc) : -1;
        const size_t at = (static_cast<size_t>(bh) * a.S_out + max(r, 0)) * D;
        bool have = ok && n > 0;
        // mma_done and not dq_done: that one has a phase per tile, and its parity alone does
        // not tell the last phase from the one before the last but one
        if (have && !__all_sync(0xffffffffu, mbar_wait(mma_done, 0, abort_flag))) {
            have = false;
            if (!*abort_flag) { report(a.status, DEV_TIMEOUT); *abort_flag = 1; }
        }
        // sums and mean keys of the two halves of the columns, or of all warps, meet in
        // the K ring, which nothing reads or fills any more
        float *sUsed = reinterpret_cast<float *>(sK), *sAll = sUsed + 256, *sMean = sAll + 256;  // [2][128] twice, [8][D + 1]
        float *sEven = sMean + 8 * (D + 1);                                                       // [D]
        if (have) {
            sUsed[hf * 128 + row] = used_sum[0] + used_sum[1];
            sAll[hf * 128 + row] = mine;
            #pragma unroll
            for (int e = 0; e < CPL; ++e) sMean[warp * (D + 1) + CPL * lane + e] = center[e];
            if (lane == 0) sMean[warp * (D + 1) + D] = mass;
        }
        named_barrier(1, 256);
        if constexpr (!WINDOW) {
            if (have && threadIdx.x < D) {
                float t = 0.f;
                for (int x = 0; x < 8; ++x) t += sMean[x * (D + 1) + threadIdx.x];
                sEven[threadIdx.x] = t / static_cast<float>(w.count);
            }
            named_barrier(1, 256);
        }
        if (have) {
            if (rows_live) {
                tc_fence_after();
                // the center first, then times the row's sum: a mass as small as fp32 has (all
                // weight on columns that do not count for it) would take the sum to infinity
                [[maybe_unused]] float inv = 0.f;
                [[maybe_unused]] const float *c0 = sMean + wq * (D + 1), *c1 = sMean + (wq + 4) * (D + 1);
                if constexpr (WINDOW) {
                    const float total = c0[D] + c1[D];
                    inv = total > 0.f ? 1.f / total : 0.f;
                }
                float used = sUsed[row] + sUsed[128 + row];
                // part of a softmax over more keys: what dX lost in rounding alone, if that is known
                const float sum = sAll[row] + sAll[128 + row];
                if (row < BS && p < a.Pw && !(fabsf(sum) <= chain_load(a.slack + static_cast<size_t>(bh) * a.Pw + p)))
                    used -= sum;
                #pragma unroll
                for (int c = 0; c < D / 64; ++c) {
                    uint32_t x[32];
                    const int col = hf * (D / 2) + 32 * c;
                    tmem_ld32(t_lane + C::DQ_COL + col, x);
                    tmem_ld_wait();
                    #pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        const float c = !WINDOW ? sEven[col + e] : (c0[col + e] + c1[col + e]) * inv;
                        x[e] = __float_as_uint(fmaf(-used, c, __uint_as_float(x[e])));
                    }
                    if (r >= 0) bwd_store32(x, a.scale, a.d0, a.out_f32, at + col);
                }
            }
        } else if (n == 0 && r >= 0 && hf == 0) {
            bwd_zero_row(a.d0, a.out_f32, at, D);  // an invalid list
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
    using C = DqCfg<D>;
    auto kern = bwd_dq_kernel<D, BS, WINDOW, TILED, BIAS>;
    constexpr int smem = C::SMEM + (BIAS ? kMaxBuckets * 4 : 0);
    static_assert(smem <= 232448, "shared memory");
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return check_cuda(e, "cudaFuncSetAttribute(attention backward, dQ)");
    return check_cuda(launch_kernel(true, kern, dim3(a.nt, a.BH), dim3(kBwdThreads), smem, st, bwd_maps<TILED>(maps), a),
                      "attention backward launch (dQ)");
}

template <int D, bool TILED>
vsa_status pick_lists(const BwdMaps &maps, const BwdArgs &a, int block, cudaStream_t st) {
    if (block == 128) return run<D, 128, false, TILED, false>(maps, a, st);
    return block == 64 ? run<D, 64, false, TILED, false>(maps, a, st)
                       : run<D, 32, false, TILED, false>(maps, a, st);
}

template <int D>
vsa_status pick(const BwdMaps &maps, const BwdArgs &a, int block, bool window, bool tiled, bool bias, cudaStream_t st) {
    if (window)
        return bias ? run<D, 128, true, false, true>(maps, a, st) : run<D, 128, true, false, false>(maps, a, st);
    return tiled ? pick_lists<D, true>(maps, a, block, st) : pick_lists<D, false>(maps, a, block, st);
}

}  // namespace

vsa_status launch_bwd_dq(const BwdMaps &maps, const BwdArgs &a, int D, int block, bool window, bool tiled, bool bias,
                         cudaStream_t st) {
    return D == 128 ? pick<128>(maps, a, block, window, tiled, bias, st) : pick<64>(maps, a, block, window, tiled, bias, st);
}

}  // namespace vsa
