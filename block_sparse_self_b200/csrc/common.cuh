// common.cuh -- device helpers shared by the libvsa kernels (sm_100a only):
// status reporting, bounded mbarrier waits, TMA tile loads, tcgen05
// (tensor-memory MMA) wrappers and shared-memory matrix descriptors.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/vsa.h"

namespace vsa {

// ---------------------------------------------------------------------------
// Device status word.  Kernels record the first failure with atomicCAS so
// that the earliest code wins; vsa_device_status() reads and clears it.
// ---------------------------------------------------------------------------
enum : int { DEV_OK = 0, DEV_RUNTIME = VSA_ERR_RUNTIME, DEV_TIMEOUT = VSA_ERR_TIMEOUT };

__device__ __forceinline__ void report(int *status, int code) {
    if (status) atomicCAS(status, 0, code);
}

// Default limit for any on-device wait: 2 s of device time.
constexpr uint64_t kWaitLimitNs = 2000000000ull;

// ---------------------------------------------------------------------------
// Shared-memory addresses, fences
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint32_t smem_u32(const void *p) {
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

__device__ __forceinline__ uint64_t global_timer_ns() {
    uint64_t t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}

// Make generic-proxy shared-memory writes visible to the async proxy
// (TMA, tensor core).
__device__ __forceinline__ void fence_proxy_async_smem() {
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// ---------------------------------------------------------------------------
// mbarrier
// ---------------------------------------------------------------------------
__device__ __forceinline__ void mbar_init(uint64_t *bar, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(count) : "memory");
}

__device__ __forceinline__ void fence_mbar_init() {
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}

__device__ __forceinline__ void mbar_arrive(uint64_t *bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

__device__ __forceinline__ void mbar_arrive_expect_tx(uint64_t *bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(bar)), "r"(bytes)
                 : "memory");
}

__device__ __forceinline__ bool mbar_try_wait(uint64_t *bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}

// Wait until the phase with the given parity has completed.  Gives up when
// `abort` (a shared flag) becomes non-zero or after limit_ns of device time;
// returns false in both cases.
__device__ __forceinline__ bool mbar_wait(uint64_t *bar, uint32_t parity, volatile int *abort,
                                          uint64_t limit_ns = kWaitLimitNs) {
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = global_timer_ns();
    while (true) {
        #pragma unroll 1
        for (int i = 0; i < 32; ++i)
            if (mbar_try_wait(bar, parity)) return true;
        if (abort && *abort) return false;
        if (global_timer_ns() - t0 > limit_ns) return false;
    }
}

// ---------------------------------------------------------------------------
// TMA (cp.async.bulk.tensor) tile loads into shared memory
// ---------------------------------------------------------------------------
__device__ __forceinline__ void tma_prefetch_desc(const CUtensorMap *map) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}

__device__ __forceinline__ void tma_load_3d(void *dst, const CUtensorMap *map, uint64_t *bar, int c0, int c1,
                                            int c2) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2)
        : "memory");
}

// 3-D tile store from shared memory (bulk-group completion); coordinates
// innermost first, none negative.
__device__ __forceinline__ void tma_store_3d(const CUtensorMap *map, const void *src, int c0, int c1, int c2) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];"
                 ::"l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(src)), "r"(c0), "r"(c1), "r"(c2)
                 : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
// at most N bulk groups still reading their shared-memory source
template <int N>
__device__ __forceinline__ void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory"); }
// all bulk groups complete (their writes performed)
__device__ __forceinline__ void bulk_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// 5-D tile load; coordinates innermost first.
__device__ __forceinline__ void tma_load_5d(void *dst, const CUtensorMap *map, uint64_t *bar, int c0, int c1, int c2,
                                            int c3, int c4) {
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4)
        : "memory");
}

// ---------------------------------------------------------------------------
// Division by a divisor fixed before the launch, as a multiply-high, an add
// and a shift (Granlund and Montgomery, "Division by invariant integers using
// multiplication", 1994): with l = ceil(log2 d) and
// mul = floor(2^32 (2^l - d) / d) + 1, n / d = (umulhi(mul, n) + n) >> l for
// every 32-bit n (the sum is taken in 64 bits).  Runtime divisions otherwise
// go through the reciprocal unit, which the softmax keeps busy.
// ---------------------------------------------------------------------------
struct FastDiv {
    uint32_t d, mul, shift;
};

inline FastDiv make_fastdiv(uint32_t d) {
    uint32_t l = 0;
    while ((uint64_t{1} << l) < d) ++l;
    const uint64_t mul = ((uint64_t{1} << 32) * ((uint64_t{1} << l) - d)) / d + 1;
    return FastDiv{d, static_cast<uint32_t>(mul), l};
}

__device__ __forceinline__ uint32_t fdiv(uint32_t n, const FastDiv &f) {
    return static_cast<uint32_t>((static_cast<uint64_t>(__umulhi(f.mul, n)) + n) >> f.shift);
}

// ---------------------------------------------------------------------------
// Tile-contiguous order ("ADR-0001", step 6; "Adaptive tiling (SPADE)",
// Recipe): position p holds the T-major token tile_token(p).  Tiles come in
// row-major tile order, the tokens of a tile in T-major order.
// ---------------------------------------------------------------------------
// (t, h, w) of position p in a grid of H x W frames (every axis a multiple of the tile's)
__device__ __forceinline__ void tile_coords(int p, int H, int W, int tt, int th, int tw, int &t, int &h, int &w) {
    const int vol = tt * th * tw;
    const int tile = p / vol, r = p - tile * vol;
    const int nth = H / th, ntw = W / tw;
    const int ct = tile / (nth * ntw);
    const int rem = tile - ct * (nth * ntw);
    const int ch = rem / ntw, cw = rem - ch * ntw;
    const int dt = r / (th * tw);
    const int r2 = r - dt * (th * tw);
    const int dh = r2 / tw, dw = r2 - dh * tw;
    t = ct * tt + dt;
    h = ch * th + dh;
    w = cw * tw + dw;
}

__device__ __forceinline__ int tile_token(int p, int H, int W, int tt, int th, int tw) {
    int t, h, w;
    tile_coords(p, H, W, tt, th, tw, t, h, w);
    return (t * H + h) * W + w;
}

// tile_token with every division by a per-tiling constant done as a
// multiply-shift (FastDiv); the divisors come from make_tile_divs on the host.
struct TileDivs {
    FastDiv vol, nthw, ntw, thw, tw;  // tile volume, tiles per frame, tiles per tile row, th*tw, tw
    int tt, th, H, W;
};

inline TileDivs make_tile_divs(int H, int W, int tt, int th, int tw) {
    TileDivs d;
    d.vol = make_fastdiv(static_cast<uint32_t>(tt * th * tw));
    d.nthw = make_fastdiv(static_cast<uint32_t>((H / th) * (W / tw)));
    d.ntw = make_fastdiv(static_cast<uint32_t>(W / tw));
    d.thw = make_fastdiv(static_cast<uint32_t>(th * tw));
    d.tw = make_fastdiv(static_cast<uint32_t>(tw));
    d.tt = tt;
    d.th = th;
    d.H = H;
    d.W = W;
    return d;
}

__device__ __forceinline__ void tile_coords_fast(uint32_t p, const TileDivs &d, uint32_t &t, uint32_t &h,
                                                 uint32_t &w) {
    const uint32_t tile = fdiv(p, d.vol), r = p - tile * d.vol.d;
    const uint32_t ct = fdiv(tile, d.nthw), rem = tile - ct * d.nthw.d;
    const uint32_t ch = fdiv(rem, d.ntw), cw = rem - ch * d.ntw.d;
    const uint32_t dt = fdiv(r, d.thw), r2 = r - dt * d.thw.d;
    const uint32_t dh = fdiv(r2, d.tw), dw = r2 - dh * d.tw.d;
    t = ct * d.tt + dt;
    h = ch * d.th + dh;
    w = cw * d.tw.d + dw;
}

__device__ __forceinline__ uint32_t tile_token_fast(uint32_t p, const TileDivs &d) {
    uint32_t t, h, w;
    tile_coords_fast(p, d, t, h, w);
    return (t * d.H + h) * d.W + w;
}

// A grid that the candidate tiles do not divide is zero-padded on each axis
// ("Adaptive tiling (SPADE)", Deviations and notes): positions and tilings
// refer to the padded grid (tile_coords over it), tensors hold only the real
// (T, H, W) tokens.  The real token at padded coordinates, or -1 for padding.
struct RealGrid {
    int T, H, W;
};
__device__ __forceinline__ int real_token(uint32_t t, uint32_t h, uint32_t w, const RealGrid &g) {
    if (t >= static_cast<uint32_t>(g.T) || h >= static_cast<uint32_t>(g.H) || w >= static_cast<uint32_t>(g.W)) return -1;
    return static_cast<int>((t * g.H + h) * g.W + w);
}

// ---------------------------------------------------------------------------
// tcgen05: tensor memory allocation, MMA, commit, loads and stores
// ---------------------------------------------------------------------------
__device__ __forceinline__ void tmem_alloc(uint32_t *dst_smem, uint32_t ncols) {  // whole warp
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst_smem)),
                 "r"(ncols)
                 : "memory");
}
__device__ __forceinline__ void tmem_relinquish() {  // whole warp
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc(uint32_t taddr, uint32_t ncols) {  // whole warp
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
__device__ __forceinline__ void tc_fence_before() {
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after() {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}

// One lane of a converged warp, the same on every call.  Code that issues
// tcgen05.mma goes behind this and not behind a lane number: the compiler then
// knows that a single thread is left and feeds the instruction's uniform
// operands directly.  Behind `lane == 0` a 128 x 128 x 16 MMA took 89 cycles to
// issue, behind elect.sync 60, i.e. its execution time (measured on the
// backward pass's dQ kernel without its element-wise work).
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

// D[tmem] (+)= A[smem desc] * B[smem desc]^T, bf16 inputs, fp32 accumulate.
__device__ __forceinline__ void umma_bf16(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                          uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// D[tmem] (+)= A[tmem] * B[smem desc]^T, bf16 inputs (A K-major in tensor
// memory: row m in lane m, elements k, k+1 packed in column k/2), fp32 accumulate.
__device__ __forceinline__ void umma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                             uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Arrive on `bar` once every tcgen05.mma issued so far by this thread completes.
__device__ __forceinline__ void umma_commit(uint64_t *bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                     smem_u32(bar))
                 : "memory");
}

// 32 lanes x 32 consecutive 32-bit columns: lane i of the warp gets row
// (lane base + i), columns [col, col + 32).
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
          "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]),
          "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]),
          "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
        "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
        "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]),
        "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]),
        "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]),
                 "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}
__device__ __forceinline__ void tmem_ld_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// ---------------------------------------------------------------------------
// Shared-memory matrix descriptor (tcgen05 format) for the 128-byte swizzle
// layout that a TMA load with CU_TENSOR_MAP_SWIZZLE_128B produces: rows of
// 128 bytes, groups of 8 rows 1024 bytes apart, 16-byte chunks XOR-swizzled
// by (row % 8).  The tile base must be 1024-byte aligned.
//   K-major operand:  lbo unused (16), sbo = 1024 (8-row group stride).
//   MN-major operand: lbo = stride between 64-element MN chunks,
//                     sbo = 1024 (stride between groups of 8 K rows).
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint64_t sdesc_sw128(uint32_t saddr, uint32_t lbo_bytes, uint32_t sbo_bytes) {
    uint64_t d = 0;
    d |= static_cast<uint64_t>((saddr >> 4) & 0x3FFFu);
    d |= static_cast<uint64_t>((lbo_bytes >> 4) & 0x3FFFu) << 16;
    d |= static_cast<uint64_t>((sbo_bytes >> 4) & 0x3FFFu) << 32;
    d |= static_cast<uint64_t>(1) << 46;  // descriptor version for sm_100
    d |= static_cast<uint64_t>(2) << 61;  // 128-byte swizzle
    return d;
}

// Instruction descriptor for kind::f16 with bf16 A and B, fp32 D, A K-major.
__host__ __device__ constexpr uint32_t idesc_bf16_f32(int M, int N, bool b_mn_major) {
    return (1u << 4)                              // D format: f32
           | (1u << 7)                            // A format: bf16
           | (1u << 10)                           // B format: bf16
           | ((b_mn_major ? 1u : 0u) << 16)       // B major-ness
           | (static_cast<uint32_t>(N >> 3) << 17)  // N / 8
           | (static_cast<uint32_t>(M >> 4) << 24); // M / 16
}

// ---------------------------------------------------------------------------
// Small numeric helpers
// ---------------------------------------------------------------------------
__device__ __forceinline__ float ex2_approx(float x) {  // hardware 2^x
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Two-wide fp32 arithmetic (one instruction for a pair; each half rounds
// exactly as the scalar operation would).
__device__ __forceinline__ uint64_t f32x2(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void f32x2_split(uint64_t v, float &lo, float &hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add_f32x2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// Bits [lo, hi) of the 32 columns that start at `base`.
__device__ __forceinline__ uint32_t span_bits(int base, int lo, int hi) {
    const int x = min(max(lo - base, 0), 32), y = min(max(hi - base, 0), 32);
    const uint32_t below_y = y >= 32 ? ~0u : (1u << y) - 1u, below_x = x >= 32 ? ~0u : (1u << x) - 1u;
    return below_y & ~below_x;
}

__device__ __forceinline__ float fmax3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// Named barrier over `count` threads (a multiple of 32); id 0 is __syncthreads.
__device__ __forceinline__ void named_barrier(int id, int count) {
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(count) : "memory");
}

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
    __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t *>(&v);
}

// 32 values x f less their bf16 rounding, rounded to bf16 themselves: with the
// rounded values they hold x f to 16 significant bits.
__device__ __forceinline__ void store_remainder(const uint32_t (&x)[32], float f, __nv_bfloat16 *out) {
    uint4 *dst = reinterpret_cast<uint4 *>(out);
    #pragma unroll
    for (int e = 0; e < 4; ++e) {
        uint32_t r[4];
        #pragma unroll
        for (int c = 0; c < 4; ++c) {
            const float a = __uint_as_float(x[8 * e + 2 * c]) * f, b = __uint_as_float(x[8 * e + 2 * c + 1]) * f;
            const uint32_t hi = pack_bf16x2(a, b);
            r[c] = pack_bf16x2(a - __uint_as_float(hi << 16), b - __uint_as_float(hi & 0xffff0000u));
        }
        dst[e] = make_uint4(r[0], r[1], r[2], r[3]);
    }
}

// acc_lo += low bf16 of pk, acc_hi += high bf16 of pk: sm_100 mixed-precision
// adds (the bf16 operand widens exactly, then one fp32 rounding), with no
// separate unpacking of the pair.
__device__ __forceinline__ void add_bf16x2_f32(uint32_t pk, float &acc_lo, float &acc_hi) {
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\t"
        "add.rn.f32.bf16 %0, lo, %0;\n\tadd.rn.f32.bf16 %1, hi, %1;\n\t}"
        : "+f"(acc_lo), "+f"(acc_hi)
        : "r"(pk));
}

}  // namespace vsa
