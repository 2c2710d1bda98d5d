// transpose_lists.cu -- block lists turned round: for each key block the query
// blocks that list it, ascending, as offsets and one run of entries per list.
//
// All work goes over a bit matrix (nb x nb bits per list, one word per key
// block and 32 query blocks): set the bits of the lists, count and scan the
// bits of each key block, write the set bits out in order.  A bit has no order
// to lose, so the result is the same whatever order the lists are read in, and
// no entry is sorted.
//
// A list of up to 128 blocks is turned by one CTA in shared memory: one launch,
// no workspace.  Longer ones go through global memory in three kernels, spread
// over the SMs.  What bounds both is latency (launches, then the lists' rows),
// not bytes.  24 lists, one CTA each against three kernels: 7 blocks 3.6 us against
// 5.0, 64 blocks 5.9 against 7.6, 120 blocks 9.0 against 8.6, 160 blocks 10.8 against
// 9.1, 240 blocks 17.3 against 8.9, 960 blocks 66.7 against 19.4 (launches in a row
// in a graph; called one by one three launches take the host 19.5 us and one 13.4).
#include "chain.cuh"
#include "common.cuh"
#include "internal.h"

namespace vsa {

namespace {

constexpr int kKeysAtOnce = 8192;  // key blocks whose words a CTA holds (32 KB)

// A warp reads and checks one query block's list: its first 128 entries, 32 u +
// lane in v[u], with all loads in flight at once; false if it is invalid (it
// then names nothing).
__device__ __forceinline__ bool list_row(const int32_t *row, int n, int nb, int cap, int lane, int (&v)[4]) {
    bool ok = n >= 0 && n <= cap;
    #pragma unroll
    for (int u = 0; u < 4; ++u) v[u] = ok && 32 * u + lane < n ? __ldg(row + 32 * u + lane) : -1;
    int last = -1;  // the entry before this run of 32
    #pragma unroll
    for (int u = 0; u < 4; ++u) {
        const int up = __shfl_up_sync(0xffffffffu, v[u], 1);
        if (32 * u + lane < n) ok = ok && v[u] >= 0 && v[u] < nb && (lane == 0 ? last : up) < v[u];
        last = __shfl_sync(0xffffffffu, v[u], 31);
    }
    for (int j = 128 + lane; ok && j < n; j += 32) {
        const int x = __ldg(row + j);
        ok = x >= 0 && x < nb && __ldg(row + j - 1) < x;
    }
    return __all_sync(0xffffffffu, ok) != 0;
}

// One CTA per (32 query blocks, list).
__global__ void __launch_bounds__(256) list_bits_kernel(const int32_t *__restrict__ idx, const int32_t *__restrict__ cnt,
                                                        int nb, int cap, uint32_t *__restrict__ bits, int *status) {
    extern __shared__ uint32_t word[];
    const int col = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const size_t list = blockIdx.y;
    grid_release();
    uint32_t *out = bits + (list * gridDim.x + col) * nb;
    for (int k0 = 0; k0 < nb; k0 += kKeysAtOnce) {
        const int keys = min(kKeysAtOnce, nb - k0);
        for (int k = threadIdx.x; k < keys; k += 256) word[k] = 0u;
        __syncthreads();
        for (int r = warp; r < 32; r += 8) {
            const int q = col * 32 + r;
            if (q >= nb) break;
            const int n = __ldg(cnt + list * nb + q);
            const int32_t *row = idx + (list * nb + q) * cap;
            int v[4];
            if (!list_row(row, n, nb, cap, lane, v)) {
                if (lane == 0 && k0 == 0) report(status, DEV_RUNTIME);
                continue;
            }
            #pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int x = v[u] - k0;
                if (32 * u + lane < n && x >= 0 && x < keys) atomicOr(&word[x], 1u << r);
            }
            for (int j = 128 + lane; j < n; j += 32) {
                const int x = __ldg(row + j) - k0;
                if (x >= 0 && x < keys) atomicOr(&word[x], 1u << r);
            }
        }
        __syncthreads();
        for (int k = threadIdx.x; k < keys; k += 256) out[k0 + k] = word[k];
        __syncthreads();
    }
    grid_wait();
}

// One CTA per list: offsets[k] = entries of the key blocks before k.
__global__ void __launch_bounds__(1024) list_offsets_kernel(const uint32_t *bits, int nb, int cols, int32_t *offsets) {
    __shared__ int warp_sum[32];
    const size_t list = blockIdx.x;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t *b = bits + list * cols * nb;
    int32_t *off = offsets + list * (nb + 1);
    grid_release();
    grid_wait();
    int before = 0;
    for (int k0 = 0; k0 < nb; k0 += 1024) {
        const int k = k0 + threadIdx.x;
        int c = 0;
        if (k < nb) {
            #pragma unroll 8
            for (int i = 0; i < cols; ++i) c += __popc(chain_load(b + static_cast<size_t>(i) * nb + k));
        }
        int s = c;
        #pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int t = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s += t;
        }
        if (lane == 31) warp_sum[warp] = s;
        __syncthreads();
        if (warp == 0) {
            int w = warp_sum[lane];
            #pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int t = __shfl_up_sync(0xffffffffu, w, o);
                if (lane >= o) w += t;
            }
            warp_sum[lane] = w;
        }
        __syncthreads();
        if (warp > 0) s += warp_sum[warp - 1];
        if (k < nb) off[k] = before + s - c;
        before += warp_sum[31];
        __syncthreads();
    }
    if (threadIdx.x == 0) off[nb] = before;
}

// One warp per (key block, list); also -1 behind the last entry when asked.
__global__ void __launch_bounds__(256) list_rows_kernel(const uint32_t *bits, const int32_t *offsets, int nb, int cols,
                                                        int cap, int fill, int32_t *rows) {
    const int key = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    const size_t list = blockIdx.y;
    grid_release();
    grid_wait();
    if (key >= nb) return;
    const uint32_t *b = bits + list * cols * nb + key;
    int32_t *out = rows + list * nb * cap;
    int at = chain_load(offsets + list * (nb + 1) + key);
    for (int c0 = 0; c0 < cols; c0 += 32) {
        const int c = c0 + lane;
        uint32_t w = c < cols ? chain_load(b + static_cast<size_t>(c) * nb) : 0u;
        int s = __popc(w);
        const int mine = s;
        #pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int t = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s += t;
        }
        for (int e = at + s - mine; w; ++e, w &= w - 1) out[e] = c * 32 + __ffs(w) - 1;
        at += __shfl_sync(0xffffffffu, s, 31);
    }
    if (fill) {
        const int total = chain_load(offsets + list * (nb + 1) + nb);
        for (int e = key * cap + lane; e < (key + 1) * cap; e += 32)
            if (e >= total) out[e] = -1;
    }
}

constexpr int kOneCtaBlocks = 128;
// words per column of the matrix in shared memory: odd, so that a warp that
// reads one key's words of 32 columns touches 32 banks
__host__ __device__ constexpr int one_cta_stride(int nb) { return nb | 1; }

// One CTA per list.
__global__ void __launch_bounds__(1024) list_turn_kernel(const int32_t *__restrict__ idx, const int32_t *__restrict__ cnt,
                                                         int nb, int cap, int32_t *__restrict__ offsets,
                                                         int32_t *__restrict__ rows, int fill, int *status) {
    extern __shared__ uint32_t word[];  // [cols][stride]
    __shared__ int warp_sum[32];
    __shared__ int start[kOneCtaBlocks];
    const int cols = (nb + 31) / 32, stride = one_cta_stride(nb);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const size_t list = blockIdx.x;
    grid_release();
    for (int e = threadIdx.x; e < cols * stride; e += 1024) word[e] = 0u;
    __syncthreads();
    for (int q = warp; q < nb; q += 32) {
        const int n = __ldg(cnt + list * nb + q);
        const int32_t *row = idx + (list * nb + q) * cap;
        int v[4];
        if (!list_row(row, n, nb, cap, lane, v)) {
            if (lane == 0) report(status, DEV_RUNTIME);
            continue;
        }
        uint32_t *col = word + (q >> 5) * stride;
        const uint32_t bit = 1u << (q & 31);
        #pragma unroll
        for (int u = 0; u < 4; ++u)
            if (32 * u + lane < n) atomicOr(col + v[u], bit);
        for (int j = 128 + lane; j < n; j += 32) atomicOr(col + __ldg(row + j), bit);
    }
    __syncthreads();
    static_assert(kOneCtaBlocks <= 1024, "one key block per thread");
    const int k1 = threadIdx.x;
    int c1 = 0;
    if (k1 < nb)
        for (int i = 0; i < cols; ++i) c1 += __popc(word[i * stride + k1]);
    int s1 = c1;
    #pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(0xffffffffu, s1, o);
        if (lane >= o) s1 += t;
    }
    if (lane == 31) warp_sum[warp] = s1;
    __syncthreads();
    int before = 0;  // of this warp's key blocks, then of all
    for (int w = 0; w < warp; ++w) before += warp_sum[w];
    if (k1 < nb) {
        start[k1] = before + s1 - c1;
        offsets[list * (nb + 1) + k1] = before + s1 - c1;
    }
    __syncthreads();
    before = 0;
    for (int w = 0; w < 32; ++w) before += warp_sum[w];
    if (threadIdx.x == 0) offsets[list * (nb + 1) + nb] = before;
    int32_t *out = rows + list * nb * cap;
    for (int k = warp; k < nb; k += 32) {
        int at = start[k];
        for (int c0 = 0; c0 < cols; c0 += 32) {
            const int c = c0 + lane;
            uint32_t w = c < cols ? word[c * stride + k] : 0u;
            int s = __popc(w);
            const int mine = s;
            #pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int t = __shfl_up_sync(0xffffffffu, s, o);
                if (lane >= o) s += t;
            }
            for (int e = at + s - mine; w; ++e, w &= w - 1) out[e] = c * 32 + __ffs(w) - 1;
            at += __shfl_sync(0xffffffffu, s, 31);
        }
    }
    if (fill)
        for (int e = before + threadIdx.x; e < nb * cap; e += 1024) out[e] = -1;
    grid_wait();
}

}  // namespace

size_t transpose_lists_workspace_bytes(int lists, int nb) {
    return nb <= kOneCtaBlocks ? 0 : static_cast<size_t>(lists) * ((nb + 31) / 32) * nb * 4;
}

cudaError_t launch_transpose_lists(const int32_t *idx, const int32_t *cnt, int lists, int nb, int cap, int32_t *offsets,
                                   int32_t *rows, bool fill, void *workspace, int *status, bool chained, cudaStream_t st) {
    const int cols = (nb + 31) / 32;
    if (nb <= kOneCtaBlocks) {
        const int smem = cols * one_cta_stride(nb) * 4;  // at most 2 KB
        return launch_kernel(chained, list_turn_kernel, dim3(lists), dim3(1024), smem, st, idx, cnt, nb, cap, offsets, rows,
                             fill ? 1 : 0, status);
    }
    uint32_t *bits = static_cast<uint32_t *>(workspace);
    cudaError_t e = launch_kernel(chained, list_bits_kernel, dim3(cols, lists), dim3(256),
                                  (nb < kKeysAtOnce ? nb : kKeysAtOnce) * 4, st, idx, cnt, nb, cap, bits, status);
    if (e == cudaSuccess) e = launch_kernel(true, list_offsets_kernel, dim3(lists), dim3(1024), 0, st, bits, nb, cols, offsets);
    if (e == cudaSuccess)
        e = launch_kernel(true, list_rows_kernel, dim3((nb + 7) / 8, lists), dim3(256), 0, st, bits, offsets, nb, cols, cap,
                          fill ? 1 : 0, rows);
    return e;
}

}  // namespace vsa
