// transpose_lists.cu -- block lists turned round: for each key block the query
// blocks that list it, ascending, as offsets and one run of entries per list.
//
// Three small kernels over a bit matrix (nb x nb bits per list, one word per
// key block and 32 query blocks): set the bits of 32 query blocks' lists in
// shared memory and write them out; count and scan the bits of each key
// block; write the set bits out in order.  A bit has no order to lose, so the
// result is the same whatever order the lists are read in, and no entry is
// sorted.  The work is a few hundred thousand to a few million entries: what
// bounds it is the three launches, then L2.
#include "common.cuh"
#include "internal.h"

namespace vsa {

namespace {

constexpr int kKeysAtOnce = 8192;  // key blocks whose words a CTA holds (32 KB)

// One CTA per (32 query blocks, list).
__global__ void __launch_bounds__(256) list_bits_kernel(const int32_t *__restrict__ idx, const int32_t *__restrict__ cnt,
                                                        int nb, int cap, uint32_t *__restrict__ bits, int *status) {
    extern __shared__ uint32_t word[];
    const int col = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const size_t list = blockIdx.y;
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
            bool ok = n >= 0 && n <= cap;
            for (int j = lane; ok && j < n; j += 32) {
                const int v = __ldg(row + j);
                ok = v >= 0 && v < nb && (j == 0 || __ldg(row + j - 1) < v);
            }
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) {  // an invalid list names nothing
                if (lane == 0 && k0 == 0) report(status, DEV_RUNTIME);
                continue;
            }
            for (int j = lane; j < n; j += 32) {
                const int v = __ldg(row + j) - k0;
                if (v >= 0 && v < keys) atomicOr(&word[v], 1u << r);
            }
        }
        __syncthreads();
        for (int k = threadIdx.x; k < keys; k += 256) out[k0 + k] = word[k];
        __syncthreads();
    }
}

// One CTA per list: offsets[k] = entries of the key blocks before k.
__global__ void __launch_bounds__(1024) list_offsets_kernel(const uint32_t *__restrict__ bits, int nb, int cols,
                                                            int32_t *__restrict__ offsets) {
    __shared__ int warp_sum[32];
    const size_t list = blockIdx.x;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t *b = bits + list * cols * nb;
    int32_t *off = offsets + list * (nb + 1);
    int before = 0;
    for (int k0 = 0; k0 < nb; k0 += 1024) {
        const int k = k0 + threadIdx.x;
        int c = 0;
        if (k < nb) {
            #pragma unroll 8
            for (int i = 0; i < cols; ++i) c += __popc(__ldg(b + static_cast<size_t>(i) * nb + k));
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
__global__ void __launch_bounds__(256) list_rows_kernel(const uint32_t *__restrict__ bits,
                                                        const int32_t *__restrict__ offsets, int nb, int cols, int cap,
                                                        int fill, int32_t *__restrict__ rows) {
    const int key = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    const size_t list = blockIdx.y;
    if (key >= nb) return;
    const uint32_t *b = bits + list * cols * nb + key;
    int32_t *out = rows + list * nb * cap;
    int at = __ldg(offsets + list * (nb + 1) + key);
    for (int c0 = 0; c0 < cols; c0 += 32) {
        const int c = c0 + lane;
        uint32_t w = c < cols ? __ldg(b + static_cast<size_t>(c) * nb) : 0u;
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
        const int total = __ldg(offsets + list * (nb + 1) + nb);
        for (int e = key * cap + lane; e < (key + 1) * cap; e += 32)
            if (e >= total) out[e] = -1;
    }
}

}  // namespace

size_t transpose_lists_workspace_bytes(int lists, int nb) {
    return static_cast<size_t>(lists) * ((nb + 31) / 32) * nb * 4;
}

cudaError_t launch_transpose_lists(const int32_t *idx, const int32_t *cnt, int lists, int nb, int cap, int32_t *offsets,
                                   int32_t *rows, bool fill, void *workspace, int *status, cudaStream_t st) {
    uint32_t *bits = static_cast<uint32_t *>(workspace);
    const int cols = (nb + 31) / 32;
    list_bits_kernel<<<dim3(cols, lists), 256, (nb < kKeysAtOnce ? nb : kKeysAtOnce) * 4, st>>>(idx, cnt, nb, cap, bits,
                                                                                              status);
    list_offsets_kernel<<<lists, 1024, 0, st>>>(bits, nb, cols, offsets);
    list_rows_kernel<<<dim3((nb + 7) / 8, lists), 256, 0, st>>>(bits, offsets, nb, cols, cap, fill ? 1 : 0, rows);
    return cudaGetLastError();
}

}  // namespace vsa
