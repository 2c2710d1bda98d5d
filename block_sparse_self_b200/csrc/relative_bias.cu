// relative_bias.cu -- the learned relative position bias of window attention:
// its buckets, its values by offset, and the last step of its gradient.
//
// A pair (query i, key j) of head h gets table[bucket(j - i)][h] added to its
// scaled logit.  With n = buckets / 2, e = n / 2 (rounded down) and
//   f(d) = d for d < e, else min(n - 1, e + floor((n - e) ln(d / e) / ln(far / e))),
// bucket(r) = f(|r|) + (n if r > 0).  f steps up where d reaches
// e (far / e)^(t / (n - e)); those borders are rounded up to whole numbers on
// the host (exactly), so the kernels only compare integers.
//
// The attention kernels read bucket(r) as a byte, for |r| <= R = min(far, S)
// (larger offsets fall into the last bucket of their side), and each head's
// values tab[h][b] = log2(e) table[b][h].
//
// Entries of a size at which fp32 no longer holds a logit beside them (a mask by
// -1e9) are moved closer.  The softmax of a row does not change when all its logits
// move together, and not either when a distance between them that leaves the lower
// one no weight becomes another such distance.  So where a head's entries, in order,
// leave a gap of more than 2839, the gap becomes 2839, and a head whose largest entry
// is beyond +-2839 moves to 0 as a whole: in the table's own units, where distances of
// close entries are exact.  A row that sees only entries below such a gap then has
// logits of about 2^12 (2839 log2 e), whose roundings move its probabilities by 2^-12
// of themselves, where at 1e9 nothing was left of them: P recomputed from lse summed
// to anything between 0.2 and 5200.
// Every row sees its own key, so nothing below that key's bucket needs an order of
// its own: all that is more than the gap below it is put at the gap.
#include <math.h>

#include "chain.cuh"
#include "common.cuh"
#include "internal.h"

namespace vsa {

namespace {

struct Borders {
    int e, n, steps;   // f(d) = d below e; then e + the borders that d has reached
    int at[128];
};

// A whole number of up to 2048 bits.
struct Whole {
    uint32_t w[64] = {1};
    int n = 1;  // words in use
    Whole &times(uint32_t x, int power) {
        for (; power > 0; --power) {
            uint64_t carry = 0;
            for (int i = 0; i < n; ++i) {
                carry += static_cast<uint64_t>(w[i]) * x;
                w[i] = static_cast<uint32_t>(carry);
                carry >>= 32;
            }
            if (carry) w[n++] = static_cast<uint32_t>(carry);
        }
        return *this;
    }
    bool operator>=(const Whole &o) const {
        if (n != o.n) return n > o.n;
        for (int i = n - 1; i > 0; --i)
            if (w[i] != o.w[i]) return w[i] > o.w[i];
        return w[0] >= o.w[0];
    }
};

// Whether d >= e (far / e)^(t / m), by whole numbers: d^m >= e^(m-t) far^t (at most
// 25 x 64 bits).
bool reaches(int d, int e, int far, int t, int m) {
    return Whole().times(d, m) >= Whole().times(e, m - t).times(far, t);
}

Borders make_borders(int buckets, int far) {
    Borders b{};
    b.n = buckets / 2;
    b.e = b.n / 2;
    const int m = b.n - b.e;
    for (int t = 1; t < m; ++t) {
        const long double x = static_cast<long double>(b.e) *
                              powl(static_cast<long double>(far) / b.e, static_cast<long double>(t) / m);
        // a border next to a whole number is that number or a little above it, which
        // no rounded power tells
        const int near = static_cast<int>(rintl(x));
        b.at[b.steps++] = fabsl(x - near) > 1e-12L * x ? static_cast<int>(ceill(x))
                                                       : reaches(near, b.e, far, t, m) ? near : near + 1;
    }
    return b;
}

__device__ __forceinline__ int bucket_of(int r, const Borders &b) {
    const int d = r < 0 ? -r : r;
    int f = d;
    if (d >= b.e) {
        f = b.e;
        for (int t = 0; t < b.steps; ++t) f += d >= b.at[t];
    }
    return f + (r > 0 ? b.n : 0);
}

__global__ void buckets_kernel(const Borders b, int far, int32_t *__restrict__ out) {
    const int x = blockIdx.x * 256 + threadIdx.x;
    if (x <= 2 * far) out[x] = bucket_of(x - far, b);
}

constexpr int kMost = 256;           // buckets
constexpr float kGap = 2839.f;       // the most that is left of a gap, and of the largest entry
constexpr float kMask = -0x1p127f;   // entries below it mask (times log2 e they would leave fp32)

__device__ __forceinline__ bool is_finite(float x) { return fabsf(x) <= 3.402823466e38f; }

// s[0 .. n): one head's entries, s[0] that of a row's own key.  Where
// this thread's entry goes (see above); called by all threads of the CTA.
__device__ float closer(const float *s, int n, int k, float top, float low, float *sorted, float *place) {
    const float mine = s[k];
    const float self = is_finite(s[0]) ? s[0] : low;
    const bool counts = k < n && is_finite(mine) && mine >= self;
    int rank = 0, m = 0;
    for (int j = 0; j < n; ++j) {
        const float x = s[j];
        if (!is_finite(x) || x < self) continue;
        ++m;
        if (x > mine || (x == mine && j < k)) ++rank;
    }
    if (counts) sorted[rank] = mine;  // descending
    __syncthreads();
    if (threadIdx.x == 0) {
        // entries of a run without a wide gap keep their distances to its first
        float first = top, at = fabsf(top) <= kGap ? top : 0.f;
        for (int j = 0; j < m; ++j) {
            if (j > 0 && sorted[j - 1] - sorted[j] > kGap) {
                at = place[j - 1] - kGap;
                first = sorted[j];
            }
            place[j] = at == first ? sorted[j] : at - (first - sorted[j]);
        }
    }
    __syncthreads();
    if (counts) return place[rank];
    if (!is_finite(mine)) return mine;
    const float at = place[m - 1];
    return at == self ? fmaxf(mine, self - kGap) : at - fminf(self - mine, kGap);
}

// The first `per_bucket` CTAs write the buckets of the offsets, the others one head's values each.
template <typename T>
__global__ void __launch_bounds__(kMost) expand_kernel(const Borders b, const T *__restrict__ table, int H, int buckets,
                                                       int R, int per_bucket, float *__restrict__ tab,
                                                       uint8_t *__restrict__ bm) {
    __shared__ float s[kMost], sorted[kMost], place[kMost], tops[kMost / 32], lows[kMost / 32];
    const int k = threadIdx.x, h = static_cast<int>(blockIdx.x) - per_bucket;
    grid_release();
    if (h < 0) {
        const int x = blockIdx.x * kMost + k;
        if (x <= 2 * R) bm[x] = static_cast<uint8_t>(bucket_of(x - R, b));
        return;
    }
    float x = -INFINITY;
    if (k < buckets) x = static_cast<float>(table[static_cast<size_t>(k) * H + h]);
    if (x < kMask) x = -INFINITY;
    s[k] = x;
    float top = is_finite(x) ? x : -INFINITY, low = is_finite(x) ? x : INFINITY;
    #pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        low = fminf(low, __shfl_xor_sync(0xffffffffu, low, o));
    }
    if ((k & 31) == 0) {
        tops[k >> 5] = top;
        lows[k >> 5] = low;
    }
    __syncthreads();
    #pragma unroll
    for (int w = 0; w < kMost / 32; ++w) {
        top = fmaxf(top, tops[w]);
        low = fminf(low, lows[w]);
    }
    // usual entries stay as they are; a head of masks alone has neither top nor low
    if (top > -INFINITY && (top - low > kGap || fabsf(top) > kGap)) x = closer(s, buckets, k, top, low, sorted, place);
    if (k < buckets) tab[static_cast<size_t>(h) * buckets + k] = x * 1.4426950408889634f;
}

// dtable[b][h]: the partial sums [B, H, per, buckets] over the batch and the
// key tiles, in a fixed order and in 64 bits.
template <typename T>
__global__ void __launch_bounds__(1024) dbias_kernel(const float *part, int B, int H, int per, int buckets,
                                                     T *__restrict__ dtable) {
    __shared__ double sum[32][33];
    const int b = blockIdx.x * 32 + threadIdx.x, h = blockIdx.y;
    grid_wait();
    double s = 0.0;
    if (b < buckets)
        for (int i = threadIdx.y; i < B * per; i += 32) {
            const int n = i / per;
            s += chain_load(part + ((static_cast<size_t>(n) * H + h) * per + (i - n * per)) * buckets + b);
        }
    sum[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.y == 0 && b < buckets) {
        for (int y = 1; y < 32; ++y) s += sum[y][threadIdx.x];
        dtable[static_cast<size_t>(b) * H + h] = static_cast<T>(static_cast<float>(s));
    }
}

size_t up256(size_t x) { return (x + 255) & ~size_t(255); }

}  // namespace

int bias_reach(int S, int far) { return far < S ? far : S; }

size_t bias_workspace_bytes(int H, int S, int buckets, int far) {
    return up256(static_cast<size_t>(H) * buckets * 4) + up256(2 * static_cast<size_t>(bias_reach(S, far)) + 1);
}

cudaError_t launch_bias_expand(const void *table, bool f32, int H, int S, int buckets, int far, void *workspace,
                               const float **tab, const uint8_t **bm, cudaStream_t st) {
    const int R = bias_reach(S, far);
    float *t = static_cast<float *>(workspace);
    uint8_t *m = static_cast<uint8_t *>(workspace) + up256(static_cast<size_t>(H) * buckets * 4);
    const Borders b = make_borders(buckets, far);
    const int per_bucket = (2 * R + kMost) / kMost, grid = per_bucket + H;
    if (f32)
        expand_kernel<<<grid, kMost, 0, st>>>(b, static_cast<const float *>(table), H, buckets, R, per_bucket, t, m);
    else
        expand_kernel<<<grid, kMost, 0, st>>>(b, static_cast<const __nv_bfloat16 *>(table), H, buckets, R, per_bucket, t, m);
    *tab = t;
    *bm = m + R;  // offset 0
    return cudaGetLastError();
}

cudaError_t launch_bias_buckets(int buckets, int far, int32_t *out, cudaStream_t st) {
    buckets_kernel<<<(2 * far + 256) / 256, 256, 0, st>>>(make_borders(buckets, far), far, out);
    return cudaGetLastError();
}

cudaError_t launch_dbias(const float *part, int B, int H, int per, int buckets, void *dtable, bool f32,
                         cudaStream_t st) {
    const dim3 grid((buckets + 31) / 32, H), block(32, 32);
    if (f32) return launch_kernel(true, dbias_kernel<float>, grid, block, 0, st, part, B, H, per, buckets, static_cast<float *>(dtable));
    return launch_kernel(true, dbias_kernel<__nv_bfloat16>, grid, block, 0, st, part, B, H, per, buckets,
                         static_cast<__nv_bfloat16 *>(dtable));
}

}  // namespace vsa
