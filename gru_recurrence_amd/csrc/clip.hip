// clip.hip -- global norm of a list of gradients, and clipping by it.
//
//   norm = sqrt(sum g^2),  out = g min(1, max_norm / norm)
//
// Two passes, as the factor needs every value: the first leaves one sum of
// squares for each workgroup, the second adds those up (every workgroup for
// itself, in the same order) and scales.  The list travels in the kernels'
// arguments, kGroup tensors a launch: nothing of it has to be in device memory
// or outlive the call, so that a captured call replays what it was given.
//
// Squares are summed in 64 bits: the largest float32 squared is far inside
// them, so only a value that is not finite gives such a sum, and there is
// arithmetic to spare (two 64-bit operations for 2 or 4 bytes read).
#include <algorithm>

#include "row.h"

namespace rnn355 {
namespace lm {

namespace {

constexpr int kThreads = 256, kUnits = 4;  // 16-byte units of a thread in a chunk
constexpr int kChunkBytes = kThreads * kUnits * 16;
constexpr int kGroup = 96;   // tensors of one launch
constexpr int kSlots = 2048; // sums kept: the first pass has at most that many workgroups

struct Group {
    const void *p[kGroup];
    void *out[kGroup];
    int64_t n[kGroup];
    int32_t first[kGroup + 1];  // chunk at which a tensor starts
    uint8_t bf16[kGroup];
    int count;
};

// Workgroup sum of 64-bit values, the same in every thread.
__device__ __forceinline__ double block_sum(double v, double *tmp) {
#pragma unroll
    for (int o = 32; o; o >>= 1) v += __shfl_xor(v, o);
    if ((threadIdx.x & 63) == 0) tmp[threadIdx.x >> 6] = v;
    __syncthreads();
    double all = 0.0;
#pragma unroll
    for (int i = 0; i < kThreads / 64; ++i) all += tmp[i];
    return all;
}

// Tensor of a chunk.
__device__ __forceinline__ int find(const Group &g, int chunk) {
    int lo = 0, hi = g.count - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (g.first[mid] <= chunk)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

template <typename T>
__device__ __forceinline__ double chunk_squares(const T *p, int64_t n, int ch) {
    constexpr int N = 16 / sizeof(T);
    const int off = (int)(((uintptr_t)p & 15) / sizeof(T));
    const T *base = p - off;
    double s = 0.0;
#pragma unroll
    for (int j = 0; j < kUnits; ++j) {
        const int64_t u = ((int64_t)ch * kUnits + j) * kThreads + threadIdx.x, i0 = u * N - off;
        if (i0 >= 0 && i0 + N <= n) {
            const Unit<T, N> q = *(const Unit<T, N> *)(base + u * N);
#pragma unroll
            for (int e = 0; e < N; ++e) {
                const double v = to_f32<T>(q.v[e]);
                s = fma(v, v, s);
            }
        } else if (i0 < n) {
            for (int e = 0; e < N; ++e)
                if (i0 + e >= 0 && i0 + e < n) {
                    const double v = to_f32<T>(p[i0 + e]);
                    s = fma(v, v, s);
                }
        }
    }
    return s;
}

__global__ __launch_bounds__(kThreads) void norm_kernel(Group g, double *slot, int add) {
    __shared__ double tmp[kThreads / 64];
    const int all = g.first[g.count];
    double s = 0.0;
    for (int ch = blockIdx.x; ch < all; ch += gridDim.x) {
        const int t = find(g, ch);
        s += g.bf16[t] ? chunk_squares((const uint16_t *)g.p[t], g.n[t], ch - g.first[t])
                       : chunk_squares((const float *)g.p[t], g.n[t], ch - g.first[t]);
    }
    s = block_sum(s, tmp);
    if (threadIdx.x == 0) slot[blockIdx.x] = add ? slot[blockIdx.x] + s : s;
}

__device__ __forceinline__ double total(const double *slot, int slots, double *tmp) {
    double s = 0.0;
    for (int i = threadIdx.x; i < slots; i += kThreads) s += slot[i];
    return block_sum(s, tmp);
}

__global__ __launch_bounds__(kThreads) void norm_only_kernel(const double *slot, int slots, float *norm) {
    __shared__ double tmp[kThreads / 64];
    const double s = total(slot, slots, tmp);
    if (threadIdx.x == 0) norm[0] = (float)sqrt(s);
}

template <typename T>
__device__ __forceinline__ void chunk_scale(const T *p, T *out, int64_t n, int ch, float c) {
    constexpr int N = 16 / sizeof(T);
    const int off = (int)(((uintptr_t)p & 15) / sizeof(T));
    const bool whole = (int)(((uintptr_t)out & 15) / sizeof(T)) == off;
    const T *base = p - off;
#pragma unroll
    for (int j = 0; j < kUnits; ++j) {
        const int64_t u = ((int64_t)ch * kUnits + j) * kThreads + threadIdx.x, i0 = u * N - off;
        if (i0 >= 0 && i0 + N <= n) {
            Unit<T, N> q = *(const Unit<T, N> *)(base + u * N);
#pragma unroll
            for (int e = 0; e < N; ++e) q.v[e] = from_f32<T>(to_f32<T>(q.v[e]) * c);
            if (whole) {
                *(Unit<T, N> *)(out + i0) = q;
            } else {
#pragma unroll
                for (int e = 0; e < N; ++e) out[i0 + e] = q.v[e];
            }
        } else if (i0 < n) {
            for (int e = 0; e < N; ++e)
                if (i0 + e >= 0 && i0 + e < n) out[i0 + e] = from_f32<T>(to_f32<T>(p[i0 + e]) * c);
        }
    }
}

__global__ __launch_bounds__(kThreads) void scale_kernel(Group g, const double *slot, int slots,
                                                         float max_norm, float *norm) {
    __shared__ double tmp[kThreads / 64];
    const double s = total(slot, slots, tmp), n = sqrt(s);
    if (norm && blockIdx.x == 0 && threadIdx.x == 0) norm[0] = (float)n;
    const bool over = n > (double)max_norm && n < (double)INFINITY;
    const float c = over ? (float)((double)max_norm / n) : 1.0f;
    const int all = g.first[g.count];
    for (int ch = blockIdx.x; ch < all; ch += gridDim.x) {
        const int t = find(g, ch);
        if (!over && !g.out[t]) continue;  // in place, as it is
        void *out = g.out[t] ? g.out[t] : const_cast<void *>(g.p[t]);
        if (g.bf16[t])
            chunk_scale((const uint16_t *)g.p[t], (uint16_t *)out, g.n[t], ch - g.first[t], c);
        else
            chunk_scale((const float *)g.p[t], (float *)out, g.n[t], ch - g.first[t], c);
    }
}

// Chunks of a tensor, wherever it starts in its 16 bytes.
int64_t tensor_chunks(const rnn_grad &t) {
    const int64_t e = t.dtype == RNN_BF16 ? 2 : 4;
    return t.n ? (t.n * e + (int64_t)((uintptr_t)t.data & 15) + kChunkBytes - 1) / kChunkBytes : 0;
}

// The next tensors of the list, from `at` on: as many as a group takes.
int fill(Group *g, int count, const rnn_grad *list, int at) {
    g->count = 0;
    int64_t chunks = 0;
    while (at < count && g->count < kGroup) {
        const rnn_grad &t = list[at++];
        if (t.n == 0) continue;
        const int i = g->count++;
        g->p[i] = t.data;
        g->out[i] = t.out == t.data ? nullptr : t.out;
        g->n[i] = t.n;
        g->bf16[i] = t.dtype == RNN_BF16;
        g->first[i] = (int32_t)chunks;
        chunks += tensor_chunks(t);
    }
    g->first[g->count] = (int32_t)chunks;
    return at;
}

}  // namespace

size_t clip_bytes() { return kSlots * sizeof(double); }

hipError_t launch_clip(int count, const rnn_grad *list, float max_norm, float *norm, void *ws,
                       hipStream_t s) {
    double *slot = (double *)ws;
    Group g;
    int64_t most = 0;  // chunks of the largest group
    int groups = 0;
    for (int at = 0; at < count || !groups; ++groups) {
        at = fill(&g, count, list, at);
        most = std::max<int64_t>(most, g.first[g.count]);
    }
    // the first launch writes all sums that a later one adds to
    const int slots = (int)std::min<int64_t>(kSlots, std::max<int64_t>(1, most));
    for (int at = 0, i = 0; i < groups; ++i) {
        at = fill(&g, count, list, at);
        const int grid = i ? std::min(slots, std::max(1, g.first[g.count])) : slots;
        hipLaunchKernelGGL(norm_kernel, dim3(grid), dim3(kThreads), 0, s, g, slot, i > 0);
    }
    if (max_norm < 0.0f) {
        hipLaunchKernelGGL(norm_only_kernel, dim3(1), dim3(kThreads), 0, s, slot, slots, norm);
        return hipGetLastError();
    }
    for (int at = 0, i = 0; i < groups; ++i) {
        at = fill(&g, count, list, at);
        const int grid = std::min(slots, std::max(1, g.first[g.count]));
        hipLaunchKernelGGL(scale_kernel, dim3(grid), dim3(kThreads), 0, s, g, slot, slots, max_norm,
                           i ? nullptr : norm);
    }
    return hipGetLastError();
}

}  // namespace lm
}  // namespace rnn355
