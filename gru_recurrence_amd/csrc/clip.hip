// clip.hip -- global norm of a list of gradients, and clipping by it.
//
//   norm = sqrt(sum g^2),  out = g min(1, max_norm / norm)
//
// Two passes, as the factor needs every value: the first leaves one sum of
// squares for each workgroup, the second adds those up (every workgroup for
// itself, in the same order) and scales.  A list that one workgroup reads in a
// microsecond takes one launch.  The list travels in the kernels' arguments,
// kGroup tensors a launch: nothing of it has to be in device memory or outlive
// the call, so that a captured call replays what it was given.
//
// Memory bounds it: a workgroup takes an equal share of the list, in pieces of a
// 16-byte unit to a thread, kAhead of them in flight.  The first pass leaves what it
// can in the last-level cache; the second reads and stores past the caches.  86
// million float32: 171 us, 6.05 TB/s over the two readings and the writing (the second
// reading through the caches 185, its stores too 217, the first past them 192; the
// second from the list's end makes no difference).
//
// Squares are summed in 64 bits: the largest float32 squared is far inside
// them, so only a value that is not finite gives such a sum, and there is
// arithmetic to spare (two 64-bit operations for 2 or 4 bytes read).  So is the
// product with the factor (86 million float32 170 us as with a float32 factor).
#include <algorithm>

#include "row.h"

namespace rnn355 {
namespace lm {

namespace {

typedef uint32_t u4 __attribute__((ext_vector_type(4)));

constexpr int kThreads = 256, kAhead = 8;
constexpr int kPiece = kThreads * 16;  // bytes
constexpr int kGroup = 96;    // tensors of one launch
constexpr int kSlots = 2048;  // sums kept: the first pass has at most that many workgroups
constexpr int kOne = 1024;    // threads of a single workgroup that does it all
constexpr int kOnePieces = 32;

struct Group {
    const void *p[kGroup];
    void *out[kGroup];
    int64_t n[kGroup];
    int32_t first[kGroup + 1];  // piece at which a tensor starts
    uint8_t bf16[kGroup];
    int count;
};

// Workgroup sum of 64-bit values, the same in every thread.
template <int NT>
__device__ __forceinline__ double block_sum(double v, double *tmp) {
#pragma unroll
    for (int o = 32; o; o >>= 1) v += __shfl_xor(v, o);
    if ((threadIdx.x & 63) == 0) tmp[threadIdx.x >> 6] = v;
    __syncthreads();
    double all = 0.0;
#pragma unroll
    for (int i = 0; i < NT / 64; ++i) all += tmp[i];
    return all;
}

// Tensor of a piece.
__device__ __forceinline__ int find(const Group &g, int piece) {
    int lo = 0, hi = g.count - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (g.first[mid] <= piece)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

// A tensor as units from the aligned address at or before its start.
template <typename T>
struct Units {
    static constexpr int N = 16 / sizeof(T);
    const T *base;
    int64_t n;
    int off;
    __device__ __forceinline__ Units(const void *p, int64_t n_) : n(n_) {
        off = (int)(((uintptr_t)p & 15) / sizeof(T));
        base = (const T *)p - off;
    }
    // whether units [lo, hi) are all whole
    __device__ __forceinline__ bool whole(int64_t lo, int64_t hi) const { return lo * N >= off && hi * N - off <= n; }
};

template <typename T>
__device__ __forceinline__ double unit_squares(const Unit<T, 16 / sizeof(T)> &q, double s) {
#pragma unroll
    for (int e = 0; e < (int)(16 / sizeof(T)); ++e) {
        const double v = to_f32<T>(q.v[e]);
        s = fma(v, v, s);
    }
    return s;
}

// Sum of squares of units [lo, hi) of a tensor, NT threads.
template <typename T, int NT>
__device__ __forceinline__ double squares(const void *p, int64_t n, int64_t lo, int64_t hi) {
    constexpr int N = Units<T>::N;
    const Units<T> t(p, n);
    double s = 0.0;
    for (int64_t at = lo; at < hi;) {
        if (at + NT * kAhead <= hi && t.whole(at, at + NT * kAhead)) {
            Unit<T, N> q[kAhead];
#pragma unroll
            for (int j = 0; j < kAhead; ++j) q[j] = *(const Unit<T, N> *)(t.base + (at + j * NT + threadIdx.x) * N);
#pragma unroll
            for (int j = 0; j < kAhead; ++j) s = unit_squares<T>(q[j], s);
            at += NT * kAhead;
            continue;
        }
        const int64_t u = at + threadIdx.x, i0 = u * N - t.off;
        if (u < hi && i0 >= 0 && i0 + N <= n) {
            s = unit_squares<T>(*(const Unit<T, N> *)(t.base + u * N), s);
        } else if (u < hi) {
            for (int e = 0; e < N; ++e)
                if (i0 + e >= 0 && i0 + e < n) {
                    const double v = to_f32<T>(t.base[u * N + e]);
                    s = fma(v, v, s);
                }
        }
        at += NT;
    }
    return s;
}

// g c, rounded once (a factor below float32's normal numbers would lose its bits there).
// bf16 by way of 21 bits of the product, the last of them set where anything is cut off
// behind: those are exact in float32 (normal numbers), and lie on a middle of two bf16
// numbers only where the product does.
template <typename T>
__device__ __forceinline__ T scaled(T g, double c) {
    double v = (double)to_f32<T>(g) * c;
    if constexpr (sizeof(T) == 2) {
        const uint64_t b = (uint64_t)__double_as_longlong(v);
        const uint32_t hi = (uint32_t)(b >> 32) | min((uint32_t)b, 1u);
        v = __longlong_as_double((long long)((uint64_t)hi << 32));
    }
    return from_f32<T>((float)v);
}

template <typename T>
__device__ __forceinline__ void store(T *out, Unit<T, 16 / sizeof(T)> q, double c, bool whole) {
    constexpr int N = 16 / sizeof(T);
#pragma unroll
    for (int e = 0; e < N; ++e) q.v[e] = scaled<T>(q.v[e], c);
    if (whole) {
        __builtin_nontemporal_store(__builtin_bit_cast(u4, q), (u4 *)out);
    } else {
#pragma unroll
        for (int e = 0; e < N; ++e) out[e] = q.v[e];
    }
}

// out = c p over units [lo, hi), NT threads.
template <typename T, int NT>
__device__ __forceinline__ void scale(const void *p, void *out_, int64_t n, int64_t lo, int64_t hi, double c) {
    constexpr int N = Units<T>::N;
    const Units<T> t(p, n);
    T *out = (T *)out_ - t.off;
    const bool same = ((uintptr_t)out & 15) == 0;  // at the same place of its 16 bytes
    for (int64_t at = lo; at < hi;) {
        if (at + NT * kAhead <= hi && t.whole(at, at + NT * kAhead)) {
            Unit<T, N> q[kAhead];
#pragma unroll
            for (int j = 0; j < kAhead; ++j)
                q[j] = __builtin_bit_cast(
                    Unit<T, N>, __builtin_nontemporal_load((const u4 *)(t.base + (at + j * NT + threadIdx.x) * N)));
#pragma unroll
            for (int j = 0; j < kAhead; ++j) store<T>(out + (at + j * NT + threadIdx.x) * N, q[j], c, same);
            at += NT * kAhead;
            continue;
        }
        const int64_t u = at + threadIdx.x, i0 = u * N - t.off;
        if (u < hi && i0 >= 0 && i0 + N <= n) {
            store<T>(out + u * N, *(const Unit<T, N> *)(t.base + u * N), c, same);
        } else if (u < hi) {
            for (int e = 0; e < N; ++e)
                if (i0 + e >= 0 && i0 + e < n) out[u * N + e] = scaled<T>(t.base[u * N + e], c);
        }
        at += NT;
    }
}

// Pieces [lo, hi) of the list, tensor by tensor: f(tensor, first unit, unit behind the last).
template <typename F>
__device__ __forceinline__ void each(const Group &g, int lo, int hi, F f) {
    if (lo >= hi) return;
    for (int t = find(g, lo); lo < hi; ++t) {
        const int to = min(g.first[t + 1], hi);
        f(t, (int64_t)(lo - g.first[t]) * kThreads, (int64_t)(to - g.first[t]) * kThreads);
        lo = to;
    }
}

// A workgroup's share of the pieces.
__device__ __forceinline__ void share(int all, int &lo, int &hi) {
    lo = (int)((int64_t)all * blockIdx.x / gridDim.x);
    hi = (int)((int64_t)all * (blockIdx.x + 1) / gridDim.x);
}

template <int NT>
__device__ __forceinline__ double share_squares(const Group &g, int lo, int hi) {
    double s = 0.0;
    each(g, lo, hi, [&](int t, int64_t a, int64_t b) {
        s += g.bf16[t] ? squares<uint16_t, NT>(g.p[t], g.n[t], a, b) : squares<float, NT>(g.p[t], g.n[t], a, b);
    });
    return s;
}

// The factor of a sum of squares, and whether the values change.
__device__ __forceinline__ bool factor(double s, double max_norm, double &c) {
    const double n = sqrt(s);
    const bool over = n > max_norm && n < (double)INFINITY;
    c = over ? max_norm / n : 1.0;
    return over;
}

template <int NT>
__device__ __forceinline__ void share_scale(const Group &g, int lo, int hi, bool over, double c) {
    each(g, lo, hi, [&](int t, int64_t a, int64_t b) {
        if (!over && !g.out[t]) return;  // in place, as it is
        void *out = g.out[t] ? g.out[t] : const_cast<void *>(g.p[t]);
        if (g.bf16[t])
            scale<uint16_t, NT>(g.p[t], out, g.n[t], a, b, c);
        else
            scale<float, NT>(g.p[t], out, g.n[t], a, b, c);
    });
}

__global__ __launch_bounds__(kThreads) void norm_kernel(Group g, double *slot, int add) {
    __shared__ double tmp[kThreads / 64];
    int lo, hi;
    share(g.first[g.count], lo, hi);
    const double s = block_sum<kThreads>(share_squares<kThreads>(g, lo, hi), tmp);
    if (threadIdx.x == 0) slot[blockIdx.x] = add ? slot[blockIdx.x] + s : s;
}

__device__ __forceinline__ double total(const double *slot, int slots, double *tmp) {
    double v[kSlots / kThreads], s = 0.0;
#pragma unroll
    for (int j = 0; j < kSlots / kThreads; ++j) {
        const int i = j * kThreads + (int)threadIdx.x;
        v[j] = i < slots ? slot[i] : 0.0;
    }
#pragma unroll
    for (int j = 0; j < kSlots / kThreads; ++j) s += v[j];
    return block_sum<kThreads>(s, tmp);
}

__global__ __launch_bounds__(kThreads) void norm_only_kernel(const double *slot, int slots, float *norm) {
    __shared__ double tmp[kThreads / 64];
    const double s = total(slot, slots, tmp);
    if (threadIdx.x == 0) norm[0] = (float)sqrt(s);
}

__global__ __launch_bounds__(kThreads) void scale_kernel(Group g, const double *slot, int slots,
                                                         double max_norm, float *norm) {
    __shared__ double tmp[kThreads / 64];
    const double s = total(slot, slots, tmp);
    if (norm && blockIdx.x == 0 && threadIdx.x == 0) norm[0] = (float)sqrt(s);
    double c;
    const bool over = factor(s, max_norm, c);
    int lo, hi;
    share(g.first[g.count], lo, hi);
    share_scale<kThreads>(g, lo, hi, over, c);
}

// A list of few pieces.  max_norm < 0: the norm alone.
__global__ __launch_bounds__(kOne) void one_kernel(Group g, double max_norm, float *norm) {
    __shared__ double tmp[kOne / 64];
    const int all = g.first[g.count];
    const double s = block_sum<kOne>(share_squares<kOne>(g, 0, all), tmp);
    if (threadIdx.x == 0) norm[0] = (float)sqrt(s);
    if (max_norm < 0.0) return;
    double c;
    const bool over = factor(s, max_norm, c);
    share_scale<kOne>(g, 0, all, over, c);
}

// Pieces of a tensor, wherever it starts in its 16 bytes.
int64_t pieces(const rnn_grad &t) {
    const int64_t e = t.dtype == RNN_BF16 ? 2 : 4;
    return t.n ? (t.n * e + (int64_t)((uintptr_t)t.data & 15) + kPiece - 1) / kPiece : 0;
}

// The next tensors of the list, from `at` on: as many as a group takes.
int fill(Group *g, int count, const rnn_grad *list, int at) {
    g->count = 0;
    int64_t n = 0;
    while (at < count && g->count < kGroup) {
        const rnn_grad &t = list[at++];
        if (t.n == 0) continue;
        const int i = g->count++;
        g->p[i] = t.data;
        g->out[i] = t.out == t.data ? nullptr : t.out;
        g->n[i] = t.n;
        g->bf16[i] = t.dtype == RNN_BF16;
        g->first[i] = (int32_t)n;
        n += pieces(t);
    }
    g->first[g->count] = (int32_t)n;
    return at;
}

// Workgroups of a launch over a group: a share is no less than kAhead pieces where the
// list is short.
int grid_of(const Group &g, int most) {
    const int n = g.first[g.count];
    return std::max(1, std::min(most, n < kSlots ? n : std::max(n / kAhead, kSlots / 2)));
}

}  // namespace

size_t clip_bytes() { return kSlots * sizeof(double); }

hipError_t launch_clip(int count, const rnn_grad *list, double max_norm, float *norm, void *ws,
                       hipStream_t s) {
    double *slot = (double *)ws;
    Group g;
    int groups = 0, slots = 1;
    for (int at = 0; at < count || !groups; ++groups) {
        at = fill(&g, count, list, at);
        slots = std::max(slots, grid_of(g, kSlots));
    }
    if (groups == 1 && g.first[g.count] <= kOnePieces) {
        hipLaunchKernelGGL(one_kernel, dim3(1), dim3(kOne), 0, s, g, max_norm, norm);
        return hipGetLastError();
    }
    // the first launch writes all sums that a later one adds to
    for (int at = 0, i = 0; i < groups; ++i) {
        if (groups > 1) at = fill(&g, count, list, at);
        hipLaunchKernelGGL(norm_kernel, dim3(i ? grid_of(g, slots) : slots), dim3(kThreads), 0, s, g, slot, i > 0);
    }
    if (max_norm < 0.0) {
        hipLaunchKernelGGL(norm_only_kernel, dim3(1), dim3(kThreads), 0, s, slot, slots, norm);
        return hipGetLastError();
    }
    for (int at = 0, i = 0; i < groups; ++i) {
        if (groups > 1) at = fill(&g, count, list, at);
        hipLaunchKernelGGL(scale_kernel, dim3(i ? grid_of(g, slots) : slots), dim3(kThreads), 0, s, g, slot, slots,
                           max_norm, i ? nullptr : norm);
    }
    return hipGetLastError();
}

}  // namespace lm
}  // namespace rnn355
