// logprob.hip -- log probabilities of given tokens with entropy and the top
// alternatives, and their gradient.
//
// For a row l[0..V) of logits and a token y, with m = max l:
//   lse = m + log s,  s = sum_v e^(l_v - m)
//   logp = l_y - lse,  H = log s - t / s,  t = sum_v (l_v - m) e^(l_v - m)
//   top: the K largest l_v, ties to the lowest index, as l_v - lse
// and backward, p_v = e^(l_v - lse):
//   dl_v = dlogp ([v = y] - p_v) - dH p_v (l_v - lse + H)
//
// The forward reads every logit once (but see the alternatives): a workgroup holds a chunk of a row in
// registers, 32 values to a thread, takes the chunk's maximum, sums and K
// candidates from there, and a second launch joins a row's chunks (only where
// V needs more than one).  Chunks of 8192 values rather than whole rows: a few
// rows with a long vocabulary then fill the chip, and small workgroups hide
// each other's reductions (4096 rows of 32000 float32: 92 us and 7 for the
// join; chunks of 32768 with 1024 threads, no join: 122).  All sums are
// float32.  1001 rows of 50001 bf16 take 35 us, 31 of which are the issue of
// their 16.6 million vector instructions (four cycles each on 1024 SIMDs): there
// the arithmetic of the sums and the selection bounds it, not memory.
//
// The K candidates of a chunk: the K-th largest of the maxima of 16, 32 or 64
// groups of threads (at least twice K, or 64) is a bound that at least K
// entries reach, and few more do.  Those that reach it are collected (any
// order) and ranked by counting over the unique keys (value, index), so the
// result does not depend on the order.  Where ties at the bound let more than kCand through (a mask rules out the
// chunk, or all but fewer than K of its groups), those above it are collected
// and the lowest indices of those that equal it added (4096 rows of 32000
// float32, one block of 8192 ids ruled out: 161 us for 100 without; the search
// below took 2490).  Where more than kCand lie above it (in fewer than K
// groups), the K-th key is found by bisection over value and index.  (The chunk is read again for either: held on to, it cost the
// ordinary path its registers.)
#include <algorithm>
#include <mutex>

#include "lm.h"
#include "row.h"

namespace rnn355 {
namespace lm {

namespace {

constexpr int kThreads = 256, kPer = 32, kChunk = kThreads * kPer;
constexpr int kCand = 1024;
// e^z is 0 in float32 from z = -104 down; z is held above this where it
// multiplies e^z, as 0 * -inf would be NaN
constexpr float kFloor = -200.0f;

// Order-preserving key of a value: -0 equals +0, NaN above everything.
__device__ __forceinline__ uint32_t order_key(float x) {
    if (x != x) return 0xFFFFFFFFu;
    const uint32_t b = __float_as_uint(x + 0.0f);
    return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float key_value(uint32_t k) {
    if (k == 0xFFFFFFFFu) return __uint_as_float(0x7FC00000u);
    return __uint_as_float((k & 0x80000000u) ? k ^ 0x80000000u : ~k);
}
__device__ __forceinline__ uint64_t pair_key(float x, int idx) {
    return ((uint64_t)order_key(x) << 32) | (uint32_t)~(uint32_t)idx;
}

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
    for (int o = 32; o; o >>= 1) v = fmaxf(v, __shfl_xor(v, o));
    return v;
}
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int o = 32; o; o >>= 1) v += __shfl_xor(v, o);
    return v;
}

// What a chunk leaves for the join.
struct Part {
    float m, s, t, pad;
};

struct Final {
    float lse, ent;
};
// s, t relative to m -> lse, entropy.  A row with nothing allowed (m = -inf):
// lse -inf, entropy 0.
__device__ __forceinline__ Final finish(float m, float s, float t) {
    if (m == -INFINITY && s == 0.0f) return {-INFINITY, 0.0f};
    const float ls = logf(s);
    return {m + ls, ls - t / s};
}
__device__ __forceinline__ float minus_lse(float x, float lse) {
    return lse == -INFINITY ? -INFINITY : x - lse;
}

template <typename T>
__device__ __forceinline__ void write_row(const LogpArgs &a, int row, const Final &f) {
    const int64_t id = a.i64 ? ((const int64_t *)a.tok)[row] : (int64_t)((const int32_t *)a.tok)[row];
    float lp = 0.0f;  // no token
    if (id >= 0 && id < a.V)
        lp = minus_lse(to_f32<T>(((const T *)a.logits)[(int64_t)row * a.ld + id]), f.lse);
    a.logp[row] = lp;
    if (a.entropy) a.entropy[row] = f.ent;
    if (a.lse) a.lse[row] = f.lse;
}

// Ranks n unique keys (LDS, 16-byte aligned, room for an even number) by
// counting and hands (rank, key) of the K largest to out.  Four threads share
// a key's comparisons.
template <int NT, typename F>
__device__ __forceinline__ void rank_keys(uint64_t *key, int n, int K, F out) {
    const int part = threadIdx.x & 3;
    if (n & 1) {
        if (threadIdx.x == 0) key[n] = 0;  // below every key
        __syncthreads();
    }
    for (int i = threadIdx.x >> 2; i < n; i += NT / 4) {
        const uint64_t mine = key[i];
        const ulonglong2 *pair = (const ulonglong2 *)key;
        int r = 0;
#pragma unroll 4
        for (int j = part; j < (n + 1) / 2; j += 4) {
            const ulonglong2 q = pair[j];
            r += (q.x > mine) + (q.y > mine);
        }
        r += __shfl_xor(r, 1);
        r += __shfl_xor(r, 2);
        if (part == 0 && r < K) out(r, mine);
    }
}

// Number of threads' entries that satisfy a predicate, over the workgroup.
template <int NT>
__device__ __forceinline__ int block_count(int mine, int *tmp) {
#pragma unroll
    for (int o = 32; o; o >>= 1) mine += __shfl_xor(mine, o);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) tmp[threadIdx.x >> 6] = mine;
    __syncthreads();
    int all = 0;
#pragma unroll
    for (int i = 0; i < NT / 64; ++i) all += tmp[i];
    return all;
}

// The K largest keys of a chunk, exactly, in `cand`; returns their number (K,
// or the chunk's entries if those are fewer).
template <typename T, int NT>
__device__ __forceinline__ int exact_top(Row<T> r, int u0, int K, uint64_t *cand, int *ncand, int *tmp) {
    constexpr int N = Row<T>::N, U = kPer / N;
    const int tid = threadIdx.x;
    // entries of this thread that satisfy a predicate on (value key, index)
    auto count = [&](auto pred) {
        int k = 0;
#pragma unroll 1
        for (int j = 0; j < U; ++j) {
            const int u = u0 + j * NT + tid, i0 = u * N - r.off;
            float x[N];
            r.load(u, x);
#pragma unroll
            for (int e = 0; e < N; ++e)
                k += i0 + e >= 0 && i0 + e < r.V && pred(order_key(x[e]), i0 + e);
        }
        return block_count<NT>(k, tmp);
    };
    // the largest value key that at least K entries reach
    uint32_t vk = 0;
#pragma unroll 1
    for (int b = 31; b >= 0; --b) {
        const uint32_t c = vk | (1u << b);
        if (count([&](uint32_t k, int) { return k >= c; }) >= K) vk = c;
    }
    // and the lowest index bound that completes K among its equals
    const int need = K - count([&](uint32_t k, int) { return k > vk; });
    int lo = 0, hi = r.V - 1;
#pragma unroll 1
    while (lo < hi) {
        const int mid = lo + (hi - lo) / 2;
        if (count([&](uint32_t k, int i) { return k == vk && i <= mid; }) >= need)
            hi = mid;
        else
            lo = mid + 1;
    }
    if (tid == 0) *ncand = 0;
    __syncthreads();
    count([&](uint32_t k, int i) {
        if (k > vk || (k == vk && i <= lo)) cand[atomicAdd(ncand, 1)] = ((uint64_t)k << 32) | (uint32_t)~(uint32_t)i;
        return false;
    });
    __syncthreads();
    return *ncand;
}

// The same where `tau`, which more than kCand entries of the chunk reach, lets
// at most that many above it: those, and of the entries that equal it the lowest
// indices.  (Masks are such ties: a chunk that -inf or the type's lowest value
// rules out but for fewer than K of its groups has that value for its bound.)
// Reads the chunk once more, and again as far as the equal entries are needed.
template <typename T, int NT>
__device__ __forceinline__ int tied_top(Row<T> r, int u0, int K, float tau, uint64_t *cand, int *ncand,
                                        int *tmp) {
    constexpr int N = Row<T>::N, U = kPer / N;
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
    __syncthreads();
    if (tid == 0) *ncand = 0;
    __syncthreads();
#pragma unroll 1
    for (int j = 0; j < U; ++j) {
        const int u = u0 + j * NT + tid, i0 = u * N - r.off;
        float x[N];
        r.load(u, x);
#pragma unroll
        for (int e = 0; e < N; ++e)
            if (!(x[e] <= tau) && i0 + e >= 0 && i0 + e < r.V) {
                const int at = atomicAdd(ncand, 1);
                if (at < kCand) cand[at] = pair_key(x[e], i0 + e);
            }
    }
    __syncthreads();
    int n = *ncand;
    if (n > kCand) return exact_top<T, NT>(r, u0, K, cand, ncand, tmp);
#pragma unroll 1
    for (int j = 0; j < U && n < K; ++j) {  // indices grow with j, the thread, e
        const int u = u0 + j * NT + tid, i0 = u * N - r.off;
        float x[N];
        r.load(u, x);
        int mine = 0;
#pragma unroll
        for (int e = 0; e < N; ++e) mine += x[e] == tau && i0 + e >= 0 && i0 + e < r.V;
        int at = mine;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const int y = __shfl_up(at, o);
            if (lane >= o) at += y;
        }
        if (lane == 63) tmp[w] = at;
        __syncthreads();
        at += n - mine;
        int all = 0;
#pragma unroll
        for (int i = 0; i < NT / 64; ++i) {
            at += i < w ? tmp[i] : 0;
            all += tmp[i];
        }
#pragma unroll
        for (int e = 0; e < N; ++e)
            if (x[e] == tau && i0 + e >= 0 && i0 + e < r.V) {
                if (at < K) cand[at] = pair_key(x[e], i0 + e);
                ++at;
            }
        n = min(n + all, K);
        __syncthreads();
    }
    return n;
}

template <typename T, bool TOP>
__global__ __launch_bounds__(kThreads) void logp_kernel(LogpArgs a, int nch) {
    constexpr int NT = kThreads, N = Row<T>::N, U = kPer / N, W = NT / 64;
    __shared__ float wm[W], ws[W], wt[W];
    __shared__ float tm[W][64];
    __shared__ __attribute__((aligned(16))) uint64_t cand[TOP ? kCand + 2 : 2];
    __shared__ int ncand, tmp[W];
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
    const int row = blockIdx.x / nch, ch = blockIdx.x - row * nch;
    const Row<T> r((const T *)a.logits + (int64_t)row * a.ld, a.V);
    const int u0 = ch * (NT * kPer / N);
    float x[kPer];
    r.template load_all<U>(u0 + tid, NT, x);

    float m = x[0];
#pragma unroll
    for (int i = 1; i < kPer; ++i) m = fmaxf(m, x[i]);
    const int groups = a.K <= 8 ? 16 : a.K <= 16 ? 32 : 64;
    if constexpr (TOP) {
        float q = m != m ? INFINITY : m;  // nothing but NaN: a bound all the same
        tm[w][lane] = q;
        if (tid == 0) ncand = 0;
    }
    m = wave_max(m);
    if (lane == 0) wm[w] = m;
    __syncthreads();
    m = wm[0];
#pragma unroll
    for (int i = 1; i < W; ++i) m = fmaxf(m, wm[i]);
    // a chunk of nothing but -inf: weights e^(-inf - 0) = 0
    const float ref = m == -INFINITY ? 0.0f : m;
    float s = 0.0f, t = 0.0f;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const float z = x[i] - ref, e = exp_fast(z);
        s += e;
        t += e * fmaxf(z, kFloor);
    }
    s = wave_sum(s);
    t = wave_sum(t);
    if (lane == 0) ws[w] = s, wt[w] = t;
    float tau = 0.0f;
    if constexpr (TOP) {
        // the K-th largest group maximum: the least of those with fewer than K above
        // (groups by lane, so that a chunk that is hardly filled still fills them)
        float mine = fmaxf(fmaxf(tm[0][lane], tm[1][lane]), fmaxf(tm[2][lane], tm[3][lane]));
        if (groups <= 32) mine = fmaxf(mine, __shfl_xor(mine, 32));
        if (groups <= 16) mine = fmaxf(mine, __shfl_xor(mine, 16));
        int above = 0;
#pragma unroll 8
        for (int j = 0; j < groups; ++j)
            above += __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(mine), j)) > mine;
        tau = __uint_as_float(
            __builtin_amdgcn_readfirstlane(__float_as_uint(-wave_max(above < a.K ? -mine : -INFINITY))));
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            if (!(x[i] < tau)) {
                const int idx = (u0 + (i / N) * NT + tid) * N + (i % N) - r.off;
                if (idx >= 0 && idx < a.V) {
                    const int at = atomicAdd(&ncand, 1);
                    if (at < kCand) cand[at] = pair_key(x[i], idx);
                }
            }
        }
    }
    __syncthreads();
    s = t = 0.0f;
#pragma unroll
    for (int i = 0; i < W; ++i) s += ws[i], t += wt[i];
    const Final f = finish(m, s, t);
    if (tid == 0) {
        if (nch == 1)
            write_row<T>(a, row, f);
        else
            ((Part *)a.ws)[blockIdx.x] = Part{m, s, t, 0.0f};
    }
    if constexpr (TOP) {
        int n = ncand;
        if (n > kCand) n = tied_top<T, NT>(r, u0, a.K, tau, cand, &ncand, tmp);
        if (nch == 1) {
            rank_keys<NT>(cand, n, a.K, [&](int k, uint64_t key) {
                a.top_id[(int64_t)row * a.K + k] = (int)~(uint32_t)key;
                a.top_logp[(int64_t)row * a.K + k] =
                    minus_lse(key_value((uint32_t)(key >> 32)), f.lse);
            });
        } else {
            uint64_t *out = (uint64_t *)((Part *)a.ws + (int64_t)a.M * nch) + (int64_t)blockIdx.x * a.K;
            // a chunk with fewer than K entries leaves the lowest key for the rest
            for (int k = n + tid; k < a.K; k += NT) out[k] = 0;
            rank_keys<NT>(cand, n, a.K, [&](int k, uint64_t key) { out[k] = key; });
        }
    }
}

// Joins the chunks of a row.
template <typename T, int NT>
__global__ __launch_bounds__(NT) void logp_join_kernel(LogpArgs a, int nch) {
    constexpr int CAP = NT == 64 ? 256 : kCand;
    extern __shared__ __attribute__((aligned(16))) uint64_t keys[];
    const int row = blockIdx.x, tid = threadIdx.x;
    const Part *p = (const Part *)a.ws + (int64_t)row * nch;
    const uint64_t *in = (const uint64_t *)((const Part *)a.ws + (int64_t)a.M * nch) +
                         (int64_t)row * nch * a.K;
    for (int i = tid; i < nch * a.K; i += NT) keys[i] = in[i];
    // a lane to a chunk, two where there are more than 64 (V <= 1000000: at most 123)
    const int lane = tid & 63;
    Part q[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
        q[i] = i * 64 + lane < nch ? p[i * 64 + lane] : Part{-INFINITY, 0.0f, 0.0f, 0.0f};
    const float m = wave_max(fmaxf(q[0].m, q[1].m));
    float s = 0.0f, t = 0.0f;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        if (q[i].m == -INFINITY && q[i].s == 0.0f) continue;  // nothing allowed in it
        const float d = q[i].m - m, e = exp_fast(d);
        s += q[i].s * e;
        t += (q[i].t + q[i].s * fmaxf(d, kFloor)) * e;
    }
    s = wave_sum(s);
    t = wave_sum(t);
    const Final f = finish(m, s, t);
    if (tid == 0) write_row<T>(a, row, f);
    if (a.K == 0) return;
    // a chunk whose last key is the largest of the last keys has K of them at or
    // above that bound: only keys that reach it can be among the row's K
    __shared__ __attribute__((aligned(16))) uint64_t kept[CAP + 2];
    __shared__ int nkept;
    if (tid == 0) nkept = 0;
    __syncthreads();
    uint64_t bound = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i)
        if (i * 64 + lane < nch) bound = max(bound, keys[(i * 64 + lane) * a.K + a.K - 1]);
#pragma unroll
    for (int o = 32; o; o >>= 1) bound = max(bound, (uint64_t)__shfl_xor((unsigned long long)bound, o));
    for (int i = tid; i < nch * a.K; i += NT)
        if (keys[i] >= bound) {
            const int at = atomicAdd(&nkept, 1);
            if (at < CAP) kept[at] = keys[i];
        }
    __syncthreads();
    const int n = nkept;
    rank_keys<NT>(n <= CAP ? kept : keys, n <= CAP ? n : nch * a.K, a.K, [&](int k, uint64_t key) {
        if (key == 0) return;
        a.top_id[(int64_t)row * a.K + k] = (int)~(uint32_t)key;
        a.top_logp[(int64_t)row * a.K + k] = minus_lse(key_value((uint32_t)(key >> 32)), f.lse);
    });
}

// dl for 4 units of 256 threads each: one pass, bound by memory.  The gradient
// is stored past the caches, which the logits' other readers keep (4096 rows of
// 32000 float32: 181 us against 191, 5.8 TB/s).
template <typename T>
__global__ __launch_bounds__(kThreads) void logp_bwd_kernel(LogpBwdArgs a, int nch) {
    constexpr int N = Row<T>::N;
    const int row = blockIdx.x / nch, ch = blockIdx.x - row * nch;
    const Row<T> r((const T *)a.logits + (int64_t)row * a.ld, a.V);
    T *out = (T *)a.dlogits + (int64_t)row * a.ldd;
    const bool whole = (int)(((uintptr_t)out & 15) / sizeof(T)) == r.off;  // same place in its 16 bytes
    const float lse = a.lse[row];
    float dy = a.dlogp ? a.dlogp[row] : 0.0f;
    const float dh = a.dent ? a.dent[row] : 0.0f, H = a.dent ? a.entropy[row] : 0.0f;
    const int64_t id = a.i64 ? ((const int64_t *)a.tok)[row] : (int64_t)((const int32_t *)a.tok)[row];
    const int y = id >= 0 && id < a.V ? (int)id : -1;
    if (y < 0) dy = 0.0f;  // no token: its log probability is the constant 0
    const bool none = lse == -INFINITY;  // nothing allowed: no gradient
    float x[4][N];
    const int u0 = ch * 4 * kThreads + threadIdx.x;
#pragma unroll
    for (int j = 0; j < 4; ++j) r.load(u0 + j * kThreads, x[j]);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int u = u0 + j * kThreads, i0 = u * N - r.off;
        if (i0 >= a.V) break;
        Unit<T, N> o;
#pragma unroll
        for (int e = 0; e < N; ++e) {
            const float lp = x[j][e] - lse, p = exp_fast(lp);
            // at p = 0 (ruled out, or underflow) p log p is 0, not 0 * -inf
            float d = -p * (dy + dh * (fmaxf(lp, kFloor) + H));
            if (i0 + e == y) d += dy;
            o.v[e] = from_f32<T>(none ? 0.0f : d);
        }
        if (whole && i0 >= 0 && i0 + N <= a.V) {
            typedef uint32_t u4 __attribute__((ext_vector_type(4)));
            __builtin_nontemporal_store(__builtin_bit_cast(u4, o), (u4 *)(out + i0));
        } else {
#pragma unroll
            for (int e = 0; e < N; ++e)
                if (i0 + e >= 0 && i0 + e < a.V) out[i0 + e] = o.v[e];
        }
    }
}

template <typename T>
hipError_t logp_t(const LogpArgs &a, hipStream_t s) {
    const int nch = chunks(a.V, kChunk, sizeof(T));
    const dim3 grid((unsigned)((long)a.M * nch)), thr(kThreads);
    if (a.K)
        hipLaunchKernelGGL((logp_kernel<T, true>), grid, thr, 0, s, a, nch);
    else
        hipLaunchKernelGGL((logp_kernel<T, false>), grid, thr, 0, s, a, nch);
    if (nch > 1) {
        // a wave joins a row where its keys are few: more rows are then in flight
        const size_t lds = ((size_t)nch * a.K + 2) * 8;
        if (nch * a.K <= 256) {
            hipLaunchKernelGGL((logp_join_kernel<T, 64>), dim3((unsigned)a.M), dim3(64), lds, s, a, nch);
        } else {
            hipError_t e = hipGetLastError();
            if (e != hipSuccess) return e;
            // with its kept keys this passes 64 KiB from V of about 909000 at K = 64
            // on, which must be allowed once per kernel
            static std::once_flag once;
            static hipError_t attr = hipSuccess;
            std::call_once(once, [] {
                attr = hipFuncSetAttribute(reinterpret_cast<const void *>(&logp_join_kernel<T, 256>),
                                           hipFuncAttributeMaxDynamicSharedMemorySize,
                                           (int)((chunks(kMaxVocab, kChunk, sizeof(T)) * kMaxTop + 2) * 8));
            });
            if (attr != hipSuccess) return attr;
            hipLaunchKernelGGL((logp_join_kernel<T, 256>), dim3((unsigned)a.M), dim3(256), lds, s, a, nch);
        }
    }
    return hipGetLastError();
}

template <typename T>
hipError_t logp_bwd_t(const LogpBwdArgs &a, hipStream_t s) {
    const int nch = chunks(a.V, 4 * kThreads * Row<T>::N, sizeof(T));
    hipLaunchKernelGGL(logp_bwd_kernel<T>, dim3((unsigned)((long)a.M * nch)), dim3(kThreads), 0, s,
                       a, nch);
    return hipGetLastError();
}

}  // namespace

size_t logp_bytes(int M, int V, int K) {
    // the larger chunk count of the two types
    const long nch = chunks(V, kChunk, 2);
    return nch > 1 ? (size_t)M * nch * (sizeof(Part) + 8 * (size_t)K) : 0;
}

// The join has at most as many workgroups as the rows have chunks.
bool logp_grid_ok(int M, int V, bool bf16) {
    return grid_ok((long)M * chunks(V, kChunk, bf16 ? 2 : 4), kThreads);
}

bool logp_bwd_grid_ok(int M, int V, bool bf16) {
    const int per = 4 * kThreads * (bf16 ? Row<uint16_t>::N : Row<float>::N);
    return grid_ok((long)M * chunks(V, per, bf16 ? 2 : 4), kThreads);
}

hipError_t launch_logp(const LogpArgs &a, bool bf16, hipStream_t s) {
    return bf16 ? logp_t<uint16_t>(a, s) : logp_t<float>(a, s);
}

hipError_t launch_logp_bwd(const LogpBwdArgs &a, bool bf16, hipStream_t s) {
    return bf16 ? logp_bwd_t<uint16_t>(a, s) : logp_bwd_t<float>(a, s);
}

}  // namespace lm
}  // namespace rnn355
