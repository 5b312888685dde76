// row.h -- rows of contiguous values that start at any element, read as 16-byte
// units (logprob.hip, verify.hip, clip.hip).
#pragma once

#include "lm.h"

namespace rnn355 {
namespace lm {

// A row seen as 16-byte units from the aligned address at or before its
// start: entry i of unit u is value u*N + i - off.
template <typename T>
struct Row {
    static constexpr int N = 16 / sizeof(T);
    const T *base;
    int off, V;
    __device__ Row(const T *row, int V_) : V(V_) {
        off = (int)(((uintptr_t)row & 15) / sizeof(T));
        base = row - off;
    }
    // Units u, u + step, ... (n of them).  Whole units load without a branch, the
    // row's nearest whole unit in the place of others, so that all loads are in
    // flight at once; the few units across the row's ends are then read again.
    template <int n>
    __device__ void load_all(int u, int step, float *x) const {
        const int first = (off + N - 1) / N, last = (V + off) / N - 1;
        if (last < first) {  // no whole unit
#pragma unroll
            for (int j = 0; j < n; ++j) load(u + j * step, x + j * N);
            return;
        }
        Unit<T, N> q[n];
#pragma unroll
        for (int j = 0; j < n; ++j)
            q[j] = *(const Unit<T, N> *)(base + (int64_t)min(max(u + j * step, first), last) * N);
#pragma unroll
        for (int j = 0; j < n; ++j) {
#pragma unroll
            for (int e = 0; e < N; ++e) x[j * N + e] = to_f32<T>(q[j].v[e]);
            const int v = u + j * step;
            if (v < first || v > last) load(v, x + j * N);
        }
    }
    // N values of unit u; entries outside the row are -inf
    __device__ void load(int u, float *x) const {
        const int i0 = u * N - off;
        if (i0 >= 0 && i0 + N <= V) {
            const Unit<T, N> q = *(const Unit<T, N> *)(base + (int64_t)u * N);
#pragma unroll
            for (int e = 0; e < N; ++e) x[e] = to_f32<T>(q.v[e]);
        } else {
#pragma unroll
            for (int e = 0; e < N; ++e)
                x[e] = i0 + e >= 0 && i0 + e < V ? to_f32<T>(base[(int64_t)u * N + e]) : -INFINITY;
        }
    }
};

// chunks of `per` values that a row of V takes wherever it starts in its 16 bytes
inline int chunks(int V, int per, size_t elt) {
    return (int)(((long)V + (long)(16 / elt) - 1 + per - 1) / per);
}

}  // namespace lm
}  // namespace rnn355
