// lm.h -- launch interface of the operators around the recurrence of a
// language model: embedding lookup and its gradient (embed.hip), token log
// probabilities and their gradient (logprob.hip), linear attention with a
// decay for each head (linattn.hip).  api_lm.hip checks the arguments and
// calls these.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "common.h"

namespace rnn355 {
namespace lm {

// bf16 (as its bits) or float32 values, N of them loaded or stored at once.
template <typename T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32<uint16_t>(uint16_t v) { return bf16_to_f32(v); }
template <>
__device__ __forceinline__ float to_f32<float>(float v) { return v; }
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ uint16_t from_f32<uint16_t>(float v) { return f32_to_bf16_rne(v); }
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }

template <typename T, int N>
struct alignas(sizeof(T) * N) Unit {
    T v[N];
};

// Token ids [T][B] at element strides st, sb, int32 or int64.
struct Ids {
    const void *p;
    int64_t st, sb;
    int T, B;
    int i64;
};

// An id outside [0, V) reads as V ("no token").
__device__ __forceinline__ int load_id(const Ids &t, int m, int V) {
    const int r = m / t.B, b = m - r * t.B;
    const int64_t at = (int64_t)r * t.st + (int64_t)b * t.sb;
    const int64_t id = t.i64 ? ((const int64_t *)t.p)[at] : (int64_t)((const int32_t *)t.p)[at];
    return id < 0 || id >= V ? V : (int)id;
}

// A launch has fewer than 2^32 threads in a dimension.  Each operator's
// *_grid_ok says whether all launches of a call do.
inline bool grid_ok(int64_t blocks, int threads) { return blocks * threads < ((int64_t)1 << 32); }

// ---- embedding (embed.hip)
bool embed_fwd_grid_ok(int M, int D, bool bf16, const void *table, int64_t ld);
bool embed_bwd_grid_ok(int M, int V, int D);
hipError_t launch_embed_fwd(const Ids &ids, int V, int D, bool bf16, const void *table,
                            int64_t ld, float scale, void *x, hipStream_t s);
size_t embed_bwd_bytes(int M, int V, int D);
hipError_t launch_embed_bwd(const Ids &ids, int V, int D, bool bf16, const void *dx, float scale,
                            float *dtable, void *ws, hipStream_t s);

// ---- token log probabilities (logprob.hip)
constexpr int kMaxTop = 64, kMaxVocab = 1000000;
struct LogpArgs {
    int M, V, K;
    const void *logits;
    int64_t ld;
    const void *tok;
    int i64;
    float *logp, *entropy, *lse;  // entropy, lse may be null
    float *top_logp;
    int *top_id;
    void *ws;
};
size_t logp_bytes(int M, int V, int K);
bool logp_grid_ok(int M, int V, bool bf16);
bool logp_bwd_grid_ok(int M, int V, bool bf16);
hipError_t launch_logp(const LogpArgs &a, bool bf16, hipStream_t s);
struct LogpBwdArgs {
    int M, V;
    const void *logits;
    int64_t ld;
    const void *tok;
    int i64;
    const float *lse, *entropy, *dlogp, *dent;  // dlogp, dent may be null (0)
    void *dlogits;
    int64_t ldd;
};
hipError_t launch_logp_bwd(const LogpBwdArgs &a, bool bf16, hipStream_t s);

// ---- linear attention with a decay for each head (linattn.hip)
// A sequence operand: row (t, b) at p + t*st + b*sb (elements), heads x D
// values contiguous in it.
struct LinSeq {
    const void *p;
    int64_t st, sb;
};
struct LinDims {
    int T, B, NH, NKV, Dk, Dv;
};
bool lin_fwd_grid_ok(const LinDims &d, bool bf16);
bool lin_step_grid_ok(const LinDims &d);
bool lin_bwd_grid_ok(const LinDims &d, bool bf16);
size_t lin_fwd_bytes(const LinDims &d, bool bf16);
size_t lin_bwd_bytes(const LinDims &d, bool bf16);
hipError_t launch_lin_fwd(const LinDims &d, bool bf16, LinSeq q, LinSeq k, LinSeq v,
                          const float *g, float scale, const float *S0, void *o, float *ST,
                          void *ws, hipStream_t s);
hipError_t launch_lin_step(const LinDims &d, bool bf16, LinSeq q, LinSeq k, LinSeq v,
                           const float *g, float scale, const float *S0, void *o, float *S1,
                           hipStream_t s);
hipError_t launch_lin_bwd(const LinDims &d, bool bf16, LinSeq q, LinSeq k, LinSeq v,
                          const float *g, float scale, const float *S0, LinSeq dO,
                          const float *dST, void *dq, void *dk, void *dv, float *dS0, void *ws,
                          hipStream_t s);

}  // namespace lm
}  // namespace rnn355
