// gated.hip -- gated linear recurrence: forward, single token, backward.
//
//   h_t = a_t h_{t-1} + b_t,  elementwise;  a, b from the gate's form:
//   logit  a = sigmoid(f), b = (1 - a) x:  h + u (x - h) with u = sigmoid(-f), so
//          that neither a gate near 1 nor one near 0 loses its small side
//   decay  a = f, b = x
#include "lm.h"

namespace rnn355 {
namespace lm {

namespace {

constexpr int kThreads = 256;

// 1 - sigmoid(f)
__device__ __forceinline__ float shut(float f) { return rcp_fast(1.0f + exp_fast(f)); }

template <bool LOGIT>
__device__ __forceinline__ float advance(float f, float x, float h) {
    return LOGIT ? fmaf(shut(f), x - h, h) : fmaf(f, h, x);
}

template <typename T, bool LOGIT>
__global__ __launch_bounds__(kThreads) void gated_fwd_kernel(GatedDims d, LinSeq f, LinSeq x,
                                                             const float *h0, const int *lens,
                                                             SeqOut out, float *hT) {
    const int64_t c = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (c >= (int64_t)d.B * d.D) return;
    const int b = (int)(c / d.D), i = (int)(c - (int64_t)b * d.D);
    const int len = lens ? min(max(lens[b], 0), d.T) : d.T;
    float h = h0 ? h0[c] : 0.0f;
    for (int t = 0; t < d.T; ++t) {
        if (t < len)
            h = advance<LOGIT>(to_f32<T>(((const T *)f.p)[t * f.st + b * f.sb + i]),
                               to_f32<T>(((const T *)x.p)[t * x.st + b * x.sb + i]), h);
        ((T *)out.p)[t * out.st + b * out.sb + i] = from_f32<T>(t < len ? h : 0.0f);
    }
    if (hT) hT[c] = h;
}

template <typename T, bool LOGIT>
__global__ __launch_bounds__(kThreads) void gated_step_kernel(GatedDims d, LinSeq f, LinSeq x,
                                                              const float *h, SeqOut y, float *h_out) {
    const int64_t c = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (c >= (int64_t)d.B * d.D) return;
    const int b = (int)(c / d.D), i = (int)(c - (int64_t)b * d.D);
    const float n = advance<LOGIT>(to_f32<T>(((const T *)f.p)[b * f.sb + i]),
                                   to_f32<T>(((const T *)x.p)[b * x.sb + i]), h[c]);
    h_out[c] = n;
    if (y.p) ((T *)y.p)[b * y.sb + i] = from_f32<T>(n);
}

template <typename T, bool LOGIT>
__global__ __launch_bounds__(kThreads) void gated_bwd_kernel(GatedDims d, LinSeq f, LinSeq x, LinSeq h,
                                                             LinSeq dh, const float *h0,
                                                             const float *dhT, const int *lens,
                                                             SeqOut df, SeqOut dx, float *dh0) {
    const int64_t c = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (c >= (int64_t)d.B * d.D) return;
    const int b = (int)(c / d.D), i = (int)(c - (int64_t)b * d.D);
    const int len = lens ? min(max(lens[b], 0), d.T) : d.T;
    float e = dhT ? dhT[c] : 0.0f;  // a_{t+1} g_{t+1}
    for (int t = d.T - 1; t >= 0; --t) {
        float of = 0.0f, ox = 0.0f;
        if (t < len) {
            const float g = e + to_f32<T>(((const T *)dh.p)[t * dh.st + b * dh.sb + i]);
            const float before = t ? to_f32<T>(((const T *)h.p)[(t - 1) * h.st + b * h.sb + i])
                                   : h0 ? h0[c] : 0.0f;
            const float fv = to_f32<T>(((const T *)f.p)[t * f.st + b * f.sb + i]);
            if (LOGIT) {
                const float u = shut(fv), a = shut(-fv);
                const float xv = to_f32<T>(((const T *)x.p)[t * x.st + b * x.sb + i]);
                ox = u * g;
                e = a * g;
                of = e * u * (before - xv);
            } else {
                ox = g;
                of = g * before;
                e = fv * g;
            }
        }
        ((T *)df.p)[t * df.st + b * df.sb + i] = from_f32<T>(of);
        ((T *)dx.p)[t * dx.st + b * dx.sb + i] = from_f32<T>(ox);
    }
    if (dh0) dh0[c] = e;
}

unsigned blocks(const GatedDims &d) { return (unsigned)(((int64_t)d.B * d.D + kThreads - 1) / kThreads); }

}  // namespace

// B * D <= 2^30: one thread to a channel is always a legal launch.
bool gated_grid_ok(const GatedDims &, bool, bool) { return true; }
bool gated_step_grid_ok(const GatedDims &) { return true; }
size_t gated_bytes(const GatedDims &, bool, bool) { return 0; }

#define GATED_LAUNCH(kernel, ...)                                                                       \
    do {                                                                                                \
        const dim3 grid(blocks(d)), thr(kThreads);                                                      \
        if (bf16) {                                                                                     \
            if (d.logit) hipLaunchKernelGGL((kernel<uint16_t, true>), grid, thr, 0, s, __VA_ARGS__);    \
            else hipLaunchKernelGGL((kernel<uint16_t, false>), grid, thr, 0, s, __VA_ARGS__);           \
        } else {                                                                                        \
            if (d.logit) hipLaunchKernelGGL((kernel<float, true>), grid, thr, 0, s, __VA_ARGS__);       \
            else hipLaunchKernelGGL((kernel<float, false>), grid, thr, 0, s, __VA_ARGS__);              \
        }                                                                                               \
    } while (0)

hipError_t launch_gated_fwd(const GatedDims &d, bool bf16, LinSeq f, LinSeq x, const float *h0,
                            const int *lens, SeqOut h, float *hT, void *, hipStream_t s) {
    GATED_LAUNCH(gated_fwd_kernel, d, f, x, h0, lens, h, hT);
    return hipGetLastError();
}

hipError_t launch_gated_step(const GatedDims &d, bool bf16, LinSeq f, LinSeq x, const float *h,
                             SeqOut y, float *h_out, hipStream_t s) {
    GATED_LAUNCH(gated_step_kernel, d, f, x, h, y, h_out);
    return hipGetLastError();
}

hipError_t launch_gated_bwd(const GatedDims &d, bool bf16, LinSeq f, LinSeq x, LinSeq h, LinSeq dh,
                            const float *h0, const float *dhT, const int *lens, SeqOut df, SeqOut dx,
                            float *dh0, void *, hipStream_t s) {
    GATED_LAUNCH(gated_bwd_kernel, d, f, x, h, dh, h0, dhT, lens, df, dx, dh0);
    return hipGetLastError();
}

}  // namespace lm
}  // namespace rnn355
