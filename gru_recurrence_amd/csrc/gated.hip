// gated.hip -- gated linear recurrence: forward, single token, backward.
//
//   h_t = a_t h_{t-1} + b_t,  elementwise;  a, b from the gate's form:
//   logit  a = sigmoid(f), b = (1 - a) x:  h + u (x - h) with u = sigmoid(-f), so
//          that a gate near 1 does not lose its small side: a constant x is a
//          fixed point, and the memory 1 / (1 - a) is right to float32
//   decay  a = f, b = x
// Steps compose: (A1, B1) then (A2, B2) is (A2 A1, A2 B1 + B2).  Backward is the same
// kind of recurrence from the end: e_t = a_t (dh_t + e_{t+1}).
//
// Memory bounds it.  A wave walks a piece of the time axis, 64 lanes of VEC channels,
// with the next steps' loads in flight; the waves of a workgroup have neighbouring
// pieces.  Where the channels alone do not fill the chip the time axis is cut and the
// call takes two launches: the first composes each piece's steps (forward f and x,
// backward f and dh) and leaves the piece's (A, B) and each workgroup's; the second
// composes what lies before a piece and runs its steps from there.  The second reading
// is for the most part the last-level cache's, so a call whose inputs exceed that runs
// over chunks of the time axis.  The order of all products is the dimensions' alone.
#include <algorithm>
#include <type_traits>

#include "lm.h"

namespace rnn355 {
namespace lm {

namespace {

constexpr int kThreads = 512, kWaves = kThreads / 64;

// How a launch is cut: T steps, C channels (D in a row), R steps to a wave, P waves
// along time (kWaves for each workgroup), ntile tiles of channels.
struct Cut {
    int T, D, C;
    int R, P, ntile;
    int off;          // the chunk's first step in the sequence
    float2 *word;     // [P][C] (A, B) of a wave's piece
    float2 *total;    // [P / kWaves][C] of a workgroup's
    float *start;     // [C] state that the chunk begins with
    float *state;     // [C] state that it ends with
};

// A h + B; a state of 0 takes no part, whatever the product of the decays is.
__device__ __forceinline__ float apply(float A, float B, float h) { return h == 0.0f ? B : fmaf(A, h, B); }

// 1 - sigmoid(f)
__device__ __forceinline__ float shut(float f) { return rcp_fast(1.0f + exp_fast(f)); }

// Where a wave works: channels c0 .. c0 + VEC of the call (c: the same, inside), steps
// [lo, hi) in the order of the recurrence, the row's steps that count.
template <int VEC>
struct Spot {
    int c0, c, b, i, len, lo, hi, p, group;
    __device__ __forceinline__ Spot(const Cut &k, const int *lens, bool cut) {
        const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        // a workgroup's waves: one tile and neighbouring pieces, or one piece and neighbouring tiles
        group = cut ? (int)(blockIdx.x / (unsigned)k.ntile) : 0;
        const int tile = cut ? (int)(blockIdx.x - (unsigned)group * k.ntile) : (int)blockIdx.x * kWaves + w;
        p = cut ? group * kWaves + w : 0;
        c0 = (tile * 64 + lane) * VEC;
        c = min(c0, k.C - VEC);
        b = c / k.D;
        i = c - b * k.D;
        len = lens ? min(max(lens[b] - k.off, 0), k.T) : k.T;
        lo = (int)min((int64_t)p * k.R, (int64_t)k.T);
        hi = (int)min((int64_t)(p + 1) * k.R, (int64_t)k.T);
    }
};

template <typename T, int VEC>
__device__ __forceinline__ const T *row_at(const LinSeq &q, int b, int i) {
    return (const T *)q.p + (int64_t)b * q.sb + i;
}

// The steps of a wave in batches of U, the next batch's loads under way while one is
// worked on: load(buffer, first step), work(buffer, first step).
template <int U, typename Buf, typename L, typename W>
__device__ __forceinline__ void batches(int lo, int hi, Buf &q, L load, W work) {
    for (int t = lo; t < hi; t += U) {
        Buf now = q;
        if (t + U < hi) load(q, t + U);
        work(now, t);
    }
}

// A piece's (A, B) to memory, the workgroup's composed from all its waves'.  With the
// first piece goes the state that the chunk begins with.
template <int VEC>
__device__ __forceinline__ void leave(const Cut &k, const Spot<VEC> &s, const float *A, const float *B,
                                      const float *start0) {
    __shared__ float2 agg[kWaves][64 * VEC];
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), at = lane * VEC;
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
        float2 q = make_float2(A[v], B[v]);
        if (s.p == 0) {
            const float h = start0 ? start0[s.c + v] : 0.0f;
            if (s.c0 < k.C) k.start[s.c + v] = h;
            q = make_float2(0.0f, apply(A[v], B[v], h));
        }
        agg[w][at + v] = q;
        if (s.c0 < k.C) k.word[(int64_t)s.p * k.C + s.c + v] = q;
    }
    __syncthreads();
    if (w == 0 && s.c0 < k.C) {
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            float tA = 1.0f, tB = 0.0f;
#pragma unroll
            for (int i = 0; i < kWaves; ++i) {
                const float2 q = agg[i][at + v];
                tB = apply(q.x, q.y, tB);
                tA *= q.x;
            }
            k.total[(int64_t)s.group * k.C + s.c + v] = make_float2(tA, tB);
        }
    }
}

// The state before a piece: the totals of the workgroups before, a share of them to
// each wave, then the pieces before it in the workgroup.
template <int VEC>
__device__ __forceinline__ void begin(const Cut &k, const Spot<VEC> &s, float *h) {
    __shared__ float2 agg[kWaves][64 * VEC], car[kWaves][64 * VEC];
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), at = lane * VEC;
    float A[VEC], B[VEC];
    float2 mine[VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
        mine[v] = k.word[(int64_t)s.p * k.C + s.c + v];
        h[v] = s.p == 0 ? k.start[s.c + v] : 0.0f;
        A[v] = 1.0f, B[v] = 0.0f;
    }
    const int lo = s.group * w / kWaves, hi = s.group * (w + 1) / kWaves;
    for (int j = lo; j < hi; j += 4) {
        float2 q[4][VEC];
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int v = 0; v < VEC; ++v) q[e][v] = k.total[(int64_t)min(j + e, hi - 1) * k.C + s.c + v];
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (j + e < hi) {
#pragma unroll
                for (int v = 0; v < VEC; ++v) {
                    B[v] = apply(q[e][v].x, q[e][v].y, B[v]);
                    A[v] *= q[e][v].x;
                }
            }
    }
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
        agg[w][at + v] = mine[v];
        car[w][at + v] = make_float2(A[v], B[v]);
    }
    lds_barrier();
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
#pragma unroll
        for (int j = 0; j < kWaves; ++j) {
            const float2 q = car[j][at + v];
            if (s.group > 0) h[v] = apply(q.x, q.y, h[v]);
        }
        for (int j = 0; j < w; ++j) {
            const float2 q = agg[j][at + v];
            h[v] = apply(q.x, q.y, h[v]);
        }
    }
}

struct FwdArgs {
    Cut k;
    LinSeq f, x;
    const float *h0;
    const int *lens;
    SeqOut h;
};

template <typename T, int VEC, int U>
struct FwdBuf {
    Unit<T, VEC> f[U], x[U];
};

template <typename T, int VEC, int U>
struct FwdLoad {
    const T *f, *x;
    int64_t sf, sx;
    int last, len;
    __device__ __forceinline__ FwdLoad(const FwdArgs &a, const Spot<VEC> &s)
        : f(row_at<T, VEC>(a.f, s.b, s.i)), x(row_at<T, VEC>(a.x, s.b, s.i)), sf(a.f.st), sx(a.x.st),
          last(a.k.T - 1), len(s.len) {}
    __device__ __forceinline__ void operator()(FwdBuf<T, VEC, U> &q, int t0) const {
        if (!__any(t0 < len)) return;  // nothing of it counts
#pragma unroll
        for (int j = 0; j < U; ++j) {
            const int64_t t = min(t0 + j, last);
            q.f[j] = *(const Unit<T, VEC> *)(f + t * sf);
            q.x[j] = *(const Unit<T, VEC> *)(x + t * sx);
        }
    }
};

template <bool LOGIT>
__device__ __forceinline__ float advance(float f, float x, float h) {
    return LOGIT ? fmaf(shut(f), x - h, h) : fmaf(f, h, x);
}

// First launch, forward.
template <typename T, bool LOGIT, int VEC, int U>
__global__ __launch_bounds__(kThreads) void gated_sum_kernel(FwdArgs a) {
    const Cut &k = a.k;
    const Spot<VEC> s(k, a.lens, true);
    const FwdLoad<T, VEC, U> load(a, s);
    float A[VEC], B[VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) A[v] = 1.0f, B[v] = 0.0f;
    FwdBuf<T, VEC, U> q;
    if (s.lo < s.hi) load(q, s.lo);
    batches<U>(s.lo, s.hi, q, load, [&](const FwdBuf<T, VEC, U> &now, int t0) {
        const int end = min(s.hi, s.len);
        const bool full = __all(t0 + U <= end);
#pragma unroll
        for (int j = 0; j < U; ++j)
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                const float f = to_f32<T>(now.f[j].v[v]), x = to_f32<T>(now.x[j].v[v]);
                const float g = LOGIT ? shut(f) : f;
                const float bn = LOGIT ? fmaf(g, x - B[v], B[v]) : fmaf(g, B[v], x);
                const float an = LOGIT ? fmaf(-g, A[v], A[v]) : A[v] * g;
                const bool on = full || t0 + j < end;
                B[v] = on ? bn : B[v];
                A[v] = on ? an : A[v];
            }
    });
    leave<VEC>(k, s, A, B, a.h0);
}

// Second launch, or the only one (CUT false: a wave walks the whole sequence).
template <typename T, bool LOGIT, int VEC, int U, bool CUT>
__global__ __launch_bounds__(kThreads) void gated_fwd_kernel(FwdArgs a) {
    const Cut &k = a.k;
    const Spot<VEC> s(k, a.lens, CUT);
    if (!CUT && s.c0 - (int)(threadIdx.x & 63) * VEC >= k.C) return;  // no tile for this wave
    const FwdLoad<T, VEC, U> load(a, s);
    FwdBuf<T, VEC, U> q;
    if (s.lo < s.hi) load(q, s.lo);
    float h[VEC];
    if (CUT) {
        begin<VEC>(k, s, h);
    } else {
#pragma unroll
        for (int v = 0; v < VEC; ++v) h[v] = a.h0 ? a.h0[s.c + v] : 0.0f;
    }
    T *out = (T *)a.h.p + (int64_t)s.b * a.h.sb + s.i;
    batches<U>(s.lo, s.hi, q, load, [&](const FwdBuf<T, VEC, U> &now, int t0) {
        const bool full = __all(t0 + U <= min(s.hi, s.len));
#pragma unroll
        for (int j = 0; j < U; ++j) {
            const bool on = full || t0 + j < min(s.hi, s.len);
            Unit<T, VEC> o;
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                const float hn = advance<LOGIT>(to_f32<T>(now.f[j].v[v]), to_f32<T>(now.x[j].v[v]), h[v]);
                h[v] = on ? hn : h[v];
                o.v[v] = from_f32<T>(on ? hn : 0.0f);
            }
            if (t0 + j < s.hi && s.c0 < k.C) *(Unit<T, VEC> *)(out + (int64_t)(t0 + j) * a.h.st) = o;
        }
    });
    if (k.state && s.p == k.P - 1 && s.c0 < k.C) {
#pragma unroll
        for (int v = 0; v < VEC; ++v) k.state[s.c + v] = h[v];
    }
}

template <typename T, bool LOGIT>
__global__ __launch_bounds__(256) void gated_step_kernel(GatedDims d, LinSeq f, LinSeq x, const float *h,
                                                         SeqOut y, float *h_out) {
    const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (c >= (int64_t)d.B * d.D) return;
    const int b = (int)(c / d.D), i = (int)(c - (int64_t)b * d.D);
    const float n = advance<LOGIT>(to_f32<T>(((const T *)f.p)[b * f.sb + i]), to_f32<T>(((const T *)x.p)[b * x.sb + i]),
                                   h[c]);
    h_out[c] = n;
    if (y.p) ((T *)y.p)[b * y.sb + i] = from_f32<T>(n);
}

// Backward: step r of the recurrence is t = T - 1 - r; the state is e = a_{t+1} g_{t+1},
// g_t = dh_t + e, e' = a_t g_t.
struct BwdArgs {
    Cut k;
    LinSeq f, x, h, dh;
    const float *h0, *dhT;
    const int *lens;
    SeqOut df, dx;
};

template <typename T, int VEC, int U>
struct BwdBuf {
    Unit<T, VEC> f[U], dh[U];
};
template <typename T, int VEC, int U>
struct BwdMore : BwdBuf<T, VEC, U> {
    Unit<T, VEC> x[U], h[U];
};

template <typename T, bool LOGIT, int VEC, int U>
struct BwdLoad {
    const T *f, *dh, *x, *h;
    int64_t sf, sd, sx, sh;
    int last, len;
    bool head;  // the chunk holds the sequence's first step
    __device__ __forceinline__ BwdLoad(const BwdArgs &a, const Spot<VEC> &s)
        : f(row_at<T, VEC>(a.f, s.b, s.i)), dh(row_at<T, VEC>(a.dh, s.b, s.i)), x(row_at<T, VEC>(a.x, s.b, s.i)),
          h(row_at<T, VEC>(a.h, s.b, s.i)), sf(a.f.st), sd(a.dh.st), sx(a.x.st), sh(a.h.st), last(a.k.T - 1),
          len(s.len), head(a.k.off == 0) {}
    __device__ __forceinline__ bool none(int r0) const { return !__any(last - (r0 + U - 1) < len); }
    __device__ __forceinline__ void operator()(BwdBuf<T, VEC, U> &q, int r0) const {
        if (none(r0)) return;
#pragma unroll
        for (int j = 0; j < U; ++j) {
            const int64_t t = max(last - (r0 + j), 0);
            q.f[j] = *(const Unit<T, VEC> *)(f + t * sf);
            q.dh[j] = *(const Unit<T, VEC> *)(dh + t * sd);
        }
    }
    __device__ __forceinline__ void operator()(BwdMore<T, VEC, U> &q, int r0) const {
        if (none(r0)) return;
        (*this)((BwdBuf<T, VEC, U> &)q, r0);
#pragma unroll
        for (int j = 0; j < U; ++j) {
            const int64_t t = max(last - (r0 + j), 0);
            if (LOGIT) q.x[j] = *(const Unit<T, VEC> *)(x + t * sx);
            // h_{t-1}; before the sequence's first step it is h0
            q.h[j] = *(const Unit<T, VEC> *)(h + (t == 0 && head ? 0 : t - 1) * sh);
        }
    }
};

template <typename T, bool LOGIT, int VEC, int U>
__global__ __launch_bounds__(kThreads) void gated_bwd_sum_kernel(BwdArgs a) {
    const Cut &k = a.k;
    const Spot<VEC> s(k, a.lens, true);
    const BwdLoad<T, LOGIT, VEC, U> load(a, s);
    float A[VEC], B[VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) A[v] = 1.0f, B[v] = 0.0f;
    BwdBuf<T, VEC, U> q;
    if (s.lo < s.hi) load(q, s.lo);
    batches<U>(s.lo, s.hi, q, load, [&](const BwdBuf<T, VEC, U> &now, int r0) {
        const bool full = __all(r0 + U <= s.hi && k.T - 1 - r0 < s.len);
#pragma unroll
        for (int j = 0; j < U; ++j)
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                const float f = to_f32<T>(now.f[j].v[v]), g = LOGIT ? shut(f) : f;
                const float d = B[v] + to_f32<T>(now.dh[j].v[v]);
                const float bn = LOGIT ? fmaf(-g, d, d) : g * d, an = LOGIT ? fmaf(-g, A[v], A[v]) : A[v] * g;
                const bool on = full || (r0 + j < s.hi && k.T - 1 - (r0 + j) < s.len);
                B[v] = on ? bn : B[v];
                A[v] = on ? an : A[v];
            }
    });
    leave<VEC>(k, s, A, B, a.dhT);
}

template <typename T, bool LOGIT, int VEC, int U, bool CUT>
__global__ __launch_bounds__(kThreads) void gated_bwd_kernel(BwdArgs a) {
    const Cut &k = a.k;
    const Spot<VEC> s(k, a.lens, CUT);
    if (!CUT && s.c0 - (int)(threadIdx.x & 63) * VEC >= k.C) return;
    const BwdLoad<T, LOGIT, VEC, U> load(a, s);
    BwdMore<T, VEC, U> q;
    if (s.lo < s.hi) load(q, s.lo);
    float e[VEC];
    if (CUT) {
        begin<VEC>(k, s, e);
    } else {
#pragma unroll
        for (int v = 0; v < VEC; ++v) e[v] = a.dhT ? a.dhT[s.c + v] : 0.0f;
    }
    T *of = (T *)a.df.p + (int64_t)s.b * a.df.sb + s.i, *ox = (T *)a.dx.p + (int64_t)s.b * a.dx.sb + s.i;
    batches<U>(s.lo, s.hi, q, load, [&](const BwdMore<T, VEC, U> &now, int r0) {
        const bool full = __all(r0 + U <= s.hi && k.T - 1 - r0 < s.len);
#pragma unroll
        for (int j = 0; j < U; ++j) {
            const int t = k.T - 1 - (r0 + j);
            const bool on = full || (r0 + j < s.hi && t < s.len);
            Unit<T, VEC> vf, vx;
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                const float f = to_f32<T>(now.f[j].v[v]), g = e[v] + to_f32<T>(now.dh[j].v[v]);
                float before = to_f32<T>(now.h[j].v[v]);
                if (t == 0 && k.off == 0) before = a.h0 ? a.h0[s.c + v] : 0.0f;
                float df, dx, en;
                if (LOGIT) {
                    // a u to full relative accuracy where either is small
                    const float ex = exp_fast(f), u = rcp_fast(1.0f + ex);
                    dx = u * g;
                    df = fminf(ex, 3e38f) * u * dx * (before - to_f32<T>(now.x[j].v[v]));
                    en = fmaf(-u, g, g);
                } else {
                    dx = g;
                    df = g * before;
                    en = f * g;
                }
                e[v] = on ? en : e[v];
                vf.v[v] = from_f32<T>(on ? df : 0.0f);
                vx.v[v] = from_f32<T>(on ? dx : 0.0f);
            }
            if (r0 + j < s.hi && s.c0 < k.C) {
                *(Unit<T, VEC> *)(of + (int64_t)t * a.df.st) = vf;
                *(Unit<T, VEC> *)(ox + (int64_t)t * a.dx.st) = vx;
            }
        }
    });
    if (k.state && s.p == k.P - 1 && s.c0 < k.C) {
#pragma unroll
        for (int v = 0; v < VEC; ++v) k.state[s.c + v] = e[v];
    }
}

// ------------------------------------------------------------------- plan
constexpr int kUnroll = 8, kUnrollBwd = 4;
constexpr int kMinSteps = 16;              // of a piece
constexpr int kFill = 6144;                // waves that fill the chip
constexpr int kMaxGroups = 256;            // workgroups along time: each reads the totals before it
constexpr int64_t kCacheBytes = 160 << 20; // of a chunk's inputs to the first launch

struct Plan {
    int vec, ntile;
    int P, R;       // waves along time in a chunk (1: not cut), steps of each
    int chunk, n;   // steps of a chunk, chunks
};

Plan plan(const GatedDims &d, bool bf16, int vec) {
    Plan p{};
    const int64_t C = (int64_t)d.B * d.D;
    p.vec = vec;
    p.ntile = (int)((C + 64 * vec - 1) / (64 * vec));
    const int64_t fit = std::max<int64_t>(kCacheBytes / (2 * C * (bf16 ? 2 : 4)), kWaves * kMinSteps);
    p.chunk = d.T, p.n = 1, p.P = 1, p.R = d.T;
    if (p.ntile >= kFill || d.T <= 2 * kMinSteps) return p;
    p.n = (int)((d.T + fit - 1) / fit);
    p.chunk = (d.T + p.n - 1) / p.n;
    p.n = (d.T + p.chunk - 1) / p.chunk;
    const int64_t want = std::min<int64_t>((kFill + p.ntile - 1) / p.ntile, (int64_t)kMaxGroups * kWaves);
    int64_t R = std::max<int64_t>((p.chunk + want - 1) / want, kMinSteps);
    R = (R + kUnroll - 1) / kUnroll * kUnroll;
    p.R = (int)R;
    p.P = (int)(((p.chunk + R - 1) / R + kWaves - 1) / kWaves * kWaves);
    return p;
}

// Bytes of the workspace: words, totals, the chunk's first and last state.
int64_t space(const Plan &p, int64_t C) {
    if (p.P == 1) return 0;
    return ((int64_t)(p.P + p.P / kWaves) * C * 8 + 2 * C * 4 + 15) / 16 * 16;
}

Cut cut(const GatedDims &d, const Plan &p, void *ws) {
    Cut k{};
    k.T = d.T, k.D = d.D, k.C = d.B * d.D;
    k.R = p.R, k.P = p.P, k.ntile = p.ntile;
    k.word = (float2 *)ws;
    k.total = k.word + (int64_t)p.P * k.C;
    k.start = (float *)(k.total + (int64_t)(p.P / kWaves) * k.C);
    k.state = k.start + k.C;
    return k;
}

// Whether two channels of every row stand together at a multiple of their size.
bool pairs(int D, size_t e, std::initializer_list<LinSeq> seqs) {
    if (D % 2) return false;
    for (const LinSeq &s : seqs)
        if ((uintptr_t)s.p % (2 * e) || s.st % 2 || s.sb % 2) return false;
    return true;
}
LinSeq in(const SeqOut &o) { return LinSeq{o.p, o.st, o.sb}; }
// A sequence from step t on.
LinSeq from(LinSeq s, int t, bool bf16) {
    s.p = (const char *)s.p + (int64_t)t * s.st * (bf16 ? 2 : 4);
    return s;
}
SeqOut from(SeqOut s, int t, bool bf16) {
    s.p = (char *)s.p + (int64_t)t * s.st * (bf16 ? 2 : 4);
    return s;
}

// Runs a call: its launches over each chunk, in the order of the recurrence.  args(cut,
// first step, start, lens) makes a launch's arguments, sum and main launch it.
template <typename A, typename S, typename M>
hipError_t run(const GatedDims &d, const Plan &p, void *ws, const float *start, float *end, bool bwd, A args, S sum,
               M main) {
    const Cut whole = cut(d, p, ws);
    const unsigned one = (unsigned)((p.ntile + kWaves - 1) / kWaves);
    const unsigned grid = p.P == 1 ? one : (unsigned)((int64_t)p.ntile * (p.P / kWaves));
    for (int i = 0; i < p.n; ++i) {
        Cut k = whole;
        k.off = (bwd ? p.n - 1 - i : i) * p.chunk;
        k.T = std::min(p.chunk, d.T - k.off);
        // a chunk after the first begins with the state that the one before it left
        const float *from_ = i ? whole.state : start;
        if (i == p.n - 1) k.state = end;
        const auto a = args(k, from_);
        if (p.P > 1) sum(a, grid);
        main(a, grid);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

// Calls go(type tag, logit tag, vec tag).
template <int V>
using Int = std::integral_constant<int, V>;
template <typename F>
void by_kind(bool bf16, bool logit, int vec, F go) {
    auto gate = [&](auto type, auto v) {
        if (logit) go(type, std::true_type{}, v);
        else go(type, std::false_type{}, v);
    };
    if (!bf16) gate(float{}, Int<1>{});
    else if (vec == 2) gate(uint16_t{}, Int<2>{});
    else gate(uint16_t{}, Int<1>{});
}

}  // namespace

// No launch nears 2^32 threads: B * D <= 2^30 channels, a thread or less to each where time
// is not cut, and about kFill waves where it is.
size_t gated_bytes(const GatedDims &d, bool bf16) {
    // a bf16 call may have either number of channels to a lane
    int64_t n = 0;
    for (int vec = 1; vec <= (bf16 ? 2 : 1); ++vec) n = std::max(n, space(plan(d, bf16, vec), (int64_t)d.B * d.D));
    return (size_t)n;
}

hipError_t launch_gated_fwd(const GatedDims &d, bool bf16, LinSeq f, LinSeq x, const float *h0,
                            const int *lens, SeqOut h, float *hT, void *ws, hipStream_t s) {
    const Plan p = plan(d, bf16, bf16 && pairs(d.D, 2, {f, x, in(h)}) ? 2 : 1);
    hipError_t e = hipSuccess;
    by_kind(bf16, d.logit, p.vec, [&](auto type, auto logit, auto vec) {
        using T = decltype(type);
        constexpr bool L = decltype(logit)::value;
        constexpr int V = decltype(vec)::value;
        e = run(d, p, ws, h0, hT, false,
                [&](const Cut &k, const float *start) {
                    return FwdArgs{k, from(f, k.off, bf16), from(x, k.off, bf16), start, lens, from(h, k.off, bf16)};
                },
                [&](const FwdArgs &a, unsigned grid) {
                    hipLaunchKernelGGL((gated_sum_kernel<T, L, V, kUnroll>), dim3(grid), dim3(kThreads), 0, s, a);
                },
                [&](const FwdArgs &a, unsigned grid) {
                    if (p.P > 1)
                        hipLaunchKernelGGL((gated_fwd_kernel<T, L, V, kUnroll, true>), dim3(grid), dim3(kThreads), 0, s, a);
                    else
                        hipLaunchKernelGGL((gated_fwd_kernel<T, L, V, kUnroll, false>), dim3(grid), dim3(kThreads), 0, s, a);
                });
    });
    return e;
}

hipError_t launch_gated_step(const GatedDims &d, bool bf16, LinSeq f, LinSeq x, const float *h,
                             SeqOut y, float *h_out, hipStream_t s) {
    const dim3 grid((unsigned)(((int64_t)d.B * d.D + 255) / 256)), thr(256);
    by_kind(bf16, d.logit, 1, [&](auto type, auto logit, auto) {
        hipLaunchKernelGGL((gated_step_kernel<decltype(type), decltype(logit)::value>), grid, thr, 0, s, d, f, x, h, y,
                           h_out);
    });
    return hipGetLastError();
}

hipError_t launch_gated_bwd(const GatedDims &d, bool bf16, LinSeq f, LinSeq x, LinSeq h, LinSeq dh,
                            const float *h0, const float *dhT, const int *lens, SeqOut df, SeqOut dx,
                            float *dh0, void *ws, hipStream_t s) {
    if (!d.logit) x = f;  // not read
    const Plan p = plan(d, bf16, bf16 && pairs(d.D, 2, {f, x, h, dh, in(df), in(dx)}) ? 2 : 1);
    hipError_t e = hipSuccess;
    by_kind(bf16, d.logit, p.vec, [&](auto type, auto logit, auto vec) {
        using T = decltype(type);
        constexpr bool L = decltype(logit)::value;
        constexpr int V = decltype(vec)::value;
        e = run(d, p, ws, dhT, dh0, true,
                [&](const Cut &k, const float *start) {
                    return BwdArgs{k, from(f, k.off, bf16), from(x, k.off, bf16), from(h, k.off, bf16),
                                   from(dh, k.off, bf16), h0, start, lens, from(df, k.off, bf16), from(dx, k.off, bf16)};
                },
                [&](const BwdArgs &a, unsigned grid) {
                    hipLaunchKernelGGL((gated_bwd_sum_kernel<T, L, V, kUnroll>), dim3(grid), dim3(kThreads), 0, s, a);
                },
                [&](const BwdArgs &a, unsigned grid) {
                    if (p.P > 1)
                        hipLaunchKernelGGL((gated_bwd_kernel<T, L, V, kUnrollBwd, true>), dim3(grid), dim3(kThreads), 0, s, a);
                    else
                        hipLaunchKernelGGL((gated_bwd_kernel<T, L, V, kUnrollBwd, false>), dim3(grid), dim3(kThreads), 0, s, a);
                });
    });
    return e;
}

}  // namespace lm
}  // namespace rnn355
