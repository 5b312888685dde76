// verify.hip -- verification of drafted tokens against the target's logits.
//
//   p_k = softmax(l_k / T), q_k the same of the draft's logits (or 1 at the draft)
//   accept draft k while u_k q_k(x_k) < p_k(x_k); then draw from
//   w = max(p - q, 0) of the refused row, or w = p of the last one:
//   the lowest i with sum_{j <= i} w_j > u_K sum w
//
// Three launches.  The first reads every row once, a chunk of it to a workgroup,
// and leaves the chunk's maximum and sum of weights.  The second joins those,
// decides how many drafts stand (each workgroup of a sequence for itself) and
// sums w over the chunks of the row to draw from.  The third finds the chunk in
// which the sum passes u and the entry in it.
//
// Weights and sums are 64-bit.  The borders between a vocabulary's V entries lie
// 1/V of the sum apart on average; a sum of 32-bit terms is off by 1e-7 of it, so
// that about one draw in a hundred at V = 128000 would depend on how it was added
// up.  With 64 bits (weights to 2e-14, below) that is one in 10^8.
#include <algorithm>

#include "row.h"

namespace rnn355 {
namespace lm {

namespace {

constexpr int kThreads = 256, kPer = 16, kChunk = kThreads * kPer, kWaves = kThreads / 64;
constexpr double kLog2eD = 1.4426950408889634;

// 2^t for t <= 0 to a relative 1.6e-14, exactly 1 at 0 and 0 below -1075; a NaN gives
// any value.  t = n + r with n the nearest whole number, 2^r = 1 + r q(r) with q of
// degree 8 fitted on Chebyshev nodes of [-1/2, 1/2] by least squares on the relative
// error, reweighted towards equal ripple.
__device__ __forceinline__ double pow2(double t) {
    t = fmax(t, -2000.0);
    const double big = 6755399441055744.0;  // 1.5 * 2^52: its lowest bits then hold n
    const double s = t + big;
    const double r = t - (s - big);
    double q = 0x1.b3de036db3bd6p-24;
    q = fma(q, r, 0x1.63e698d29c93cp-20);
    q = fma(q, r, 0x1.ffce2ff794fdcp-17);
    q = fma(q, r, 0x1.430897f0af9dbp-13);
    q = fma(q, r, 0x1.5d87fd93724e7p-10);
    q = fma(q, r, 0x1.3b2ab72413c05p-7);
    q = fma(q, r, 0x1.c6b08d70c88e9p-5);
    q = fma(q, r, 0x1.ebfbdff81bdf2p-3);
    q = fma(q, r, 0x1.62e42fefa37d1p-1);
    return __builtin_amdgcn_ldexp(fma(q, r, 1.0), (int)(uint32_t)__double_as_longlong(s));
}

// What a chunk of a row leaves: its maximum, the lowest index of that (only where
// the sequence is greedy) and sum of 2^((x - m) scale), NaN where the chunk holds a
// NaN or +inf.
struct Part {
    double s;
    float m;
    int at;
};

// What the second launch leaves for the third.
struct Pick {
    double scale, mp, ip, mq, iq;  // weight p = 2^((x - mp) scale) ip, q the same
    int row, acc, drop, token;     // row to draw from; draft without q to leave out (or -1);
                                   // token >= -1: already known
};

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
    for (int o = 32; o; o >>= 1) v = fmaxf(v, __shfl_xor(v, o));
    return v;
}
__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
    for (int o = 32; o; o >>= 1) v += __shfl_xor(v, o);
    return v;
}
__device__ __forceinline__ int wave_min(int v) {
#pragma unroll
    for (int o = 32; o; o >>= 1) v = min(v, __shfl_xor(v, o));
    return v;
}
__device__ __forceinline__ double block_sum(double v, double *tmp) {
    v = wave_sum(v);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) tmp[threadIdx.x >> 6] = v;
    __syncthreads();
    double all = 0.0;
#pragma unroll
    for (int i = 0; i < kWaves; ++i) all += tmp[i];
    return all;
}

__device__ __forceinline__ int drafts_of(const VerifyArgs &a, int b) {
    return a.n ? min(max(a.n[b], 0), a.K) : a.K;
}
// log2(e) / temperature, above 0 even where that is +inf; 0 for a temperature of 0
// or less (or NaN): greedy
__device__ __forceinline__ double scale_of(const VerifyArgs &a, int b) {
    if (!a.temp) return kLog2eD;
    const float t = a.temp[b];
    return t > 0.0f ? fmax(kLog2eD / (double)t, 1e-300) : 0.0;
}
template <typename T>
__device__ __forceinline__ const T *row_of(const LinSeq &s, int k, int b) {
    return (const T *)s.p + (int64_t)k * s.st + (int64_t)b * s.sb;
}

// Rows of a sequence: 0 .. K the target's, K + 1 .. 2 K the draft's.
template <typename T>
__global__ __launch_bounds__(kThreads) void verify_sum_kernel(VerifyArgs a, int nch, int rows) {
    constexpr int N = Row<T>::N, U = kPer / N;
    __shared__ float wm[kWaves];
    __shared__ double ws[kWaves];
    __shared__ int wi[kWaves], wbad[kWaves];
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
    const int64_t at = blockIdx.x;
    const int64_t rb = at / nch;
    const int ch = (int)(at - rb * nch), r = (int)(rb / a.B), b = (int)(rb - (int64_t)r * a.B);
    const int n = drafts_of(a, b);
    const double scale = scale_of(a, b);
    const bool draft = r > a.K;
    if (draft ? r - a.K - 1 >= n || scale == 0.0 : r > n) return;  // a row that nothing asks for
    const Row<T> row(draft ? row_of<T>(a.q, r - a.K - 1, b) : row_of<T>(a.logits, r, b), a.V);
    const int u0 = ch * (kChunk / N);
    float x[kPer];
    row.template load_all<U>(u0 + tid, kThreads, x);
    float m = -INFINITY;
    bool bad = false;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        m = fmaxf(m, x[i]);
        bad |= x[i] != x[i];
    }
    m = wave_max(m);
    if (lane == 0) wm[w] = m;
    bad = __any(bad);
    if (lane == 0) wbad[w] = bad;
    __syncthreads();
    m = wm[0], bad = wbad[0];
#pragma unroll
    for (int i = 1; i < kWaves; ++i) m = fmaxf(m, wm[i]), bad |= wbad[i] != 0;
    bad |= m == INFINITY;
    Part *out = (Part *)a.ws + at;
    if (scale == 0.0) {
        int first = 0x7FFFFFFF;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int idx = (u0 + (i / N) * kThreads + tid) * N + (i % N) - row.off;
            if (x[i] == m && idx >= 0 && idx < a.V) first = min(first, idx);
        }
        first = wave_min(first);
        if (lane == 0) wi[w] = first;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kWaves; ++i) first = min(first, wi[i]);
        if (tid == 0) *out = Part{bad ? NAN : m == -INFINITY ? 0.0 : 1.0, m, first};
        return;
    }
    const double ref = m == -INFINITY ? 0.0 : (double)m;
    double s = 0.0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) s += pow2(((double)x[i] - ref) * scale);
    s = wave_sum(s);
    if (lane == 0) ws[w] = s;
    __syncthreads();
    s = 0.0;
#pragma unroll
    for (int i = 0; i < kWaves; ++i) s += ws[i];
    if (tid == 0) *out = Part{bad ? NAN : s, m, 0};
}

// Joins the parts of a row, a wave to a row: maximum and sum (greedy: lowest index
// of the maximum in `at`).
struct Joined {
    double m, s;
    int at;
};
__device__ __forceinline__ Joined join(const Part *p, int nch, double scale) {
    const int lane = threadIdx.x & 63;
    float m = -INFINITY;
    for (int c = lane; c < nch; c += 64) m = fmaxf(m, p[c].m);
    m = wave_max(m);
    double s = 0.0;
    int at = 0x7FFFFFFF;
    for (int c = lane; c < nch; c += 64) {
        const Part q = p[c];
        if (q.s != q.s) s = q.s;                  // a NaN somewhere
        if (q.m == -INFINITY) continue;           // nothing allowed in it
        s += scale == 0.0 ? q.s : q.s * pow2(((double)q.m - (double)m) * scale);
        if (q.m == m) at = min(at, q.at);
    }
    return Joined{m == -INFINITY ? 0.0 : (double)m, wave_sum(s), wave_min(at)};
}

// Weights of row to draw from, entry i of value x, y (draft's).
__device__ __forceinline__ double weight(const Pick &p, float x, float y, int i, bool q) {
    double w = pow2(((double)x - p.mp) * p.scale);
    if (q) return fmax(w * p.ip - pow2(((double)y - p.mq) * p.scale) * p.iq, 0.0);
    return i == p.drop ? 0.0 : w;
}

// Values of a chunk of the row to draw from, by position: entry e of unit j of a
// thread is value (u0 + j kThreads + tid) N + e of both rows, counted from the
// target's aligned start.
template <typename T>
__device__ __forceinline__ void load_pair(const VerifyArgs &a, const Pick &p, int b, int ch, bool q,
                                          float *x, float *y, int &i0) {
    constexpr int N = Row<T>::N, U = kPer / N;
    const Row<T> row(row_of<T>(a.logits, p.row, b), a.V);
    const int u = ch * (kChunk / N) + threadIdx.x;
    row.template load_all<U>(u, kThreads, x);
    i0 = u * N - row.off;
    if (!q) return;
    const T *qr = row_of<T>(a.q, p.row, b);
    if ((int)(((uintptr_t)qr & 15) / sizeof(T)) == row.off) {
        Row<T>(qr, a.V).template load_all<U>(u, kThreads, y);
    } else {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int at = i0 + (i / N) * kThreads * N + i % N;
            y[i] = at >= 0 && at < a.V ? to_f32<T>(qr[at]) : -INFINITY;
        }
    }
}

template <typename T>
__global__ __launch_bounds__(kThreads) void verify_pick_kernel(VerifyArgs a, int nch, int rows) {
    __shared__ Joined all[2 * kMaxDrafts + 1];
    __shared__ Pick pick;
    __shared__ double tmp[kWaves];
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
    const int b = blockIdx.x / nch, ch = blockIdx.x - b * nch;
    const int n = drafts_of(a, b);
    const double scale = scale_of(a, b);
    const Part *part = (const Part *)a.ws;
    const bool greedy = scale == 0.0, has_q = a.q.p != nullptr && !greedy;
    Pick *picks = (Pick *)(part + (int64_t)rows * a.B * nch);
    double *sums = (double *)(picks + a.B);
    const int live = n + 1 + (has_q ? n : 0);
    for (int i = w; i < live; i += kWaves) {
        const int r = i <= n ? i : a.K + (i - n);
        const Joined j = join(part + ((int64_t)r * a.B + b) * nch, nch, scale);
        if (lane == 0) all[i] = j;
    }
    __syncthreads();
    if (w == 0) {
        bool ok = false;
        if (lane < n) {
            const int id = load_id(a.drafts, lane * a.B + b, a.V);
            const Joined p = all[lane];
            if (id < a.V && p.s > 0.0) {
                if (greedy) {
                    ok = id == p.at;
                } else {
                    const double px = pow2(((double)to_f32<T>(row_of<T>(a.logits, lane, b)[id]) - p.m) * scale) / p.s;
                    double qx = 1.0;
                    if (has_q) {
                        const Joined q = all[n + 1 + lane];
                        qx = q.s == 0.0 ? 0.0  // NaN: refuses
                                        : pow2(((double)to_f32<T>(row_of<T>(a.q, lane, b)[id]) - q.m) * scale) / q.s;
                    }
                    const float u = fminf(fmaxf(a.u[(int64_t)lane * a.B + b], 0.0f), 1.0f);
                    ok = (double)u * qx < px;
                }
            }
        }
        const uint64_t stood = __ballot(ok);
        const int acc = __ffsll((unsigned long long)~stood) - 1;  // n <= 63: bit 63 is never set
        if (lane == 0) {
            const Joined p = all[acc];
            Pick k{scale, p.m, 1.0 / p.s, 0.0, 0.0, acc, acc, -1, -2};
            if (!(p.s > 0.0)) k.token = -1;
            else if (greedy) k.token = p.at;
            else if (acc < n && has_q) {
                const Joined q = all[n + 1 + acc];
                k.mq = q.m;
                k.iq = q.s == 0.0 ? 0.0 : 1.0 / q.s;
                if (q.s != q.s) k.token = -1;
            } else if (acc < n) {
                k.drop = load_id(a.drafts, acc * a.B + b, a.V);
            }
            pick = k;
            if (ch == 0) picks[b] = k;
        }
    }
    __syncthreads();
    const Pick p = pick;
    if (p.token != -2) return;
    const bool q = has_q && p.acc < n;
    float x[kPer], y[kPer];
    int i0;
    load_pair<T>(a, p, b, ch, q, x, y, i0);
    double s = 0.0;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
        s += weight(p, x[i], y[i], i0 + (i / Row<T>::N) * kThreads * Row<T>::N + i % Row<T>::N, q);
    s = block_sum(s, tmp);
    if (tid == 0) sums[(int64_t)b * nch + ch] = s;
}

template <typename T>
__global__ __launch_bounds__(kThreads) void verify_draw_kernel(VerifyArgs a, int nch, int rows) {
    constexpr int N = Row<T>::N, U = kPer / N;
    __shared__ double unit[U][kWaves];
    __shared__ int found, last;
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, b = blockIdx.x;
    const int n = drafts_of(a, b);
    const Part *part = (const Part *)a.ws;
    const Pick *picks = (const Pick *)(part + (int64_t)rows * a.B * nch);
    const double *sums = (const double *)(picks + a.B) + (int64_t)b * nch;
    Pick p = picks[b];
    bool q = a.q.p != nullptr && p.scale != 0.0 && p.acc < n;
    int token = p.token;
    if (token == -2) {
        token = -1;
        double all = 0.0;
        for (int c = 0; c < nch; ++c) all += sums[c];
        const Part *pp = part + ((int64_t)p.row * a.B + b) * nch;
        const bool instead = all == 0.0;  // nothing of p - q is left: p itself
        if (instead) {
            p.drop = -1;
            q = false;
        }
        auto sum = [&](int c) {
            if (!instead) return sums[c];
            return pp[c].m == -INFINITY ? 0.0 : pp[c].s * pow2(((double)pp[c].m - p.mp) * p.scale);
        };
        if (instead)
            for (int c = 0; c < nch; ++c) all += sum(c);
        const double goal = (double)fminf(fmaxf(a.u[(int64_t)a.K * a.B + b], 0.0f), 1.0f) * all;
        // the chunk in which the sum passes the goal; at its very end the last with any weight
        double before = 0.0, s = 0.0;
        int ch = -1;
        for (int c = 0; c < nch; ++c) {
            const double v = sum(c);
            if (!(v > 0.0)) continue;
            before = s;
            s += v;
            ch = c;
            if (s > goal) break;
        }
        if (ch >= 0) {
            float x[kPer], y[kPer];
            double v[kPer], us[U];
            int i0;
            load_pair<T>(a, p, b, ch, q, x, y, i0);
#pragma unroll
            for (int j = 0; j < U; ++j) {
                us[j] = 0.0;
#pragma unroll
                for (int e = 0; e < N; ++e) {
                    const int i = j * N + e;
                    v[i] = weight(p, x[i], y[i], i0 + j * kThreads * N + e, q);
                    us[j] += v[i];
                }
                const double t = wave_sum(us[j]);
                if (lane == 0) unit[j][w] = t;
            }
            if (tid == 0) found = 0x7FFFFFFF, last = -1;
            __syncthreads();
            // indices grow with the unit j, the thread, the entry e
            double run = before;
#pragma unroll
            for (int j = 0; j < U; ++j) {
                double mine = us[j];
#pragma unroll
                for (int o = 1; o < 64; o <<= 1) {
                    const double up = __shfl_up(mine, o);
                    if (lane >= o) mine += up;
                }
                double at = run + (mine - us[j]);
                for (int i = 0; i < w; ++i) at += unit[j][i];
#pragma unroll
                for (int e = 0; e < N; ++e) {
                    const int i = j * N + e, idx = i0 + j * kThreads * N + e;
                    at += v[i];
                    if (v[i] > 0.0) {
                        atomicMax(&last, idx);
                        if (at > goal) atomicMin(&found, idx);
                    }
                }
                for (int i = 0; i < kWaves; ++i) run += unit[j][i];
            }
            __syncthreads();
            token = found != 0x7FFFFFFF ? found : last;
        }
    }
    if (tid == 0) a.accepted[b] = p.acc;
    for (int k = tid; k <= a.K; k += kThreads) {
        int t = -1;
        if (k < p.acc)
            t = load_id(a.drafts, k * a.B + b, a.V);
        else if (k == p.acc)
            t = token;
        a.tokens[(int64_t)k * a.B + b] = t;
    }
}

template <typename T>
hipError_t verify_t(const VerifyArgs &a, hipStream_t s) {
    const int nch = chunks(a.V, kChunk, sizeof(T)), rows = a.q.p ? 2 * a.K + 1 : a.K + 1;
    const dim3 thr(kThreads);
    hipLaunchKernelGGL(verify_sum_kernel<T>, dim3((unsigned)((int64_t)rows * a.B * nch)), thr, 0, s, a, nch, rows);
    hipLaunchKernelGGL(verify_pick_kernel<T>, dim3((unsigned)((int64_t)a.B * nch)), thr, 0, s, a, nch, rows);
    hipLaunchKernelGGL(verify_draw_kernel<T>, dim3((unsigned)a.B), thr, 0, s, a, nch, rows);
    return hipGetLastError();
}

}  // namespace

size_t verify_bytes(int K, int B, int V) {
    // the larger chunk count of the two types
    const size_t nch = chunks(V, kChunk, 2);
    return ((size_t)(2 * K + 1) * nch * sizeof(Part) + sizeof(Pick) + nch * sizeof(double)) * B;
}

bool verify_grid_ok(int K, int B, int V) {
    return grid_ok((int64_t)(2 * K + 1) * B * chunks(V, kChunk, 2), kThreads);
}

hipError_t launch_verify(const VerifyArgs &a, bool bf16, hipStream_t s) {
    return bf16 ? verify_t<uint16_t>(a, s) : verify_t<float>(a, s);
}

}  // namespace lm
}  // namespace rnn355
