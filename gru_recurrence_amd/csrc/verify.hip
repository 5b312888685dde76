// verify.hip -- verification of drafted tokens against the target's logits.
//
//   p_k = softmax(l_k / T), q_k the same of the draft's logits (or 1 at the draft)
//   accept draft k while u_k q_k(x_k) < p_k(x_k); then draw from
//   w = max(p - q, 0) of the refused row, or w = p of the last one:
//   the lowest i with sum_{j <= i} w_j > u_K sum w
//
// Two launches.  The first reads every row once, a chunk of it to a workgroup, and
// leaves the chunk's maximum and sum of weights.  The second joins those, decides how
// many drafts stand (each workgroup of a sequence for itself) and sums w over the
// chunks of the row to draw from; the sequence's last workgroup to finish finds the
// chunk in which the sum passes u, and the entry in it.  Sums are added in the order of
// the chunks, so nothing depends on which workgroup that is.
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

// 2^t for t <= 0 to a relative 1.6e-14, exactly 1 at 0, 0 below -1020 (and for a NaN).
// t = n + r with n the nearest whole number, 2^r = 1 + r q(r) with q of degree 8 fitted
// on Chebyshev nodes of [-1/2, 1/2] by least squares on the relative error, reweighted
// towards equal ripple; n goes into the exponent's bits.
__device__ __forceinline__ double pow2(double t) {
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
    const uint64_t p = (uint64_t)__double_as_longlong(fma(q, r, 1.0));
    const uint32_t n = (uint32_t)__double_as_longlong(s);
    const uint64_t v = p + ((uint64_t)(n << 20) << 32);
    return t >= -1020.0 ? __longlong_as_double((long long)v) : 0.0;
}

// What a chunk of a row leaves: its maximum, the lowest index of that (only where
// the sequence is greedy) and sum of 2^((x - m) scale), NaN where the chunk holds a
// NaN or +inf.
struct Part {
    double s;
    float m;
    int at;
};

// How to draw the token behind the accepted ones.
struct Pick {
    double scale, mp, ip, mq, iq;  // weight p = 2^((x - mp) scale) ip, q the same
    int acc, drop, token;          // accepted, so also the row to draw from; draft without q to
                                   // leave out (or -1); token >= -1: already known
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

// The workspace: parts [rows][B][nch], sums [B][nch], counters [B].
__device__ __forceinline__ double *chunk_sums(const VerifyArgs &a, int nch, int rows) {
    return (double *)((Part *)a.ws + (int64_t)rows * a.B * nch);
}
__device__ __forceinline__ unsigned *counter(const VerifyArgs &a, int nch, int rows) {
    return (unsigned *)(chunk_sums(a, nch, rows) + (int64_t)a.B * nch);
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
    if (r == 0 && ch == 0 && tid == 0) counter(a, nch, rows)[b] = 0;
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

// A row's parts joined: maximum and sum (greedy: lowest index of the maximum in `at`).
struct Joined {
    double m, s;
    int at;
};

// Joins rows i of a sequence, parts of row i from part(i) on, `across` lanes (a power of
// two of at least the chunks, or 64) to a row.
constexpr int kMaxParts = 4;  // of a lane: V <= 1000000 has at most 246 chunks
template <typename F>
__device__ __forceinline__ void join(int live, int nch, int across, double scale, Joined *all, F part) {
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const int each = 64 / across, sub = lane / across, l = lane - sub * across;
    for (int base = w * each; base < live; base += kWaves * each) {
        const int i = base + sub;
        Part q[kMaxParts];
        float m = -INFINITY;
#pragma unroll
        for (int j = 0; j < kMaxParts; ++j) {
            const int c = j * 64 + l;
            q[j] = Part{0.0, -INFINITY, 0x7FFFFFFF};
            if (i < live && c < nch) q[j] = part(i)[c];
            m = fmaxf(m, q[j].m);
        }
        for (int o = across >> 1; o; o >>= 1) m = fmaxf(m, __shfl_xor(m, o));
        const double ref = m == -INFINITY ? 0.0 : (double)m;
        double s = 0.0;
        int at = 0x7FFFFFFF;
#pragma unroll
        for (int j = 0; j < kMaxParts; ++j) {
            if (q[j].s != q[j].s) s = q[j].s;  // a NaN somewhere
            if (q[j].m == -INFINITY) continue; // nothing allowed in it
            s += scale == 0.0 ? q[j].s : q[j].s * pow2(((double)q[j].m - ref) * scale);
            if (q[j].m == m) at = min(at, q[j].at);
        }
        for (int o = across >> 1; o; o >>= 1) {
            s += __shfl_xor(s, o);
            at = min(at, __shfl_xor(at, o));
        }
        if (l == 0 && i < live) all[i] = Joined{ref, s, at};
    }
}

// Weight of entry i of the row to draw from, of value x, y (draft's).
__device__ __forceinline__ double weight(const Pick &p, float x, float y, int i, bool q) {
    const double w = pow2(((double)x - p.mp) * p.scale);
    if (q) return fmax(w * p.ip - pow2(((double)y - p.mq) * p.scale) * p.iq, 0.0);
    return i == p.drop ? 0.0 : w;
}

// Values of a chunk of the row to draw from (and of the draft's): unit u0 + j step + tid
// of the target's aligned start for j = 0, 1, ...; the first is entry i0.
template <typename T>
__device__ __forceinline__ void load_pair(const VerifyArgs &a, const Pick &p, int b, int u, int step, bool q,
                                          float *x, float *y, int &i0) {
    constexpr int N = Row<T>::N, U = kPer / N;
    const Row<T> row(row_of<T>(a.logits, p.acc, b), a.V);
    row.template load_all<U>(u, step, x);
    i0 = u * N - row.off;
    if (!q) return;
    const T *qr = row_of<T>(a.q, p.acc, b);
    if ((int)(((uintptr_t)qr & 15) / sizeof(T)) == row.off) {
        Row<T>(qr, a.V).template load_all<U>(u, step, y);
    } else {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int at = i0 + (i / N) * step * N + i % N;
            y[i] = at >= 0 && at < a.V ? to_f32<T>(qr[at]) : -INFINITY;
        }
    }
}

// Inclusive sum over the lanes up to one's own.
__device__ __forceinline__ double scan(double v) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const double up = __shfl_up(v, o);
        if (lane >= o) v += up;
    }
    return v;
}

// The chunk in which the sum of v (lane's chunks j 64 + lane) passes u times the whole,
// and the sum before it; at the very end the last with any weight; -1: no weight at all.
__device__ __forceinline__ int find_chunk(const double *v, float u, double &before, double &goal) {
    const int lane = threadIdx.x & 63;
    double incl[kMaxParts], run = 0.0;
#pragma unroll
    for (int j = 0; j < kMaxParts; ++j) {
        incl[j] = run + scan(v[j]);
        run = __shfl(incl[j], 63);
    }
    goal = (double)u * run;
    int ch = -1, last = -1;
#pragma unroll
    for (int j = kMaxParts - 1; j >= 0; --j) {  // the lowest that passes is found last
        const uint64_t some = __ballot(v[j] > 0.0), over = __ballot(v[j] > 0.0 && incl[j] > goal);
        if (some && last < 0) last = j * 64 + 63 - __clzll((long long)some);
        if (over) ch = j * 64 + __ffsll((unsigned long long)over) - 1;
    }
    if (ch < 0) ch = last;
    before = 0.0;
#pragma unroll
    for (int j = 0; j < kMaxParts; ++j) {
        double up = __shfl_up(incl[j], 1);
        if (lane == 0) up = j ? __shfl(incl[j ? j - 1 : 0], 63) : 0.0;
        const double at = __shfl(up, ch & 63);
        if (ch >= 0 && j == ch >> 6) before = at;
    }
    return ch;
}

// One workgroup: the token drawn from the row that p names.
template <typename T>
__device__ __forceinline__ int draw(const VerifyArgs &a, Pick p, int b, int nch, bool q, const double *sums,
                                    const Part *parts) {
    constexpr int U = kPer / Row<T>::N;
    __shared__ double total[kWaves];
    __shared__ int found, last;
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
    if (tid == 0) found = 0x7FFFFFFF, last = -1;
    const float u = fminf(fmaxf(a.u[(int64_t)a.K * a.B + b], 0.0f), 1.0f);
    double v[kMaxParts], before, goal;
#pragma unroll
    for (int j = 0; j < kMaxParts; ++j)
        v[j] = j * 64 + lane < nch
                   ? __hip_atomic_load(sums + j * 64 + lane, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT)
                   : 0.0;
    int ch = find_chunk(v, u, before, goal);
    if (ch < 0) {  // nothing of p - q is left: p itself
        p.drop = -1;
        q = false;
#pragma unroll
        for (int j = 0; j < kMaxParts; ++j) {
            const Part c = j * 64 + lane < nch ? parts[j * 64 + lane] : Part{0.0, -INFINITY, 0};
            v[j] = c.m == -INFINITY ? 0.0 : c.s * pow2(((double)c.m - p.mp) * p.scale);
        }
        ch = find_chunk(v, u, before, goal);
    }
    if (ch < 0) return -1;
    // a thread takes neighbouring entries: indices grow with the thread
    float x[kPer], y[kPer];
    double wt[kPer], s = 0.0;
    int i0;
    load_pair<T>(a, p, b, (ch * kThreads + tid) * U, 1, q, x, y, i0);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        wt[i] = weight(p, x[i], y[i], i0 + i, q);
        s += wt[i];
    }
    const double incl = scan(s);
    if (lane == 63) total[w] = incl;
    __syncthreads();
    double at = before + (incl - s);
    for (int i = 0; i < w; ++i) at += total[i];
    int mine = 0x7FFFFFFF, end = -1;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        at += wt[i];
        if (wt[i] > 0.0) {
            end = i0 + i;
            if (at > goal) mine = min(mine, i0 + i);
        }
    }
    mine = wave_min(mine);
    end = -wave_min(-end);
    if (lane == 0) {
        atomicMin(&found, mine);
        atomicMax(&last, end);
    }
    __syncthreads();
    return found != 0x7FFFFFFF ? found : last;
}

template <typename T>
__global__ __launch_bounds__(kThreads) void verify_draw_kernel(VerifyArgs a, int nch, int rows, int across) {
    constexpr int N = Row<T>::N;
    __shared__ Joined all[2 * kMaxDrafts + 1];
    __shared__ Pick pick;
    __shared__ double tmp[kWaves];
    __shared__ int done;
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
    const int b = blockIdx.x / nch, ch = blockIdx.x - b * nch;
    const int n = drafts_of(a, b);
    const double scale = scale_of(a, b);
    const Part *part = (const Part *)a.ws;
    const bool greedy = scale == 0.0, has_q = a.q.p != nullptr && !greedy;
    // the drafts' own logits, on their way while the rows are joined
    int id = a.V;
    float xd = 0.0f, yd = 0.0f, ud = 0.0f;
    if (w == 0 && lane < n) {
        id = load_id(a.drafts, lane * a.B + b, a.V);
        ud = fminf(fmaxf(a.u[(int64_t)lane * a.B + b], 0.0f), 1.0f);
        if (id < a.V && !greedy) {
            xd = to_f32<T>(row_of<T>(a.logits, lane, b)[id]);
            if (has_q) yd = to_f32<T>(row_of<T>(a.q, lane, b)[id]);
        }
    }
    join(n + 1 + (has_q ? n : 0), nch, across, scale, all,
         [&](int i) { return part + ((int64_t)(i <= n ? i : a.K + (i - n)) * a.B + b) * nch; });
    __syncthreads();
    if (w == 0) {
        bool ok = false;
        if (lane < n && id < a.V) {
            const Joined p = all[lane];
            if (greedy) {
                ok = p.s > 0.0 && id == p.at;
            } else if (p.s > 0.0) {
                const double px = pow2(((double)xd - p.m) * scale) / p.s;
                double qx = 1.0;
                if (has_q) {
                    const Joined q = all[n + 1 + lane];
                    qx = q.s == 0.0 ? 0.0 : pow2(((double)yd - q.m) * scale) / q.s;  // NaN: refuses
                }
                ok = (double)ud * qx < px;
            }
        }
        const uint64_t stood = __ballot(ok);
        const int acc = __ffsll((unsigned long long)~stood) - 1;  // n <= 63: bit 63 is never set
        if (lane == 0) {
            const Joined p = all[acc];
            Pick k{scale, p.m, 1.0 / p.s, 0.0, 0.0, acc, -1, -2};
            if (!(p.s > 0.0)) {
                k.token = -1;
            } else if (greedy) {
                k.token = p.at;
            } else if (acc < n && has_q) {
                const Joined q = all[n + 1 + acc];
                k.mq = q.m;
                k.iq = q.s == 0.0 ? 0.0 : 1.0 / q.s;
                if (q.s != q.s) k.token = -1;
            } else if (acc < n) {
                k.drop = load_id(a.drafts, acc * a.B + b, a.V);
            }
            pick = k;
        }
    }
    __syncthreads();
    const Pick p = pick;
    int token = p.token;
    if (token == -2) {
        const bool q = has_q && p.acc < n;
        float x[kPer], y[kPer];
        int i0;
        load_pair<T>(a, p, b, ch * (kChunk / N) + tid, kThreads, q, x, y, i0);
        double s = 0.0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) s += weight(p, x[i], y[i], i0 + (i / N) * kThreads * N + i % N, q);
        s = wave_sum(s);
        if (lane == 0) tmp[w] = s;
        __syncthreads();
        double *sums = chunk_sums(a, nch, rows) + (int64_t)b * nch;
        if (tid == 0) {
            s = 0.0;
#pragma unroll
            for (int i = 0; i < kWaves; ++i) s += tmp[i];
            __hip_atomic_store(sums + ch, s, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            // this sum is there before the count, all others before the last count
            done = __hip_atomic_fetch_add(counter(a, nch, rows) + b, 1u, __ATOMIC_ACQ_REL,
                                          __HIP_MEMORY_SCOPE_AGENT) == (unsigned)nch - 1;
        }
        __syncthreads();
        if (!done) return;
        token = draw<T>(a, p, b, nch, q, sums, part + ((int64_t)p.acc * a.B + b) * nch);
    } else if (ch != 0) {
        return;
    }
    if (tid == 0) a.accepted[b] = p.acc;
    if (tid <= a.K) {
        int t = -1;
        if (tid < p.acc)
            t = load_id(a.drafts, tid * a.B + b, a.V);
        else if (tid == p.acc)
            t = token;
        a.tokens[(int64_t)tid * a.B + b] = t;
    }
}

template <typename T>
hipError_t verify_t(const VerifyArgs &a, hipStream_t s) {
    const int nch = chunks(a.V, kChunk, sizeof(T)), rows = a.q.p ? 2 * a.K + 1 : a.K + 1;
    const dim3 thr(kThreads);
    hipLaunchKernelGGL(verify_sum_kernel<T>, dim3((unsigned)((int64_t)rows * a.B * nch)), thr, 0, s, a, nch, rows);
    int across = 1;
    while (across < nch && across < 64) across *= 2;
    hipLaunchKernelGGL(verify_draw_kernel<T>, dim3((unsigned)((int64_t)a.B * nch)), thr, 0, s, a, nch, rows, across);
    return hipGetLastError();
}

}  // namespace

size_t verify_bytes(int K, int B, int V) {
    // the larger chunk count of the two types
    const size_t nch = chunks(V, kChunk, 2);
    return ((size_t)(2 * K + 1) * nch * sizeof(Part) + nch * sizeof(double) + sizeof(unsigned)) * B;
}

bool verify_grid_ok(int K, int B, int V) {
    return grid_ok((int64_t)(2 * K + 1) * B * chunks(V, kChunk, 2), kThreads);
}

hipError_t launch_verify(const VerifyArgs &a, bool bf16, hipStream_t s) {
    return bf16 ? verify_t<uint16_t>(a, s) : verify_t<float>(a, s);
}

}  // namespace lm
}  // namespace rnn355
