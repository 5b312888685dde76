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
// strips of the row to draw from, a wave a strip; the sequence's last workgroup to
// finish finds the strip in which the sum passes u, and the entry in it.  In a large call
// the first launch's sums serve where w is p, and one workgroup goes from the chunk to
// the strip.  Sums are added in the order of the strips, so nothing depends on which
// workgroup is last.  A sum is one 64-bit word that says by its value that it is there; an
// ordered counter in its place would write back and empty the caches of every workgroup
// (48.1 us for 45.4 at 32 x 5 x 128000 bf16, 22.0 for 20.0 at 8 x 5 x 128000 float32).
//
// Weights and sums are 64-bit.  The borders between a vocabulary's V entries lie
// 1/V of the sum apart on average; a sum of 32-bit terms is off by 1e-7 of it, so
// that about one draw in a hundred at V = 128000 would depend on how it was added
// up.  With 64 bits (weights to 1e-12, below) that is less than one in 10^6.
#include <algorithm>

#include "row.h"

namespace rnn355 {
namespace lm {

namespace {

constexpr int kThreads = 256, kWaves = kThreads / 64;
constexpr int kHead = 128;             // bytes before the parts: the status word
constexpr uint64_t kNone = ~0ull;      // no sum yet (no sum is this NaN)
constexpr double kLog2eD = 1.4426950408889634;
// Workgroups of a draw launch from which on a row of p is left to one of them: a longer
// chain, but less work in all (64 x 1 x 128000, 2048 workgroups, 28.9 us for 33.9; 16 x 8 x
// 50001, 208 of them, 18.4 either way).
constexpr int kCrowd = 1024;
constexpr int kAtOnce = 4;             // weights side by side (a lone wave waits for each step otherwise)

// d <- 2^(d k) for d <= 0 < k to a relative 1e-12, exactly 1 at d = 0, with low = -1100 / k; 0
// below -1075 (and for a NaN).  d k = n + r with n the nearest whole number, 2^r = 1 + r q(r)
// with q of degree 7 fitted on Chebyshev nodes of [-1/2, 1/2] by least squares on the
// relative error, reweighted towards equal ripple (8e-13).  With the conversion and the
// sum 16 64-bit instructions, whose issue bounds the sums: one takes a wave 5.3 to 5.9
// cycles.  Sums of 37 million bf16 weights take 32 us, 23 of them the issue of 25 vector
// instructions a weight.  M at once: the draw launch has about a wave to a SIMD, which one
// after another would wait for each instruction (32 x 5 x 128000 47.8 us for 45.4, 16 x 8 x
// 50001 19.3 for 18.5, 1 x 5 x 32000 17.3 either way).
template <int M>
__device__ __forceinline__ void pow2s(double *d, double k, double low) {
    const double big = 6755399441055744.0;  // 1.5 * 2^52: its lowest bits then hold n
    constexpr double c[8] = {0x1.61c51b381035fp-20, 0x1.00d858d17751cp-16, 0x1.430aa865450adp-13, 0x1.5d874cfcc70f3p-10,
                             0x1.3b2ab5ed76007p-7,  0x1.c6b08dcede4ffp-5,  0x1.ebfbdff8edf23p-3,  0x1.62e42fef89cbbp-1};
    double s[M], r[M], q[M];
#pragma unroll
    for (int i = 0; i < M; ++i) d[i] = fmax(d[i], low);
#pragma unroll
    for (int i = 0; i < M; ++i) s[i] = fma(d[i], k, big);
#pragma unroll
    for (int i = 0; i < M; ++i) r[i] = big - s[i];
#pragma unroll
    for (int i = 0; i < M; ++i) r[i] = fma(d[i], k, r[i]);
#pragma unroll
    for (int i = 0; i < M; ++i) q[i] = fma(c[0], r[i], c[1]);
#pragma unroll
    for (int j = 2; j < 8; ++j) {
#pragma unroll
        for (int i = 0; i < M; ++i) q[i] = fma(q[i], r[i], c[j]);
    }
#pragma unroll
    for (int i = 0; i < M; ++i) q[i] = fma(q[i], r[i], 1.0);
#pragma unroll
    for (int i = 0; i < M; ++i) d[i] = __builtin_amdgcn_ldexp(q[i], (int)(uint32_t)__double_as_longlong(s[i]));
}
__device__ __forceinline__ double pow2(double d, double k, double low) {
    pow2s<1>(&d, k, low);
    return d;
}
__device__ __forceinline__ double lowest(double k) { return -1100.0 / k; }

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
    double scale, low, mp, ip, mq, iq;  // weight p = 2^((x - mp) scale) ip, q the same
    int acc, drop, token;          // accepted, so also the row to draw from; draft without q to
                                   // leave out (or -1); token >= -1: already known
};

// A lane's value moved along the wave (a row is 16 lanes): kShr + n by n lanes within
// its row, kLast15 and kLast31 from lane 15 of a row to the next and from lane 31 to
// rows 2 and 3, in the rows of `rows`; 0 where nothing comes.
constexpr int kShr = 0x110, kLast15 = 0x142, kLast31 = 0x143;
template <int CTRL, int ROWS = 0xF>
__device__ __forceinline__ double moved(double v) {
    const uint64_t b = (uint64_t)__double_as_longlong(v);
    const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)b, CTRL, ROWS, 0xF, false);
    const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)(b >> 32), CTRL, ROWS, 0xF, false);
    return __longlong_as_double((long long)(((uint64_t)hi << 32) | lo));
}
// Sum over the lanes up to one's own.
__device__ __forceinline__ double scan(double v) {
    v += moved<kShr + 1>(v);
    v += moved<kShr + 2>(v);
    v += moved<kShr + 4>(v);
    v += moved<kShr + 8>(v);
    v += moved<kLast15, 0xA>(v);
    v += moved<kLast31, 0xC>(v);
    return v;
}
__device__ __forceinline__ double from_lane(double v, int lane) {
    const uint64_t b = (uint64_t)__double_as_longlong(v);
    const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)b, lane);
    const uint32_t hi = __builtin_amdgcn_readlane((int)(uint32_t)(b >> 32), lane);
    return __longlong_as_double((long long)(((uint64_t)hi << 32) | lo));
}
__device__ __forceinline__ double wave_sum(double v) { return from_lane(scan(v), 63); }
template <int CTRL, int ROWS = 0xF>
__device__ __forceinline__ float larger(float v) {
    const int low = (int)0xFF800000u;  // -inf
    return fmaxf(v, __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(low, (int)__float_as_uint(v), CTRL, ROWS, 0xF, false)));
}
__device__ __forceinline__ float wave_max(float v) {
    v = larger<kShr + 1>(v);
    v = larger<kShr + 2>(v);
    v = larger<kShr + 4>(v);
    v = larger<kShr + 8>(v);
    v = larger<kLast15, 0xA>(v);
    v = larger<kLast31, 0xC>(v);
    return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(v), 63));
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

// The workspace: status word, parts [rows][B][nch], sums of strips [B][nch kWaves], counters [B].
__device__ __forceinline__ Part *parts_of(const VerifyArgs &a) { return (Part *)((char *)a.ws + kHead); }
__device__ __forceinline__ uint64_t *strip_sums(const VerifyArgs &a, int nch, int rows) {
    return (uint64_t *)(parts_of(a) + (int64_t)rows * a.B * nch);
}
__device__ __forceinline__ unsigned *counter(const VerifyArgs &a, int nch, int rows) {
    return (unsigned *)(strip_sums(a, nch, rows) + (int64_t)a.B * nch * kWaves);
}

// Rows of a sequence: 0 .. K the target's, K + 1 .. 2 K the draft's.
// Each wave takes its own maximum for reference, so that it waits for the others once.
template <typename T, int PER>
__global__ __launch_bounds__(kThreads) void verify_sum_kernel(VerifyArgs a, int nch, int rows) {
    constexpr int N = Row<T>::N, U = PER / N;
    __shared__ Part waves[kWaves];
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
    const unsigned rb = blockIdx.x / (unsigned)nch;  // fewer than 2^24 workgroups
    const int ch = (int)(blockIdx.x - rb * nch), r = (int)(rb / (unsigned)a.B), b = (int)(rb - (unsigned)r * a.B);
    const int n = drafts_of(a, b);
    const double scale = scale_of(a, b), low = lowest(scale);
    const bool draft = r > a.K, greedy = scale == 0.0;
    if (r == 0 && tid < kWaves) strip_sums(a, nch, rows)[((int64_t)b * nch + ch) * kWaves + tid] = kNone;
    if (r == 0 && ch == 0 && tid == 0) {
        counter(a, nch, rows)[b] = 0;
        if (b == 0) *(unsigned *)a.ws = 0;
    }
    if (draft ? r - a.K - 1 >= n || greedy : r > n) return;  // a row that nothing asks for
    const Row<T> row(draft ? row_of<T>(a.q, r - a.K - 1, b) : row_of<T>(a.logits, r, b), a.V);
    const int u0 = ch * (kThreads * U);
    float x[PER];
    row.template load_all<U>(u0 + tid, kThreads, x);
    float m = -INFINITY;
    bool bad = false;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        m = fmaxf(m, x[i]);
        bad |= x[i] != x[i];
    }
    m = wave_max(m);
    bad = __any(bad) || m == INFINITY;
    double s = 0.0;
    int first = 0x7FFFFFFF;
    if (greedy) {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int idx = (u0 + (i / N) * kThreads + tid) * N + (i % N) - row.off;
            if (x[i] == m && idx >= 0 && idx < a.V) first = min(first, idx);
        }
        first = wave_min(first);
        s = m == -INFINITY ? 0.0 : 1.0;
    } else {
        const double ref = m == -INFINITY ? 0.0 : (double)m;
#pragma unroll
        for (int i = 0; i < PER; i += kAtOnce) {
            double d[kAtOnce];
#pragma unroll
            for (int j = 0; j < kAtOnce; ++j) d[j] = (double)x[i + j] - ref;
            pow2s<kAtOnce>(d, scale, low);
#pragma unroll
            for (int j = 0; j < kAtOnce; ++j) s += d[j];
        }
        s = wave_sum(s);
    }
    if (lane == 0) waves[w] = Part{bad ? NAN : s, m, first};
    __syncthreads();
    if (tid == 0) {
        m = waves[0].m;
#pragma unroll
        for (int i = 1; i < kWaves; ++i) m = fmaxf(m, waves[i].m);
        s = 0.0, first = 0x7FFFFFFF;
#pragma unroll
        for (int i = 0; i < kWaves; ++i) {
            const Part q = waves[i];
            if (q.s != q.s) s = q.s;
            if (q.m == -INFINITY) continue;
            s += greedy ? q.s : q.s * pow2((double)q.m - (double)m, scale, low);
            if (q.m == m) first = min(first, q.at);
        }
        parts_of(a)[blockIdx.x] = Part{s, m, first};
    }
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
__device__ __forceinline__ void join(int live, int nch, int across, double scale, double low, Joined *all, F part) {
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
            s += scale == 0.0 ? q[j].s : q[j].s * pow2((double)q[j].m - ref, scale, low);
            if (q[j].m == m) at = min(at, q[j].at);
        }
        for (int o = across >> 1; o; o >>= 1) {
            s += __shfl_xor(s, o);
            at = min(at, __shfl_xor(at, o));
        }
        if (l == 0 && i < live) all[i] = Joined{ref, s, at};
    }
}

// Weights of M entries from i on of the row to draw from, of values x, y (draft's).  A
// difference of less than kNoise of p counts as nothing: p and q of the same distribution
// differ by up to four times 8e-13, since their sums run in another order where the rows
// start at different places of their 16 bytes (and pow2 rounds twice on a sum's way).
constexpr double kNoise = 0x1p-37;
template <int M>
__device__ __forceinline__ void weights(const Pick &p, const float *x, const float *y, int i, bool q, double *w) {
#pragma clang fp contract(off)
    double v[M];
#pragma unroll
    for (int j = 0; j < M; ++j) w[j] = (double)x[j] - p.mp;
    pow2s<M>(w, p.scale, p.low);
    if (q) {
#pragma unroll
        for (int j = 0; j < M; ++j) v[j] = (double)y[j] - p.mq;
        pow2s<M>(v, p.scale, p.low);
#pragma unroll
        for (int j = 0; j < M; ++j) {
            const double pj = w[j] * p.ip, left = pj - v[j] * p.iq;
            w[j] = left > kNoise * pj ? left : 0.0;
        }
    } else {
#pragma unroll
        for (int j = 0; j < M; ++j) w[j] = i + j == p.drop ? 0.0 : w[j];
    }
}

// NU units of the row to draw from (and of the draft's): units u, u + step, ... from the
// target's aligned start; the first holds entry i0.
template <typename T, int NU>
__device__ __forceinline__ void load_pair(const VerifyArgs &a, const Pick &p, int b, int u, int step, bool q,
                                          float *x, float *y, int &i0) {
    constexpr int N = Row<T>::N;
    const Row<T> row(row_of<T>(a.logits, p.acc, b), a.V);
    row.template load_all<NU>(u, step, x);
    i0 = u * N - row.off;
    if (!q) return;
    const T *qr = row_of<T>(a.q, p.acc, b);
    if ((int)(((uintptr_t)qr & 15) / sizeof(T)) == row.off) {
        Row<T>(qr, a.V).template load_all<NU>(u, step, y);
    } else {
#pragma unroll
        for (int i = 0; i < NU * N; ++i) {
            const int at = i0 + (i / N) * step * N + i % N;
            y[i] = at >= 0 && at < a.V ? to_f32<T>(qr[at]) : -INFINITY;
        }
    }
}

// The strip in which the sum of v (lane's strips j 64 + lane, n in all) passes u times
// the whole, and the sum before it; at the very end the last with any weight; -1: no
// weight at all.
constexpr int kMaxStrips = kMaxParts * kWaves;  // of a lane
__device__ __forceinline__ int find_strip(const double *v, int n, float u, double &before, double &goal) {
    double incl[kMaxStrips], run = 0.0;
#pragma unroll
    for (int j = 0; j < kMaxStrips; ++j) {
        incl[j] = run;
        if (j * 64 >= n) continue;
        incl[j] = run + scan(v[j]);
        run = from_lane(incl[j], 63);
    }
    goal = (double)u * run;
    int at = -1, last = -1;
#pragma unroll
    for (int j = kMaxStrips - 1; j >= 0; --j) {  // the lowest that passes is found last
        if (j * 64 >= n) continue;
        const uint64_t some = __ballot(v[j] > 0.0), over = __ballot(v[j] > 0.0 && incl[j] > goal);
        if (some && last < 0) last = j * 64 + 63 - __clzll((long long)some);
        if (over) at = j * 64 + __ffsll((unsigned long long)over) - 1;
    }
    if (at < 0) at = last;
    before = 0.0;
    if (at > 0) {
        const int c = at - 1;
#pragma unroll
        for (int j = 0; j < kMaxStrips; ++j)
            if (j == c >> 6) before = from_lane(incl[j], c & 63);
    }
    return at;
}

// One workgroup: the token drawn from the row that p names, given the sums of its strips
// of 64 U units (null where w is p) and its parts, which are those of p.  lost: LDS, 0.
template <typename T, int PER>
__device__ __forceinline__ int draw(const VerifyArgs &a, Pick p, int b, int nch, bool q, const uint64_t *sums,
                                    const Part *parts, int *lost) {
    constexpr int N = Row<T>::N, U = PER / N, NU = U >= kWaves ? U / kWaves : 1;
    __shared__ double total[kWaves];
    __shared__ int found, last;
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, strips = nch * kWaves;
    if (tid == 0) found = 0x7FFFFFFF, last = -1;
    const float u = fminf(fmaxf(a.u[(int64_t)a.K * a.B + b], 0.0f), 1.0f);
    double v[kMaxStrips], before, goal;
    int at = -1;
    if (sums) {
#pragma unroll
        for (int j = 0; j < kMaxStrips; ++j) {
            uint64_t word = 0;
            // counted already, so stored already: on its way at most
            for (unsigned spins = 0; j * 64 + lane < strips && spins < a.spins; ++spins) {
                word = __hip_atomic_load(sums + j * 64 + lane, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
                if (word != kNone) break;
            }
            v[j] = __longlong_as_double((long long)word);
        }
        at = find_strip(v, strips, u, before, goal);
        if (goal != goal) {  // a wave's wait ran out: noted, and nothing drawn, below
            *lost = 1;
            __hip_atomic_store((unsigned *)a.ws, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            at = 0;
        }
    }
    if (at < 0) {  // p itself (or nothing of p - q is left): first its chunk, then the strip
        __syncthreads();
        if (*lost) return -1;  // another wave's
        p.drop = -1;
        q = false;
#pragma unroll
        for (int j = 0; j < kMaxStrips; ++j) {
            const Part c = j * 64 + lane < nch ? parts[j * 64 + lane] : Part{0.0, -INFINITY, 0};
            // above 0 where its largest entry's weight, the same power of two, is
            v[j] = c.m == -INFINITY ? 0.0 : c.s * pow2((double)c.m - p.mp, p.scale, p.low);
        }
        const int ch = find_strip(v, nch, u, before, goal);
        if (ch < 0) return -1;
        float x[PER], y[PER];
        int i0;
        load_pair<T, U>(a, p, b, (ch * kWaves + w) * 64 * U + lane, 64, false, x, y, i0);
        double s = 0.0;
#pragma unroll
        for (int i = 0; i < PER; i += kAtOnce) {
            double wt[kAtOnce];
            weights<kAtOnce>(p, x + i, y + i, 0, false, wt);
#pragma unroll
            for (int j = 0; j < kAtOnce; ++j) s += wt[j];
        }
        s = wave_sum(s);
        if (lane == 0) total[w] = s;
        __syncthreads();
        double sum = before;
        for (int i = 0; i < kWaves; ++i) {
            if (!(total[i] > 0.0)) continue;
            at = ch * kWaves + i;
            before = sum;
            sum += total[i];
            if (sum > goal) break;
        }
        __syncthreads();
        if (at < 0) return -1;
    }
    // a thread takes NU neighbouring units of the strip, as far as there are any: indices
    // grow with the thread
    const bool some = tid * NU < 64 * U;
    float x[NU * N], y[NU * N];
    double wt[NU * N], s = 0.0;
    int i0;
    load_pair<T, NU>(a, p, b, at * 64 * U + (some ? tid * NU : 0), 1, q, x, y, i0);
#pragma unroll
    for (int i = 0; i < NU * N; i += kAtOnce) {
        weights<kAtOnce>(p, x + i, y + i, i0 + i, q, wt + i);
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) s += wt[i + j] = some ? wt[i + j] : 0.0;
    }
    const double incl = scan(s);
    if (lane == 63) total[w] = incl;
    __syncthreads();
    double sum = before + (incl - s);
    for (int i = 0; i < w; ++i) sum += total[i];
    int mine = 0x7FFFFFFF, end = -1;
#pragma unroll
    for (int i = 0; i < NU * N; ++i) {
        sum += wt[i];
        if (wt[i] > 0.0) {
            end = i0 + i;
            if (sum > goal) mine = min(mine, i0 + i);
        }
    }
    mine = wave_min(mine);
    end = -wave_min(-end);
    if (lane == 0) {
        atomicMin(&found, mine);
        atomicMax(&last, end);
    }
    __syncthreads();
    if (*lost) return -1;
    return found != 0x7FFFFFFF ? found : last;
}

template <typename T, int PER>
__global__ __launch_bounds__(kThreads) void verify_draw_kernel(VerifyArgs a, int nch, int rows, int across) {
    constexpr int N = Row<T>::N, U = PER / N;
    __shared__ Joined all[2 * kMaxDrafts + 1];
    __shared__ Pick pick;
    __shared__ int done, lost;
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
    const int b = blockIdx.x / nch, ch = blockIdx.x - b * nch;
    const int n = drafts_of(a, b);
    const double scale = scale_of(a, b), low = lowest(scale);
    const Part *part = parts_of(a);
    if (tid == 0) lost = 0;
    const bool greedy = scale == 0.0, has_q = a.q.p != nullptr && !greedy;
    const bool crowd = a.B * nch >= kCrowd;
    if (ch != 0 && (greedy || (n == 0 && crowd))) return;  // one workgroup's work, below
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
    join(n + 1 + (has_q ? n : 0), nch, across, scale, low, all,
         [&](int i) { return part + ((int64_t)(i <= n ? i : a.K + (i - n)) * a.B + b) * nch; });
    __syncthreads();
    if (w == 0) {
        bool ok = false;
        if (lane < n && id < a.V) {
            const Joined p = all[lane];
            if (greedy) {
                ok = p.s > 0.0 && id == p.at;
            } else if (p.s > 0.0) {
                const double px = pow2((double)xd - p.m, scale, low) / p.s;
                double qx = 1.0;
                if (has_q) {
                    const Joined q = all[n + 1 + lane];
                    qx = q.s == 0.0 ? 0.0 : pow2((double)yd - q.m, scale, low) / q.s;  // NaN: refuses
                }
                ok = (double)ud * qx < px;
            }
        }
        const uint64_t stood = __ballot(ok);
        const int acc = __ffsll((unsigned long long)~stood) - 1;  // n <= 63: bit 63 is never set
        if (lane == 0) {
            const Joined p = all[acc];
            Pick k{scale, low, p.m, 1.0 / p.s, 0.0, 0.0, acc, -1, -2};
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
        const bool q = has_q && p.acc < n, own = crowd && !q && p.drop < 0;  // w is p
        if (own && ch != 0) return;
        uint64_t *sums = own ? nullptr : strip_sums(a, nch, rows) + (int64_t)b * nch * kWaves;
        if (!own) {
            float x[PER], y[PER];
            int i0;
            load_pair<T, U>(a, p, b, (ch * kWaves + w) * 64 * U + lane, 64, q, x, y, i0);
            double s = 0.0;
#pragma unroll
            for (int i = 0; i < PER; i += kAtOnce) {
                double wt[kAtOnce];
                weights<kAtOnce>(p, x + i, y + i, i0 + (i / N) * 64 * N + i % N, q, wt);
#pragma unroll
                for (int j = 0; j < kAtOnce; ++j) s += wt[j];
            }
            s = wave_sum(s);
            if (lane == 0)
                __hip_atomic_store(sums + ch * kWaves + w, (uint64_t)__double_as_longlong(s), __ATOMIC_RELAXED,
                                   __HIP_MEMORY_SCOPE_AGENT);
            __syncthreads();
            if (tid == 0)
                done = __hip_atomic_fetch_add(counter(a, nch, rows) + b, 1u, __ATOMIC_RELAXED,
                                              __HIP_MEMORY_SCOPE_AGENT) == (unsigned)nch - 1;
            __syncthreads();
            if (!done) return;
        }
        token = draw<T, PER>(a, p, b, nch, q, sums, part + ((int64_t)p.acc * a.B + b) * nch, &lost);
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

// Values of a thread: 32 where that leaves the first launch sixteen workgroups a CU, for
// half the fixed work of a chunk (32 x 5 x 128000: 45.4 us for 53), else 16, which
// spread a small call further (16 x 8 x 50001: 18.5 us for 22.2; 1 x 5 x 32000 17 either
// way; a call of one row a sequence, 64 x 1 x 128000, would be faster with 32, 24.4 for 28.9).
constexpr int kFew = 16, kMany = 32;

template <typename T, int PER>
hipError_t verify_t(const VerifyArgs &a, hipStream_t s) {
    const int nch = chunks(a.V, kThreads * PER, sizeof(T)), rows = a.q.p ? 2 * a.K + 1 : a.K + 1;
    const dim3 thr(kThreads);
    hipLaunchKernelGGL((verify_sum_kernel<T, PER>), dim3((unsigned)((int64_t)rows * a.B * nch)), thr, 0, s, a, nch, rows);
    int across = 1;
    while (across < nch && across < 64) across *= 2;
    hipLaunchKernelGGL((verify_draw_kernel<T, PER>), dim3((unsigned)((int64_t)a.B * nch)), thr, 0, s, a, nch, rows, across);
    return hipGetLastError();
}

template <typename T>
hipError_t verify_by_size(const VerifyArgs &a, hipStream_t s) {
    const int64_t rows = a.q.p ? 2 * a.K + 1 : a.K + 1;
    return rows * a.B * chunks(a.V, kThreads * kMany, sizeof(T)) >= 4096 ? verify_t<T, kMany>(a, s)
                                                                          : verify_t<T, kFew>(a, s);
}

}  // namespace

size_t verify_bytes(int K, int B, int V) {
    // the larger chunk count of the two types and sizes
    const size_t nch = chunks(V, kThreads * kFew, 2);
    const size_t each = (size_t)(2 * K + 1) * nch * sizeof(Part) + nch * kWaves * sizeof(double) + sizeof(unsigned);
    return std::max<size_t>(4096, kHead + each * B);  // rnn_workspace_status takes no less than 4 KiB
}

bool verify_grid_ok(int K, int B, int V) {
    return grid_ok((int64_t)(2 * K + 1) * B * chunks(V, kThreads * kFew, 2), kThreads);
}

hipError_t launch_verify(const VerifyArgs &a, bool bf16, hipStream_t s) {
    return bf16 ? verify_by_size<uint16_t>(a, s) : verify_by_size<float>(a, s);
}

}  // namespace lm
}  // namespace rnn355
