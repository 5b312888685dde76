// gated.hip -- gated linear recurrence: forward, single token, backward.
//
//   h_t = a_t h_{t-1} + b_t,  elementwise;  a, b from the gate's form:
//   logit  a = sigmoid(f), b = (1 - a) x, by the smaller side of the gate, which is right to
//          (2 |f| + 6) 2^-24 of itself (the exponent's product and constant are rounded to
//          float32) and 0 below float32's normal numbers (|f| > 87.3):  h + u (x - h) with
//          u = sigmoid(-f) where a > 1/2, so that a constant x is a fixed point and the
//          memory 1 / (1 - a) is as right as u;  x - a (x - h) elsewhere, so that a closed
//          gate leaves of a state, or lets through of a gradient, what it should and no
//          rounding of the rest
//   decay  a = f, b = x
// Steps compose: (A1, B1) then (A2, B2) is (A2 A1, A2 B1 + B2).  Backward is the same
// kind of recurrence from the end: e_t = a_t (dh_t + e_{t+1}).
//
// Every operand is read once and every output written once; memory bounds it.  A
// workgroup takes a tile of 64 lanes of VEC channels by kWaves S steps (a wave S of
// them) in registers: the gates in float32, the rest as loaded.  Each thread composes
// its S steps; a segment's total goes to memory, the carry into it is composed from
// the totals of the segments before it, and the steps run again from the carry, from
// the same registers.  Where it pays (shape, below) a workgroup has all steps of fewer
// channels, and nothing goes through memory.
//
// Segments wait for each other inside one launch: a workgroup draws its segment from
// its tile's counter, so that whatever it waits for belongs to workgroups that run
// already and wait for earlier segments only; the first waits for none.  (One counter
// for all serves a workgroup every 13 ns: 6144 workgroups then took 94 us.)  A total
// is one 64-bit word for each channel, which says by being other than 0 that it is
// there (written and read whole, so nothing else needs an order).  Past kGroup
// segments the last of a group of about sqrt(segments) publishes the group's total,
// so that a segment reads no more than twice that many words.  The order of all
// products is the dimensions' and the alignment's alone.
//
// 32768 x 1 x 768 float32 forward 65 us and 5 to clear the words (4.6 TB/s), backward of
// 1000 x 16 x 1024 bf16 46 and 5 (4.3 TB/s): the workgroups on the chip load together and
// then wait together, a join (3 to 5 us of a workgroup's 8 to 12) long.  An earlier form of
// 8 steps took 80 and 66 us for the calls, and 56 and 45 with its joins left out.  Two
// launches, totals first and the inputs read twice, wait for nothing but took 100 and 57
// us for the calls' 70 and 51 at the time; workgroups that stay and load their next tile
// while they wait for a carry, 87 and 72; tiles of 32 lanes 73 and 58 with the best of 8,
// 12 and 16 steps for each; rows of 128 bytes and 1024 threads 73 and 52, of 256 bytes 67
// and 55 (but 8192 x 16 x 2048 bf16 385 for 324).  1024 x 16 x 768 bf16 forward, one
// workgroup to a sequence, 17.7 us (4.3 TB/s): all load, then all store.
//
// Stores go past the caches, but for the backward pass of bf16 (8192 x 16 x 2048 forward
// 350 us for 338, 32768 x 1 x 768 float32 backward 131 for 126; 1000 x 16 x 1024 bf16
// backward however 49.3 for 50.9).
#include <algorithm>
#include <type_traits>

#include "host.h"
#include "lm.h"

namespace rnn355 {
namespace lm {

namespace {

constexpr int kThreads = 512, kWaves = kThreads / 64;
constexpr int kAll = 1024;   // most threads where one workgroup has all of a sequence
constexpr int kNarrow = 16;  // its lanes along the channels
constexpr int kGroup = 16;
constexpr int kKept = 10;  // steps of sixteen whose gates four channels keep: as many as 128 registers
                           // hold (1024 x 16 x 768 bf16 18.1 us in a graph; 8 19.3, one 21.6)
constexpr int kHead = 128;           // bytes before the counters: the status word

// How a call is cut, and the words that its segments exchange.
struct Cut {
    int T, D, C;      // steps, channels of a row, channels of all rows
    int nseg, ntile;  // segments of time, tiles of channels
    int G;            // segments of a group
    int pitch;        // words between the tiles' counters
    unsigned spins;   // polls of a wait before it is given up (seconds), and noted in flag
    unsigned *flag;   // the status word; null: no workspace
    unsigned *counter;
    uint64_t *word, *gword;  // [segment][channel], [group][channel]
};

__device__ __forceinline__ uint64_t pack(float A, float B) {
    const uint64_t w = ((uint64_t)__float_as_uint(A) << 32) | __float_as_uint(B);
    return w ? w : (uint64_t)0x80000000u << 32;  // (-0, 0) for (0, 0)
}
__device__ __forceinline__ void publish(uint64_t *p, float A, float B) {
    __hip_atomic_store(p, pack(A, B), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
// A gate from its logit: the smaller of sigmoid(f) and sigmoid(-f), with the sign of -f:
// the gate is open (u stored) where that is set, +inf's zero among them.
__device__ __forceinline__ float side(float f) {
    const float e = exp_fast(-fabsf(f));
    return copysignf(e * rcp_fast(1.0f + e), -f);
}
__device__ __forceinline__ float by_side(float s, float open, float shut) {
    return __float_as_int(s) < 0 ? open : shut;
}
// a h + (1 - a) x and a h for the gate s.  s (x - h) as s x less s h, whose rounding the
// first takes along: x - h may leave float32 where h and x do not, and what lies between
// them does not either.
__device__ __forceinline__ float mix(float s, float h, float x) { return by_side(s, h, x) - fmaf(s, x, -(s * h)); }
__device__ __forceinline__ float part_of(float s, float h) { return fmaf(s, h, by_side(s, h, 0.0f)); }

// This workgroup's segment and tile of channels.  Workgroups go round the eight XCDs:
// where a tile's rows are short of a few cache lines (LN < 64), neighbouring tiles go to
// one of them.
template <int LN>
__device__ __forceinline__ void place(const Cut &k, int &seg, int &tile) {
    __shared__ unsigned drawn;
    seg = 0;
    if (LN < 64) {
        const int xcd = blockIdx.x & 7, each = k.ntile >> 3, more = k.ntile & 7;
        tile = xcd * each + min(xcd, more) + (int)(blockIdx.x >> 3);
        return;
    }
    tile = blockIdx.x % k.ntile;
    if (k.nseg > 1) {
        if (threadIdx.x == 0)
            drawn = __hip_atomic_fetch_add(k.counter + (int64_t)tile * k.pitch, 1u, __ATOMIC_RELAXED,
                                           __HIP_MEMORY_SCOPE_AGENT);
        __syncthreads();
        seg = __builtin_amdgcn_readfirstlane(drawn);
    }
}

// A call of one segment waits for nothing and has no launch that clears its workspace:
// the first workgroup clears the status word.
__device__ __forceinline__ void no_waits(const Cut &k) {
    if (k.nseg == 1 && k.flag && blockIdx.x == 0 && threadIdx.x == 0) *k.flag = 0;
}

// Parts along time of a workgroup with LN lanes along the channels, and a thread's.
template <int LN, int NT>
constexpr int parts() { return NT / LN; }
template <int LN>
__device__ __forceinline__ int part() {
    const int p = threadIdx.x / LN;
    return LN == 64 ? __builtin_amdgcn_readfirstlane(p) : p;
}

// From the threads' own (A, B) to the state that each begins with.  agg, car: LDS.
// Returns the state before the thread's first step in h.
// start: the recurrence's initial state, in the first part of segment 0.  Nobody
// else reads that, and all that follows waits for what this part makes of it, so
// the last state may be written over the first.

// One segment, LN < 64: a scan over the wave's parts, then the waves before.
template <int VEC, int LN, int NT>
__device__ __forceinline__ void join(const float *A, const float *B, const float *start,
                                     float2 (*agg)[LN * VEC], float *h) {
    constexpr int P = 64 / LN;
    const int p = (threadIdx.x & 63) / LN, at = (threadIdx.x & (LN - 1)) * VEC;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const bool first = threadIdx.x < LN;
    float sA[VEC], sB[VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
        sA[v] = first ? 0.0f : A[v];
        sB[v] = first ? fmaf(A[v], start[v], B[v]) : B[v];
    }
#pragma unroll
    for (int o = 1; o < P; o *= 2)
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            const float qA = __shfl_up(sA[v], o * LN), qB = __shfl_up(sB[v], o * LN);
            if (p >= o) {
                sB[v] = fmaf(sA[v], qB, sB[v]);
                sA[v] *= qA;
            }
        }
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
        if (p == P - 1) agg[wave][at + v] = make_float2(sA[v], sB[v]);
        h[v] = 0.0f;
    }
    lds_barrier();
#pragma unroll
    for (int i = 0; i < NT / 64 - 1; ++i) {
        if (i >= wave) break;
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            const float2 q = agg[i][at + v];
            h[v] = fmaf(q.x, h[v], q.y);
        }
    }
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
        const float qA = __shfl_up(sA[v], LN), qB = __shfl_up(sB[v], LN);
        if (p) h[v] = fmaf(qA, h[v], qB);
        if (first) h[v] = start[v];
    }
}

// LN = 64: a part is a wave.
template <int VEC>
__device__ __forceinline__ void join(const Cut &k, int seg, int c0, const float *A, const float *B,
                                     const float *start, float2 (*agg)[64 * VEC],
                                     float2 (*car)[64 * VEC], float *h) {
    const int lane = threadIdx.x & 63, w = part<64>(), at = lane * VEC;
    const bool first = seg == 0 && w == 0;
#pragma unroll
    for (int v = 0; v < VEC; ++v)
        agg[w][at + v] = first ? make_float2(0.0f, fmaf(A[v], start[v], B[v])) : make_float2(A[v], B[v]);
    lds_barrier();
    // the steps of this workgroup before this part
    float pA[VEC], pB[VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) pA[v] = 1.0f, pB[v] = first ? start[v] : 0.0f;
#pragma unroll
    for (int i = 0; i < kWaves - 1; ++i) {
        if (i >= w) break;
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            const float2 q = agg[i][at + v];
            pB[v] = fmaf(q.x, pB[v], q.y);
            pA[v] *= q.x;
        }
    }
    const bool last = seg == k.nseg - 1;
    float tA[VEC], tB[VEC];  // the whole segment, in the last wave
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
        tA[v] = seg == 0 ? 0.0f : pA[v] * A[v];
        tB[v] = fmaf(A[v], pB[v], B[v]);
        if (w == kWaves - 1 && !last && c0 + v < k.C) publish(k.word + (int64_t)seg * k.C + c0 + v, tA[v], tB[v]);
    }
    if (seg == 0) {
#pragma unroll
        for (int v = 0; v < VEC; ++v) h[v] = pB[v];
        return;
    }
    // the segments before: whole groups by the first half of the waves, those of the
    // own group by the second (by all waves where there is no group before)
    const int group = seg / k.G, inside = seg - group * k.G;
    const int half = group ? kWaves / 2 : 0;
    const bool mine = w >= half;
    const int n = mine ? inside : group, parts = mine ? kWaves - half : half, part = mine ? w - half : w;
    const uint64_t *words = mine ? k.word + (int64_t)(seg - inside) * k.C : k.gword;
    const int lo = (int)((int64_t)n * part / parts), hi = (int)((int64_t)n * (part + 1) / parts);
    float cA[VEC], cB[VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) cA[v] = 1.0f, cB[v] = 0.0f;
    const int c = min(c0, k.C - VEC);
    for (int j = lo; j < hi; j += 4) {
        uint64_t q[4][VEC];
        unsigned spins = 0, left = (1u << min(hi - j, 4)) - 1;  // words still to come
        while (true) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (left & (1u << i)) {
#pragma unroll
                    for (int v = 0; v < VEC; ++v)
                        q[i][v] = __hip_atomic_load(words + (int64_t)(j + i) * k.C + c + v, __ATOMIC_RELAXED,
                                                    __HIP_MEMORY_SCOPE_AGENT);
                }
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (left & (1u << i)) {
                    bool there = true;
#pragma unroll
                    for (int v = 0; v < VEC; ++v) there &= q[i][v] != 0;
                    if (__all(there)) left &= ~(1u << i);
                }
            if (!left) break;
            if (++spins >= k.spins) {
                __hip_atomic_store(k.flag, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
                break;
            }
            __builtin_amdgcn_s_sleep(1);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (j + i < hi) {
#pragma unroll
                for (int v = 0; v < VEC; ++v) {
                    const float a = __uint_as_float((uint32_t)(q[i][v] >> 32));
                    cB[v] = fmaf(a, cB[v], __uint_as_float((uint32_t)q[i][v]));
                    cA[v] *= a;
                }
            }
    }
#pragma unroll
    for (int v = 0; v < VEC; ++v) car[w][at + v] = make_float2(cA[v], cB[v]);
    lds_barrier();
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
        h[v] = 0.0f;
#pragma unroll
        for (int i = 0; i < kWaves; ++i) {
            const float2 q = car[i][at + v];
            h[v] = fmaf(q.x, h[v], q.y);
        }
    }
    if (w == kWaves - 1 && !last && inside == k.G - 1) {  // the group's total
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            float gA = 1.0f, gB = 0.0f;
            for (int i = half; i < kWaves; ++i) {
                const float2 q = car[i][at + v];
                gB = fmaf(q.x, gB, q.y);
                gA *= q.x;
            }
            if (c0 + v < k.C)
                publish(k.gword + (int64_t)group * k.C + c0 + v, group ? tA[v] * gA : 0.0f, fmaf(tA[v], gB, tB[v]));
        }
    }
#pragma unroll
    for (int v = 0; v < VEC; ++v) h[v] = fmaf(pA[v], h[v], pB[v]);
}

struct FwdArgs {
    Cut k;
    LinSeq f, x;
    const float *h0;
    const int *lens;
    SeqOut h;
    float *hT;
};

// Makes the compiler take a register's value as new, so that its conversion to float32
// is computed again where it is needed again, in place of being kept.
template <typename V>
__device__ __forceinline__ void forget(V &q) {
    if constexpr (sizeof(V) == 2) {
        uint32_t r = __builtin_bit_cast(uint16_t, q);
        asm volatile("" : "+v"(r));
        q = __builtin_bit_cast(V, (uint16_t)r);
    } else {
        uint32_t r[sizeof(V) / 4];
        __builtin_memcpy(r, &q, sizeof q);
#pragma unroll
        for (uint32_t &i : r) asm volatile("" : "+v"(i));
        __builtin_memcpy(&q, r, sizeof q);
    }
}

// f(true_type) or f(false_type): the steps of a tile that counts whole need no masks.
template <typename F>
__device__ __forceinline__ void by_flag(bool flag, F f) {
    if (flag)
        f(std::true_type{});
    else
        f(std::false_type{});
}

// Stores values in the sequence's type (two at once to bf16); PAST: past the caches.
template <bool PAST, typename T, int VEC>
__device__ __forceinline__ void put(T *p, const float *v) {
    typedef Unit<T, VEC> V;
    typedef std::conditional_t<sizeof(V) == 2, uint16_t, std::conditional_t<sizeof(V) == 4, uint32_t, uint64_t>> W;
    V o;
    if constexpr (sizeof(T) == 2 && VEC % 2 == 0) {
        typedef float f2 __attribute__((ext_vector_type(2)));
        typedef __bf16 b2 __attribute__((ext_vector_type(2)));
        b2 two[VEC / 2];
#pragma unroll
        for (int i = 0; i < VEC / 2; ++i) two[i] = __builtin_convertvector((f2){v[2 * i], v[2 * i + 1]}, b2);
        __builtin_memcpy(&o, two, sizeof o);
    } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) o.v[i] = from_f32<T>(v[i]);
    }
    if (PAST)
        __builtin_nontemporal_store(__builtin_bit_cast(W, o), (W *)p);
    else
        *(V *)p = o;
}

template <typename T, bool LOGIT, int VEC, int S, int LN, int NT>
__global__ __launch_bounds__(NT, 4) void gated_fwd_kernel(FwdArgs a) {
    typedef Unit<T, VEC> V;
    __shared__ float2 agg[NT / 64][LN * VEC], car[LN == 64 ? kWaves : 1][LN * VEC];
    const Cut &k = a.k;
    int seg, tile;
    place<LN>(k, seg, tile);
    const int lane = threadIdx.x & (LN - 1), w = part<LN>();
    const int c0 = (tile * LN + lane) * VEC, c = min(c0, k.C - VEC);
    const int b = c / k.D, i = c - b * k.D;
    const int len = a.lens ? min(max(a.lens[b], 0), k.T) : k.T;
    const int t0 = (seg * parts<LN, NT>() + w) * S;  // the grid's limit keeps this in 31 bits
    V fr[S], xr[S];
    if (__any(t0 < len)) {
        const T *fp = (const T *)a.f.p + (int64_t)b * a.f.sb + i, *xp = (const T *)a.x.p + (int64_t)b * a.x.sb + i;
#pragma unroll
        for (int s = 0; s < S; ++s) {
            const int64_t t = min(t0 + s, k.T - 1);
            fr[s] = *(const V *)(fp + t * a.f.st);
            xr[s] = *(const V *)(xp + t * a.x.st);
        }
    }
    // what a step keeps beside x: the gate's side (logit) or a (decay); with four channels
    // there are registers for some, and the other steps keep f
    constexpr int keep = VEC < 4 ? S : kKept;
    float g[keep][VEC], A[VEC], B[VEC], h[VEC], start[VEC];
    auto gate = [&](int s, int v) {
        const float fv = to_f32<T>(fr[s].v[v]);
        return LOGIT ? side(fv) : fv;
    };
#pragma unroll
    for (int s = 0; s < keep; ++s)
#pragma unroll
        for (int v = 0; v < VEC; ++v) g[s][v] = gate(s, v);
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
        A[v] = 1.0f, B[v] = 0.0f;
        start[v] = seg == 0 && w == 0 && a.h0 ? a.h0[c + v] : 0.0f;
    }
    const bool full = __all(t0 + S <= len);
    by_flag(full, [&](auto all) {
#pragma unroll
        for (int s = 0; s < S; ++s)
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                if (!all.value && t0 + s >= len) continue;
                const float xv = to_f32<T>(xr[s].v[v]), gv = s < keep ? g[s < keep ? s : 0][v] : gate(s, v);
                B[v] = LOGIT ? mix(gv, B[v], xv) : fmaf(gv, B[v], xv);
                A[v] = LOGIT ? part_of(gv, A[v]) : A[v] * gv;
            }
    });
#pragma unroll
    for (int s = 0; s < S; ++s) {
        forget(xr[s]);
        if (s >= keep) forget(fr[s]);
    }
    if constexpr (LN == 64)
        join<VEC>(k, seg, c0, A, B, start, agg, car, h);
    else
        join<VEC, LN, NT>(A, B, start, agg, h);
    T *out = (T *)a.h.p + (int64_t)b * a.h.sb + i;
    by_flag(full, [&](auto all) {
#pragma unroll
        for (int s = 0; s < S; ++s) {
            float o[VEC];
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                const float xv = to_f32<T>(xr[s].v[v]), gv = s < keep ? g[s < keep ? s : 0][v] : gate(s, v);
                const float hn = LOGIT ? mix(gv, h[v], xv) : fmaf(gv, h[v], xv);
                const bool on = all.value || t0 + s < len;
                h[v] = on ? hn : h[v];
                o[v] = on ? hn : 0.0f;
            }
            if ((all.value || t0 + s < k.T) && c0 < k.C) put<true, T, VEC>(out + (int64_t)(t0 + s) * a.h.st, o);
        }
    });
    if (a.hT && seg == k.nseg - 1 && w == parts<LN, NT>() - 1 && c0 < k.C) {
#pragma unroll
        for (int v = 0; v < VEC; ++v) a.hT[c + v] = h[v];
    }
    no_waits(k);
}

template <typename T, bool LOGIT>
__global__ __launch_bounds__(256) void gated_step_kernel(GatedDims d, LinSeq f, LinSeq x, const float *h,
                                                         SeqOut y, float *h_out) {
    const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (c >= (int64_t)d.B * d.D) return;
    const int b = (int)(c / d.D), i = (int)(c - (int64_t)b * d.D);
    const float fv = to_f32<T>(((const T *)f.p)[b * f.sb + i]), xv = to_f32<T>(((const T *)x.p)[b * x.sb + i]);
    const float n = LOGIT ? mix(side(fv), h[c], xv) : fmaf(fv, h[c], xv);
    h_out[c] = n;
    if (y.p) ((T *)y.p)[b * y.sb + i] = from_f32<T>(n);
}

struct BwdArgs {
    Cut k;
    LinSeq f, x, h, dh;
    const float *h0, *dhT;
    const int *lens;
    SeqOut df, dx;
    float *dh0;
};

// Backwards in time: step s of a thread is t = T - 1 - (first + s).  The state is
// e = a_{t+1} g_{t+1}; g_t = dh_t + e, e' = a_t g_t.
template <typename T, bool LOGIT, int VEC, int S, int LN, int NT>
__global__ __launch_bounds__(NT, 4) void gated_bwd_kernel(BwdArgs a) {
    typedef Unit<T, VEC> V;
    __shared__ float2 agg[NT / 64][LN * VEC], car[LN == 64 ? kWaves : 1][LN * VEC];
    const Cut &k = a.k;
    int seg, tile;
    place<LN>(k, seg, tile);
    const int lane = threadIdx.x & (LN - 1), w = part<LN>();
    const int c0 = (tile * LN + lane) * VEC, c = min(c0, k.C - VEC);
    const int b = c / k.D, i = c - b * k.D;
    const int len = a.lens ? min(max(a.lens[b], 0), k.T) : k.T;
    const int t0 = k.T - 1 - (seg * parts<LN, NT>() + w) * S;  // the thread's last step in time; may be below 0
    V fr[S], dr[S], xr[S], hr[S];
    if (__any(t0 - (S - 1) < len && t0 >= 0)) {
        const T *fp = (const T *)a.f.p + (int64_t)b * a.f.sb + i, *dp = (const T *)a.dh.p + (int64_t)b * a.dh.sb + i;
        const T *xp = (const T *)a.x.p + (int64_t)b * a.x.sb + i, *hp = (const T *)a.h.p + (int64_t)b * a.h.sb + i;
#pragma unroll
        for (int s = 0; s < S; ++s) {
            const int64_t t = max(t0 - s, 0);
            fr[s] = *(const V *)(fp + t * a.f.st);
            dr[s] = *(const V *)(dp + t * a.dh.st);
        }
#pragma unroll
        for (int s = 0; s < S; ++s) {
            const int64_t t = max(t0 - s, 0);
            if (LOGIT) xr[s] = *(const V *)(xp + t * a.x.st);
            hr[s] = *(const V *)(hp + max(t - 1, (int64_t)0) * a.h.st);
        }
    }
    // what a step keeps beside dh, x and h: the gate's side (logit) or a (decay)
    float g[S][VEC], A[VEC], B[VEC], start[VEC], e[VEC];
#pragma unroll
    for (int s = 0; s < S; ++s)
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            const float fv = to_f32<T>(fr[s].v[v]);
            g[s][v] = LOGIT ? side(fv) : fv;
        }
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
        A[v] = 1.0f, B[v] = 0.0f;
        start[v] = seg == 0 && w == 0 && a.dhT ? a.dhT[c + v] : 0.0f;
    }
    // steps outside the sequence, or before its start, do not count
    const bool full = __all(t0 < len && t0 - (S - 1) >= 0);
    by_flag(full, [&](auto all) {
#pragma unroll
        for (int s = 0; s < S; ++s)
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                if (!all.value && (t0 - s >= len || t0 - s < 0)) continue;
                const float q = B[v] + to_f32<T>(dr[s].v[v]);
                B[v] = LOGIT ? part_of(g[s][v], q) : g[s][v] * q;
                A[v] = LOGIT ? part_of(g[s][v], A[v]) : A[v] * g[s][v];
            }
    });
#pragma unroll
    for (int s = 0; s < S; ++s) forget(dr[s]), forget(xr[s]), forget(hr[s]);
    if constexpr (LN == 64)
        join<VEC>(k, seg, c0, A, B, start, agg, car, e);
    else
        join<VEC, LN, NT>(A, B, start, agg, e);
    T *of = (T *)a.df.p + (int64_t)b * a.df.sb + i, *ox = (T *)a.dx.p + (int64_t)b * a.dx.sb + i;
    by_flag(full, [&](auto all) {
#pragma unroll
        for (int s = 0; s < S; ++s) {
            const int t = t0 - s;
            const bool on = all.value || (t < len && t >= 0);
            float df[VEC], dx[VEC];
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                const float q = e[v] + to_f32<T>(dr[s].v[v]);
                float before = to_f32<T>(hr[s].v[v]);
                if (t == 0) before = a.h0 ? a.h0[c + v] : 0.0f;
                if (LOGIT) {
                    const float small = fabsf(g[s][v]), less = small * q, more = fmaf(-small, q, q);
                    dx[v] = by_side(g[s][v], less, more);
                    // half the difference: all of it may leave float32
                    const float half = fmaf(0.5f, before, -0.5f * to_f32<T>(xr[s].v[v]));
                    df[v] = 2.0f * (small * more) * half;
                    e[v] = on ? by_side(g[s][v], more, less) : e[v];
                } else {
                    dx[v] = q;
                    df[v] = q * before;
                    e[v] = on ? g[s][v] * q : e[v];
                }
                if (!on) df[v] = dx[v] = 0.0f;
            }
            if ((all.value || t >= 0) && c0 < k.C) {
                put<sizeof(T) == 4, T, VEC>(of + (int64_t)t * a.df.st, df);
                put<sizeof(T) == 4, T, VEC>(ox + (int64_t)t * a.dx.st, dx);
            }
        }
    });
    if (a.dh0 && seg == k.nseg - 1 && w == parts<LN, NT>() - 1 && c0 < k.C) {
#pragma unroll
        for (int v = 0; v < VEC; ++v) a.dh0[c + v] = e[v];
    }
    no_waits(k);
}

__global__ __launch_bounds__(256) void gated_clear_kernel(uint4 *p, int64_t n) {
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256)
        p[i] = make_uint4(0, 0, 0, 0);
}

// How a call is laid out: channels of a lane, steps of a thread, lanes along the channels,
// threads of a workgroup.
struct Shape {
    int vec, steps, lanes, threads;
};

int64_t tiles(const GatedDims &d, const Shape &p) {
    const int64_t wide = (int64_t)p.vec * p.lanes;
    return ((int64_t)d.B * d.D + wide - 1) / wide;
}
int64_t segments(int T, const Shape &p) {
    const int64_t tile = (int64_t)(p.threads / p.lanes) * p.steps;
    return (T + tile - 1) / tile;
}

// 16 steps a thread, backward of two channels to a lane (bf16) 8: longer segments have
// fewer words to exchange, until their registers leave too few waves to hide a join
// (forward 32768 x 1 x 768 bf16 51 us, with 8 steps 66; backward 1000 x 16 x 1024 49 us with
// 8, with 16 77).
// Where 1024 steps or fewer make more than one such segment, a workgroup may take all of
// them, with nothing to clear and nobody to wait for (times in a graph, wide for narrow or
// whole):
// narrow, in rows of a few values, while those are few: forward 1000 x 4 x 1024 bf16 12.1
// us for 11.0, 700 x 1 x 768 9.7 for 6.8, however 200 x 32 x 1024 14.1 for 19.1; backward,
// with twice the rows, sooner no longer: 200 x 8 x 1024 float32 12.5 for 10.8, however 300 x
// 16 x 768 bf16 15.2 for 25.1, past 512 steps 1024 x 2 x 768 11.3 for 16.0.  In a graph the
// narrow bf16 gradient is behind from about 10^6 values on (200 x 8 x 1024 11.4 for 14.1, 1000
// x 1 x 1024 10.1 for 13.0), call by call ahead up to the limits (17.6 for 14.4 and 14.1: a
// launch less for the host).
// whole, the forward pass of bf16 whose channels stand in fours, in rows of 128 bytes,
// where all workgroups run at once and on most CUs: 1024 x 16 x 1024 25.4 for 21.1, x 12
// 22.5 for 18.4, however x 8 15.1 for 17.1, x 20 29.7 for 33.2, and 200 x 32 x 1024, two
// segments, 14.1 for 13.8.
constexpr int steps(bool bwd, int vec) { return bwd && vec == 2 ? 8 : 16; }
Shape shape(const GatedDims &d, int vec, bool bwd) {
    const int two = std::min(vec, 2), all = d.T <= kThreads / kNarrow * 16 ? kThreads : kAll;
    const Shape wide{two, steps(bwd, two), 64, kThreads}, narrow{1, 16, kNarrow, all}, whole{4, 16, kNarrow, all};
    if (segments(d.T, wide) == 1 || segments(d.T, narrow) > 1) return wide;
    const int64_t n = tiles(d, whole), few = (int64_t)1 << (!bwd ? 22 : all == kThreads ? 21 : 20);
    if ((int64_t)d.T * d.B * d.D <= few) return narrow;
    return vec == 4 && !bwd && segments(d.T, wide) > 2 && n >= 160 && n * all <= 256 * 1024 ? whole : wide;
}
int64_t group_of(int64_t nseg) {
    if (nseg <= kGroup) return nseg;
    int64_t g = kGroup;
    while (g * g < nseg) ++g;
    return g;
}

// Counters a cache line apart while they are few; many tiles share the lines' work anyway.
int pitch(int64_t ntile) { return ntile <= 1024 ? 32 : 1; }
int64_t counter_words(int64_t ntile) { return (ntile * pitch(ntile) + 31) / 32 * 32; }

Cut cut(const GatedDims &d, const Shape &p, void *ws) {
    Cut k{};
    k.T = d.T, k.D = d.D, k.C = d.B * d.D;
    k.nseg = (int)segments(d.T, p);
    k.G = (int)group_of(k.nseg);
    k.ntile = (int)tiles(d, p);
    k.pitch = pitch(k.ntile);
    k.spins = host::spin_limit();
    k.flag = (unsigned *)ws;
    k.counter = (unsigned *)((char *)ws + kHead);
    k.word = (uint64_t *)(k.counter + counter_words(k.ntile));
    k.gword = k.word + (int64_t)k.nseg * k.C;
    return k;
}

// Bytes of the workspace, a multiple of 16; rnn_workspace_status takes no less than 4 KiB.
int64_t space(const Cut &k) {
    if (k.nseg == 1) return 0;
    const int64_t words = ((int64_t)k.nseg + (k.nseg + k.G - 1) / k.G) * k.C;
    return std::max<int64_t>(4096, kHead + 4 * counter_words(k.ntile) + (words * 8 + 15) / 16 * 16);
}

hipError_t clear(const Cut &k, hipStream_t s) {
    if (k.nseg == 1) return hipSuccess;
    const int64_t n = space(k) / 16;
    const unsigned grid = (unsigned)std::min<int64_t>((n + 255) / 256, 2048);
    hipLaunchKernelGGL(gated_clear_kernel, dim3(grid), dim3(256), 0, s, (uint4 *)k.flag, n);
    return hipGetLastError();
}

// How many channels of every row stand together at a multiple of their size: 4, 2 or 1.
int together(int D, size_t e, std::initializer_list<LinSeq> seqs) {
    int n = 4;
    for (const LinSeq &s : seqs)
        while (n > 1 && (D % n || (uintptr_t)s.p % (n * e) || s.st % n || s.sb % n)) n /= 2;
    return n;
}
LinSeq in(const SeqOut &o) { return LinSeq{o.p, o.st, o.sb}; }

// go(type, gate, channels of a lane, steps, lanes, threads) of a call, as values of their types.
template <int V>
using Int = std::integral_constant<int, V>;
template <bool BWD, typename F>
void by_shape(const Shape &p, bool bf16, bool logit, F go) {
    auto gate = [&](auto type, auto vec, auto steps, auto lanes, auto threads) {
        if (logit)
            go(type, std::true_type{}, vec, steps, lanes, threads);
        else
            go(type, std::false_type{}, vec, steps, lanes, threads);
    };
    auto all = [&](auto type, auto vec) {
        if (p.threads == kThreads)
            gate(type, vec, Int<16>{}, Int<kNarrow>{}, Int<kThreads>{});
        else
            gate(type, vec, Int<16>{}, Int<kNarrow>{}, Int<kAll>{});
    };
    auto one = [&](auto type) {
        if (p.lanes == kNarrow)
            all(type, Int<1>{});
        else
            gate(type, Int<1>{}, Int<steps(BWD, 1)>{}, Int<64>{}, Int<kThreads>{});
    };
    if (!bf16)
        one(float{});
    else if (p.vec == 1)
        one(uint16_t{});
    else if (p.vec == 2)
        gate(uint16_t{}, Int<2>{}, Int<steps(BWD, 2)>{}, Int<64>{}, Int<kThreads>{});
    else if constexpr (!BWD)
        all(uint16_t{}, Int<4>{});
}

}  // namespace

// A bf16 call may have any number of channels together.
size_t gated_bytes(const GatedDims &d, bool bf16, bool bwd) {
    int64_t n = 0;
    for (int vec = 1; vec <= (bf16 ? 4 : 1); vec *= 2) n = std::max(n, space(cut(d, shape(d, vec, bwd), nullptr)));
    return (size_t)n;
}

bool gated_grid_ok(const GatedDims &d, bool bf16, bool bwd) {
    for (int vec = 1; vec <= (bf16 ? 4 : 1); vec *= 2) {
        const Shape p = shape(d, vec, bwd);
        if (!grid_ok(segments(d.T, p) * tiles(d, p), p.threads)) return false;
    }
    return true;
}

hipError_t launch_gated_fwd(const GatedDims &d, bool bf16, LinSeq f, LinSeq x, const float *h0,
                            const int *lens, SeqOut h, float *hT, void *ws, hipStream_t s) {
    const Shape p = shape(d, bf16 ? together(d.D, 2, {f, x, in(h)}) : 1, false);
    const FwdArgs a{cut(d, p, ws), f, x, h0, lens, h, hT};
    const hipError_t e = clear(a.k, s);
    if (e != hipSuccess) return e;
    const dim3 grid((unsigned)((int64_t)a.k.nseg * a.k.ntile)), thr(p.threads);
    auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, thr, 0, s, a); };
    by_shape<false>(p, bf16, d.logit, [&](auto type, auto logit, auto vec, auto steps, auto lanes, auto threads) {
        go(gated_fwd_kernel<decltype(type), logit.value, vec.value, steps.value, lanes.value, threads.value>);
    });
    return hipGetLastError();
}

hipError_t launch_gated_step(const GatedDims &d, bool bf16, LinSeq f, LinSeq x, const float *h,
                             SeqOut y, float *h_out, hipStream_t s) {
    const dim3 grid((unsigned)(((int64_t)d.B * d.D + 255) / 256)), thr(256);
    auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, thr, 0, s, d, f, x, h, y, h_out); };
    if (bf16 && d.logit) go(gated_step_kernel<uint16_t, true>);
    if (bf16 && !d.logit) go(gated_step_kernel<uint16_t, false>);
    if (!bf16 && d.logit) go(gated_step_kernel<float, true>);
    if (!bf16 && !d.logit) go(gated_step_kernel<float, false>);
    return hipGetLastError();
}

hipError_t launch_gated_bwd(const GatedDims &d, bool bf16, LinSeq f, LinSeq x, LinSeq h, LinSeq dh,
                            const float *h0, const float *dhT, const int *lens, SeqOut df, SeqOut dx,
                            float *dh0, void *ws, hipStream_t s) {
    if (!d.logit) x = f;  // not read
    const Shape p = shape(d, bf16 ? together(d.D, 2, {f, x, h, dh, in(df), in(dx)}) : 1, true);
    const BwdArgs a{cut(d, p, ws), f, x, h, dh, h0, dhT, lens, df, dx, dh0};
    const hipError_t e = clear(a.k, s);
    if (e != hipSuccess) return e;
    const dim3 grid((unsigned)((int64_t)a.k.nseg * a.k.ntile)), thr(p.threads);
    auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, thr, 0, s, a); };
    by_shape<true>(p, bf16, d.logit, [&](auto type, auto logit, auto vec, auto steps, auto lanes, auto threads) {
        go(gated_bwd_kernel<decltype(type), logit.value, vec.value, steps.value, lanes.value, threads.value>);
    });
    return hipGetLastError();
}

}  // namespace lm
}  // namespace rnn355
