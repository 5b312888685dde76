// embed.hip -- embedding lookup with scaling, and its gradient by sorted ids.
//
//   x[m][:] = s * E[id_m][:]            (id outside [0, V): zeros)
//   dE[v][:] = s * sum_{m: id_m = v} dx[m][:]     (every row of dE written)
//
// Both are bound by memory: the lookup reads M rows and writes M rows, the
// gradient reads M rows once and writes V rows once.
//
// The gradient's sums must not depend on timing, so rows are added in the
// order of a stable sort of the ids, never by atomics:
//  1. a least-significant-digit radix sort of (id, m), stable by ranking each
//     wave's 64 items at a time with ballots; up to 4096 ids in one
//     workgroup's LDS, more in blocks (count, then scatter);
//  2. the sorted positions and the table's rows are merged into one sequence
//     (each row's end marker after its positions) that is cut into equal
//     pieces, one for each wave (the merge-path split: a binary search along
//     each cut's diagonal).  A piece reads its positions' rows and writes the
//     rows that end in it, zeros included, so neither a frequent id nor an
//     absent one unbalances this step.  The open row at a piece's end goes to a
//     carry;
//  3. the carries of each run of pieces with the same open row are added to
//     that row, in order, by one wave for each tile of columns: a sum in turn
//     over a 32nd of an id's occurrences.  So here a dominant id does cost:
//     16384 ids of 32000 x 768 float32 44 us with the skew of text, 62 with half
//     of them the same, 82 with all; 262144 ids 297, 685 and 1130.
//
// Measured: lookup of 16384 rows of 768 bf16 8.4 us (4.1 TB/s); gradient of
// 16384 ids of 32000 x 768 float32 31 us for the sums (4.8 TB/s), 17 for the
// sort's four launches, 5 for the carries.
#include <algorithm>

#include "common.h"
#include "lm.h"

namespace rnn355 {
namespace lm {

namespace {

// ------------------------------------------------------------------ lookup
// A row is `upr` units of N values; G lanes (a power of two) share a row.
template <typename T, int N>
__global__ __launch_bounds__(256) void embed_fwd_kernel(Ids ids, int V, int upr, int gshift,
                                                        const T *__restrict__ table, int64_t ld,
                                                        float scale, T *__restrict__ x) {
    const int G = 1 << gshift;
    const int64_t m64 = (int64_t)blockIdx.x * (256 >> gshift) + (threadIdx.x >> gshift);
    const int M = ids.T * ids.B;
    if (m64 >= M) return;
    const int m = (int)m64, lane = threadIdx.x & (G - 1);
    const int id = load_id(ids, m, V);
    const Unit<T, N> *src = (const Unit<T, N> *)(table + (int64_t)(id < V ? id : 0) * ld);
    Unit<T, N> *dst = (Unit<T, N> *)(x + (int64_t)m * upr * N);
    for (int c0 = lane; c0 < upr; c0 += 4 * G) {
        Unit<T, N> r[4];
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if (c0 + u * G < upr) r[u] = src[c0 + u * G];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            if (c0 + u * G >= upr) continue;
            Unit<T, N> o;
#pragma unroll
            for (int e = 0; e < N; ++e)
                o.v[e] = id < V ? from_f32<T>(to_f32<T>(r[u].v[e]) * scale) : from_f32<T>(0.0f);
            dst[c0 + u * G] = o;
        }
    }
}

// Lanes per row (their log2): the power of two that wastes the fewest in the
// last round.
int lane_shift(int upr) {
    int best = 6;
    long waste = -1;
    for (int g = 6; g >= 3; --g) {
        const long w = ((long)(upr + (1 << g) - 1) >> g << g) - upr;
        if (waste < 0 || w < waste) waste = w, best = g;
    }
    return best;
}
long row_blocks(long M, int upr) {
    const long rows = 256 >> lane_shift(upr);
    return (M + rows - 1) / rows;
}

// Values of the widest unit that divides a row and keeps every row aligned.
int row_unit(int D, size_t elt, const void *table, int64_t ld) {
    for (int n = 16 / (int)elt; n > 1; n = n > 2 ? 2 : 1)
        if (D % n == 0 && ld % n == 0 && (uintptr_t)table % (n * elt) == 0) return n;
    return 1;
}

template <typename T, int N>
hipError_t embed_fwd_n(const Ids &ids, int V, int D, const T *table, int64_t ld, float scale, T *x,
                       hipStream_t s) {
    const int upr = D / N;
    const long blocks = row_blocks((long)ids.T * ids.B, upr);
    hipLaunchKernelGGL((embed_fwd_kernel<T, N>), dim3((unsigned)blocks), dim3(256), 0, s, ids, V, upr,
                       lane_shift(upr), table, ld, scale, x);
    return hipGetLastError();
}

template <typename T>
hipError_t embed_fwd_t(const Ids &ids, int V, int D, const T *table, int64_t ld, float scale, T *x,
                       hipStream_t s) {
    constexpr int W = 16 / sizeof(T);
    switch (row_unit(D, sizeof(T), table, ld)) {
        case W: return embed_fwd_n<T, W>(ids, V, D, table, ld, scale, x, s);
        case 2: return embed_fwd_n<T, 2>(ids, V, D, table, ld, scale, x, s);
        default: return embed_fwd_n<T, 1>(ids, V, D, table, ld, scale, x, s);
    }
}

// -------------------------------------------------------------------- sort
// A workgroup sorts ROUNDS items per thread.
constexpr int kSortThreads = 1024, kSortWaves = kSortThreads / 64;
constexpr int kSortOne = 4 * kSortThreads;  // most items of the one-workgroup sort
constexpr int kMaxDigits = 512;
constexpr int kMaxBlocks = 64;  // each block adds up the others' counts

int key_bits(int V) { return 32 - __builtin_clz((unsigned)V); }  // keys 0..V
int sort_passes(int V) { return (key_bits(V) + 8) / 9; }
int digit_bits(int V) { return (key_bits(V) + sort_passes(V) - 1) / sort_passes(V); }

// Rank of each of this wave's items among the wave's earlier items of the
// same digit; cnt[digit] ends as the wave's count.  Items are dealt in order:
// wave w holds items [w*R*64, (w+1)*R*64), round r lane l the item r*64 + l of
// those.
template <int R>
__device__ __forceinline__ void rank_items(const uint32_t *key, int nmine, int shift,
                                           int rb, int *cnt, int *rank) {
    const int lane = threadIdx.x & 63;
    const uint64_t below = ((uint64_t)1 << lane) - 1;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const bool have = r * 64 + lane < nmine;
        const int d = (int)((key[r] >> shift) & ((1u << rb) - 1));
        uint64_t peers = __ballot(have);
        for (int b = 0; b < rb; ++b) {
            const uint64_t one = __ballot((d >> b) & 1);
            peers &= ((d >> b) & 1) ? one : ~one;
        }
        int before = 0;
        if (have) before = cnt[d];
        rank[r] = before + __popcll(peers & below);
        // the last of each group of peers writes the new count; the reads of
        // this round came first (one wave, LDS operations in order)
        if (have && (peers >> lane) == 1) cnt[d] = rank[r] + 1;
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
    }
}

// A digit's counts in the waves (at cnt, `ND` apart) -> `from` plus those of
// earlier waves; returns their total.
__device__ __forceinline__ int add_waves(int *cnt, int ND, int from) {
    int c[kSortWaves];
#pragma unroll
    for (int i = 0; i < kSortWaves; ++i) c[i] = cnt[i * ND];
    int s = from;
#pragma unroll
    for (int i = 0; i < kSortWaves; ++i) {
        cnt[i * ND] = s;
        s += c[i];
    }
    return s - from;
}

// Exclusive prefix sum over the first ND entries of tot (LDS), in place.
__device__ __forceinline__ void scan_digits(int *tot, int ND, int *tmp) {
    const int tid = threadIdx.x;
    int v = tid < ND ? tot[tid] : 0, x = v;
    const int lane = tid & 63, w = tid >> 6;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int y = __shfl_up(x, o);
        if (lane >= o) x += y;
    }
    if (lane == 63) tmp[w] = x;
    __syncthreads();
    int base = 0;
#pragma unroll
    for (int i = 0; i < kSortWaves; ++i) base += i < w ? tmp[i] : 0;
    if (tid < ND) tot[tid] = base + x - v;
    __syncthreads();
}

// All passes in one workgroup.
template <int R>
__global__ __launch_bounds__(kSortThreads) void sort_one_kernel(Ids ids, int V, int rb, int passes,
                                                                uint32_t *okey, uint32_t *opos) {
    __shared__ uint32_t skey[kSortThreads * R];
    __shared__ uint16_t spos[kSortThreads * R];
    __shared__ int cnt[kSortWaves * kMaxDigits];
    __shared__ int tot[kMaxDigits], tmp[kSortWaves];
    const int M = ids.T * ids.B, tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
    const int first = w * R * 64, nmine = min(max(M - first, 0), R * 64);
    const int ND = 1 << rb;
    uint32_t key[R], pos[R];
    int rank[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int i = r * 64 + lane;
        key[r] = i < nmine ? (uint32_t)load_id(ids, first + i, V) : 0;
        pos[r] = (uint32_t)(first + i);
    }
    for (int p = 0; p < passes; ++p) {
        for (int i = tid; i < kSortWaves * ND; i += kSortThreads) cnt[i] = 0;
        __syncthreads();
        rank_items<R>(key, nmine, p * rb, rb, cnt + w * ND, rank);
        __syncthreads();
        if (tid < ND) tot[tid] = add_waves(cnt + tid, ND, 0);
        __syncthreads();
        scan_digits(tot, ND, tmp);
#pragma unroll
        for (int r = 0; r < R; ++r)
            if (r * 64 + lane < nmine) {
                const int d = (int)((key[r] >> (p * rb)) & (ND - 1));
                const int at = tot[d] + cnt[w * ND + d] + rank[r];
                skey[at] = key[r];
                spos[at] = (uint16_t)pos[r];
            }
        __syncthreads();
#pragma unroll
        for (int r = 0; r < R; ++r)
            if (r * 64 + lane < nmine) {
                key[r] = skey[first + r * 64 + lane];
                pos[r] = spos[first + r * 64 + lane];
            }
    }
#pragma unroll
    for (int r = 0; r < R; ++r)
        if (r * 64 + lane < nmine) {
            okey[first + r * 64 + lane] = key[r];
            opos[first + r * 64 + lane] = pos[r];
        }
}

// One pass in blocks of n items: each block's digit counts.
__global__ __launch_bounds__(kSortThreads) void sort_count_kernel(Ids ids, int V, int shift, int rb,
                                                                  int block, const uint32_t *ikey,
                                                                  int *hist) {
    __shared__ int h[kMaxDigits];
    const int M = ids.T * ids.B, tid = threadIdx.x, ND = 1 << rb;
    if (tid < ND) h[tid] = 0;
    __syncthreads();
    const int first = blockIdx.x * block, n = min(M - first, block);
    for (int i = tid; i < n; i += kSortThreads) {
        const uint32_t k = ikey ? ikey[first + i] : (uint32_t)load_id(ids, first + i, V);
        atomicAdd(&h[(k >> shift) & (ND - 1)], 1);  // whole numbers: any order, one sum
    }
    __syncthreads();
    if (tid < ND) hist[blockIdx.x * ND + tid] = h[tid];
}

// The same pass's scatter: a block's place for a digit is the count of all
// smaller digits plus that of the digit in earlier blocks.  (A launch apart
// from the count: where each of 16 blocks counted all 16384 items itself, a
// pass took 13-18 us instead of 3.3 + 5.3.)
template <int R>
__global__ __launch_bounds__(kSortThreads) void sort_scatter_kernel(
    Ids ids, int V, int shift, int rb, const uint32_t *ikey, const uint32_t *ipos, const int *hist,
    uint32_t *okey, uint32_t *opos) {
    __shared__ int cnt[kSortWaves * kMaxDigits];
    __shared__ int tot[kMaxDigits], tmp[kSortWaves];
    const int M = ids.T * ids.B, tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
    const int ND = 1 << rb, nb = gridDim.x, blk = blockIdx.x;
    const int base = blk * kSortThreads * R, n = min(M - base, kSortThreads * R);
    const int first = w * R * 64, nmine = min(max(n - first, 0), R * 64);
    uint32_t key[R], pos[R];
    int rank[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int i = r * 64 + lane, at = base + first + i;
        key[r] = pos[r] = 0;
        if (i < nmine) {
            key[r] = ikey ? ikey[at] : (uint32_t)load_id(ids, at, V);
            pos[r] = ipos ? ipos[at] : (uint32_t)at;
        }
    }
    int mine = 0;  // the digit's count in earlier blocks
    if (tid < ND) {
        int all = 0;
#pragma unroll 16
        for (int b = 0; b < nb; ++b) {
            const int c = hist[b * ND + tid];
            all += c;
            mine += b < blk ? c : 0;
        }
        tot[tid] = all;
    }
    for (int i = tid; i < kSortWaves * ND; i += kSortThreads) cnt[i] = 0;
    __syncthreads();
    rank_items<R>(key, nmine, shift, rb, cnt + w * ND, rank);
    scan_digits(tot, ND, tmp);  // its barriers also order cnt
    if (tid < ND) add_waves(cnt + tid, ND, tot[tid] + mine);
    __syncthreads();
#pragma unroll
    for (int r = 0; r < R; ++r)
        if (r * 64 + lane < nmine) {
            const int at = cnt[w * ND + (int)((key[r] >> shift) & (ND - 1))] + rank[r];
            okey[at] = key[r];
            opos[at] = pos[r];
        }
}

// --------------------------------------------------------------- row sums
// A wave sums columns [tile*64*N, ...) of its piece: VEC lanes hold N
// neighbouring columns, otherwise N columns 64 apart (any width, any
// alignment).
// Items (positions and row ends) of one piece: 32, fewer (down to 8) where
// that would leave less than about 4096 waves.
int piece_items(long M, long V, int tiles) {
    return (int)std::min(32L, std::max(8L, (M + V + 1) * tiles / 4096));
}
constexpr int kInFlight = 8; // rows a wave has in flight

template <typename T, int N, bool VEC>
struct Cols {
    int c[N];
    bool on[N];
    __device__ Cols(int D, int tile) {
        const int lane = threadIdx.x & 63;
#pragma unroll
        for (int e = 0; e < N; ++e) {
            c[e] = tile * 64 * N + (VEC ? lane * N + e : e * 64 + lane);
            on[e] = c[e] < D;
        }
    }
    __device__ void load(const T *row, float *r) const {
        if constexpr (VEC) {
            Unit<T, N> u{};
            if (on[0]) u = *(const Unit<T, N> *)(row + c[0]);
#pragma unroll
            for (int e = 0; e < N; ++e) r[e] = to_f32<T>(u.v[e]);
        } else {
#pragma unroll
            for (int e = 0; e < N; ++e) r[e] = on[e] ? to_f32<T>(row[c[e]]) : 0.0f;
        }
    }
    __device__ void store(float *row, const float *r) const {
        if constexpr (VEC) {
            Unit<float, N> u;
#pragma unroll
            for (int e = 0; e < N; ++e) u.v[e] = r[e];
            if (on[0]) *(Unit<float, N> *)(row + c[0]) = u;
        } else {
#pragma unroll
            for (int e = 0; e < N; ++e)
                if (on[e]) row[c[e]] = r[e];
        }
    }
};

// First position of the piece that starts at item `d` of the merge of the
// positions with the row ends 0..V (position p before row end v iff
// key[p] <= v); its first row end is d minus that.  The 32 lanes of each half
// wave search together, 33 ways at a time: the loads of a plain bisection
// would follow each other.  The halves may search different cuts.
__device__ __forceinline__ int merge_cut(const uint32_t *key, int M, int V, long d) {
    int lo = (int)max(d - ((long)V + 1), 0l), hi = (int)min(d, (long)M);
    const int l = threadIdx.x & 31;
    // position p comes before the cut iff key[p] <= d - 1 - p: true, then false
    while (__any(lo < hi)) {
        const int step = (hi - lo) / 33 + 1;
        const long p = (long)lo + (long)(l + 1) * step - 1;  // the last of the lane's share
        const bool before = p < hi && (long)key[p] <= d - 1 - p;
        const uint32_t mask = (uint32_t)(__ballot(before) >> (threadIdx.x & 32));
        const int k = __popc(mask);  // lanes wholly before the cut
        lo += k * step;
        hi = min(hi, lo + step - 1);
    }
    return lo;
}

template <typename T, int N, bool VEC>
__global__ __launch_bounds__(256) void embed_sum_kernel(int M, int V, int D, int pieces, int piece,
                                                        const uint32_t *__restrict__ key,
                                                        const uint32_t *__restrict__ pos,
                                                        const T *__restrict__ dx, float scale,
                                                        float *__restrict__ dtable,
                                                        float *__restrict__ carry,
                                                        int *__restrict__ crow) {
    const int lane = threadIdx.x & 63;
    const int w = __builtin_amdgcn_readfirstlane(blockIdx.x * 4 + (threadIdx.x >> 6));
    if (w >= pieces) return;
    const long items = (long)M + V + 1;
    const long d0 = (long)w * piece, d1 = min(d0 + piece, items);
    const int cut = merge_cut(key, M, V, lane < 32 ? d0 : d1);
    const int p0 = __builtin_amdgcn_readlane(cut, 0), p1 = __builtin_amdgcn_readlane(cut, 32);
    int v = (int)(d0 - p0);
    const int v1 = (int)(d1 - p1);
    uint32_t k = V, at = 0;
    if (p0 + lane < p1) {
        k = key[p0 + lane];
        at = pos[p0 + lane];
    }
    const int np = __popcll(__ballot(k < (uint32_t)V));  // ids that are no token sort last
    const Cols<T, N, VEC> cols(D, blockIdx.y);
    float acc[N];
#pragma unroll
    for (int e = 0; e < N; ++e) acc[e] = 0.0f;
    auto put = [&](int row) {
        float o[N];
#pragma unroll
        for (int e = 0; e < N; ++e) o[e] = acc[e] * scale, acc[e] = 0.0f;
        cols.store(dtable + (int64_t)row * D, o);
    };
    for (int i = 0; i < np; i += kInFlight) {
        float r[kInFlight][N];
#pragma unroll
        for (int u = 0; u < kInFlight; ++u) {
            const int row = __builtin_amdgcn_readlane(at, min(i + u, np - 1));
            if (i + u < np) cols.load(dx + (int64_t)(uint32_t)row * D, r[u]);
        }
#pragma unroll
        for (int u = 0; u < kInFlight; ++u)
            if (i + u < np) {
                const int kk = __builtin_amdgcn_readlane(k, i + u);
                while (v < kk) put(v++);
#pragma unroll
                for (int e = 0; e < N; ++e) acc[e] += r[u][e];
            }
    }
    for (; v < v1 && v < V; ++v) put(v);
    // the open row at the end
    const bool open = np > 0 && __builtin_amdgcn_readlane(k, np - 1) == v1 && v1 < V;
    if (blockIdx.y == 0 && lane == 0) crow[w] = open ? v1 : -1;
    if (open) cols.store(carry + (int64_t)w * D, acc);
}

// Adds each run of carries to its row; a wave per piece, the run's first
// piece does the work.
template <int N, bool VEC>
__global__ __launch_bounds__(256) void embed_carry_kernel(int V, int D, int pieces, float scale,
                                                          float *__restrict__ dtable,
                                                          const float *__restrict__ carry,
                                                          const int *__restrict__ crow) {
    const int w = __builtin_amdgcn_readfirstlane(blockIdx.x * 4 + (threadIdx.x >> 6));
    if (w >= pieces) return;
    const int row = crow[w];
    if (row < 0 || (w > 0 && crow[w - 1] == row)) return;
    const Cols<float, N, VEC> cols(D, blockIdx.y);
    float acc[N];
#pragma unroll
    for (int e = 0; e < N; ++e) acc[e] = 0.0f;
    const int lane = threadIdx.x & 63;
    for (int w0 = w;; w0 += 64) {
        const bool same = w0 + lane < pieces && crow[w0 + lane] == row;
        const uint64_t mask = __ballot(same);
        const int n = mask == ~0ull ? 64 : __builtin_ctzll(~mask);
        for (int i = 0; i < n; i += kInFlight) {
            float r[kInFlight][N];
#pragma unroll
            for (int u = 0; u < kInFlight; ++u)
                if (i + u < n) cols.load(carry + (int64_t)(w0 + i + u) * D, r[u]);
#pragma unroll
            for (int u = 0; u < kInFlight; ++u)
                if (i + u < n)
#pragma unroll
                    for (int e = 0; e < N; ++e) acc[e] += r[u][e];
        }
        if (n < 64) break;
    }
    float own[N];
    cols.load(dtable + (int64_t)row * D, own);
#pragma unroll
    for (int e = 0; e < N; ++e) own[e] += acc[e] * scale;
    cols.store(dtable + (int64_t)row * D, own);
}

size_t up(size_t v) { return (v + 255) & ~(size_t)255; }
// Columns per lane: as many neighbours as fill one wave.
int cols_per_lane(int D) { return D > 128 ? 4 : D > 64 ? 2 : 1; }
int col_tiles(int D) { return (D + 64 * cols_per_lane(D) - 1) / (64 * cols_per_lane(D)); }
long pieces_of(long M, long V, int D) {
    const int piece = piece_items(M, V, col_tiles(D));
    return (M + V + 1 + piece - 1) / piece;
}

// Items per thread of the blocked sort: few blocks' counts to add up, and yet
// many blocks.
int sort_rounds(int M) {
    return M <= kMaxBlocks * kSortThreads ? 1 : M <= 4 * kMaxBlocks * kSortThreads ? 4 : 16;
}

struct BwdWs {
    size_t key[2], pos[2], hist, crow, carry, total;
};
BwdWs bwd_ws(int M, int V, int D) {
    BwdWs w{};
    size_t off = 0;
    for (int i = 0; i < 2; ++i) {
        w.key[i] = off; off += up(4 * (size_t)M);
        w.pos[i] = off; off += up(4 * (size_t)M);
        if (M <= kSortOne) { w.key[1] = w.key[0]; w.pos[1] = w.pos[0]; break; }
    }
    if (M > kSortOne) {
        const int per = kSortThreads * sort_rounds(M);
        w.hist = off; off += up(sizeof(int) * (size_t)((M + per - 1) / per) * kMaxDigits);
    }
    w.crow = off; off += up(sizeof(int) * (size_t)pieces_of(M, V, D));
    w.carry = off; off += up(sizeof(float) * (size_t)pieces_of(M, V, D) * D);
    w.total = off;
    return w;
}

template <typename T, int N, bool VEC>
hipError_t sums(int M, int V, int D, const uint32_t *key, const uint32_t *pos, const T *dx,
                float scale, float *dtable, float *carry, int *crow, hipStream_t s) {
    const int tiles = col_tiles(D), pieces = (int)pieces_of(M, V, D);
    const dim3 grid((pieces + 3) / 4, tiles);
    hipLaunchKernelGGL((embed_sum_kernel<T, N, VEC>), grid, dim3(256), 0, s, M, V, D, pieces,
                       piece_items(M, V, tiles), key, pos, dx, scale, dtable, carry, crow);
    hipLaunchKernelGGL((embed_carry_kernel<N, VEC>), grid, dim3(256), 0, s, V, D, pieces, scale,
                       dtable, carry, crow);
    return hipGetLastError();
}

template <typename T>
hipError_t sums_t(int M, int V, int D, const uint32_t *key, const uint32_t *pos, const T *dx,
                  float scale, float *dtable, float *carry, int *crow, hipStream_t s) {
    if (cols_per_lane(D) == 4)
        return D % 4 == 0 ? sums<T, 4, true>(M, V, D, key, pos, dx, scale, dtable, carry, crow, s)
                          : sums<T, 4, false>(M, V, D, key, pos, dx, scale, dtable, carry, crow, s);
    if (cols_per_lane(D) == 2)
        return D % 2 == 0 ? sums<T, 2, true>(M, V, D, key, pos, dx, scale, dtable, carry, crow, s)
                          : sums<T, 2, false>(M, V, D, key, pos, dx, scale, dtable, carry, crow, s);
    return sums<T, 1, true>(M, V, D, key, pos, dx, scale, dtable, carry, crow, s);
}

}  // namespace

bool embed_fwd_grid_ok(int M, int D, bool bf16, const void *table, int64_t ld) {
    return grid_ok(row_blocks(M, D / row_unit(D, bf16 ? 2 : 4, table, ld)), 256);
}

// The sort's launches have at most one thread for each id.
bool embed_bwd_grid_ok(int M, int V, int D) { return grid_ok((pieces_of(M, V, D) + 3) / 4, 256); }

hipError_t launch_embed_fwd(const Ids &ids, int V, int D, bool bf16, const void *table,
                            int64_t ld, float scale, void *x, hipStream_t s) {
    return bf16 ? embed_fwd_t<uint16_t>(ids, V, D, (const uint16_t *)table, ld, scale,
                                        (uint16_t *)x, s)
                : embed_fwd_t<float>(ids, V, D, (const float *)table, ld, scale, (float *)x, s);
}

size_t embed_bwd_bytes(int M, int V, int D) { return bwd_ws(M, V, D).total; }

hipError_t launch_embed_bwd(const Ids &ids, int V, int D, bool bf16, const void *dx, float scale,
                            float *dtable, void *ws, hipStream_t s) {
    const int M = ids.T * ids.B;
    const BwdWs w = bwd_ws(M, V, D);
    char *base = (char *)ws;
    const int passes = sort_passes(V), rb = digit_bits(V);
    uint32_t *key[2], *pos[2];
    for (int i = 0; i < 2; ++i) {
        key[i] = (uint32_t *)(base + w.key[i]);
        pos[i] = (uint32_t *)(base + w.pos[i]);
    }
    int last = 0;
    if (M <= kSortThreads) {
        hipLaunchKernelGGL(sort_one_kernel<1>, dim3(1), dim3(kSortThreads), 0, s, ids, V, rb, passes,
                           key[0], pos[0]);
    } else if (M <= kSortOne) {
        hipLaunchKernelGGL(sort_one_kernel<4>, dim3(1), dim3(kSortThreads), 0, s, ids, V, rb, passes,
                           key[0], pos[0]);
    } else {
        const int R = sort_rounds(M), per = kSortThreads * R;
        int *hist = (int *)(base + w.hist);
        const dim3 grid((M + per - 1) / per), thr(kSortThreads);
        for (int p = 0; p < passes; ++p) {
            const uint32_t *ik = p ? key[(p - 1) & 1] : nullptr, *ip = p ? pos[(p - 1) & 1] : nullptr;
            uint32_t *ok = key[p & 1], *op = pos[p & 1];
            hipLaunchKernelGGL(sort_count_kernel, grid, thr, 0, s, ids, V, p * rb, rb, per, ik, hist);
            if (R == 1)
                hipLaunchKernelGGL(sort_scatter_kernel<1>, grid, thr, 0, s, ids, V, p * rb, rb, ik, ip,
                                   hist, ok, op);
            else if (R == 4)
                hipLaunchKernelGGL(sort_scatter_kernel<4>, grid, thr, 0, s, ids, V, p * rb, rb, ik, ip,
                                   hist, ok, op);
            else
                hipLaunchKernelGGL(sort_scatter_kernel<16>, grid, thr, 0, s, ids, V, p * rb, rb, ik, ip,
                                   hist, ok, op);
            last = p & 1;
        }
    }
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    float *carry = (float *)(base + w.carry);
    int *crow = (int *)(base + w.crow);
    return bf16 ? sums_t<uint16_t>(M, V, D, key[last], pos[last], (const uint16_t *)dx, scale,
                                   dtable, carry, crow, s)
                : sums_t<float>(M, V, D, key[last], pos[last], (const float *)dx, scale, dtable,
                                carry, crow, s);
}

}  // namespace lm
}  // namespace rnn355
