// linattn.hip -- linear attention with a decay for each head.
//
// For each batch row and head, with a = e^g and a matrix state S [Dk][Dv]:
//   S_t = a S_{t-1} + k_t^T v_t,     o_t = scale q_t S_t        (t = 0..T-1)
// and backward, with G_t = dL/dS_t:
//   dq_t = scale S_t do_t,  G_t = scale q_t^T do_t + a G_{t+1}  (+ dS_T at T-1)
//   dk_t = G_t v_t,  dv_t = G_t^T k_t,  dS_0 = a G_0
//
// One kernel serves all of these.  It computes, over rows r in walking order,
//   o_r = os ( is sum_{j<=r} a^(r-j) (x_r . y_j) z_j + a^r x_r X )
// with a carried matrix X ("the state already decayed for the next row") and
//   X <- a^n X + is sum_j a^(n-j) y_j^T z_j    over n rows:
//   forward  x,y,z = q,k,v     X = a S_0           is = 1, os = scale
//   dq       x,y,z = do,v,k    X = a S_0^T         is = 1, os = scale
//   dk       x,y,z = v,do,q    X = dS_T^T          is = scale, os = 1, backwards in t
//   dv       x,y,z = k,q,do    X = dS_T            is = scale, os = 1, backwards in t
// (the final X of dv is dS_0; the forward's S_T takes one decay less).
//
// Rows are taken in chunks of C.  Inside a chunk the masked, decayed product
// P = (x y^T) o a^(r-j) is formed and applied to z; the rest goes through X.
// Exponents are never negative, so no decay overflows, a = 0 included.
//
// Layout: a workgroup of four or eight waves owns (batch row, head, 64 or 128
// columns of z, a segment of the rows); a wave owns 16 of the columns and the
// whole X for them.  In the 16x16 matrix instructions a lane holds, for its column,
// four consecutive rows of a result; with the operand's depth numbered so that
// a lane's eight depth elements are rows 4g..4g+3 of two neighbouring 16-row
// tiles (g = lane / 16), a result is an operand as it stands: X never leaves
// the registers, and P, which all waves need, is formed once, a tile at a time
// by one of them, and passed through LDS in operand order.  y and z are
// needed along their rows too: LDS is read through the transposing 16-bit
// loads of gfx950.
//
// Arithmetic: x, y, z as given (bf16 or float32), all sums float32.  P, X and
// the decayed z are operands of further products; in bf16 calls they are split
// in three bf16 parts (8 + 8 + 8 bits, so nothing is left out), and outputs
// carry one rounding, their own.  Two parts for P and X (2^-17 of them left out)
// took 62 us for 66 (T1024 B16 NH6 D128) and 96 for 104 (backward T1000 B8
// NH8:4 D128), but left outputs 1e-4 from a float32 evaluation rounded once,
// for 3e-5.  float32 calls use the float32 matrix instructions.
//
// Few (batch row, head) pairs leave the chip empty, so the rows are cut into
// segments: a first launch forms the segments' own X from nothing (in pieces of
// a segment where that fills the chip), a second carries X across them (where
// they are few the main launch adds them up itself), and the main launch runs
// all segments at once.
//
// Measured: T1024 B16 NH6 D128 bf16 13.6 us for the states and 52 for the main
// launch (114 MB from memory, matrix units 20% busy): bound by the latency of a
// chunk's phases, 13-14 thousand cycles for 3500 of products.  T8191 NH12 D64
// float32 16 + 8 + 33 us, matrix units 47% busy.  A token for B64 NH12 D64
// 7.0 us (3.6 TB/s).
#include <algorithm>
#include <mutex>

#include "lm.h"

namespace rnn355 {
namespace lm {

namespace {

typedef __attribute__((ext_vector_type(4))) short s16x4;
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

// One product with the sequences' heads, operands, ranges and scales.
struct Role {
    LinSeq x, y, z;
    int gx, gy, gz;         // heads that share one of the operand's (head h uses h / g)
    int Da, Db;             // depth of x.y, columns of z
    const float *init;      // X before the first row, [B][NH][Dk][Dv], or null
    int init_t;             // read it transposed
    int init_decay;         // times a
    float *fin;             // final state, [B][NH][Da][Db], or null
    int fin_less;           // with one decay less (the forward's S_T)
    int rev;                // rows run backwards in t
    float is, os;
    void *o;                // [T][B][NH][Db]
    int o_f32;              // float32 whatever the call's type (partial sums of shared heads)
    float *part;            // carried X of the segments, in fragment order
};
struct LinArgs {
    Role role[3];
    int nroles, T, B, NH;
    const float *g;
    int nseg, subs, sub_rows;  // segments of `subs` pieces of sub_rows rows
    int slices;                // of the columns of z
};

// ---- element types
template <typename T>
struct Frag;  // eight depth elements of a lane
template <>
struct Frag<uint16_t> { bf16x8 v; };
template <>
struct Frag<float> { float v[8]; };

// d += A B over a depth of 32
__device__ __forceinline__ void mma(f32x4 &d, const Frag<uint16_t> &a, const Frag<uint16_t> &b) {
    d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.v, b.v, d, 0, 0, 0);
}
__device__ __forceinline__ void mma(f32x4 &d, const Frag<float> &a, const Frag<float> &b) {
#pragma unroll
    for (int e = 0; e < 8; ++e)
        d = __builtin_amdgcn_mfma_f32_16x16x4f32(a.v[e], b.v[e], d, 0, 0, 0);
}

typedef __attribute__((ext_vector_type(2))) float f32x2;
typedef __attribute__((ext_vector_type(2))) __bf16 bf16x2;
typedef __attribute__((ext_vector_type(4))) uint32_t u32x4;

// A float32 operand: as it is, or as a bf16, the bf16 of what that leaves, and
// the bf16 of what is left then (nothing beyond: 8 + 8 + 8 bits).
template <typename T>
struct Wide;
template <>
struct Wide<float> {
    Frag<float> f;
    __device__ void set(const float *x) {
#pragma unroll
        for (int e = 0; e < 8; ++e) f.v[e] = x[e];
    }
};
// a pair's bf16 parts, what they leave in x
__device__ __forceinline__ uint32_t split2(float *x) {
    const uint32_t h = __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{x[0], x[1]}, bf16x2));
    x[0] -= __uint_as_float(h << 16);
    x[1] -= __uint_as_float(h & 0xFFFF0000u);
    return h;
}
__device__ __forceinline__ void split8(Frag<uint16_t> &f, float *x) {
    const u32x4 w{split2(x), split2(x + 2), split2(x + 4), split2(x + 6)};
    f.v = __builtin_bit_cast(bf16x8, w);
}
template <>
struct Wide<uint16_t> {
    Frag<uint16_t> part[3];
    __device__ void set(float *x) {
#pragma unroll
        for (int i = 0; i < 3; ++i) split8(part[i], x);
    }
};
__device__ __forceinline__ void mma(f32x4 &d, const Frag<float> &a, const Wide<float> &b) { mma(d, a, b.f); }
__device__ __forceinline__ void mma(f32x4 &d, const Wide<float> &a, const Frag<float> &b) { mma(d, a.f, b); }
__device__ __forceinline__ void mma(f32x4 &d, const Frag<uint16_t> &a, const Wide<uint16_t> &b) {
#pragma unroll
    for (int i = 0; i < 3; ++i) mma(d, a, b.part[i]);
}
__device__ __forceinline__ void mma(f32x4 &d, const Wide<uint16_t> &a, const Frag<uint16_t> &b) {
#pragma unroll
    for (int i = 0; i < 3; ++i) mma(d, a.part[i], b);
}

// P^T in LDS: operands of depth 32 (pairs of tiles), each in lane order.  A
// tile is half an operand: four of a lane's eight elements.
template <typename T>
constexpr int kOperand = sizeof(T) == 2 ? 3 * 64 * 16 : 2 * 64 * 16;  // bytes of one
__device__ __forceinline__ void put_half(char *o, int half, float *x, uint16_t) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        uint2 w;
        w.x = split2(x), w.y = split2(x + 2);
        *(uint2 *)(o + i * 1024 + lane * 16 + half * 8) = w;
    }
}
__device__ __forceinline__ void put_half(char *o, int half, float *x, float) {
    *(float4 *)(o + half * 1024 + (threadIdx.x & 63) * 16) = make_float4(x[0], x[1], x[2], x[3]);
}
// One of its parts: products take them one after another.
template <typename T>
constexpr int kParts = sizeof(T) == 2 ? 3 : 1;
__device__ __forceinline__ void get_part(Frag<uint16_t> &f, const char *o, int i) {
    f.v = *(const bf16x8 *)(o + i * 1024 + (threadIdx.x & 63) * 16);
}
__device__ __forceinline__ void get_part(Frag<float> &f, const char *o, int) {
    const int lane = threadIdx.x & 63;
    const float4 a = *(const float4 *)(o + lane * 16), b = *(const float4 *)(o + 1024 + lane * 16);
    f.v[0] = a.x; f.v[1] = a.y; f.v[2] = a.z; f.v[3] = a.w;
    f.v[4] = b.x; f.v[5] = b.y; f.v[6] = b.z; f.v[7] = b.w;
}

// Depth elements of row `row`, depths [32 kb, 32 kb + 32), from a row-major
// LDS tile.  Tiles that are only read this way (x) keep each lane's eight
// together in bf16 calls: one 16-byte read, where two of 8 bytes would meet in
// the same banks.
__device__ __forceinline__ int x_col(int k, uint16_t) {
    return (k & ~31) | ((k & 12) << 1) | ((k & 16) >> 2) | (k & 3);
}
__device__ __forceinline__ int x_col(int k, float) { return k; }
__device__ __forceinline__ void put_x(uint16_t *t, int c, const uint4 &v) {
    *(uint2 *)(t + x_col(c, uint16_t())) = make_uint2(v.x, v.y);
    *(uint2 *)(t + x_col(c + 4, uint16_t())) = make_uint2(v.z, v.w);
}
__device__ __forceinline__ void put_x(float *t, int c, const uint4 &v) { *(uint4 *)(t + c) = v; }
__device__ __forceinline__ void along_x(Frag<uint16_t> &f, const uint16_t *t, int ld, int row, int kb, int g) {
    f.v = *(const bf16x8 *)(t + row * ld + kb * 32 + 8 * g);
}
__device__ __forceinline__ void along(Frag<uint16_t> &f, const uint16_t *t, int ld, int row, int kb, int g) {
    const uint2 a = *(const uint2 *)(t + row * ld + kb * 32 + 4 * g);
    const uint2 b = *(const uint2 *)(t + row * ld + kb * 32 + 16 + 4 * g);
    const uint4 w = make_uint4(a.x, a.y, b.x, b.y);
    f.v = __builtin_bit_cast(bf16x8, w);
}
__device__ __forceinline__ void along(Frag<float> &f, const float *t, int ld, int row, int kb, int g) {
    const float4 a = *(const float4 *)(t + row * ld + kb * 32 + 4 * g);
    const float4 b = *(const float4 *)(t + row * ld + kb * 32 + 16 + 4 * g);
    f.v[0] = a.x; f.v[1] = a.y; f.v[2] = a.z; f.v[3] = a.w;
    f.v[4] = b.x; f.v[5] = b.y; f.v[6] = b.z; f.v[7] = b.w;
}
__device__ __forceinline__ void along_x(Frag<float> &f, const float *t, int ld, int row, int kb, int g) {
    along(f, t, ld, row, kb, g);
}
// Depth runs over the tile's rows [32 kb, 32 kb + 32) at column col0 + lane % 16.
__device__ __forceinline__ void across(Frag<uint16_t> &f, const uint16_t *t, int ld, int col0, int kb,
                                       int g, int c) {
    // each 16 lanes: four rows of 16 columns in, four rows of one column out
    const uint16_t *p = t + (kb * 32 + 4 * g + (c >> 2)) * ld + col0 + 4 * (c & 3);
    const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)p);
    const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(p + 16 * ld));
    const __attribute__((ext_vector_type(8))) short w = __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
    f.v = __builtin_bit_cast(bf16x8, w);
}
__device__ __forceinline__ void across(Frag<float> &f, const float *t, int ld, int col0, int kb, int g,
                                       int c) {
#pragma unroll
    for (int e = 0; e < 8; ++e) f.v[e] = t[(kb * 32 + (e >> 2) * 16 + 4 * g + (e & 3)) * ld + col0 + c];
}
__device__ __forceinline__ void unpack(float *x, const Frag<uint16_t> &f) {
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = (float)f.v[e];
}
__device__ __forceinline__ void unpack(float *x, const Frag<float> &f) {
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = f.v[e];
}

// Whether a sequence's rows are whole 16-byte pieces and a chunk of them lies
// within 32 bits of its first.
template <typename T>
bool pieces_ok(const LinSeq &q, int D) {
    constexpr int N = 16 / sizeof(T);
    return ((uintptr_t)q.p & 15) == 0 && q.st % N == 0 && q.sb % N == 0 && D % N == 0 && q.st >= 0 &&
           q.st < (1ll << 23);
}

// A [C][W] tile of a sequence operand: rows row0.. of n (walking order, t =
// rev ? T-1-row : row), columns [0, D) of `src`, zeros outside.  FAST (see
// lin_kernel): 16-byte pieces wait in registers between fetch() and put(), R
// per thread, loaded without a branch (rows outside come from inside and are
// dropped by put) so that all are in flight at once.  Otherwise put() reads the
// tile value by value.
template <typename T, int C, int W, int THREADS, bool FAST>
struct Tile {
    static constexpr int N = 16 / sizeof(T), PR = W / N, RS = THREADS / PR, R = (C + RS - 1) / RS;
    static_assert(THREADS % PR == 0 && (C % RS == 0 || RS > C), "a thread's pieces share their columns");
    const T *src;
    int64_t st;
    int D, T_, rev;
    uint4 r[FAST ? R : 1];
    __device__ void init(const T *src_, int64_t st_, int Tn, int rev_, int D_) {
        src = src_;
        st = st_;
        T_ = Tn;
        rev = rev_;
        D = D_;
    }
    __device__ void fetch(int row0, int n) {
        if constexpr (FAST) {
            const int row = threadIdx.x / PR, c = (threadIdx.x % PR) * N;
            const int64_t t0 = rev ? T_ - row0 - C : row0;  // lowest t of a whole chunk
            const char *base = (const char *)(src + t0 * st);
            const uint32_t pitch = (uint32_t)st * sizeof(T), at = (c < D ? c : 0) * sizeof(T);
#pragma unroll
            for (int i = 0; i < R; ++i) {
                const int k = min(row + i * RS, n - 1);
                r[i] = *(const uint4 *)(base + ((uint32_t)(rev ? C - 1 - k : k) * pitch + at));
            }
        }
    }
    template <bool X = false>
    __device__ void put(T *t, int ld, int row0, int n) const {
        if constexpr (FAST) {
            const int row = threadIdx.x / PR, c = (threadIdx.x % PR) * N;
            const bool all = n == C && D == W;  // nothing outside the tile
#pragma unroll
            for (int i = 0; i < R; ++i) {
                if (RS > C && row >= C) break;  // more threads than pieces
                uint4 v = r[i];
                if (!all && !(row + i * RS < n && c < D)) v = make_uint4(0, 0, 0, 0);
                T *at = t + (row + i * RS) * ld;
                if constexpr (X)
                    put_x(at, c, v);
                else
                    *(uint4 *)(at + c) = v;
            }
        } else {
#pragma unroll 1
            for (int q = threadIdx.x; q < C * W; q += THREADS) {
                const int i = q / W, k = q % W;
                t[i * ld + (X ? x_col(k, T()) : k)] =
                    i < n && k < D ? src[(int64_t)(rev ? T_ - 1 - row0 - i : row0 + i) * st + k]
                                   : from_f32<T>(0.0f);
            }
        }
    }
};

// Four neighbouring values at p[at], one base for all threads.
__device__ __forceinline__ void store4(float *p, uint32_t at, const f32x4 &v) {
    *(f32x4 *)((char *)p + at * 4u) = v;
}
__device__ __forceinline__ void store4(uint16_t *p, uint32_t at, const f32x4 &v) {
    uint2 u;
    u.x = __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{v[0], v[1]}, bf16x2));
    u.y = __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{v[2], v[3]}, bf16x2));
    *(uint2 *)((char *)p + at * 2u) = u;
}

template <typename T>
struct Shape;
// Rows of a chunk; values of padding to a row of an LDS tile.  A tile that is
// read along its rows puts 16 rows 16 bytes apart over the 64 banks; the
// transposing 16-bit reads take 32 bytes of 8 rows at a time, so theirs are 32
// bytes apart.
template <>
struct Shape<uint16_t> { static constexpr int C = 64, pad = 16, padx = 8; };
template <>
struct Shape<float> { static constexpr int C = 32, pad = 4, padx = 4; };

// Where each part of the workgroup's LDS starts.
template <typename T, int DA, int NW, bool STATE>
struct Lds {
    static constexpr int C = Shape<T>::C, RT = C / 16;
    static constexpr int LD = DA + Shape<T>::pad, LDZ = 16 * NW + Shape<T>::pad,
                         LDX = DA + Shape<T>::padx;
    // operands of P: depth blocks up to each 16-row tile's own
    static constexpr int operands = (RT / 2) * (RT / 2 + 1);
    static constexpr size_t y = 0, z = y + sizeof(T) * C * LD, w = z + sizeof(T) * C * LDZ,
                            x = w + sizeof(float) * C, p = x + sizeof(T) * C * LDX,
                            bytes = STATE ? x : p + operands * kOperand<T>;
};

// Fragment order of one workgroup's X: [wave][DA/16 tiles][lane][4].
template <int DA, int NW>
__device__ __forceinline__ int64_t part_at(const LinArgs &a, int bh, int slice, int seg, int tile) {
    const int w = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int64_t wg = ((int64_t)bh * a.slices + slice) * a.nseg * a.subs + seg;
    return (((wg * NW + w) * (DA / 16) + tile) * 64 + lane) * 4;
}

// log2 of the decay e^g; kept finite, so that 0 times it is 0 (a = 0).  NaN
// stays (fmaxf would make it a decay of 0).
__device__ __forceinline__ float log2_decay(float g) {
    const float g2 = g * kLog2e;
    return g2 < -1e30f ? -1e30f : g2;
}

// Up to three pieces before the last segment, a workgroup adds up the earlier
// ones' X itself; past that their reading costs more than a launch.
__host__ __device__ __forceinline__ bool folds(const LinArgs &a) { return (a.nseg - 1) * a.subs <= 3; }

// STATE: only the piece's own X, from nothing (the first: from the initial
// state), into its slot of `part`.
// Registers for two workgroups to a CU where their LDS allows it: in a grid of
// many, one's barriers and loads then hide behind the other's products (B64 NH8
// T1024 D128 175 us against 190 with the registers of one; backward B16 NH6 129
// against 156).  A grid of one to a CU gains nothing (T1024 B16 NH6 66 for 65).
// FAST: every operand in whole 16-byte pieces and z in whole 16-column tiles
// (the host's rule); the general form, which reads value by value, then stays
// out of the registers of the ordinary one (7 rows of 1968 tokens, 6 heads of
// 48 x 32 in bf16: 32 us against 106).
template <typename T, int DA, int NW, bool STATE, bool FAST>
__global__ __launch_bounds__(64 * NW, (DA <= 128 && 2 * Lds<T, DA, NW, STATE>::bytes <= 160 * 1024 ? 2 : 1) * NW / 4)
void lin_kernel(LinArgs a) {
    using L = Lds<T, DA, NW, STATE>;
    constexpr int C = L::C, LD = L::LD, LDZ = L::LDZ, LDX = L::LDX, COLS = 16 * NW;
    constexpr int KB = DA / 32, RB = C / 32, RT = C / 16, DT = DA / 16;
    extern __shared__ __attribute__((aligned(16))) char smem[];
    T *ys = (T *)(smem + L::y), *zs = (T *)(smem + L::z), *xs = (T *)(smem + L::x);
    float *wz = (float *)(smem + L::w);  // decays of z's rows towards the next chunk
    char *ps = smem + L::p;

    const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, c = lane & 15;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    // slices of one (role, row, head, segment) go to the same XCD (workgroups
    // go round the eight of them), where they share x and y in its L2
    const int nsegs = STATE ? (a.nseg - 1) * a.subs : a.nseg;
    const int groups = a.nroles * a.B * a.NH * nsegs;
    // (quotients come from the vector units; all of this is the same for a wave)
    auto div = [](int p, int q) { return __builtin_amdgcn_readfirstlane(p / q); };
    const int outer = div(blockIdx.x >> 3, a.slices), slice = (blockIdx.x >> 3) - outer * a.slices;
    const int grp = outer * 8 + (blockIdx.x & 7);
    if (grp >= groups) return;
    const int rest = div(grp, nsegs), seg = grp - rest * nsegs;
    const int role = div(rest, a.B * a.NH), bh = rest - role * a.B * a.NH;
    const Role R = a.role[role];
    const int b = div(bh, a.NH), h = bh - b * a.NH;
    const int col0 = slice * COLS;
    if (col0 >= R.Db) return;
    const int nc = min(R.Db - col0, COLS);

    Tile<T, C, DA, 64 * NW, FAST> tx, ty;
    Tile<T, C, COLS, 64 * NW, FAST> tz;
    if constexpr (!STATE)
        tx.init((const T *)R.x.p + (int64_t)b * R.x.sb + (int64_t)div(h, R.gx) * R.Da, R.x.st, a.T, R.rev, R.Da);
    ty.init((const T *)R.y.p + (int64_t)b * R.y.sb + (int64_t)div(h, R.gy) * R.Da, R.y.st, a.T, R.rev, R.Da);
    tz.init((const T *)R.z.p + (int64_t)b * R.z.sb + (int64_t)div(h, R.gz) * R.Db + col0, R.z.st, a.T, R.rev, nc);

    const float g2 = log2_decay(a.g[h]);
    auto power = [&](int n) { return __builtin_amdgcn_exp2f(g2 * (float)n); };

    const float powc = power(c);

    const int rows = STATE ? a.sub_rows : a.subs * a.sub_rows;
    const int row_lo = seg * rows, row_hi = min(row_lo + rows, a.T);

    // element r of X[t]: depth 16 t + 4 g + r, column wcol + c of the slice
    f32x4 X[DT];
    const int wcol = 16 * w;
    const bool wave_on = wcol < nc;
#pragma unroll
    for (int t = 0; t < DT; ++t) X[t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    // The initial state: from where the caller has it by the one workgroup that
    // starts there.  With several segments that is the first piece's, in the
    // launch before; it also leaves a copy in slot 0 for the main launch, whose
    // last segment may be writing the final state over the initial one by then.
    if (R.init && seg == 0 && STATE == (a.nseg > 1)) {
        const float f = R.init_decay ? power(1) : 1.0f;
        const float *S = R.init + (int64_t)bh * R.Da * R.Db;
        const int sd = R.init_t ? 1 : R.Db, sc = R.init_t ? R.Da : 1;
        const int col = col0 + wcol + c;
        // loads without a branch, from inside the state
        const float *Sc = S + min(col, R.Db - 1) * sc;
#pragma unroll
        for (int t = 0; t < DT; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int d = 16 * t + 4 * g + r;
                const float v = Sc[min(d, R.Da - 1) * sd];
                X[t][r] = d < R.Da && col < R.Db ? f * v : 0.0f;
            }
        if constexpr (STATE) {
#pragma unroll
            for (int t = 0; t < DT; ++t)
                *(f32x4 *)(R.part + part_at<DA, NW>(a, bh, slice, 0, t)) = X[t];
        }
    }
    if constexpr (!STATE) {
        // what comes before: the initial state for the first segment; for others
        // the earlier pieces' X, carried by a launch of its own or added up here
        const float fs = power(a.sub_rows);
        const int before = seg * a.subs;
        const int from0 = a.nseg == 1 || (seg == 0 && !R.init) ? before + 1 : seg == 0 ? 0 : folds(a) ? 1 : before;
        for (int from = from0; from <= before; ++from) {
            f32x4 v[DT];
#pragma unroll
            for (int t = 0; t < DT; ++t) v[t] = *(const f32x4 *)(R.part + part_at<DA, NW>(a, bh, slice, from, t));
            // X is no plain copy of loads: those are then waited for here, where a
            // wait inside the loop would be for the next chunk's loads as well
#pragma unroll
            for (int t = 0; t < DT; ++t)
#pragma unroll
                for (int r = 0; r < 4; ++r) X[t][r] = fs * X[t][r] + v[t][r];
        }
        // the tiles above the diagonal that share an operand with one on it
        for (int i = tid; i < L::operands * kOperand<T> / 16; i += 64 * NW)
            ((uint4 *)ps)[i] = make_uint4(0, 0, 0, 0);
    }

    auto fetch = [&](int row0) {
        const int n = min(C, row_hi - row0);
        ty.fetch(row0, n);
        tz.fetch(row0, n);
        if constexpr (!STATE) tx.fetch(row0, n);
    };
    fetch(row_lo);
    for (int row0 = row_lo; row0 < row_hi; row0 += C) {
        const int n = min(C, row_hi - row0);
        const bool last = row0 + C >= a.T;
        // rows that X moves on by; the forward's final state takes one decay less
        const int m = n - (last && R.fin_less ? 1 : 0);
        lds_barrier();
        ty.put(ys, LD, row0, n);
        tz.put(zs, LDZ, row0, n);
        if constexpr (!STATE) tx.template put<true>(xs, LDX, row0, n);
        if (tid < C) wz[tid] = R.is * power(max(m - tid, 0));  // rows past n are zero in z
        lds_barrier();

        // the next chunk's loads have this chunk's whole time (T1024 B16 NH6 D128 66 us
        // against 71 issued after P.z, B64 NH8 175 against 183)
        if (row0 + C < row_hi) fetch(row0 + C);
        f32x4 o[STATE ? 1 : RT];
        if constexpr (!STATE) {
            // P^T, tile by tile: rows j of y, columns i of x
            for (int p = w; p < RT * (RT + 1) / 2; p += NW) {
                int it = 0;
                while ((it + 1) * (it + 2) / 2 <= p) ++it;
                const int jt = p - it * (it + 1) / 2;
                if (it * 16 >= n) break;
                f32x4 d{0.0f, 0.0f, 0.0f, 0.0f};
                constexpr int PM = sizeof(T) == 2 ? 4 : 1, PB = KB < PM ? KB : PM;  // depth blocks read at a time
#pragma unroll
                for (int k0 = 0; k0 < KB; k0 += PB) {
                    Frag<T> yf[PB], xf[PB];
#pragma unroll
                    for (int kb = 0; kb < PB; ++kb) {
                        along(yf[kb], ys, LD, jt * 16 + c, k0 + kb, g);
                        along_x(xf[kb], xs, LDX, it * 16 + c, k0 + kb, g);
                    }
                    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                    for (int kb = 0; kb < PB; ++kb) mma(d, yf[kb], xf[kb]);
                }
                mfma_chain_end();
                float e[4];
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int lag = (it - jt) * 16 + c - 4 * g - r;
                    e[r] = lag >= 0 ? d[r] * (R.is * power(max(lag, 0))) : 0.0f;
                }
                // operands before this tile row's: 1, 1, 2, 2, ... each
                put_half(ps + ((it / 2) * (it / 2 + 1) + (it & 1) * (it / 2 + 1) + jt / 2) * kOperand<T>,
                         jt & 1, e, T());
            }
            // what the carried X gives
#pragma unroll
            for (int it = 0; it < RT; ++it) o[it] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
            if (wave_on) {
                // reads of LDS run AX operands ahead of the products
                constexpr int AX = 2, NX = KB * RT;
                Frag<T> xf[AX + 1];
                Wide<T> Xw;
#pragma unroll
                for (int i = 0; i < AX; ++i) along_x(xf[i], xs, LDX, (i % RT) * 16 + c, i / RT, g);
#pragma unroll
                for (int i = 0; i < NX; ++i) {
                    const int kb = i / RT, j = i + AX;
                    if (j < NX) along_x(xf[j % (AX + 1)], xs, LDX, (j % RT) * 16 + c, j / RT, g);
                    __builtin_amdgcn_sched_barrier(0);
                    if (i % RT == 0) {
                        float e[8];
#pragma unroll
                        for (int r = 0; r < 4; ++r) e[r] = X[2 * kb][r], e[4 + r] = X[2 * kb + 1][r];
                        Xw.set(e);
                    }
                    mma(o[i % RT], Xw, xf[i % (AX + 1)]);
                    __builtin_amdgcn_sched_barrier(0);
                }
                mfma_chain_end();
#pragma unroll
                for (int it = 0; it < RT; ++it) {
                    const float f = power(it * 16) * powc;
#pragma unroll
                    for (int r = 0; r < 4; ++r) o[it][r] *= f;
                }
            }
            lds_barrier();
        }
        if (!wave_on) continue;

        // this wave's columns of z, depth along the chunk's rows
        Frag<T> zf[RB];
#pragma unroll
        for (int kb = 0; kb < RB; ++kb) across(zf[kb], zs, LDZ, wcol, kb, g, c);

        if constexpr (!STATE) {
            // operand q belongs to tile row (0, 1, 2, 2, 3, 3)[q], depth block (0, 0, 0, 1, 0, 1)[q]
            constexpr int NP = L::operands * kParts<T>;
            Frag<T> pf[3];
            get_part(pf[0], ps, 0);
            if (NP > 1) get_part(pf[1], ps + 1 / kParts<T> * kOperand<T>, 1 % kParts<T>);
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                const int q = i / kParts<T>, j = i + 2;
                if (j < NP) get_part(pf[j % 3], ps + j / kParts<T> * kOperand<T>, j % kParts<T>);
                __builtin_amdgcn_sched_barrier(0);
                mma(o[q < 2 ? q : 1 + q / 2], zf[q < 2 ? 0 : q & 1], pf[i % 3]);
                __builtin_amdgcn_sched_barrier(0);
            }
            mfma_chain_end();
            // lane: row it*16 + c, columns wcol + 4 g ..+3
            // 16 rows lie within 32 bits of each other (the host's check)
            const uint32_t pitch = (uint32_t)(a.B * a.NH * R.Db);
            const uint32_t mine = (uint32_t)(R.rev ? 15 - c : c) * pitch + (uint32_t)(wcol + 4 * g);
            const int64_t at = ((int64_t)b * a.NH + h) * R.Db + col0;
#pragma unroll
            for (int it = 0; it < RT; ++it) {
                if (it * 16 + c >= n) continue;
#pragma unroll
                for (int r = 0; r < 4; ++r) o[it][r] *= R.os;
                const int row = row0 + it * 16;
                const int64_t base = at + (int64_t)(R.rev ? a.T - row - 16 : row) * pitch;
                if constexpr (FAST) {
                    if (R.o_f32)
                        store4((float *)R.o + base, mine, o[it]);
                    else
                        store4((T *)R.o + base, mine, o[it]);
                } else {
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        if (wcol + 4 * g + r < nc) {
                            if (R.o_f32)
                                ((float *)R.o)[base + mine + r] = o[it][r];
                            else
                                ((T *)R.o)[base + mine + r] = from_f32<T>(o[it][r]);
                        }
                }
            }
        }
        // X <- a^m X + y^T (decayed z)
        if (STATE || row0 + C < row_hi || (last && R.fin)) {
            const float f = power(m);
#pragma unroll
            for (int t = 0; t < DT; ++t)
#pragma unroll
                for (int r = 0; r < 4; ++r) X[t][r] *= f;
#pragma unroll
            for (int kb = 0; kb < RB; ++kb) {
                const float4 wa = *(const float4 *)(wz + kb * 32 + 4 * g);
                const float4 wb = *(const float4 *)(wz + kb * 32 + 16 + 4 * g);
                const float ww[8] = {wa.x, wa.y, wa.z, wa.w, wb.x, wb.y, wb.z, wb.w};
                float e[8];
                unpack(e, zf[kb]);
#pragma unroll
                for (int i = 0; i < 8; ++i) e[i] *= ww[i];
                Wide<T> zw;
                zw.set(e);
                // reads of LDS run a tile ahead of the products
                constexpr int YA = 1;
                Frag<T> yf[2][YA];
#pragma unroll
                for (int u = 0; u < YA; ++u) across(yf[0][u], ys, LD, 16 * u, kb, g, c);
#pragma unroll
                for (int t0 = 0; t0 < DT; t0 += YA) {
                    if (t0 + YA < DT)
#pragma unroll
                        for (int u = 0; u < YA; ++u)
                            across(yf[(t0 / YA + 1) & 1][u], ys, LD, 16 * (t0 + YA + u), kb, g, c);
                    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                    for (int u = 0; u < YA; ++u) mma(X[t0 + u], yf[(t0 / YA) & 1][u], zw);
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
            mfma_chain_end();
        }
    }
    if constexpr (STATE) {
        // this piece's own X, in the slot of the piece it is carried into
#pragma unroll
        for (int t = 0; t < DT; ++t)
            *(f32x4 *)(R.part + part_at<DA, NW>(a, bh, slice, seg + 1, t)) = X[t];
    } else if (R.fin && seg == a.nseg - 1 && wave_on) {
        float *S = R.fin + (int64_t)bh * R.Da * R.Db;
        const int col = col0 + wcol + c;
#pragma unroll
        for (int t = 0; t < DT; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int d = 16 * t + 4 * g + r;
                if (d < R.Da && col < R.Db) S[(int64_t)d * R.Db + col] = X[t][r];
            }
    }
}

// Carries X across pieces in place: slot s holds piece s-1's own X (the first
// with the initial state in it) and gets sum_{s' < s} a^(L (s-1-s')) of them, L
// rows to a piece.  E: values of one
// workgroup's X.
__global__ __launch_bounds__(256) void lin_carry_kernel(LinArgs a, int E) {
    constexpr int kAhead = 16;  // pieces loaded at a time
    const int slots = a.nseg * a.subs, last = (a.nseg - 1) * a.subs;
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t per = (int64_t)a.B * a.NH * a.slices * E;
    if (i >= per * a.nroles) return;
    const Role &R = a.role[i / per];
    const int64_t j = i % per, wg = j / E;
    const int h = (int)(wg / a.slices % a.NH);
    const float f = __builtin_amdgcn_exp2f(log2_decay(a.g[h]) * (float)a.sub_rows);
    float *p = R.part + wg * slots * E + j % E;
    float X = 0.0f;
    for (int s = 1; s <= last; s += kAhead) {
        float own[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) own[u] = p[(int64_t)min(s + u, last) * E];
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
            if (s + u <= last) p[(int64_t)(s + u) * E] = X = f * X + own[u];
    }
}

// Gradients of a shared head: the sum over its `grp` heads, in order; V values
// of one head to a thread, dk in the first workgroups and dv in the rest.
struct ShareArgs {
    const float *in[2];
    void *out[2];
    int64_t n[2];  // outputs / V
    int D[2], grp;
};
template <typename T, int V>
__global__ __launch_bounds__(256) void lin_share_kernel(ShareArgs a, unsigned blocks0) {
    const int which = blockIdx.x >= blocks0;
    const int64_t i = (int64_t)(blockIdx.x - (which ? blocks0 : 0)) * 256 + threadIdx.x;
    if (i >= a.n[which]) return;
    const int per = a.D[which] / V;
    const int64_t head = i / per;
    const Unit<float, V> *p = (const Unit<float, V> *)a.in[which] + head * a.grp * per + i % per;
    Unit<float, V> s = p[0];
    for (int j = 1; j < a.grp; ++j) {
        const Unit<float, V> x = p[(int64_t)j * per];
#pragma unroll
        for (int e = 0; e < V; ++e) s.v[e] += x.v[e];
    }
    Unit<T, V> o;
#pragma unroll
    for (int e = 0; e < V; ++e) o.v[e] = from_f32<T>(s.v[e]);
    ((Unit<T, V> *)a.out[which])[i] = o;
}

constexpr int kStepCols = 64;

// One token: S' = a S + k^T v, o = scale q S'.  A workgroup owns 64 columns of
// a (row, head)'s state, 16 lanes of 4 columns by 16 groups of rows.
template <typename T, bool VEC>
__global__ __launch_bounds__(256) void lin_step_kernel(LinDims d, LinSeq q, LinSeq k, LinSeq v,
                                                       const float *g, float scale, const float *S0,
                                                       T *o, float *S1, int slices) {
    __shared__ float sum[16][kStepCols];
    const int bh = blockIdx.x / slices, col0 = (blockIdx.x % slices) * kStepCols;
    const int b = bh / d.NH, h = bh % d.NH, hk = h / (d.NH / d.NKV);
    const int lane = threadIdx.x & 15, grp = threadIdx.x >> 4;
    const T *qp = (const T *)q.p + (int64_t)b * q.sb + (int64_t)h * d.Dk;
    const T *kp = (const T *)k.p + (int64_t)b * k.sb + (int64_t)hk * d.Dk;
    const T *vp = (const T *)v.p + (int64_t)b * v.sb + (int64_t)hk * d.Dv;
    const float a = exp_fast(g[h]);
    const int c = col0 + 4 * lane, n = min(d.Dv - c, 4);
    float vv[4], acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int e = 0; e < 4; ++e) vv[e] = e < n ? to_f32<T>(vp[c + e]) : 0.0f;
    const int64_t base = (int64_t)bh * d.Dk * d.Dv + c;
#pragma unroll 4
    for (int r = grp; r < d.Dk; r += 16) {
        const float kk = to_f32<T>(kp[r]), qq = to_f32<T>(qp[r]);
        const int64_t at = base + (int64_t)r * d.Dv;
        float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        if (S0) {
            if constexpr (VEC) {
                if (n > 0) {
                    const float4 w = *(const float4 *)(S0 + at);
                    s[0] = w.x; s[1] = w.y; s[2] = w.z; s[3] = w.w;
                }
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (e < n) s[e] = S0[at + e];
            }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            s[e] = a * s[e] + kk * vv[e];
            acc[e] += qq * s[e];
        }
        if (S1) {
            if constexpr (VEC) {
                if (n > 0) *(float4 *)(S1 + at) = make_float4(s[0], s[1], s[2], s[3]);
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (e < n) S1[at + e] = s[e];
            }
        }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) sum[grp][4 * lane + e] = acc[e];
    __syncthreads();
    if (threadIdx.x < kStepCols && col0 + (int)threadIdx.x < d.Dv) {
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i) s += sum[i][threadIdx.x];
        o[((int64_t)b * d.NH + h) * d.Dv + col0 + threadIdx.x] = from_f32<T>(s * scale);
    }
}

// ------------------------------------------------------------------- host
size_t up(size_t v) { return (v + 255) & ~(size_t)255; }
int pad_depth(int d) { return d <= 32 ? 32 : d <= 64 ? 64 : d <= 128 ? 128 : 256; }
// Waves (of 16 columns) of a workgroup: eight where there are the columns, as
// they share P and the staged x and y.
int waves_of(int Db) { return Db > 64 ? 8 : 4; }
int slices_of(int Db, int NW) { return (Db + 16 * NW - 1) / (16 * NW); }

// Segments: enough workgroups for the chip's 256 CUs, one of eight waves or
// three of four to a CU, and at least two chunks to a segment, which costs
// another pass over y and z and a state.  That pass cuts a segment into pieces
// where there are few of them.  Measured, us, for the workgroups aimed at:
//   eight waves, bf16 D128                 256    512
//     T1024 B16 NH6                         66     70
//     T4096 B2 NH8                          54     63
//     backward T1000 B8 NH8:4              104    118
//   four waves, D64                        256    512    768   1024
//     bf16 T8191 B1 NH12                  45.5   40.2   39.1   38.5
//     bf16 T4096 B2 NH4                   27.6   28.9   28.9   28.7
//     bf16 backward T8191 B1 NH12         94.9   70.2   67.3   73.3
//     float32 T8191 B1 NH12               59.5   56.3   55.0   54.9
//     float32 T1024 B16 NH12              84.8   91.1   82.5   93.7
struct Cut {
    int nseg, subs, rows;  // rows of a piece
};
Cut cut(int T, int C, long wgs, int NW) {
    const int chunks = (T + C - 1) / C;
    const long target = NW == 8 ? 256 : 768;
    long want = std::max(1L, target / std::max(1L, wgs));
    want = std::min(want, (long)std::max(1, chunks / 2));
    const int per = (int)((chunks + want - 1) / want);
    const int nseg = (chunks + per - 1) / per;
    if (nseg == 1) return {1, 1, per * C};
    long subs = std::max(1L, target / (wgs * (nseg - 1)));
    subs = std::min(subs, (long)per);
    const int rows = (int)((per + subs - 1) / subs);
    subs = (per + rows - 1) / rows;
    const int whole = (int)subs * rows;  // chunks of a segment, rounded up to its pieces
    return {(chunks + whole - 1) / whole, (int)subs, rows * C};
}

size_t part_bytes(const LinDims &d, int DA, int NW, int slices, const Cut &c) {
    return c.nseg > 1 ? up(sizeof(float) * (size_t)d.B * d.NH * slices * c.nseg * c.subs * DA * 16 * NW) : 0;
}

// Workgroups of a launch over `segs` segments: the slices of eight (role, row,
// head, segment) go together.
long lin_blocks(int nroles, int B, int NH, int segs, int slices) {
    return ((long)nroles * B * NH * segs + 7) / 8 * 8 * slices;
}

template <typename T, int DA, int NW, bool STATE, bool FAST>
hipError_t lin_launch(const LinArgs &a, hipStream_t s) {
    constexpr size_t lds = Lds<T, DA, NW, STATE>::bytes;
    static std::once_flag once;
    static hipError_t attr = hipSuccess;
    std::call_once(once, [] {
        attr = hipFuncSetAttribute(reinterpret_cast<const void *>(&lin_kernel<T, DA, NW, STATE, FAST>),
                                   hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
    });
    if (attr != hipSuccess) return attr;
    const long blocks =
        lin_blocks(a.nroles, a.B, a.NH, STATE ? (a.nseg - 1) * a.subs : a.nseg, a.slices);
    hipLaunchKernelGGL((lin_kernel<T, DA, NW, STATE, FAST>), dim3((unsigned)blocks), dim3(64 * NW), lds, s,
                       a);
    return hipGetLastError();
}

template <typename T, int DA, int NW, bool FAST>
hipError_t lin_run(const LinArgs &a, hipStream_t s) {
    if (a.nseg > 1) {
        hipError_t e = lin_launch<T, DA, NW, true, FAST>(a, s);
        if (e != hipSuccess) return e;
        if (!folds(a)) {
            const int E = DA * 16 * NW;
            const long n = (long)a.nroles * a.B * a.NH * a.slices * E;
            hipLaunchKernelGGL(lin_carry_kernel, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, s, a, E);
            e = hipGetLastError();
            if (e != hipSuccess) return e;
        }
    }
    return lin_launch<T, DA, NW, false, FAST>(a, s);
}

template <typename T, int NW, bool FAST>
hipError_t lin_run_depth(const LinArgs &a, int DA, hipStream_t s) {
    switch (DA) {
        case 32: return lin_run<T, 32, NW, FAST>(a, s);
        case 64: return lin_run<T, 64, NW, FAST>(a, s);
        case 128: return lin_run<T, 128, NW, FAST>(a, s);
        default: return lin_run<T, 256, NW, FAST>(a, s);
    }
}

template <typename T>
hipError_t lin_run_type(const LinArgs &a, int DA, int NW, hipStream_t s) {
    bool fast = true;
    for (int i = 0; i < a.nroles; ++i) {
        const Role &r = a.role[i];
        fast = fast && r.Db % 16 == 0 && pieces_ok<T>(r.x, r.Da) && pieces_ok<T>(r.y, r.Da) &&
               pieces_ok<T>(r.z, r.Db);
    }
    if (NW == 8) return fast ? lin_run_depth<T, 8, true>(a, DA, s) : lin_run_depth<T, 8, false>(a, DA, s);
    return fast ? lin_run_depth<T, 4, true>(a, DA, s) : lin_run_depth<T, 4, false>(a, DA, s);
}

hipError_t lin_run_any(const LinArgs &a, bool bf16, int DA, int NW, hipStream_t s) {
    return bf16 ? lin_run_type<uint16_t>(a, DA, NW, s) : lin_run_type<float>(a, DA, NW, s);
}

int chunk_of(bool bf16) { return bf16 ? Shape<uint16_t>::C : Shape<float>::C; }

// The backward's launches: roles with the same padded depth share one.
struct BwdPlan {
    int n;             // launches
    int roles[2];      // roles of each
    int DA[2], NW[2], slices[2];
    Cut c[2];
    size_t part[2], shared_k, shared_v, total;
};
BwdPlan bwd_plan(const LinDims &d, bool bf16) {
    BwdPlan p{};
    // dq, dk: depth Dv, columns Dk;  dv: depth Dk, columns Dv
    const int da = pad_depth(d.Dv), db = pad_depth(d.Dk), C = chunk_of(bf16);
    const long bh = (long)d.B * d.NH;
    size_t off = 0;
    if (da == db) {
        const int D = std::max(d.Dk, d.Dv);
        p.n = 1;
        p.roles[0] = 3;
        p.DA[0] = da;
        p.NW[0] = waves_of(D);
        p.slices[0] = slices_of(D, p.NW[0]);
    } else {
        p.n = 2;
        p.roles[0] = 2;
        p.DA[0] = da;
        p.NW[0] = waves_of(d.Dk);
        p.slices[0] = slices_of(d.Dk, p.NW[0]);
        p.roles[1] = 1;
        p.DA[1] = db;
        p.NW[1] = waves_of(d.Dv);
        p.slices[1] = slices_of(d.Dv, p.NW[1]);
    }
    for (int i = 0; i < p.n; ++i) {
        p.c[i] = cut(d.T, C, bh * p.slices[i] * p.roles[i], p.NW[i]);
        p.part[i] = off;
        off += p.roles[i] * part_bytes(d, p.DA[i], p.NW[i], p.slices[i], p.c[i]);
    }
    p.shared_k = p.shared_v = off;
    if (d.NH != d.NKV) {
        const size_t n = (size_t)d.T * d.B * d.NH;
        p.shared_k = off; off += up(sizeof(float) * n * d.Dk);
        p.shared_v = off; off += up(sizeof(float) * n * d.Dv);
    }
    p.total = off;
    return p;
}

// Values of a head to a thread, and the workgroups of one array's n outputs.
int share_unit(const LinDims &d) { return d.Dk % 4 == 0 && d.Dv % 4 == 0 ? 4 : 1; }
long share_blocks(int64_t n, int V) { return (long)((n / V + 255) / 256); }

template <typename T, int V>
hipError_t share(ShareArgs a, hipStream_t s) {
    const long b0 = share_blocks(a.n[0], V), b1 = share_blocks(a.n[1], V);
    for (int i = 0; i < 2; ++i) a.n[i] /= V;
    hipLaunchKernelGGL((lin_share_kernel<T, V>), dim3((unsigned)(b0 + b1)), dim3(256), 0, s, a, (unsigned)b0);
    return hipGetLastError();
}

int step_slices(const LinDims &d) { return (d.Dv + kStepCols - 1) / kStepCols; }

}  // namespace

bool lin_step_grid_ok(const LinDims &d) { return grid_ok((long)d.B * d.NH * step_slices(d), 256); }

// The main launches only: those of the states have at most the 768 workgroups
// that cut() aims at for each segment, the carries a thread for a value of
// their X.
bool lin_fwd_grid_ok(const LinDims &d, bool bf16) {
    if (d.T == 1) return lin_step_grid_ok(d);
    const int NW = waves_of(d.Dv), sl = slices_of(d.Dv, NW);
    const Cut c = cut(d.T, chunk_of(bf16), (long)d.B * d.NH * sl, NW);
    return grid_ok(lin_blocks(1, d.B, d.NH, c.nseg, sl), 64 * NW);
}

bool lin_bwd_grid_ok(const LinDims &d, bool bf16) {
    const BwdPlan p = bwd_plan(d, bf16);
    for (int i = 0; i < p.n; ++i)
        if (!grid_ok(lin_blocks(p.roles[i], d.B, d.NH, p.c[i].nseg, p.slices[i]), 64 * p.NW[i])) return false;
    const int64_t n = (int64_t)d.T * d.B * d.NKV;
    const int V = share_unit(d);
    return d.NH == d.NKV || grid_ok(share_blocks(n * d.Dk, V) + share_blocks(n * d.Dv, V), 256);
}

size_t lin_fwd_bytes(const LinDims &d, bool bf16) {
    const int DA = pad_depth(d.Dk), NW = waves_of(d.Dv), sl = slices_of(d.Dv, NW);
    return part_bytes(d, DA, NW, sl, cut(d.T, chunk_of(bf16), (long)d.B * d.NH * sl, NW));
}

size_t lin_bwd_bytes(const LinDims &d, bool bf16) { return bwd_plan(d, bf16).total; }

hipError_t launch_lin_step(const LinDims &d, bool bf16, LinSeq q, LinSeq k, LinSeq v,
                           const float *g, float scale, const float *S0, void *o, float *S1,
                           hipStream_t s) {
    const int sl = step_slices(d);
    const dim3 grid((unsigned)((long)d.B * d.NH * sl)), thr(256);
    const bool vec = d.Dv % 4 == 0;
    if (bf16 && vec)
        hipLaunchKernelGGL((lin_step_kernel<uint16_t, true>), grid, thr, 0, s, d, q, k, v, g, scale,
                           S0, (uint16_t *)o, S1, sl);
    else if (bf16)
        hipLaunchKernelGGL((lin_step_kernel<uint16_t, false>), grid, thr, 0, s, d, q, k, v, g, scale,
                           S0, (uint16_t *)o, S1, sl);
    else if (vec)
        hipLaunchKernelGGL((lin_step_kernel<float, true>), grid, thr, 0, s, d, q, k, v, g, scale, S0,
                           (float *)o, S1, sl);
    else
        hipLaunchKernelGGL((lin_step_kernel<float, false>), grid, thr, 0, s, d, q, k, v, g, scale, S0,
                           (float *)o, S1, sl);
    return hipGetLastError();
}

hipError_t launch_lin_fwd(const LinDims &d, bool bf16, LinSeq q, LinSeq k, LinSeq v,
                          const float *g, float scale, const float *S0, void *o, float *ST,
                          void *ws, hipStream_t s) {
    if (d.T == 1) return launch_lin_step(d, bf16, q, k, v, g, scale, S0, o, ST, s);
    LinArgs a{};
    const int grp = d.NH / d.NKV, DA = pad_depth(d.Dk), NW = waves_of(d.Dv);
    a.nroles = 1;
    a.T = d.T; a.B = d.B; a.NH = d.NH;
    a.g = g;
    a.slices = slices_of(d.Dv, NW);
    const Cut c = cut(d.T, chunk_of(bf16), (long)d.B * d.NH * a.slices, NW);
    a.nseg = c.nseg;
    a.subs = c.subs;
    a.sub_rows = c.rows;
    a.role[0] = Role{q, k, v, 1, grp, grp, d.Dk, d.Dv, S0, 0, 1, ST, 1, 0, 1.0f, scale, o, 0,
                     (float *)ws};
    return lin_run_any(a, bf16, DA, NW, s);
}

hipError_t launch_lin_bwd(const LinDims &d, bool bf16, LinSeq q, LinSeq k, LinSeq v,
                          const float *g, float scale, const float *S0, LinSeq dO,
                          const float *dST, void *dq, void *dk, void *dv, float *dS0, void *ws,
                          hipStream_t s) {
    const BwdPlan p = bwd_plan(d, bf16);
    const int grp = d.NH / d.NKV;
    char *base = (char *)ws;
    float *pk = (float *)(base + p.shared_k), *pv = (float *)(base + p.shared_v);
    const Role rq{dO, v, k, 1, grp, grp, d.Dv, d.Dk, S0, 1, 1, nullptr, 0, 0, 1.0f, scale, dq, 0, nullptr};
    const Role rk{v, dO, q, grp, 1, 1, d.Dv, d.Dk, dST, 1, 0, nullptr, 0, 1, scale, 1.0f,
                  grp > 1 ? (void *)pk : dk, grp > 1, nullptr};
    const Role rv{k, q, dO, grp, 1, 1, d.Dk, d.Dv, dST, 0, 0, dS0, 0, 1, scale, 1.0f,
                  grp > 1 ? (void *)pv : dv, grp > 1, nullptr};
    const Role *order[3] = {&rq, &rk, &rv};
    int next = 0;
    for (int i = 0; i < p.n; ++i) {
        LinArgs a{};
        a.nroles = p.roles[i];
        a.T = d.T; a.B = d.B; a.NH = d.NH;
        a.g = g;
        a.slices = p.slices[i];
        a.nseg = p.c[i].nseg;
        a.subs = p.c[i].subs;
        a.sub_rows = p.c[i].rows;
        const size_t each = part_bytes(d, p.DA[i], p.NW[i], p.slices[i], p.c[i]);
        for (int j = 0; j < a.nroles; ++j) {
            a.role[j] = *order[next++];
            a.role[j].part = (float *)(base + p.part[i] + j * each);
        }
        hipError_t e = lin_run_any(a, bf16, p.DA[i], p.NW[i], s);
        if (e != hipSuccess) return e;
    }
    if (grp > 1) {
        const int64_t n = (int64_t)d.T * d.B * d.NKV;
        const ShareArgs a{{pk, pv}, {dk, dv}, {n * d.Dk, n * d.Dv}, {d.Dk, d.Dv}, grp};
        if (share_unit(d) == 4)
            return bf16 ? share<uint16_t, 4>(a, s) : share<float, 4>(a, s);
        return bf16 ? share<uint16_t, 1>(a, s) : share<float, 1>(a, s);
    }
    return hipSuccess;
}

}  // namespace lm
}  // namespace rnn355
