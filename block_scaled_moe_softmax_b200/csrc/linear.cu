// linear.cu -- out = act(x w^T + bias) + residual and its gradient, dense or over the segments of
// the grouped layout (segment e: rows pad_offsets[e] .. + counts[e], a multiple of 128 apart, with
// weights w[e] and bias[e]; the rows behind counts[e] are neither read into a result nor written).
//
//   z = x w^T + b          dz = dout * act'(z)
//   out = act(z) + res     dx = dz w      dw = dz^T x      db = sum over rows of dz
//
// dz is rounded once to the operands' type, which the products take (db sums it before that).  float32 dout
// of float16 operands may lie outside float16's range, so dz is scaled by a power of two before that rounding,
// one of each segment, and the products' sums by its inverse.
#include "../../include/moe_mx.h"
#include "host.cuh"
#include "kernels.cuh"
#include "pair.cuh"
#include "routed.cuh"
#include "vec.cuh"

#include <type_traits>

namespace moe_mx {

namespace {

// ---------------------------------------------------------------- activations
// 1 / (1 + e^-v) to a few parts in 2^24, and far below 0 as if v were off by a few parts in 2^24 of its own
// (|v| 2^-23 of the result, as much as rounding v itself moves it): __expf rounds its argument's product with
// log2(e).  0 once e^-v overflows.
__device__ __forceinline__ float sigmoid(float v) { return __fdividef(1.f, 1.f + __expf(-v)); }

// gelu in its tanh form: 0.5 z (1 + tanh u) = z sigmoid(2u), u = sqrt(2/pi) (z + 0.044715 z^3)
constexpr float kGelu2A = 1.5957691216057308f; // 2 sqrt(2/pi)
constexpr float kGeluC = 0.044715f;

__device__ __forceinline__ float act_fwd(float z, int act)
{
    if (act == kActSilu)
        return z * sigmoid(z);
    if (act == kActGelu)
        return z * sigmoid(kGelu2A * (z + kGeluC * z * z * z));
    return z;
}

__device__ __forceinline__ float act_grad(float z, int act)
{
    if (act == kActSilu) {
        const float q = sigmoid(z);
        return q * (1.f + z * (1.f - q));
    }
    if (act == kActGelu) {
        const float q = sigmoid(kGelu2A * (z + kGeluC * z * z * z));
        const float qq = q * (1.f - q); // 0 far from 0, where z * z may overflow
        return qq == 0.f ? q : q + z * qq * kGelu2A * (1.f + 3.f * kGeluC * z * z);
    }
    return 1.f;
}

// ---------------------------------------------------------------- segments
struct Segments {
    const int32_t *counts, *pad_offsets;
    int E; // 0: one dense segment of M rows
    int64_t M;
};

// Valid rows of expert e's segment, and its first row (none of a segment that starts outside the buffer).
__device__ __forceinline__ int segment_rows(const Segments &s, int e, int &first)
{
    first = s.pad_offsets[e];
    if (first < 0 || first >= s.M)
        return 0;
    return max(0, min(s.counts[e], (int)(s.M - first)));
}

// The segment holding row `r0` (a multiple of 64): its expert, and the end of its valid rows.
__device__ __forceinline__ bool find_segment(const Segments &s, int64_t r0, int &e, int64_t &end)
{
    e = 0;
    if (s.E == 0) {
        end = s.M;
        return r0 < s.M;
    }
    int lo = 0, hi = s.E; // the last e with pad_offsets[e] <= r0
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (s.pad_offsets[mid] <= r0)
            lo = mid;
        else
            hi = mid;
    }
    e = lo;
    int first;
    const int rows = segment_rows(s, e, first);
    end = (int64_t)first + rows;
    return r0 >= first && r0 < end;
}

template <typename F> void by_half(int type, F f)
{
    if (type == kTypeF16)
        f(__half());
    else
        f(__nv_bfloat16());
}

// ---------------------------------------------------------------- matrix product
// D[m, n] = sum_k A[m, k] B[n, k] on tcgen05, two CTAs to a 256 x BN tile (cta_group::2): each holds
// 128 rows of A and half of B's rows in shared memory and 128 rows of the accumulator in its TMEM.
// Warp 0 (and warp 2) copies 64-deep k blocks of A and B in with TMA, warp 1 of the leader issues the MMAs,
// warps 4..11 take a finished accumulator out while the next tile's runs in the other half of TMEM,
// and warp 3 finds the tiles ahead of them all (kAhead).  (One warp that found its tiles and issued four copies a
// k block took 0.3 us a block and 1.1 us a tile: longer than the MMAs of a short product.)
//
// Operands with k contiguous (x and w of the forward pass, dz in dx) are K-major tiles; those with
// k along the rows (w in dx; dz and x in dw) are read as they lie, as M- or N-major tiles.
//
// kSwap computes the transpose of a tile: 256 weight rows are the A operand and the tokens the B
// operand, as many of them (a multiple of 32, up to 256) as the tile has.  A segment of 40 tokens then
// costs the MMAs of 64 tokens and loads no rows of padding, where a tile of 256 token rows takes all
// of them: the grouped products and small dense ones run so.
struct Gemm {
    Segments seg;
    int seg_k;            // the segments run over k (dw) instead of the rows
    int M, n_cols, K;     // rows and columns of D, depth (dense, or of a rows-segmented product)
    int kb_split;         // k blocks of one split (dense only), split s writes plane s of out
    int mt, nt, splits;   // tiles of a dense product, or of one expert's when the segments run over k
    int tok;              // kSwap, dense: tokens of a tile
    int gated;            // swiglu: gate and up rows in one tile (of B halves; kSwap: 16 by 16 rows of A)
    int fmt;              // 0: f16, 1: bf16
    int run_log;          // log2 of the k blocks that one accumulator sums (!kSum)
    // epilogue
    const float *bias;
    const void *residual;
    void *out, *preact;
    int act, N;           // columns of preact, and of each expert's bias
    int type, out_type, vec;
    int wide_a, wide_b;   // an M- or N-major operand of whole 64-element groups: one copy takes all of them
    const float *unscale; // a gradient's factor of each expert's sums, or nullptr
    int64_t d_expert;     // elements from one expert's D to the next's (seg_k)
    float4 *held;         // sums of tiles of more than one run, kHeld of every epilogue warp (kHeldBytes in all)
};

constexpr int kTileM = 256, kBk = 64, kMaxSeg = kMaxExperts;
constexpr int kThreads = 384, kEpiWarps = 8;
constexpr int kPairs = 74; // SM pairs of the 148-SM part the plans are made for
constexpr int kHeldChunk = 32 * 32 / 4, kHeld = 4 * kHeldChunk; // float4s of 32 x 32 values; of a warp's four
constexpr int64_t kHeldBytes = (int64_t)kPairs * 2 * kEpiWarps * kHeld * 16;
constexpr int kRing = 4, kTileInts = 12; // tiles decoded ahead, and the words of one
constexpr unsigned long long kWaitNs = 2000000000ull, kDrainNs = 200000000ull;

template <int BN, bool kSwap> struct Cfg {
    static constexpr int kABytes = 128 * kBk * 2, kBBytes = BN / 2 * kBk * 2, kStage = kABytes + kBBytes;
    // BN = 256: the experts' tile counts take the sixth stage's room where rows are segmented
    static constexpr bool kPrefix = kSwap || BN == 128;
    static constexpr int kStages = BN == 256 ? (kPrefix ? 5 : 6) : BN == 192 ? 6 : 7;
    static constexpr int kOffEpi = kStages * kStage, kOffBar = kOffEpi + kEpiWarps * 4096;
    // barriers: full, empty per stage, 2 acc_full, 2 acc_empty, mma_done, and full, empty of the tile ring;
    // then the TMEM address, the ring, and the experts' tile counts
    static constexpr int kNumBar = 2 * kStages + 5 + 2 * kRing;
    static constexpr int kOffRing = (kOffBar + kNumBar * 8 + 8 + 15) / 16 * 16;
    static constexpr int kOffPrefix = kOffRing + kRing * kTileInts * 4;
    static constexpr int kSmem = kOffPrefix + (kPrefix ? (kMaxSeg + 1) * 4 : 0) + 1024; // + alignment of the base
    static_assert(kSmem <= 227 * 1024, "shared memory of one CTA");
};

struct Tile {
    int e, row, row_end; // first row of D, and the end of the rows that are stored
    int n0;              // first column of D
    int k0, nkb, rem;    // first k (element), k blocks, valid rows of the last (0: all)
    int split;
    int tok;             // kSwap: tokens of the tile, a multiple of 32
};

// Token tiles of a segment, equally long: at most `most` tokens each, rounded up to 32.
__device__ __forceinline__ int token_tiles(int rows, int most, int &tok)
{
    const int tiles = (rows + most - 1) / most;
    tok = tiles ? ((rows + tiles - 1) / tiles + 31) / 32 * 32 : 0;
    return tiles;
}

// The t-th tile.  Rows-segmented: prefix[e] holds the number of tiles of the experts before e, tiles run
// over an expert's row tiles first, so that neighbouring pairs read the same weights.
template <int BN, bool kSwap, int kMostTok>
__device__ __forceinline__ bool get_tile(const Gemm &g, const int32_t *prefix, int t, Tile &o)
{
    const int bn = g.gated ? (kSwap ? 128 : BN / 2) : BN; // columns of D in a tile
    o.rem = 0, o.split = 0;
    if (g.seg.E == 0) {
        const int per = g.mt * g.nt;
        o.split = t / per;
        if (o.split >= g.splits)
            return false;
        t -= o.split * per;
        o.e = 0, o.row = t % g.mt * (kSwap ? g.tok : kTileM), o.row_end = g.M, o.n0 = t / g.mt * bn;
        o.tok = min(g.tok, (g.M - o.row + 31) / 32 * 32);
        const int kb = (g.K + kBk - 1) / kBk, lo = o.split * g.kb_split;
        o.k0 = lo * kBk, o.nkb = min(g.kb_split, kb - lo);
        return true;
    }
    if (!kSwap && g.seg_k) {
        const int per = g.mt * g.nt;
        o.e = t / per;
        if (o.e >= g.seg.E)
            return false;
        t -= o.e * per;
        o.row = t % g.mt * kTileM, o.row_end = g.M, o.n0 = t / g.mt * bn;
        int first;
        const int rows = segment_rows(g.seg, o.e, first);
        o.k0 = first, o.nkb = (rows + kBk - 1) / kBk, o.rem = rows % kBk;
        return true;
    }
    if (t >= prefix[g.seg.E])
        return false;
    int lo = 0, hi = g.seg.E; // the last e with prefix[e] <= t
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (prefix[mid] <= t)
            lo = mid;
        else
            hi = mid;
    }
    int first, tok = kTileM;
    const int rows = segment_rows(g.seg, lo, first);
    const int mt = kSwap ? token_tiles(rows, kMostTok, tok) : (rows + kTileM - 1) / kTileM;
    t -= prefix[lo];
    o.e = lo, o.row = first + t % mt * tok, o.row_end = first + rows, o.n0 = t / mt * bn;
    o.tok = min(tok, (o.row_end - o.row + 31) / 32 * 32);
    o.k0 = 0, o.nkb = (g.K + kBk - 1) / kBk;
    return true;
}

// What the epilogue of a product needs (shared by the kernels).
struct Epi {
    const float *bias;    // of this expert, or nullptr
    const void *residual;
    void *out, *preact;
    int act, N, n_cols, type, out_type, vec;
};

// R rows of 8 columns from column n: offsets of the first in out (and residual) and in preact, elements
// from one to the next, and which are stored (bit j).
struct Rows {
    size_t o, po;
    int so, spo, n;
    uint32_t ok;
    __device__ __forceinline__ bool has(int j) const { return (ok >> j) & 1u; }
    __device__ __forceinline__ size_t at(int j) const { return o + (size_t)j * so; }
};

// Residual values (16-bit) of R rows x 8 columns, loaded ahead of their use.
template <int R> struct Ahead {
    uint4 a[R];
    __device__ __forceinline__ void load(const Epi &g, const Rows &w)
    {
        if (!g.residual)
            return;
        const uint16_t *p = static_cast<const uint16_t *>(g.residual);
#pragma unroll
        for (int j = 0; j < R; ++j)
            if (w.has(j))
                a[j] = *reinterpret_cast<const uint4 *>(p + w.at(j));
    }
};

template <typename T, int R> __device__ __forceinline__ void add_rows(const Ahead<R> &ahead, float (&v)[R][8])
{
#pragma unroll
    for (int j = 0; j < R; ++j) {
        Raw<T, 8> r;
        float f[8];
        r.v = ahead.a[j];
        r.get(f);
#pragma unroll
        for (int i = 0; i < 8; ++i) // rows not stored hold what they hold
            v[j][i] += f[i];
    }
}

template <typename T, int R>
__device__ __forceinline__ void put_rows(T *p, int step, const Rows &w, const float (&v)[R][8])
{
#pragma unroll
    for (int j = 0; j < R; ++j)
        if (w.has(j))
            Raw<T, 8>::put(p + (size_t)j * step, v[j]);
}

template <int R>
__device__ __forceinline__ void put_preact(size_t off, const Epi &g, const Rows &w, const float (&v)[R][8])
{
    if (g.type == kTypeF16)
        put_rows<__half, R>(static_cast<__half *>(g.preact) + off, w.spo, w, v);
    else
        put_rows<__nv_bfloat16, R>(static_cast<__nv_bfloat16 *>(g.preact) + off, w.spo, w, v);
}

template <int R> __device__ __forceinline__ void add_bias(const float *b, const Epi &g, const Rows &w, float (&v)[R][8])
{
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float f = w.n + i < g.n_cols ? b[w.n + i] : 0.f;
#pragma unroll
        for (int j = 0; j < R; ++j)
            v[j][i] += f;
    }
}

// Bias, preact, activation, residual and store of z (kGated: swiglu, with up).  Every choice is made
// once for all rows: choosing per value cost 3000 cycles per 32 x 32 block in branches alone.
template <int R, bool kGated>
__device__ __forceinline__ void finish(const Epi &g, const Rows &w, float (&z)[R][8], float (&up)[R][8],
                                       const Ahead<R> &ahead)
{
    if (g.bias) {
        add_bias<R>(g.bias, g, w, z);
        if (kGated)
            add_bias<R>(g.bias + g.n_cols, g, w, up);
    }
    if (g.preact) {
        put_preact<R>(w.po, g, w, z);
        if (kGated)
            put_preact<R>(w.po + g.n_cols, g, w, up);
    }
    if (kGated) {
#pragma unroll
        for (int j = 0; j < R; ++j)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                z[j][i] *= sigmoid(z[j][i]) * up[j][i];
    } else if (g.act == kActSilu) {
#pragma unroll
        for (int j = 0; j < R; ++j)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                z[j][i] = act_fwd(z[j][i], kActSilu);
    } else if (g.act == kActGelu) {
#pragma unroll
        for (int j = 0; j < R; ++j)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                z[j][i] = act_fwd(z[j][i], kActGelu);
    }
    if (g.out_type == kTypeF16) {
        if (g.residual)
            add_rows<__half, R>(ahead, z);
        put_rows<__half, R>(static_cast<__half *>(g.out) + w.o, w.so, w, z);
    } else {
        if (g.residual)
            add_rows<__nv_bfloat16, R>(ahead, z);
        put_rows<__nv_bfloat16, R>(static_cast<__nv_bfloat16 *>(g.out) + w.o, w.so, w, z);
    }
}

template <typename T>
__device__ __forceinline__ void put_column(void *out, size_t off, int step, int rows, const float (&v)[32])
{
    T *p = static_cast<T *>(out) + off;
#pragma unroll
    for (int x = 0; x < 32; ++x, p += step)
        if (x < rows)
            *p = from_f32<T>(v[x]);
}

template <typename T> __device__ __forceinline__ void add_column(const void *res, size_t off, int step, int rows, float (&v)[32])
{
    const T *p = static_cast<const T *>(res) + off;
#pragma unroll
    for (int x = 0; x < 32; x += 16) { // sixteen loads at a time
        T f[16];
#pragma unroll
        for (int i = 0; i < 16; ++i, p += step)
            f[i] = x + i < rows ? *p : from_f32<T>(0.f);
#pragma unroll
        for (int i = 0; i < 16; ++i)
            v[x + i] += to_f32<T>(f[i]);
    }
}

template <typename T>
__device__ __forceinline__ void end_column(const Epi &g, size_t off, int rows, float (&v)[32])
{
    if (g.residual)
        add_column<T>(g.residual, off, g.n_cols, rows, v);
    put_column<T>(g.out, off, g.n_cols, rows, v);
}

// The same for float32 outputs and for those whose rows do not start on 16 bytes: a lane has column n of
// `rows` rows (0: none) from row m, so that a warp's store is a piece of one row.  With eight columns a lane,
// ragged ones were stored one at a time, 32 pieces of eight rows: 780 rows by 912 -> 1470 18 us, 10 us so (9 us
// at 1472).  Aligned float32 rows, eight columns a lane in two 16-byte stores: 483 rows by 872 -> 384 11.3 us,
// 9.8 us so.  d: where the output starts.
template <bool kGated>
__device__ __forceinline__ void finish_column(const Epi &g, size_t d, int m, int n, int rows, float (&z)[32], float (&up)[32])
{
    if (rows <= 0)
        return;
    if (g.bias) {
        const float b = g.bias[n], bu = kGated ? g.bias[g.n_cols + n] : 0.f;
#pragma unroll
        for (int x = 0; x < 32; ++x) {
            z[x] += b;
            if (kGated)
                up[x] += bu;
        }
    }
    if (g.preact) {
        const size_t off = (size_t)m * g.N + n;
        if (g.type == kTypeF16) {
            put_column<__half>(g.preact, off, g.N, rows, z);
            if (kGated)
                put_column<__half>(g.preact, off + g.n_cols, g.N, rows, up);
        } else {
            put_column<__nv_bfloat16>(g.preact, off, g.N, rows, z);
            if (kGated)
                put_column<__nv_bfloat16>(g.preact, off + g.n_cols, g.N, rows, up);
        }
    }
    if (kGated) {
#pragma unroll
        for (int x = 0; x < 32; ++x)
            z[x] *= sigmoid(z[x]) * up[x];
    } else if (g.act == kActSilu) {
#pragma unroll
        for (int x = 0; x < 32; ++x)
            z[x] = act_fwd(z[x], kActSilu);
    } else if (g.act == kActGelu) {
#pragma unroll
        for (int x = 0; x < 32; ++x)
            z[x] = act_fwd(z[x], kActGelu);
    }
    const size_t off = d + (size_t)m * g.n_cols + n;
    if (g.out_type == kTypeF32)
        end_column<float>(g, off, rows, z);
    else if (g.out_type == kTypeF16)
        end_column<__half>(g, off, rows, z);
    else
        end_column<__nv_bfloat16>(g, off, rows, z);
}

// The same for one value: row m, column n.
template <typename T, bool kGated>
__device__ __forceinline__ void finish_value(const Epi &e, size_t m, int n, float z, float up)
{
    if (e.bias) {
        z += e.bias[n];
        if (kGated)
            up += e.bias[e.n_cols + n];
    }
    if (e.preact) {
        T *p = static_cast<T *>(e.preact) + m * e.N + n;
        *p = from_f32<T>(z);
        if (kGated)
            p[e.n_cols] = from_f32<T>(up);
    }
    float v = kGated ? z * sigmoid(z) * up : act_fwd(z, e.act);
    const size_t o = m * e.n_cols + n;
    if (e.out_type == kTypeF32) {
        if (e.residual)
            v += static_cast<const float *>(e.residual)[o];
        static_cast<float *>(e.out)[o] = v;
    } else {
        if (e.residual)
            v += to_f32<T>(static_cast<const T *>(e.residual)[o]);
        static_cast<T *>(e.out)[o] = from_f32<T>(v);
    }
}

// Bias and activation of 64 columns of one row from column n.
__device__ __forceinline__ void bias_act(const Epi &g, int n, uint32_t (&r0)[32], uint32_t (&r1)[32])
{
    if (g.bias) {
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            r0[i] = __float_as_uint(__uint_as_float(r0[i]) + (n + i < g.n_cols ? g.bias[n + i] : 0.f));
            r1[i] = __float_as_uint(__uint_as_float(r1[i]) + (n + 32 + i < g.n_cols ? g.bias[n + 32 + i] : 0.f));
        }
    }
    if (g.act == kActSilu) {
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            r0[i] = __float_as_uint(act_fwd(__uint_as_float(r0[i]), kActSilu));
            r1[i] = __float_as_uint(act_fwd(__uint_as_float(r1[i]), kActSilu));
        }
    } else if (g.act == kActGelu) {
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            r0[i] = __float_as_uint(act_fwd(__uint_as_float(r0[i]), kActGelu));
            r1[i] = __float_as_uint(act_fwd(__uint_as_float(r1[i]), kActGelu));
        }
    }
}

// The tensor core adds into its float32 accumulator by truncation: a chain over K = 7168 is off by
// 8e-6 in relative norm (measured), where a rounding sum is by 9e-7, and a sum of products of one sign by
// 6.5e-9 of itself per k.  Products with float32 outputs therefore hand the accumulator over every kChain k
// blocks (kSum) and the epilogue's warps keep the sum in registers.  Other products do so every 2^run_log
// k blocks, where such a chain is off by a ninth of half a step of the output's type (8192 of k and 5.3e-5 for
// float16, 65536 and 4.3e-4 for bf16), and keep the sum in the workspace (Gemm::held): dw sums over as many rows as
// there are, and in one chain of 300,000 rows of one sign a float16 one was off by 2e-3.  A handover costs
// about 9 us (4096 x 4096 weights' gradient over 65536 rows: 1510 us in one chain, 1570 in eight).
constexpr int kChain = 8;
inline int run_log(int type) { return type == kTypeF16 ? 7 : 10; }

// Recorded by a wait that gave up, until linear_status reads it.  No wait looks at it: a product that failed
// must not cut short the waits of a later call, or of one on another stream.
__device__ uint32_t g_linear_err;

__device__ __forceinline__ bool wait_phase(uint32_t bar, uint32_t parity)
{
    if (mbar_wait_bounded(bar, parity, nullptr, kWaitNs))
        return true;
    atomicOr(&g_linear_err, kErrTimeout);
    return false;
}

// kSwap: token rows in boxes of 16, 32 and 64 rows.  dw of grouped rows: each expert's last k block of
// A and of B with zeros behind its rows, 64 rows an expert (after_kernel).
struct MoreMaps {
    CUtensorMap m[3];
};

template <int BN, bool kAMn, bool kBMn, bool kSum, bool kSwap>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    gemm_kernel(const Gemm g, const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                const __grid_constant__ MoreMaps map_c)
{
    using C = Cfg<BN, kSwap>;
    constexpr bool kPlain = kSwap ? kAMn : kBMn;  // a gradient: no bias, preact, activation or residual
    constexpr int kMostTok = kSum ? 128 : 256;    // kSwap: tokens of a tile (kSum keeps them in registers)
    // M- or N-major operands may take two copies each: warp 2 issues B's (one warp for both is 2 % faster where
    // each is one copy)
    constexpr bool kSplit = kAMn || kBMn;
    // Tiles are found ahead by warp 3; dense products with k contiguous, whose tiles take no search, let each
    // warp find its own.  Measured: 8192 x 7168 x 2048 130 us so, 140 with warp 3; experts' products
    // (search, short k) 1 to 5 % faster with warp 3.
    constexpr bool kAhead = kSwap || kSplit || BN == 128;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    uint8_t *const sm = smem_raw + (base - smem_u32(smem_raw));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    constexpr int S = C::kStages;
    const uint32_t bar0 = base + C::kOffBar;
    auto full = [&](int s) { return bar0 + 8u * s; };
    auto empty = [&](int s) { return bar0 + 8u * (S + s); };
    auto acc_full = [&](int b) { return bar0 + 8u * (2 * S + b); };
    auto acc_empty = [&](int b) { return bar0 + 8u * (2 * S + 2 + b); };
    const uint32_t mma_done = bar0 + 8u * (2 * S + 4), tmem_slot = bar0 + 8u * C::kNumBar;
    auto tile_full = [&](uint32_t r) { return bar0 + 8u * (2 * S + 5 + r); };
    auto tile_empty = [&](uint32_t r) { return bar0 + 8u * (2 * S + 5 + kRing + r); };
    int4 *const ring = reinterpret_cast<int4 *>(sm + C::kOffRing);
    const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
    // A dense product's first tile depends on nothing in memory: found while the barriers are set up (its
    // divisions and the first reads of the arguments take most of a microsecond)
    Tile t;
    const bool early = g.seg.E == 0;
    bool some = early && get_tile<BN, kSwap, kMostTok>(g, nullptr, pair, t);
    int32_t *const prefix = reinterpret_cast<int32_t *>(sm + C::kOffPrefix); // kPrefix only

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(full(s), 2);  // each CTA's copies
            mbar_init(empty(s), 1); // the commit of the MMAs that read the stage
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(acc_full(b), 1);
            mbar_init(acc_empty(b), 2 * kEpiWarps);
        }
        mbar_init(mma_done, 1);
        for (int r = 0; r < kRing; ++r) {
            mbar_init(tile_full(r), 1);
            mbar_init(tile_empty(r), kEpiWarps + (rank == 0 ? 2 : 1) + (kSplit ? 1 : 0)); // the warps that read tiles
        }
        fence_mbar_init();
        prefetch_tensormap(&map_a);
        prefetch_tensormap(&map_b);
    }
    if (warp == 2)
        tmem_alloc_pair(tmem_slot, 512);
    grid_dep_wait(); // everything this kernel reads, and the buffers it writes
    tc_fence_before();
    __syncthreads();
    cluster_sync(); // barriers of both CTAs are set up
    tc_fence_after();
    grid_dep_launch(); // this CTA holds its TMEM: a kernel launched early cannot take it first
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(sm + C::kOffBar + 8 * C::kNumBar);
    // The c-th tile of this pair (whole warp); false after the last, or if a wait gave up.
    auto next = [&](uint32_t &c) {
        if (!kAhead) { // dense: the first is found already
            if (c > 0)
                some = get_tile<BN, kSwap, kMostTok>(g, prefix, pair + (int)c * pairs, t);
            ++c;
            return some;
        }
        const uint32_t r = c % kRing;
        if (!__all_sync(0xFFFFFFFFu, wait_phase(tile_full(r), (c / kRing) & 1)))
            return false;
        const int4 x = ring[r * 3], y = ring[r * 3 + 1], z = ring[r * 3 + 2];
        __syncwarp();
        if (lane == 0)
            mbar_arrive(tile_empty(r));
        ++c;
        t.e = x.x, t.row = x.y, t.row_end = x.z, t.n0 = x.w;
        t.k0 = y.x, t.nkb = y.y, t.rem = y.z, t.split = y.w;
        t.tok = z.x;
        return t.nkb >= 0;
    };
    uint32_t c = 0;
    bool ok = true;

    if (warp == 0 || (kSplit && warp == 2)) {
        // ------------------------------------------------------------ copies: A, and B
        uint32_t it = 0, stage = 0, phase = 1; // k blocks issued, and the next one's stage and (inverted) phase
        while (ok && next(c)) {
            const int a_row = t.row + (int)rank * 128; // kSwap: weight rows (columns of D) from n0
            const int w_row = t.n0 + (int)rank * (g.gated ? 64 : 128), tok0 = t.row + (int)rank * (t.tok / 2);
            // kSwap: one box of 16, 32, 64 or 128 token rows, the least that holds the tile's half (a copy
            // of exactly its rows, 16 at a time, costs more in copies issued than it saves in bytes:
            // 0.54 against 0.37 us a k block at 224 tokens)
            const int box_log = t.tok > 128 ? 3 : t.tok > 64 ? 2 : t.tok > 32 ? 1 : 0;
            const uint32_t bytes = C::kABytes + (kSwap ? 2048u << box_log : C::kBBytes);
            const int b_row = g.gated ? (int)rank * g.n_cols + t.n0 : t.n0 + (int)rank * (BN / 2);
            auto copy = [&](int kb, uint32_t s) {
                const int k = t.k0 + kb * kBk;
                const uint32_t bar = map_rank(full(s), 0);
                // the last block of a segment whose rows end inside it: its copy filled up with zeros
                const bool cut = kAMn && kBMn && t.rem && kb == t.nkb - 1;
                const int kr = cut ? t.e * kBk : k;
                const uint32_t sa = base + s * C::kStage, sb = sa + C::kABytes;
                if (!kSplit || warp == 0) {
                    if (kAMn) {
                        const CUtensorMap *m = !kSwap && cut ? &map_c.m[0] : &map_a;
                        const int row = kSwap ? w_row : a_row, e = kSwap ? t.e : 0;
                        if (g.wide_a)
                            tma_pair_4d(sa, m, 0, kr, row / 64, e, bar);
                        else
                            for (int j = 0; j < 2; ++j)
                                tma_pair_3d(sa + j * 8192, m, row + j * 64, kr, e, bar);
                    } else if (kSwap && g.gated) {
                        tma_pair_5d(sa, &map_a, k, 0, 0, w_row / 16, t.e, bar);
                    } else if (kSwap) {
                        tma_pair_3d(sa, &map_a, k, w_row, t.e, bar);
                    } else {
                        tma_pair_2d(sa, &map_a, k, a_row, bar);
                    }
                }
                if (kSplit && warp == 0) {
                } else if (kSwap) {
                    tma_pair_2d(sb, box_log == 3 ? &map_b : &map_c.m[box_log], k, tok0, bar);
                } else if (kBMn) {
                    const CUtensorMap *m = cut ? &map_c.m[1] : &map_b;
                    const int e = g.seg_k ? 0 : t.e;
                    if (g.wide_b)
                        tma_pair_4d(sb, m, 0, kr, b_row / 64, e, bar);
                    else
                        for (int j = 0; j < BN / 128; ++j)
                            tma_pair_3d(sb + j * 8192, m, b_row + j * 64, kr, e, bar);
                } else {
                    tma_pair_3d(sb, &map_b, k, b_row, t.e, bar);
                }
            };
            // A round of waits and copies takes the warp about 460 cycles: longer than the MMAs of a block of
            // 128 columns, whose blocks are therefore taken two at a time (512 x 4096 -> 4096 22.1 -> 18.6 us).
            // Wider tiles keep the second stage's copy in flight instead (8192 x 7168 -> 384 in 192 columns
            // 49 us one at a time, 53 us two).
            constexpr int kRound = BN == 128 ? 2 : 1;
            for (int kb = 0; kb < t.nkb; kb += kRound) {
                const bool two = kRound == 2 && kb + 1 < t.nkb;
                const uint32_t s0 = stage, p0 = phase;
                uint32_t s1 = s0 + 1, p1 = p0;
                if (s1 == S)
                    s1 = 0, p1 ^= 1;
                if (!__all_sync(0xFFFFFFFFu, wait_phase(empty(s0), p0) && (!two || wait_phase(empty(s1), p1)))) {
                    ok = false;
                    break;
                }
                if (elect_lane()) {
                    // one arrival for both operands; B's bytes may land before it, which the barrier counts
                    if (warp == 0) {
                        mbar_arrive_expect_tx_relaxed(map_rank(full(s0), 0), bytes);
                        if (two)
                            mbar_arrive_expect_tx_relaxed(map_rank(full(s1), 0), bytes);
                    }
                    copy(kb, s0);
                    if (two)
                        copy(kb + 1, s1);
                }
                __syncwarp();
                stage = two ? s1 + 1 : s1, phase = p1;
                if (two && stage == S)
                    stage = 0, phase ^= 1;
                it += two ? 2 : 1;
            }
        }
        // Before either CTA may exit, every copy has landed (all report to the leader's barriers; a wait
        // that gave up leaves some unread) and every commit has reached this CTA's barriers.
        if (warp == 0) {
            for (int j = 0; j < S; ++j)
                if (it > (uint32_t)j) {
                    const uint32_t last = it - 1 - j;
                    if (rank == 0)
                        mbar_wait_bounded(full(last % S), (last / S) & 1, nullptr, kDrainNs);
                    mbar_wait_bounded(empty(last % S), (last / S) & 1, nullptr, kDrainNs);
                }
            if (rank == 1)
                mbar_wait_bounded(mma_done, 0, nullptr, kDrainNs); // the leader's last commit
        }
    } else if (kAhead && warp == 3) {
        // ------------------------------------------------------------ tiles
        if (C::kPrefix && g.seg.E && !g.seg_k) {
            int run = 0;
            for (int e0 = 0; e0 < g.seg.E; e0 += 32) {
                const int e = e0 + lane;
                int n = 0;
                if (e < g.seg.E) {
                    int first;
                    const int rows = segment_rows(g.seg, e, first);
                    int tok;
                    n = (kSwap ? token_tiles(rows, kMostTok, tok) : (rows + kTileM - 1) / kTileM) * g.nt;
                }
                int incl = n;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int y = __shfl_up_sync(0xFFFFFFFFu, incl, o);
                    if (lane >= o)
                        incl += y;
                }
                if (e < g.seg.E)
                    prefix[e] = run + incl - n;
                run += __shfl_sync(0xFFFFFFFFu, incl, 31);
            }
            if (lane == 0)
                prefix[g.seg.E] = run;
            __syncwarp();
        }
        bool more = true;
        for (int i = pair; more; i += pairs, ++c) {
            more = early && c == 0 ? some : get_tile<BN, kSwap, kMostTok>(g, prefix, i, t);
            const uint32_t r = c % kRing;
            if (!__all_sync(0xFFFFFFFFu, wait_phase(tile_empty(r), ((c / kRing) & 1) ^ 1)))
                break;
            if (lane == 0) {
                ring[r * 3] = make_int4(t.e, t.row, t.row_end, t.n0);
                ring[r * 3 + 1] = make_int4(t.k0, more ? t.nkb : -1, t.rem, t.split);
                ring[r * 3 + 2] = make_int4(t.tok, 0, 0, 0);
                mbar_arrive(tile_full(r));
            }
            __syncwarp();
        }
    } else if (warp == 1 && rank == 0) {
        // ------------------------------------------------------------ MMAs
        uint32_t n = 0, stage = 0, phase = 0;
        const uint64_t da0 = kAMn ? smem_desc_mn_sw128(base, 8192) : smem_desc_sw128(base);
        const uint64_t db0 = kBMn ? smem_desc_mn_sw128(base + C::kABytes, 8192) : smem_desc_sw128(base + C::kABytes);
        while (ok && next(c)) {
            const uint32_t idesc = idesc_f16(g.fmt, kAMn, kBMn, kTileM, kSwap ? t.tok : BN);
            for (int kb = 0; ok && kb < t.nkb;) {
                const int buf = n & 1;
                if (!__all_sync(0xFFFFFFFFu, wait_phase(acc_empty(buf), ((n >> 1) & 1) ^ 1))) {
                    ok = false;
                    break;
                }
                ++n;
                tc_fence_after();
                const int first = kb, end = min(t.nkb, kb + (kSum ? kChain : 1 << g.run_log));
                while (ok && kb < end) {
                    // unrolled over the stages, whose descriptors are then constants apart (about 100 cycles less
                    // a block; descriptors are affine in the address, which stays below 2^18)
#pragma unroll
                    for (int s = 0; s < S; ++s) {
                        if (s != (int)stage || kb >= end)
                            continue;
                        if (!__all_sync(0xFFFFFFFFu, wait_phase(full(s), phase))) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        if (elect_lane()) {
                            // 16 of k: 32 bytes of a K-major row, or two 1024-byte groups of 8 k
#pragma unroll
                            for (int q = 0; q < kBk / 16; ++q)
                                umma_f16_pair(tmem + 256u * buf, da0 + (s * (C::kStage >> 4) + q * (kAMn ? 128 : 2)),
                                              db0 + (s * (C::kStage >> 4) + q * (kBMn ? 128 : 2)), idesc,
                                              kb > first || q > 0);
                            umma_commit_pair(empty(s));
                            if (kb == end - 1)
                                umma_commit_pair(acc_full(buf));
                        }
                        __syncwarp();
                        ++kb;
                        ++stage;
                    }
                    if (stage == S)
                        stage = 0, phase ^= 1;
                }
            }
        }
        // every MMA has completed before TMEM is released
        if (elect_lane())
            umma_commit_pair(mma_done);
        __syncwarp();
        mbar_wait_bounded(mma_done, 0, nullptr, kDrainNs);
    } else if (warp >= 4) {
        // ------------------------------------------------------------ epilogue
        const int q = warp & 3, half = (warp - 4) >> 2;
        float *const stg = reinterpret_cast<float *>(sm + C::kOffEpi + (warp - 4) * 4096);
        const int cols = g.gated ? BN / 4 : BN / 2; // columns of D this warp takes
        const int rl = lane >> 2, c8 = (lane & 3) * 8;
        uint32_t n = 0;
        // 32 columns of this warp's 32 rows (lane: row) through shared memory: lane l then holds row
        // 8 j + l / 4, columns 8 (l % 4) .. + 7
        auto turn = [&](const uint32_t (&r)[32], float (&v)[4][8]) {
            float4 *own = reinterpret_cast<float4 *>(stg + lane * 32);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                own[j ^ (lane & 7)] = make_float4(__uint_as_float(r[4 * j]), __uint_as_float(r[4 * j + 1]),
                                                  __uint_as_float(r[4 * j + 2]), __uint_as_float(r[4 * j + 3]));
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int row = i * 8 + rl;
                const float4 *src = reinterpret_cast<const float4 *>(stg + row * 32);
                const float4 a = src[(c8 / 4) ^ (row & 7)], b = src[(c8 / 4 + 1) ^ (row & 7)];
                v[i][0] = a.x, v[i][1] = a.y, v[i][2] = a.z, v[i][3] = a.w;
                v[i][4] = b.x, v[i][5] = b.y, v[i][6] = b.z, v[i][7] = b.w;
            }
            __syncwarp();
        };
        // 32 columns of this warp's 32 rows (lane: row) to lane: column
        auto turn_columns = [&](const uint32_t (&r)[32], float (&v)[32]) {
            float4 *own = reinterpret_cast<float4 *>(stg + lane * 32);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                own[j ^ (lane & 7)] = make_float4(__uint_as_float(r[4 * j]), __uint_as_float(r[4 * j + 1]),
                                                  __uint_as_float(r[4 * j + 2]), __uint_as_float(r[4 * j + 3]));
            __syncwarp();
#pragma unroll
            for (int x = 0; x < 32; ++x)
                v[x] = stg[x * 32 + (((lane >> 2) ^ (x & 7)) << 2) + (lane & 3)];
            __syncwarp();
        };
        // Accumulator n of this pair is complete; `free_acc` gives its TMEM back to the MMAs.
        auto wait_acc = [&]() {
            ok = __all_sync(0xFFFFFFFFu, wait_phase(acc_full(n & 1), (n >> 1) & 1));
            tc_fence_after();
            return ok;
        };
        auto free_acc = [&]() {
            tc_fence_before();
            __syncwarp();
            if (lane == 0)
                mbar_arrive_relaxed(map_rank(acc_empty(n & 1), 0)); // its TMEM reads are done (wait::ld)
            ++n;
        };
        // The sums of a tile of more than one run (!kSum): those of all its runs but the last, 32 x 32 at a
        // time from column `col(i)` of TMEM, i < chunks, go to this warp's part of the workspace.  A lane reads
        // what it wrote.  `settle` makes the last run's sums the tile's: adds the ones held and scales a gradient.
        float4 *const held = g.held + ((size_t)blockIdx.x * kEpiWarps + (warp - 4)) * kHeld + lane;
        int runs = 0; // of this tile, before its last
        const float *const factors = kPlain ? g.unscale : nullptr;
        float factor = 1.f; // of this tile's sums, a power of two
        bool as_is = true;  // this tile's sums need nothing settled
        auto add_held = [&](int i, uint32_t (&r)[32]) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float4 h = held[i * kHeldChunk + j * 32];
                r[4 * j] = __float_as_uint(__uint_as_float(r[4 * j]) + h.x);
                r[4 * j + 1] = __float_as_uint(__uint_as_float(r[4 * j + 1]) + h.y);
                r[4 * j + 2] = __float_as_uint(__uint_as_float(r[4 * j + 2]) + h.z);
                r[4 * j + 3] = __float_as_uint(__uint_as_float(r[4 * j + 3]) + h.w);
            }
        };
        auto hold_runs = [&](int nkb, int chunks, auto col) {
            const int most = (nkb - 1) >> g.run_log;
            for (runs = 0; runs < most; ++runs) {
                if (!wait_acc())
                    return false;
                for (int i = 0; i < chunks; ++i) {
                    uint32_t r[32];
                    tmem_ld32(tmem + 256u * (n & 1) + ((uint32_t)(q * 32) << 16) + col(i), r);
                    tmem_wait_ld();
                    if (runs)
                        add_held(i, r); // of the runs before
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        held[i * kHeldChunk + j * 32] =
                            make_float4(__uint_as_float(r[4 * j]), __uint_as_float(r[4 * j + 1]),
                                        __uint_as_float(r[4 * j + 2]), __uint_as_float(r[4 * j + 3]));
                }
                free_acc();
            }
            as_is = runs <= 0 && !factors;
            return true;
        };
        auto settle = [&](int i, uint32_t (&r)[32]) {
            if (as_is)
                return;
            if (runs)
                add_held(i, r);
#pragma unroll
            for (int x = 0; x < 32; ++x)
                r[x] = __float_as_uint(__uint_as_float(r[x]) * factor);
        };
        while (ok && next(c)) {
            // gradients have no bias, preact, activation or residual
            const Epi ep = kPlain ? Epi{nullptr, nullptr, g.out, nullptr, kActNone, g.N, g.n_cols, g.type, g.out_type, g.vec}
                                : Epi{g.bias ? g.bias + (size_t)t.e * g.N : nullptr, g.residual, g.out, g.preact, g.act,
                                      g.N, g.n_cols, g.type, g.out_type, g.vec};
            if (factors)
                factor = factors[t.e];
            const bool columns = kSum || !ep.vec || ep.out_type == kTypeF32; // kSum: of float32 outputs
            const size_t d_off = g.seg_k ? (size_t)t.e * g.d_expert : (size_t)t.split * g.M * g.n_cols;
            if constexpr (kSwap) {
                // lane: a column of D; chunk c: tokens 32 c .. + 31, taken by the warp halves in turn
                const bool gated = !kPlain && g.gated;
                const uint32_t acc0 = (uint32_t)(q * 32) << 16;
                // [token][column] through shared memory; groups of 4 columns change place by the token
                // so that neither side meets bank conflicts
                auto put = [&](const uint32_t (&r)[32]) {
#pragma unroll
                    for (int x = 0; x < 32; ++x) {
                        const int sw = (x & 1) | ((x & 2) << 1);
                        stg[x * 32 + (((lane >> 2) ^ sw) << 2) + (lane & 3)] = __uint_as_float(r[x]);
                    }
                    __syncwarp();
                };
                auto get8 = [&](int token, int col, float (&f)[8]) {
                    const int sw = (token & 1) | ((token & 2) << 1);
                    const float4 *src = reinterpret_cast<const float4 *>(stg + token * 32);
                    const float4 a = src[(col / 4) ^ sw], b = src[(col / 4 + 1) ^ sw];
                    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w;
                    f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
                };
                Rows w;
                Ahead<4> ahead;
                Ahead<2> ahead2;
                auto place = [&](int c) {
                    // gated: 2 lanes to a token's 16 columns, tokens 16 apart; else 4 lanes to 32, 8 apart
                    const int step = gated ? 16 : 8;
                    const int m = t.row + c * 32 + (gated ? lane >> 1 : rl);
                    w.n = gated ? t.n0 + (int)rank * 64 + q * 16 + (lane & 1) * 8 : t.n0 + (int)rank * 128 + q * 32 + c8;
                    w.ok = 0;
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        w.ok |= m + j * step < t.row_end && w.n < g.n_cols ? 1u << j : 0u;
                    w.so = step * g.n_cols, w.spo = step * g.N;
                    w.o = d_off + (size_t)m * g.n_cols + w.n;
                    w.po = (size_t)m * g.N + w.n;
                    if (gated)
                        ahead2.load(ep, w);
                    else
                        ahead.load(ep, w);
                };
                auto done = [&](int c, const uint32_t (&r)[32]) {
                    if (columns) { // a lane has a column of 32 tokens as it is
                        const int m = t.row + c * 32;
                        const int col = gated ? t.n0 + (int)rank * 64 + q * 16 + (lane & 15)
                                              : t.n0 + (int)rank * 128 + q * 32 + lane;
                        const int rows = col < g.n_cols ? min(32, t.row_end - m) : 0;
                        float v[32], up[32];
#pragma unroll
                        for (int x = 0; x < 32; ++x)
                            v[x] = __uint_as_float(r[x]);
                        if (gated) { // the up half lies 16 lanes on
#pragma unroll
                            for (int x = 0; x < 32; ++x)
                                up[x] = __shfl_down_sync(0xFFFFFFFFu, v[x], 16);
                            finish_column<true>(ep, d_off, m, col, lane < 16 ? rows : 0, v, up);
                        } else {
                            finish_column<false>(ep, d_off, m, col, rows, v, v);
                        }
                        return;
                    }
                    put(r);
                    if (gated) {
                        float v[2][8], up[2][8];
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            get8(j * 16 + (lane >> 1), (lane & 1) * 8, v[j]);
                            get8(j * 16 + (lane >> 1), 16 + (lane & 1) * 8, up[j]);
                        }
                        __syncwarp();
                        finish<2, true>(ep, w, v, up, ahead2);
                    } else {
                        float v[4][8];
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            get8(j * 8 + rl, c8, v[j]);
                        __syncwarp();
                        finish<4, false>(ep, w, v, v, ahead);
                    }
                };
                const int chunks = t.tok / 32;
                if constexpr (kSum) {
                    uint32_t sum[2][32];
#pragma unroll
                    for (int c = 0; c < 2; ++c)
#pragma unroll
                        for (int x = 0; x < 32; ++x)
                            sum[c][x] = 0u;
                    for (int kb = 0; ok && kb < t.nkb; kb += kChain) {
                        if (!wait_acc())
                            break;
#pragma unroll
                        for (int c = 0; c < 2; ++c)
                            if (half + 2 * c < chunks) {
                                uint32_t r[32];
                                tmem_ld32(tmem + 256u * (n & 1) + acc0 + (half + 2 * c) * 32, r);
                                tmem_wait_ld();
#pragma unroll
                                for (int x = 0; x < 32; ++x)
                                    sum[c][x] = __float_as_uint(__uint_as_float(sum[c][x]) + __uint_as_float(r[x]));
                            }
                        free_acc();
                    }
                    if (!ok)
                        break;
#pragma unroll
                    for (int c = 0; c < 2; ++c)
                        if (half + 2 * c < chunks)
                            done(half + 2 * c, sum[c]);
                } else {
                    if (!hold_runs(t.nkb, (chunks - half + 1) / 2, [&](int i) { return (half + 2 * i) * 32; }))
                        break;
                    if (half < chunks && !columns)
                        place(half);
                    if (!wait_acc())
                        break;
                    if (half >= chunks)
                        free_acc();
                    for (int c = half; c < chunks; c += 2) {
                        if (c > half && !columns)
                            place(c);
                        uint32_t r[32];
                        tmem_ld32(tmem + 256u * (n & 1) + acc0 + c * 32, r);
                        tmem_wait_ld();
                        settle(c / 2, r);
                        if (c + 2 >= chunks)
                            free_acc();
                        done(c, r);
                    }
                }
                continue;
            }
            const int row0 = t.row + (int)rank * 128 + q * 32 + rl;
            Ahead<4> ahead;
            Rows w;
            w.so = 8 * g.n_cols, w.spo = 8 * g.N;
            auto place = [&](int c) { // this lane's four rows at column c of the tile
                w.n = t.n0 + c + c8;
                w.ok = 0;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    w.ok |= row0 + j * 8 < t.row_end && w.n < g.n_cols ? 1u << j : 0u;
                w.o = d_off + (size_t)row0 * g.n_cols + w.n;
                w.po = (size_t)row0 * g.N + w.n;
                ahead.load(ep, w);
            };
            const uint32_t lanes = (uint32_t)(q * 32) << 16;
            // `columns`: this warp's rows of column c + lane of the tile
            const int row32 = row0 - rl;
            auto column_rows = [&](int c) { return t.n0 + c + lane < g.n_cols ? min(32, t.row_end - row32) : 0; };
            if constexpr (kSum) {
                // columns lc .. of D (gated: and the same of the up half) summed over the chains
                constexpr int kChunks = BN / 64;
                const bool gated = kChunks % 2 == 0 && g.gated; // the plan gates no tile of 192 columns
                uint32_t sum[kChunks][32];
#pragma unroll
                for (int c = 0; c < kChunks; ++c)
#pragma unroll
                    for (int x = 0; x < 32; ++x)
                        sum[c][x] = 0u;
                // chunk c's first accumulator column: this warp's half, or its gate and up columns
                auto acc_col = [&](int c) {
                    return gated ? (c % (kChunks / 2)) * 32 + half * (BN / 4) + (c >= kChunks / 2 ? BN / 2 : 0)
                                   : half * (BN / 2) + c * 32;
                };
                for (int kb = 0; ok && kb < t.nkb; kb += kChain) {
                    if (!wait_acc())
                        break;
                    const uint32_t acc = tmem + 256u * (n & 1) + lanes;
#pragma unroll
                    for (int c = 0; c < kChunks; ++c) {
                        uint32_t r0[16], r1[16];
                        tmem_ld16(acc + acc_col(c), r0);
                        tmem_ld16(acc + acc_col(c) + 16, r1);
                        tmem_wait_ld();
#pragma unroll
                        for (int x = 0; x < 16; ++x) {
                            sum[c][x] = __float_as_uint(__uint_as_float(sum[c][x]) + __uint_as_float(r0[x]));
                            sum[c][x + 16] = __float_as_uint(__uint_as_float(sum[c][x + 16]) + __uint_as_float(r1[x]));
                        }
                    }
                    free_acc();
                }
                if (!ok)
                    break;
                if (gated) {
#pragma unroll
                    for (int c = 0; c < kChunks / 2; ++c) {
                        float z[32], up[32];
                        const int lc = half * cols + c * 32;
                        turn_columns(sum[c], z);
                        turn_columns(sum[c + kChunks / 2], up);
                        finish_column<true>(ep, d_off, row32, t.n0 + lc + lane, column_rows(lc), z, up);
                    }
                } else {
#pragma unroll
                    for (int c = 0; c < kChunks; ++c) {
                        float z[32];
                        const int lc = half * cols + c * 32;
                        turn_columns(sum[c], z);
                        finish_column<false>(ep, d_off, row32, t.n0 + lc + lane, column_rows(lc), z, z);
                    }
                }
            } else {
                constexpr int kChunks = BN / 64; // gated: half of them of the up half
                const bool gated = !kPlain && g.gated;
                if (!hold_runs(t.nkb, kChunks, [&](int i) {
                        return half * cols + (gated && i >= kChunks / 2 ? BN / 2 + (i - kChunks / 2) * 32 : i * 32);
                    }))
                    break;
                if (!columns && cols % 64 == 0 && !ep.residual && !ep.preact &&
                    !gated) {
                    // One 16-bit output: bias, activation and rounding where the values lie (lane: row), turned
                    // 64 columns at a time as 16-bit values, stored as whole 128-byte lines.  Half the
                    // shared-memory traffic of float32 blocks of 32 columns; it bounds products of short k, such
                    // as gradients, and is what a single wave waits for at its end.
                    if (t.nkb > 0 && !wait_acc())
                        break;
                    uint4 *const line = reinterpret_cast<uint4 *>(stg);
                    uint16_t *const out = static_cast<uint16_t *>(g.out) + d_off;
                    const int r8 = lane >> 3, l8 = lane & 7;
                    for (int c = 0; c < cols; c += 64) {
                        const int lc = half * cols + c;
                        uint32_t r0[32] = {}, r1[32] = {};
                        if (t.nkb > 0) {
                            tmem_ld32(tmem + 256u * (n & 1) + lanes + lc, r0);
                            tmem_ld32(tmem + 256u * (n & 1) + lanes + lc + 32, r1);
                            tmem_wait_ld();
                            settle(c / 32, r0);
                            settle(c / 32 + 1, r1);
                            if (c + 64 >= cols)
                                free_acc();
                        }
                        if (!kPlain)
                            bias_act(ep, t.n0 + lc, r0, r1);
                        auto pack = [&](auto zero) {
                            using T = decltype(zero);
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                uint32_t a[4], b[4];
#pragma unroll
                                for (int x = 0; x < 4; ++x) {
                                    a[x] = pack2(__uint_as_float(r0[8 * j + 2 * x]), __uint_as_float(r0[8 * j + 2 * x + 1]), T());
                                    b[x] = pack2(__uint_as_float(r1[8 * j + 2 * x]), __uint_as_float(r1[8 * j + 2 * x + 1]), T());
                                }
                                line[lane * 8 + (j ^ (lane & 7))] = make_uint4(a[0], a[1], a[2], a[3]);
                                line[lane * 8 + ((j + 4) ^ (lane & 7))] = make_uint4(b[0], b[1], b[2], b[3]);
                            }
                        };
                        if (g.type == kTypeF16)
                            pack(__half());
                        else
                            pack(__nv_bfloat16());
                        __syncwarp();
                        const int nn = t.n0 + lc + l8 * 8;
                        uint4 v[8];
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            v[j] = line[(j * 4 + r8) * 8 + (l8 ^ ((j * 4 + r8) & 7))];
                        __syncwarp();
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const int m = t.row + (int)rank * 128 + q * 32 + j * 4 + r8;
                            if (m < t.row_end && nn < g.n_cols)
                                *reinterpret_cast<uint4 *>(out + (size_t)m * g.n_cols + nn) = v[j];
                        }
                    }
                    continue;
                }
                auto take = [&](uint32_t col, int chunk, float (&f)[4][8]) {
                    uint32_t r[32];
                    tmem_ld32(tmem + 256u * (n & 1) + lanes + col, r);
                    tmem_wait_ld();
                    settle(chunk, r);
                    turn(r, f);
                };
                auto take_columns = [&](uint32_t col, int chunk, float (&f)[32]) {
                    uint32_t r[32];
                    tmem_ld32(tmem + 256u * (n & 1) + lanes + col, r);
                    tmem_wait_ld();
                    settle(chunk, r);
                    turn_columns(r, f);
                };
                for (int c = 0; c < cols; c += 32) {
                    const int lc = half * cols + c; // column within the tile
                    if (columns) {
                        if (c == 0 && t.nkb > 0 && !wait_acc())
                            break;
                        float z[32] = {}, u[32] = {};
                        if (t.nkb > 0) {
                            take_columns(lc, c / 32, z);
                            if (gated)
                                take_columns(BN / 2 + lc, kChunks / 2 + c / 32, u);
                            if (c + 32 >= cols)
                                free_acc();
                        }
                        if (gated)
                            finish_column<true>(ep, d_off, row32, t.n0 + lc + lane, column_rows(lc), z, u);
                        else
                            finish_column<false>(ep, d_off, row32, t.n0 + lc + lane, column_rows(lc), z, u);
                        continue;
                    }
                    place(lc);
                    if (c == 0 && t.nkb > 0 && !wait_acc())
                        break;
                    float v[4][8] = {}, up[4][8] = {};
                    if (t.nkb > 0)
                        take(lc, c / 32, v);
                    if (gated) {
                        if (t.nkb > 0) {
                            take(BN / 2 + lc, kChunks / 2 + c / 32, up);
                            if (c + 32 >= cols)
                                free_acc();
                        }
                        finish<4, true>(ep, w, v, up, ahead);
                    } else {
                        if (t.nkb > 0 && c + 32 >= cols)
                            free_acc();
                        finish<4, false>(ep, w, v, up, ahead);
                    }
                }
            }
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    tc_fence_after();
    if (warp == 2) {
        tmem_relinquish_pair();
        tmem_dealloc_pair(tmem, 512);
    }
}

// ---------------------------------------------------------------- split products
// out = epilogue(sum over the splits' float32 planes, in order); one thread per value, eight loads at a time.
// Latency bounds it: 100 rows by 7168 -> 384, 23 planes, 15 us with the product, 18 us with eight columns a thread;
// -> 387, whose columns were loaded one by one there, 11 us and 21 us.
template <typename T, bool kGated>
__global__ void __launch_bounds__(256) reduce_kernel(const float *planes, int splits, int M, Epi g)
{
    grid_dep_wait();
    grid_dep_launch();
    const uint32_t i = blockIdx.x * 256 + threadIdx.x; // plan_dense splits products of less than 2^31 values alone
    const uint32_t m = i / (uint32_t)g.n_cols, n = i % (uint32_t)g.n_cols;
    if (m >= (uint32_t)M)
        return;
    const size_t plane = (size_t)M * g.N;
    const float *p = planes + (size_t)m * g.N + n;
    float z = 0.f, up = 0.f;
    for (int s = 0; s < splits; s += 8) {
        float a[8], b[8];
#pragma unroll
        for (int j = 0; j < 8; ++j, p += plane) {
            a[j] = s + j < splits ? p[0] : 0.f;
            b[j] = kGated && s + j < splits ? p[g.n_cols] : 0.f;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
            z += a[j], up += b[j];
    }
    finish_value<T, kGated>(g, m, (int)n, z, up);
}

// ---------------------------------------------------------------- unaligned rows
// TMA reads rows that start on 16 bytes: operands whose row length is not a multiple of 8 are first
// copied to rows of the next multiple (the pad is not read: the tensor map ends at the true length).
struct PackArgs {
    const uint16_t *src[2]; // x, w; nullptr: no copy
    uint16_t *dst[2];
    int64_t rows[2];
    int cols, ld;
    Segments seg;           // of x's rows: padding is left out
};

constexpr int kPackCols = 1024; // of a warp: a lane has four chunks of 8 in flight

// A warp per piece of a row (grid y: x or w); a lane copies 8 elements at a time from aligned words that its
// row may start in the middle of.  Latency bounds it: 780 + 1470 rows of 909 4.2 us, 9.7 us with a CTA a row
// and a chunk at a time.
__global__ void __launch_bounds__(256) pack_kernel(const PackArgs a)
{
    grid_dep_wait();
    grid_dep_launch();
    const int o = a.src[0] ? blockIdx.y : 1, lane = threadIdx.x & 31;
    const int pieces = (a.cols + kPackCols - 1) / kPackCols;
    const int64_t items = a.rows[o] * pieces;
    for (int64_t i = blockIdx.x * 8 + (threadIdx.x >> 5); i < items; i += gridDim.x * 8) {
        const int64_t r = i / pieces;
        int e;
        int64_t end;
        if (o == 0 && a.seg.E && !find_segment(a.seg, r, e, end))
            continue;
        const int first = (int)(i % pieces) * kPackCols, last = min(a.cols, first + kPackCols);
        const uint16_t *src = a.src[o] + r * a.cols;
        uint16_t *dst = a.dst[o] + r * a.ld;
        const bool odd = reinterpret_cast<uintptr_t>(src) & 2;
        uint32_t v[4][5];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            // odd: the words around the eight.  The first holds the element before them, which is in the
            // buffer (an odd row is not the first), and the last ends with the eighth
            const int c = first + lane * 8 + j * 256;
            const uint32_t *p = reinterpret_cast<const uint32_t *>(src + c - (odd ? 1 : 0));
#pragma unroll
            for (int x = 0; x < 4; ++x)
                v[j][x] = c + 8 <= last ? p[x] : 0u;
            v[j][4] = odd && c + 8 <= last ? src[c + 7] : 0u;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int c = first + lane * 8 + j * 256;
            if (c + 8 > last)
                continue;
            if (odd)
#pragma unroll
                for (int x = 0; x < 4; ++x)
                    v[j][x] = __funnelshift_r(v[j][x], v[j][x + 1], 16);
            *reinterpret_cast<uint4 *>(dst + c) = make_uint4(v[j][0], v[j][1], v[j][2], v[j][3]);
        }
        const int rest = (last & ~7) + lane; // pieces start at multiples of 8
        if (rest < last)
            dst[rest] = src[rest];
    }
}

// x and w (either may be absent) with aligned rows; nothing to do when K is a multiple of 8.
cudaError_t launch_pack(const void *&x, int64_t x_rows, const Segments &seg, char *x_ws, const void *&w, int64_t w_rows,
                        char *w_ws, int K, cudaStream_t s)
{
    if (K % 8 == 0 || (!x && !w))
        return cudaSuccess;
    PackArgs a{};
    a.src[0] = static_cast<const uint16_t *>(x), a.src[1] = static_cast<const uint16_t *>(w);
    a.dst[0] = reinterpret_cast<uint16_t *>(x_ws), a.dst[1] = reinterpret_cast<uint16_t *>(w_ws);
    a.rows[0] = x_rows, a.rows[1] = w_rows;
    a.cols = K, a.ld = (int)round_up(K, 8), a.seg = seg;
    const int64_t most = !x ? w_rows : !w ? x_rows : x_rows > w_rows ? x_rows : w_rows;
    const int64_t ctas = (most * ((K + kPackCols - 1) / kPackCols) + 7) / 8;
    const dim3 grid((unsigned)(ctas < 148 * 8 ? ctas : 148 * 8), x && w ? 2 : 1);
    if (x)
        x = x_ws;
    if (w)
        w = w_ws;
    return launch_kernel(pack_kernel, grid, dim3(256), 0, s, true, a);
}

// ---------------------------------------------------------------- launch
// The shape of a dense [M, cols] product over kb blocks of k, by the estimated cycles: a 64-deep block of a
// 256 x BN tile (BN weight rows, or BN tokens for kSwap) takes about 256 + BN cycles (its MMAs 2 BN,
// its loads from L2 (16 KB + 64 BN bytes) / 64 a cycle), a tile about 1500 to start and finish, and
// a split product writes and reads its float32 planes and launches a second kernel.
struct Plan {
    int bn, splits;
    bool sum;  // the sum over chains of kChain k blocks kept in registers (at most 192 columns, or 128 tokens)
    int tok;   // kSwap: tokens of a tile; else 0
};
constexpr int64_t kMostSplit = (int64_t)1 << 31; // reduce_kernel counts the values of D in 32 bits
Plan plan_dense(int64_t M, int cols, int kb, bool gated, bool mn, bool f32, bool swap)
{
    Plan best{256, 1, false, 0};
    if (M == 0 || kb == 0)
        return best;
    double best_t = 1e30;
    auto consider = [&](int bn, int tok, int64_t row_tiles, int col_tiles, int width) {
        for (int s : {1, 2, 3, 4, 6, 8, 12, 18, 24, 36}) {
            if (s > 1 && (kb / s < 3 || M * cols >= kMostSplit))
                break;
            const int64_t kbs = (kb + s - 1) / s;
            const bool sum = f32 && kbs > kChain;
            if (sum && width > (tok ? 128 : 192))
                continue;
            const int64_t tiles = row_tiles * col_tiles * ((kb + kbs - 1) / kbs);
            double t = (double)((tiles + kPairs - 1) / kPairs) * ((double)kbs * (256 + width) + 1500);
            if (s > 1)
                t += 5000 + (double)s * M * cols * 8 / 4000;
            if (t < best_t)
                best_t = t, best = Plan{bn, s, sum, tok};
        }
    };
    // A tile of rows holds 256, one of tokens no more than there are.  100 x 7168 -> 384 12.6 us as rows, 8.9 as
    // tokens; 200 x 2048 -> 1024 11.5 and 9.9; full tiles, 256 x 4096 -> 4096, 19.8 and 20.1.  Up to 128 columns
    // the same holds the other way round (128 x 1024 -> 128 6.7 us, 7.6 as tokens).
    const bool rows = !swap || M > 224 || cols <= 128;
    for (int bn : {256, 192, 128})
        if (rows && (bn != 192 || !(gated || mn))) // halves of 96 columns
            consider(bn, 0, (M + kTileM - 1) / kTileM, (cols + bn - 1) / bn, bn);
    if (swap)
        for (int most : {256, 128}) {
            const int64_t tiles = (M + most - 1) / most;
            const int tok = (int)round_up((M + tiles - 1) / tiles, 32);
            consider(256, tok, (M + tok - 1) / tok, (cols + 255) / 256, tok);
        }
    return best;
}

// ---------------------------------------------------------------- a few rows
// A few rows of x (a decode step): the product streams w once and its time is w's bytes over the
// memory rate, or launch latency.  Weight rows are the A operand of 16 x 8 x 16 warp MMAs, tokens the
// B operand; a warp takes kR x 16 weight rows over a slice of k, the 8 warps of a CTA and the CTAs of a
// cluster share k, and the partial sums meet in shared memory (a fixed order, one launch, where
// a split tile product writes planes and launches a second kernel: 16.7 -> 8.6 us a call of
// 384 x 7168, most of it the host's).  Within a 32-element k block lane t of a row's four holds elements
// 8t .. 8t + 7 of both operands (one 16-byte load), which the two MMAs take in the same order.
constexpr int kSmallWarps = 8, kMaxCluster = 8;

template <typename T>
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1)
{
    if constexpr (sizeof(T) == sizeof(__half) && !__is_same(T, __nv_bfloat16))
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

struct SmallArgs {
    const void *x, *w;
    int M, N, K, k_warp; // k_warp: elements of k of one warp (a multiple of 32)
    Epi epi;
};

// kR: 16-row weight tiles of a CTA (swiglu: a gate and an up tile); kNb: 8-token groups; kShort: the MMAs
// truncate their sums, as the tile product's do (kChain), so chains of 32 kU of k are summed by float32 adds.
// For float32 outputs of more than kSmallChain of k a warp: 16 rows by 7168 -> 4096, 896 of k a warp, a
// relative error of 8.6e-7 in one chain, 1.4e-7 in short ones, both 16 us (with SwiGLU, 8 rows: 8.4e-7 and
// 2.5e-7, 15.4 us).  A 16-bit output's own rounding is larger up to a tile product's run; short chains everywhere
// cost 48 rows by 1408 -> 2816 8.8 -> 12.7 us, in registers.
constexpr int kSmallChain = 256;

template <typename T, int kR, int kNb, bool kGated, bool kShort>
__global__ void __launch_bounds__(kSmallWarps * 32) small_kernel(const SmallArgs a)
{
    constexpr int kOut = kR * 16 * kNb * 8; // partial sums of a CTA: [weight row][token]
    __shared__ float part[kSmallWarps][kOut];
    __shared__ float total[kOut];
    grid_dep_wait();
    grid_dep_launch();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    uint32_t ranks, rank = cluster_rank();
    asm volatile("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(ranks));
    const int tile = blockIdx.x / ranks;
    const int n0 = tile * (kGated ? 16 : kR * 16); // first column of D
    const int cols = a.epi.n_cols;
    const T *w = static_cast<const T *>(a.w), *x = static_cast<const T *>(a.x);
    const T *wp[2 * kR], *xp[kNb];
    bool wok[2 * kR], xok[kNb];
#pragma unroll
    for (int r = 0; r < 2 * kR; ++r) {
        const int n = kGated ? n0 + (r & 1) * 8 + g : n0 + r * 8 + g;
        wok[r] = n < cols;
        wp[r] = w + (size_t)(wok[r] ? n + (kGated && r >= 2 ? cols : 0) : 0) * a.K + 8 * t;
    }
#pragma unroll
    for (int b = 0; b < kNb; ++b) {
        xok[b] = b * 8 + g < a.M;
        xp[b] = x + (size_t)(xok[b] ? b * 8 + g : 0) * a.K + 8 * t;
    }
    float acc[kR][kNb][4] = {};
    const int k0 = (int)(rank * kSmallWarps + warp) * a.k_warp, k1 = min(a.K, k0 + a.k_warp);
    float sum[kR][kNb][4] = {}; // kShort: of the chains before
    constexpr int kU = kNb <= 2 ? 4 : 2; // k blocks of 32 in flight
    for (int k = k0; k < k1; k += 32 * kU) {
        uint4 wv[kU][2 * kR], xv[kU][kNb];
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int ku = k + 32 * u;
            const bool in = ku + 8 * t < k1; // K is a multiple of 8: 8 elements are in or out together
#pragma unroll
            for (int r = 0; r < 2 * kR; ++r)
                wv[u][r] = in && wok[r] ? load_once(wp[r] + ku) : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int b = 0; b < kNb; ++b)
                xv[u][b] = in && xok[b] ? *reinterpret_cast<const uint4 *>(xp[b] + ku) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int u = 0; u < kU; ++u)
#pragma unroll
            for (int r = 0; r < kR; ++r)
#pragma unroll
                for (int b = 0; b < kNb; ++b) {
                    const uint4 lo = wv[u][2 * r], hi = wv[u][2 * r + 1], v = xv[u][b];
                    mma16816<T>(acc[r][b], lo.x, hi.x, lo.y, hi.y, v.x, v.y);
                    mma16816<T>(acc[r][b], lo.z, hi.z, lo.w, hi.w, v.z, v.w);
                }
        if (kShort)
#pragma unroll
            for (int r = 0; r < kR; ++r)
#pragma unroll
                for (int b = 0; b < kNb; ++b)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        sum[r][b][i] += acc[r][b][i];
                        acc[r][b][i] = 0.f;
                    }
    }
    // element (weight row 16 r + g (+ 8), token 8 b + 2 t (+ 1))
#pragma unroll
    for (int r = 0; r < kR; ++r)
#pragma unroll
        for (int b = 0; b < kNb; ++b)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                part[warp][(r * 16 + g + (i >> 1) * 8) * (kNb * 8) + b * 8 + 2 * t + (i & 1)] =
                    kShort ? sum[r][b][i] + acc[r][b][i] : acc[r][b][i];
    __syncthreads();
    for (int i = threadIdx.x; i < kOut; i += kSmallWarps * 32) {
        float s = 0.f;
#pragma unroll
        for (int j = 0; j < kSmallWarps; ++j)
            s += part[j][i];
        total[i] = s;
    }
    if (ranks > 1)
        cluster_sync();
    else
        __syncthreads();
    if (rank == 0) {
        const Epi &e = a.epi;
        for (int i = threadIdx.x; i < (kGated ? kOut / 2 : kOut); i += kSmallWarps * 32) {
            // neighbouring threads: neighbouring columns of one token
            const int rows = kGated ? 16 : kR * 16, c = i % rows, m = i / rows, n = n0 + c;
            if (m >= a.M || n >= cols)
                continue;
            float z = 0.f, up = 0.f;
            for (uint32_t q = 0; q < ranks; ++q) {
                z += load_rank(&total[c * (kNb * 8) + m], q);
                if (kGated)
                    up += load_rank(&total[(16 + c) * (kNb * 8) + m], q);
            }
            finish_value<T, kGated>(e, m, n, z, up);
        }
    }
    if (ranks > 1)
        cluster_sync(); // the other CTAs' shared memory is read until here
}

// Whether a dense product runs as small_kernel: few rows, and rows of w of whole 16 bytes.
// - Up to 16 rows: less than 48 M weights.  Larger ones stream faster through the tile product with 32 tokens a
//   tile: 16 rows by 4096 -> 14336 (59 M) 35 us here and 25 us there, 8 rows by 4096 -> 8192 (34 M) 14 us
//   here and 17 us there.
// - Up to 64 rows (32 with SwiGLU, whose partial sums take twice the shared memory): x below 128 K elements and
//   less than 192 M multiplications, since every CTA reads its slice of all rows of x.  17 rows by 7168 -> 384
//   7.2 us here, 8.2 as split tiles, 32 rows 8.5 and 7.7, 64 rows 10.8 and 8.3; 24 rows by 2048 -> 512 5.0 and
//   6.5; 64 rows by 2048 -> 1024 8.0 and 7.4.
bool is_small(int64_t M, int64_t N, int K, bool gated)
{
    return K % 8 == 0 && (M <= 16 ? N * K < 48000000 : M <= (gated ? 32 : 64) && M * K < 128000 && M * N * K < 192000000);
}

int launch_small(const SmallArgs &args, int type, cudaStream_t s)
{
    SmallArgs a = args;
    const bool gated = a.epi.act == kActSwiglu;
    // 32 weight rows a CTA halve the reads of x; 16 where that leaves SMs without a CTA
    const bool two = gated || (a.M <= 16 && a.N >= 32 * 296);
    const int tiles = (a.epi.n_cols + (two && !gated ? 31 : 15)) / (two && !gated ? 32 : 16);
    // k is shared by the CTAs of a cluster as long as all CTAs are resident at once (their registers allow one
    // to four an SM) and each warp keeps 64 elements: 8 rows of 7168 -> 4096 with SwiGLU 15.5 us as 256
    // CTAs, 18 as 512, of which 444 are resident
    const int resident = 2 * kPairs * (a.M > 32 ? 1 : a.M > 16 ? 2 : (two ? 3 : 4) - (a.M > 8));
    int ranks = 1;
    while (ranks < kMaxCluster && tiles * ranks * 2 <= resident && a.K >= 64 * kSmallWarps * ranks * 2)
        ranks *= 2;
    a.k_warp = (int)round_up((a.K + kSmallWarps * ranks - 1) / (kSmallWarps * ranks), 32);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(tiles * ranks);
    cfg.blockDim = dim3(kSmallWarps * 32);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = ranks;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    cudaError_t ce = cudaSuccess;
    by_half(type, [&](auto zero) {
        using T = decltype(zero);
        auto pick = [&](auto is_short) {
            constexpr bool kS = decltype(is_short)::value;
            return gated ? (a.M <= 8    ? small_kernel<T, 2, 1, true, kS>
                            : a.M <= 16 ? small_kernel<T, 2, 2, true, kS>
                                        : small_kernel<T, 2, 4, true, kS>)
                   : two ? (a.M <= 8 ? small_kernel<T, 2, 1, false, kS> : small_kernel<T, 2, 2, false, kS>)
                         : (a.M <= 8    ? small_kernel<T, 1, 1, false, kS>
                            : a.M <= 16 ? small_kernel<T, 1, 2, false, kS>
                            : a.M <= 32 ? small_kernel<T, 1, 4, false, kS>
                                        : small_kernel<T, 1, 8, false, kS>);
        };
        const bool is_short = a.k_warp > (a.epi.out_type == kTypeF32 ? kSmallChain : kBk << run_log(type));
        auto kernel = is_short ? pick(std::true_type()) : pick(std::false_type());
        ce = cudaLaunchKernelEx(&cfg, kernel, a);
    });
    return ce == cudaSuccess ? MOE_MX_OK : cuda_fail(ce, "linear launch");
}

template <int BN, bool kAMn, bool kBMn, bool kSum, bool kSwap = false>
int launch_gemm(const Gemm &g, const CUtensorMap &ma, const CUtensorMap &mb, const MoreMaps &mc, int tiles, cudaStream_t s)
{
    auto kernel = gemm_kernel<BN, kAMn, kBMn, kSum, kSwap>;
    // per device and cheap; nothing to remember between calls
    cudaError_t ce = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<BN, kSwap>::kSmem);
    if (ce != cudaSuccess)
        return cuda_fail(ce, "cudaFuncSetAttribute(linear)");
    const int pairs = tiles < kPairs ? tiles : kPairs;
    ce = launch_kernel(kernel, dim3(2 * pairs), dim3(kThreads), Cfg<BN, kSwap>::kSmem, s, true, g, ma, mb, mc);
    return ce == cudaSuccess ? MOE_MX_OK : cuda_fail(ce, "linear product launch");
}

// A product's operands as the kernel reads them: pointer, contiguous extent, rows, elements per row.
struct Operand {
    const void *p;
    int64_t inner, rows, ld;
    int experts; // planes of rows (B of a rows-segmented product), else 1
};

// rank 2 (x of kSwap, one plane) or 3; box of 64 elements x box_rows rows.
int make_map(CUtensorMap *map, const Operand &o, int box_rows, bool three)
{
    const cuuint64_t dims[3] = {(cuuint64_t)o.inner, (cuuint64_t)o.rows, (cuuint64_t)o.experts};
    const cuuint64_t strides[2] = {(cuuint64_t)o.ld * 2, (cuuint64_t)o.ld * 2 * o.rows};
    const cuuint32_t box[3] = {64, (cuuint32_t)box_rows, 1};
    return encode_nd(map, CU_TENSOR_MAP_DATA_TYPE_UINT16, three ? 3 : 2, o.p, dims, strides, box);
}

// An operand whose contiguous dimension is M or N, in boxes of 64 rows of k x `groups` groups of 64 elements
// when its rows are whole groups (wide), else of one group (a group may not run over the last row's end).
int make_map_mn(CUtensorMap *map, const Operand &o, int groups, int *wide)
{
    *wide = o.inner % 64 == 0;
    if (!*wide)
        return make_map(map, o, 64, true);
    const cuuint64_t dims[4] = {64, (cuuint64_t)o.rows, (cuuint64_t)o.inner / 64, (cuuint64_t)o.experts};
    const cuuint64_t strides[3] = {(cuuint64_t)o.ld * 2, 128, (cuuint64_t)o.ld * 2 * o.rows};
    const cuuint32_t box[4] = {64, 64, (cuuint32_t)groups, 1};
    return encode_nd(map, CU_TENSOR_MAP_DATA_TYPE_UINT16, 4, o.p, dims, strides, box);
}

// tiles: an upper bound of the product's tiles (the kernel finds a grouped product's on the device)
template <bool kAMn, bool kBMn>
int run_gemm(Gemm &g, int bn, bool sum, const Operand &a, const Operand &b, int64_t tiles, cudaStream_t s,
             const MoreMaps &more = MoreMaps{})
{
    if (tiles > INT32_MAX)
        return fail(MOE_MX_ERR_UNSUPPORTED, "the product has %lld tiles", (long long)tiles);
    CUtensorMap ma, mb;
    int rc;
    if ((rc = kAMn ? make_map_mn(&ma, a, 2, &g.wide_a) : make_map(&ma, a, 128, false)) ||
        (rc = kBMn ? make_map_mn(&mb, b, bn / 128, &g.wide_b) : make_map(&mb, b, bn / 2, true)))
        return rc;
    if constexpr (!kBMn)
        if (sum)
            return bn == 192 ? launch_gemm<192, kAMn, kBMn, true>(g, ma, mb, more, (int)tiles, s)
                             : launch_gemm<128, kAMn, kBMn, true>(g, ma, mb, more, (int)tiles, s);
    if (bn == 256)
        return launch_gemm<256, kAMn, kBMn, false>(g, ma, mb, more, (int)tiles, s);
    if constexpr (!kBMn)
        if (bn == 192)
            return launch_gemm<192, kAMn, kBMn, false>(g, ma, mb, more, (int)tiles, s);
    return launch_gemm<128, kAMn, kBMn, false>(g, ma, mb, more, (int)tiles, s);
}

// The same with the weights as A: w rows (or, kWMn, its columns) and `tok` token rows of x.
template <bool kWMn>
int run_swap(Gemm &g, bool sum, const Operand &x, const Operand &w, int64_t tiles, cudaStream_t s)
{
    if (tiles > INT32_MAX)
        return fail(MOE_MX_ERR_UNSUPPORTED, "the product has %lld tiles", (long long)tiles);
    CUtensorMap ma, mb;
    MoreMaps mc;
    int rc;
    if (g.gated) {
        // 16 gate rows, then the 16 up rows of the same columns, four times: lanes of one warp hold both
        const cuuint64_t row = (cuuint64_t)w.ld * 2, half = (cuuint64_t)w.rows / 2;
        const cuuint64_t dims[5] = {(cuuint64_t)w.inner, 16, 2, half / 16, (cuuint64_t)w.experts};
        const cuuint64_t strides[4] = {row, row * half, row * 16, row * w.rows};
        const cuuint32_t box[5] = {64, 16, 2, 4, 1};
        rc = encode_nd(&ma, CU_TENSOR_MAP_DATA_TYPE_UINT16, 5, w.p, dims, strides, box);
    } else {
        rc = kWMn ? make_map_mn(&ma, w, 2, &g.wide_a) : make_map(&ma, w, 128, true);
    }
    // the boxes that the tiles may use: a dense product's are tiles of g.tok tokens, and a shorter last one
    const int most = g.seg.E ? 256 : g.tok;
    if (rc || (rc = make_map(&mb, x, most > 128 ? 128 : 16, false)))
        return rc;
    for (int i = 0; i < 3; ++i)
        if ((i == 0 || most > 16 << i) && (rc = make_map(&mc.m[i], x, 16 << i, false)))
            return rc;
    if constexpr (!kWMn)
        if (sum)
            return launch_gemm<256, kWMn, false, true, true>(g, ma, mb, mc, (int)tiles, s);
    return launch_gemm<256, kWMn, false, false, true>(g, ma, mb, mc, (int)tiles, s);
}

// ---------------------------------------------------------------- dz and the bias gradient
__device__ __forceinline__ float warp_max(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
    return v;
}

struct DzArgs {
    const void *dout, *preact;
    void *dz;           // [M, ldz] or nullptr
    float *part;        // [ceil(M / 128)][N] column sums of each 128-row block, or nullptr
    const float *scale; // of each expert's dz, or nullptr
    float *most;        // kMost: [ceil(M / 128)][ceil(n_out / 64)]
    Segments seg;
    int N, n_out, ldz, act;
};

// One CTA: 128 rows x 64 columns of dout (8 lanes x 8 columns, 32 row lanes x 4 rows).  The column
// sums of a block are added in a fixed order.  kDzMost: nothing but the largest finite |dz| of the block;
// kDzScaled: dz times its expert's scale (an instance of its own: the multiplications' registers cost the plain one
// a CTA an SM, 5.3 us -> 6.2 us at 512 x 4096).
enum DzMode { kDzPlain, kDzMost, kDzScaled };
template <typename T, typename TO, int V, DzMode kMode> __global__ void __launch_bounds__(256) dz_kernel(const DzArgs a)
{
    constexpr bool kMost = kMode == kDzMost;
    __shared__ float red[32][65];
    const int64_t m0 = (int64_t)blockIdx.x * 128;
    int e;
    int64_t end;
    grid_dep_wait();
    grid_dep_launch();
    const bool any = find_segment(a.seg, m0, e, end);
    if (!any)
        return; // a block of padding, or past the last segment
    const bool gated = a.act == kActSwiglu;
    const int cl = threadIdx.x % 8, rl = threadIdx.x / 8;
    const float scale = kMode == kDzScaled ? a.scale[e] : 1.f;
    float sum[2][8] = {}, most = 0.f;
    auto finite = [](float v) { return fabsf(v) <= 3.402823466e38f ? fabsf(v) : 0.f; };
    for (int v = 0; v < 8; v += V) {
        const int n = blockIdx.y * 64 + cl * 8 + v;
        if (n >= a.n_out)
            break;
        // the loads of all four rows before the first use
        Raw<TO, V> rd[4];
        Raw<T, V> rz[4], ru[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t m = m0 + i * 32 + rl;
            if (m >= end)
                continue;
            rd[i].load(static_cast<const TO *>(a.dout) + m * a.n_out + n);
            if (a.act != kActNone)
                rz[i].load(static_cast<const T *>(a.preact) + m * a.N + n);
            if (gated)
                ru[i].load(static_cast<const T *>(a.preact) + m * a.N + n + a.n_out);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t m = m0 + i * 32 + rl;
            if (m >= end)
                continue;
            float d[V], z[V], u[V], dz[V], du[V];
            rd[i].get(d);
            if (gated) {
                rz[i].get(z);
                ru[i].get(u);
#pragma unroll
                for (int q = 0; q < V; ++q) {
                    const float sg = sigmoid(z[q]);
                    dz[q] = d[q] * u[q] * (sg * (1.f + z[q] * (1.f - sg)));
                    du[q] = d[q] * z[q] * sg;
                    sum[0][v + q] += dz[q];
                    sum[1][v + q] += du[q];
                }
            } else {
                if (a.act != kActNone)
                    rz[i].get(z);
#pragma unroll
                for (int q = 0; q < V; ++q) {
                    dz[q] = a.act == kActNone ? d[q] : d[q] * act_grad(z[q], a.act);
                    sum[0][v + q] += dz[q];
                }
            }
            if (kMost) {
#pragma unroll
                for (int q = 0; q < V; ++q)
                    most = fmaxf(most, gated ? fmaxf(finite(dz[q]), finite(du[q])) : finite(dz[q]));
            } else if (a.dz) {
                T *o = static_cast<T *>(a.dz) + m * a.ldz + n;
                if (kMode == kDzScaled) {
#pragma unroll
                    for (int q = 0; q < V; ++q) {
                        dz[q] *= scale;
                        if (gated)
                            du[q] *= scale;
                    }
                }
                Raw<T, V>::put(o, dz);
                if (gated)
                    Raw<T, V>::put(o + a.n_out, du);
            }
        }
    }
    if (kMost) {
        __shared__ float largest[8];
        const float m = warp_max(most);
        if (threadIdx.x % 32 == 0)
            largest[threadIdx.x / 32] = m;
        __syncthreads();
        if (threadIdx.x < 32) {
            const float b = warp_max(threadIdx.x < 8 ? largest[threadIdx.x] : 0.f);
            if (threadIdx.x == 0)
                a.most[(size_t)blockIdx.x * gridDim.y + blockIdx.y] = b;
        }
        return;
    }
    if (!a.part)
        return;
    for (int h = 0; h < (gated ? 2 : 1); ++h) {
#pragma unroll
        for (int v = 0; v < 8; ++v)
            red[rl][cl * 8 + v] = h ? sum[1][v] : sum[0][v];
        __syncthreads();
        if (threadIdx.x < 64) {
            const int n = blockIdx.y * 64 + threadIdx.x;
            float t = 0.f;
            for (int r = 0; r < 32; ++r)
                t += red[r][threadIdx.x];
            if (n < a.n_out)
                a.part[(size_t)blockIdx.x * a.N + h * a.n_out + n] = t;
        }
        __syncthreads();
    }
}

// The power of two that takes a segment's largest finite |dz| to [2^14, 2^15), and its inverse (after all
// experts' scales): float16 then holds to half a step what is down to 2^-28 of the largest, and the rest to
// 2^-39 of it, whatever the range of dout.  One CTA per expert over its blocks' maxima.
__global__ void __launch_bounds__(1024) scale_kernel(const float *block_most, int per_block, Segments seg, float *scale)
{
    grid_dep_wait();
    grid_dep_launch();
    __shared__ float largest[32];
    const int e = blockIdx.x;
    int first = 0;
    const int64_t rows = seg.E ? segment_rows(seg, e, first) : seg.M;
    const int64_t n = (rows + 127) / 128 * per_block;
    const float *p = block_most + (size_t)(first / 128) * per_block;
    float m = 0.f;
#pragma unroll 4
    for (int64_t i = threadIdx.x; i < n; i += 1024)
        m = fmaxf(m, p[i]);
    m = warp_max(m);
    if (threadIdx.x % 32 == 0)
        largest[threadIdx.x / 32] = m;
    __syncthreads();
    if (threadIdx.x < 32) {
        m = warp_max(largest[threadIdx.x]);
        if (threadIdx.x == 0) {
            const int exponent = (int)(__float_as_uint(m) >> 23) - 127; // -127: zero or subnormal
            const int up = m == 0.f ? 0 : min(14 - exponent, 126);      // 14 - 127 at least
            scale[e] = __uint_as_float((uint32_t)(127 + up) << 23);
            scale[gridDim.x + e] = __uint_as_float((uint32_t)(127 - up) << 23);
        }
    }
}

// What a gradient needs of dz beside the products, in one launch.
//
// dbias[e][n]: the sum of the segment's 128-row blocks, 4 threads to a column, in a fixed order.
//
// Last k blocks: dw of grouped rows takes a segment in 64-row blocks of k.  The last one's rows behind the
// segment are padding, which may hold anything, so that block of dz and of x is copied with zeros
// behind its rows (clearing it in shared memory instead held every tile up by about a microsecond).
struct AfterArgs {
    const float *part;
    float *dbias;           // nullptr: none
    int N, bias_blocks;     // CTAs of dbias: columns / 64 per expert
    const uint16_t *src[2]; // dz, x; nullptr: no copies
    uint16_t *dst[2];       // [E][64][ld]
    int ld[2];              // elements per row, multiples of 8
    Segments seg;
};

constexpr int kCutRows = 4; // rows of a copy that one CTA takes

__global__ void __launch_bounds__(256) after_kernel(const AfterArgs a)
{
    grid_dep_wait(); // dz and its blocks' sums
    grid_dep_launch();
    __shared__ float s[4][64];
    const int e = blockIdx.y;
    int first = 0;
    const int64_t rows = a.seg.E ? segment_rows(a.seg, e, first) : a.seg.M;
    if ((int)blockIdx.x < a.bias_blocks) {
        const int c = threadIdx.x & 63, g = threadIdx.x >> 6, n = blockIdx.x * 64 + c;
        const int64_t blocks = (rows + 127) / 128;
        float t = 0.f;
        if (n < a.N) {
            const float *p = a.part + (size_t)(first / 128) * a.N + n;
#pragma unroll 4
            for (int64_t b = g; b < blocks; b += 4)
                t += p[b * a.N];
        }
        s[g][c] = t;
        __syncthreads();
        if (g == 0 && n < a.N)
            a.dbias[(size_t)e * a.N + n] = (s[0][c] + s[1][c]) + (s[2][c] + s[3][c]);
        return;
    }
    const int rem = (int)(rows % kBk);
    if (rem == 0)
        return;
    const int i = blockIdx.x - a.bias_blocks, o = i & 1, r0 = (i >> 1) * kCutRows;
    const uint16_t *src = a.src[o] + (size_t)(first + rows - rem) * a.ld[o];
    uint16_t *dst = a.dst[o] + (size_t)e * kBk * a.ld[o];
    for (int r = r0; r < r0 + kCutRows; ++r)
        for (int c = threadIdx.x * 8; c < a.ld[o]; c += 256 * 8)
            *reinterpret_cast<uint4 *>(dst + (size_t)r * a.ld[o] + c) =
                r < rem ? *reinterpret_cast<const uint4 *>(src + (size_t)r * a.ld[o] + c) : make_uint4(0, 0, 0, 0);
}

int ldz_of(int N) { return (int)round_up(N, 8); }

bool dz_is_dout(int act, int type, int dout_type, int N) { return act == kActNone && type == dout_type && N % 8 == 0; }


// Workspace parts of a call, in order; an absent part has no bytes.
struct Parts {
    int64_t at = 0;
    int64_t take(int64_t bytes)
    {
        const int64_t o = at;
        at += round_up(bytes, 256);
        return o;
    }
};

// Workspace of a product of kb k blocks whose tiles may have more than one run of them.
int64_t held_bytes(const Plan &p, int64_t kb, int type)
{
    return !p.sum && (kb + p.splits - 1) / p.splits > 1 << run_log(type) ? kHeldBytes : 0;
}

struct ForwardPlan {
    Plan p;
    int64_t x, w, planes, held, bytes;
};
ForwardPlan plan_linear(int E, int64_t M, int N, int K, int act, int type, bool f32)
{
    ForwardPlan f{};
    if (E == 0 && is_small(M, N, K, act == kActSwiglu))
        return f;
    const bool gated = act == kActSwiglu;
    const bool swap = !gated || N % 32 == 0; // gate and up rows are taken 16 by 16
    const int kb = (K + kBk - 1) / kBk;
    if (E == 0) {
        // a gated product is one of N columns in tiles of the gate's and the up's; a split one is plain
        f.p = plan_dense(M, N, kb, gated, false, f32, swap);
    } else {
        const bool sum = f32 && kb > kChain;
        f.p = Plan{swap ? 256 : 128, 1, sum, swap ? 256 : 0};
    }
    Parts ws;
    f.x = ws.take(K % 8 ? M * round_up(K, 8) * 2 : 0);
    f.w = ws.take(K % 8 ? (E ? E : 1) * (int64_t)N * round_up(K, 8) * 2 : 0);
    f.planes = ws.take(f.p.splits > 1 ? f.p.splits * M * N * 4 : 0);
    f.held = ws.take(held_bytes(f.p, kb, type));
    f.bytes = ws.at;
    return f;
}

struct BackwardPlan {
    bool direct;
    Plan dx, dw;
    int64_t part, most, scale, dz, x, w, planes, held, cut_a, cut_b, bytes;
};
bool dz_is_scaled(int type, int dout_type) { return type == kTypeF16 && dout_type == kTypeF32; }

BackwardPlan plan_backward(int E, int64_t M, int N, int K, int act, int type, int dout_type)
{
    BackwardPlan f{};
    f.direct = dz_is_dout(act, type, dout_type, N);
    f.dx = Plan{256, 1, false, 256};
    f.dw = Plan{256, 1, false, 0};
    if (E == 0)
        f.dw = plan_dense(N, K, (int)((M + kBk - 1) / kBk), false, true, false, false);
    if (E == 0 && M > 0) {
        f.dx = plan_dense(M, K, (N + kBk - 1) / kBk, false, true, false, true);
    }
    Parts ws;
    f.part = ws.take((M + 127) / 128 * N * 4);
    const bool scaled = dz_is_scaled(type, dout_type);
    f.most = ws.take(scaled ? (M + 127) / 128 * (((act == kActSwiglu ? N / 2 : N) + 63) / 64) * 4 : 0);
    f.scale = ws.take(scaled ? 2 * (E ? E : 1) * 4 : 0);
    f.dz = ws.take(f.direct ? 0 : M * ldz_of(N) * 2);
    f.x = ws.take(K % 8 ? M * round_up(K, 8) * 2 : 0);
    f.w = ws.take(K % 8 ? (E ? E : 1) * (int64_t)N * round_up(K, 8) * 2 : 0);
    // dx's planes, then (dx is summed by then) dw's
    const int64_t px = f.dx.splits > 1 ? f.dx.splits * M * K * 4 : 0;
    const int64_t pw = f.dw.splits > 1 ? (int64_t)f.dw.splits * N * K * 4 : 0;
    f.planes = ws.take(px > pw ? px : pw);
    // the sums of long tiles likewise; a grouped dw's depth is known on the device: at most all rows
    const int64_t hx = M > 0 ? held_bytes(f.dx, (N + kBk - 1) / kBk, type) : 0;
    const int64_t hw = held_bytes(f.dw, (M + kBk - 1) / kBk, type);
    f.held = ws.take(hx > hw ? hx : hw);
    f.cut_a = ws.take((int64_t)E * kBk * ldz_of(N) * 2);
    f.cut_b = ws.take((int64_t)E * kBk * round_up(K, 8) * 2);
    f.bytes = ws.at;
    return f;
}

// The sum of a split product's planes, through the epilogue.
int launch_reduce(const float *planes, int splits, int64_t M, const Epi &e, cudaStream_t s)
{
    cudaError_t ce = cudaSuccess;
    by_half(e.type, [&](auto zero) {
        using T = decltype(zero);
        auto kernel = e.act == kActSwiglu ? reduce_kernel<T, true> : reduce_kernel<T, false>;
        ce = launch_kernel(kernel, dim3((unsigned)((M * e.n_cols + 255) / 256)), dim3(256), 0, s, true, planes, splits, (int)M, e);
    });
    return ce == cudaSuccess ? MOE_MX_OK : cuda_fail(ce, "split sum launch");
}

Epi epilogue_of(const Gemm &g)
{
    return Epi{g.bias, g.residual, g.out, g.preact, g.act, g.N, g.n_cols, g.type, g.out_type, g.vec};
}

// Turn a dense product into one that writes its splits' float32 planes.
void split_out(Gemm &g, int splits, int kb, int N, void *planes)
{
    g.splits = splits;
    g.kb_split = (kb + splits - 1) / splits;
    g.splits = (kb + g.kb_split - 1) / g.kb_split;
    if (splits == 1)
        return;
    g.gated = 0, g.n_cols = N, g.act = kActNone;
    g.bias = nullptr, g.residual = nullptr, g.preact = nullptr;
    g.out = planes, g.out_type = kTypeF32;
}

} // namespace

int64_t linear_workspace(int E, int64_t M, int N, int K, int act, int type, int out_type)
{
    return plan_linear(E, M, N, K, act, type, out_type == kTypeF32).bytes;
}

int64_t linear_backward_workspace(int E, int64_t M, int N, int K, int act, int type, int dout_type)
{
    return plan_backward(E, M, N, K, act, type, dout_type).bytes;
}

void linear_plan(int which, int E, int64_t M, int N, int K, int act, int type, int io_type, int *o)
{
    if (which == 0 && E == 0 && is_small(M, N, K, act == kActSwiglu)) {
        o[0] = o[1] = o[2] = o[3] = 0;
        return;
    }
    const Plan p = which == 0   ? plan_linear(E, M, N, K, act, type, io_type == kTypeF32).p
                   : which == 1 ? plan_backward(E, M, N, K, act, type, io_type).dx
                                : plan_backward(E, M, N, K, act, type, io_type).dw;
    o[0] = p.bn, o[1] = p.tok, o[2] = p.splits, o[3] = p.sum;
}

int launch_linear(const LinearArgs &a, cudaStream_t s)
{
    if (a.E == 0 && is_small(a.M, a.N, a.K, a.act == kActSwiglu)) {
        const SmallArgs m{a.x, a.w, (int)a.M, a.N, a.K, 0,
                          Epi{a.bias, a.residual, a.out, a.preact, a.act, a.N, a.No(), a.type, a.out_type, 0}};
        return launch_small(m, a.type, s);
    }
    const ForwardPlan f = plan_linear(a.E, a.M, a.N, a.K, a.act, a.type, a.out_type == kTypeF32);
    char *ws = static_cast<char *>(a.ws);
    const int ld = (int)round_up(a.K, 8), experts = a.E ? a.E : 1;
    const Segments seg{a.counts, a.pad_offsets, a.E, a.M};
    const void *xk = a.x, *wk = a.w;
    const cudaError_t ce = launch_pack(xk, a.M, seg, ws + f.x, wk, (int64_t)experts * a.N, ws + f.w, a.K, s);
    if (ce != cudaSuccess)
        return cuda_fail(ce, "operand copy launch");
    const Operand x{xk, a.K, a.M, ld, 1};
    const Operand w{wk, a.K, a.N, ld, experts};
    Gemm g{};
    g.seg = seg;
    g.M = (int)a.M, g.n_cols = a.No(), g.N = a.N, g.K = a.K;
    g.gated = a.act == kActSwiglu, g.act = a.act, g.fmt = a.type == kTypeBf16;
    g.bias = a.bias, g.residual = a.residual, g.out = a.out, g.preact = a.preact;
    g.type = a.type, g.out_type = a.out_type, g.vec = g.n_cols % 8 == 0;
    g.run_log = run_log(a.type), g.held = reinterpret_cast<float4 *>(ws + f.held);
    const Epi ep = epilogue_of(g);
    const int kb = (a.K + kBk - 1) / kBk;
    split_out(g, f.p.splits, kb, a.N, ws + f.planes);
    int rc;
    if (f.p.tok) {
        g.nt = (g.n_cols + (g.gated ? 127 : 255)) / (g.gated ? 128 : 256);
        g.tok = f.p.tok;
        g.mt = (int)((a.M + g.tok - 1) / g.tok);
        const int most = f.p.sum ? 128 : 256; // grouped: every expert hit has at most one part-filled tile
        const int64_t mt = a.E ? a.M / most + a.E : g.mt;
        rc = run_swap<false>(g, f.p.sum, x, w, mt * g.nt * g.splits, s);
    } else {
        const int bn = g.gated ? f.p.bn / 2 : f.p.bn;
        g.nt = (g.n_cols + bn - 1) / bn;
        g.mt = (int)((a.M + kTileM - 1) / kTileM);
        const int64_t mt = a.E ? a.M / kTileM + a.E : g.mt;
        rc = run_gemm<false, false>(g, f.p.bn, f.p.sum, x, w, mt * g.nt * g.splits, s);
    }
    if (rc || g.splits == 1)
        return rc;
    return launch_reduce(reinterpret_cast<float *>(ws + f.planes), g.splits, a.M, ep, s);
}

int launch_linear_backward(const LinearBackwardArgs &a, cudaStream_t s)
{
    const Segments seg{a.counts, a.pad_offsets, a.E, a.M};
    const BackwardPlan f = plan_backward(a.E, a.M, a.N, a.K, a.act, a.type, a.dout_type);
    char *ws = static_cast<char *>(a.ws);
    float *part = reinterpret_cast<float *>(ws + f.part);
    DzArgs d{};
    d.dout = a.dout, d.preact = a.preact, d.seg = seg;
    d.N = a.N, d.n_out = a.No(), d.ldz = ldz_of(a.N), d.act = a.act;
    d.part = a.dbias ? part : nullptr;
    if (!f.direct && (a.dx || a.dw))
        d.dz = ws + f.dz;
    const int experts = a.E ? a.E : 1;
    const float *unscale = nullptr;
    if (a.M > 0 && (d.part || d.dz)) {
        const dim3 grid((unsigned)((a.M + 127) / 128), (d.n_out + 63) / 64);
        const bool vec = d.n_out % 8 == 0;
        if (d.dz && dz_is_scaled(a.type, a.dout_type)) {
            float *scale = reinterpret_cast<float *>(ws + f.scale);
            d.most = reinterpret_cast<float *>(ws + f.most);
            cudaError_t ce = launch_kernel(vec ? dz_kernel<__half, float, 8, kDzMost> : dz_kernel<__half, float, 1, kDzMost>,
                                           grid, dim3(256), 0, s, true, d);
            if (ce == cudaSuccess)
                ce = launch_kernel(scale_kernel, dim3(experts), dim3(1024), 0, s, true, d.most, (int)grid.y, seg, scale);
            d.scale = scale, unscale = scale + experts;
            if (ce == cudaSuccess)
                ce = launch_kernel(vec ? dz_kernel<__half, float, 8, kDzScaled> : dz_kernel<__half, float, 1, kDzScaled>,
                                   grid, dim3(256), 0, s, true, d);
            if (ce != cudaSuccess)
                return cuda_fail(ce, "scaled gradient launch");
        } else {
            by_half(a.type, [&](auto x) {
                using T = decltype(x);
                auto go = [&](auto y) {
                    using TO = decltype(y);
                    launch_kernel(vec ? dz_kernel<T, TO, 8, kDzPlain> : dz_kernel<T, TO, 1, kDzPlain>, grid, dim3(256), 0,
                                  s, true, d);
                };
                if (a.dout_type == kTypeF32)
                    go(float());
                else
                    go(T());
            });
        }
    }
    const void *dz = f.direct ? a.dout : d.dz;
    const int ldz = f.direct ? a.N : d.ldz, ldk = (int)round_up(a.K, 8);
    // x and w with aligned rows, where a product reads them
    const void *xk = a.dw && a.M > 0 ? a.x : nullptr, *wk = a.dx && a.M > 0 ? a.w : nullptr;
    cudaError_t pe = launch_pack(xk, a.M, seg, ws + f.x, wk, (int64_t)experts * a.N, ws + f.w, a.K, s);
    if (pe != cudaSuccess)
        return cuda_fail(pe, "operand copy launch");
    const bool cut = a.dw && a.E && a.M > 0;
    if (a.dbias || cut) {
        AfterArgs p{};
        p.seg = seg, p.part = part, p.dbias = a.dbias, p.N = a.N;
        p.bias_blocks = a.dbias ? (a.N + 63) / 64 : 0;
        if (cut) {
            p.src[0] = static_cast<const uint16_t *>(dz), p.src[1] = static_cast<const uint16_t *>(xk);
            p.dst[0] = reinterpret_cast<uint16_t *>(ws + f.cut_a), p.dst[1] = reinterpret_cast<uint16_t *>(ws + f.cut_b);
            p.ld[0] = ldz, p.ld[1] = ldk;
        }
        const dim3 grid(p.bias_blocks + (cut ? 2 * kBk / kCutRows : 0), experts);
        const cudaError_t ce = launch_kernel(after_kernel, grid, dim3(256), 0, s, true, p);
        if (ce != cudaSuccess)
            return cuda_fail(ce, "bias gradient launch");
    }
    int rc;
    if (a.dx && a.M > 0) {
        const Operand oa{dz, a.N, a.M, ldz, 1};
        const Operand ob{wk, a.K, a.N, ldk, experts};
        Gemm g{};
        g.seg = seg, g.M = (int)a.M, g.n_cols = g.N = a.K, g.K = a.N;
        g.fmt = a.type == kTypeBf16, g.out = a.dx, g.type = g.out_type = a.type, g.vec = a.K % 8 == 0;
        g.run_log = run_log(a.type), g.held = reinterpret_cast<float4 *>(ws + f.held), g.unscale = unscale;
        const int kb = (a.N + kBk - 1) / kBk;
        const Epi ep = epilogue_of(g);
        split_out(g, f.dx.splits, kb, a.K, ws + f.planes);
        if (f.dx.tok) {
            g.nt = (a.K + 255) / 256, g.tok = f.dx.tok;
            g.mt = (int)((a.M + g.tok - 1) / g.tok);
            const int64_t mt = a.E ? a.M / 256 + a.E : g.mt;
            rc = run_swap<true>(g, false, oa, ob, mt * g.nt * g.splits, s);
        } else {
            const int bn = f.dx.bn;
            g.nt = (a.K + bn - 1) / bn;
            g.mt = (int)((a.M + kTileM - 1) / kTileM);
            rc = run_gemm<false, true>(g, bn, false, oa, ob, (int64_t)g.mt * g.nt * g.splits, s);
        }
        if (rc)
            return rc;
        if (g.splits > 1 && (rc = launch_reduce(reinterpret_cast<float *>(ws + f.planes), g.splits, a.M, ep, s)))
            return rc;
    }
    if (a.dw) {
        if (a.M == 0) { // no rows: zeros
            const cudaError_t ce = cudaMemsetAsync(a.dw, 0, (size_t)experts * a.N * a.K * 2, s);
            return ce == cudaSuccess ? MOE_MX_OK : cuda_fail(ce, "cudaMemsetAsync(dw)");
        }
        const Operand oa{dz, a.N, a.M, ldz, 1};
        const Operand ob{xk, a.K, a.M, ldk, 1};
        Gemm g{};
        g.seg = seg, g.seg_k = 1, g.M = a.N, g.n_cols = g.N = a.K, g.K = (int)a.M;
        g.d_expert = (int64_t)a.N * a.K;
        g.run_log = run_log(a.type), g.held = reinterpret_cast<float4 *>(ws + f.held), g.unscale = unscale;
        g.fmt = a.type == kTypeBf16, g.out = a.dw, g.type = g.out_type = a.type, g.vec = a.K % 8 == 0;
        const Epi ep = epilogue_of(g);
        split_out(g, f.dw.splits, (int)((a.M + kBk - 1) / kBk), a.K, ws + f.planes);
        if (a.E == 0)
            g.seg_k = 0; // one segment: k ends with the rows, where the copies read zeros
        g.nt = (a.K + f.dw.bn - 1) / f.dw.bn;
        g.mt = (a.N + kTileM - 1) / kTileM;
        MoreMaps more{};
        if (a.E) {
            const Operand ca{ws + f.cut_a, a.N, (int64_t)a.E * kBk, ldz, 1}, cb{ws + f.cut_b, a.K, (int64_t)a.E * kBk, ldk, 1};
            int wide; // as of the operands themselves
            if ((rc = make_map_mn(&more.m[0], ca, 2, &wide)) || (rc = make_map_mn(&more.m[1], cb, f.dw.bn / 128, &wide)))
                return rc;
        }
        if ((rc = run_gemm<true, true>(g, f.dw.bn, false, oa, ob, (int64_t)g.mt * g.nt * (a.E ? a.E : g.splits), s, more)))
            return rc;
        if (g.splits > 1)
            return launch_reduce(reinterpret_cast<float *>(ws + f.planes), g.splits, a.N, ep, s);
    }
    return MOE_MX_OK;
}

int linear_watchdog(unsigned long long timeout_ns, cudaStream_t s)
{
    void *word = nullptr;
    const cudaError_t ce = cudaGetSymbolAddress(&word, g_linear_err);
    if (ce != cudaSuccess)
        return cuda_fail(ce, "cudaGetSymbolAddress(error word)");
    launch_watchdog(static_cast<uint32_t *>(word), timeout_ns, s);
    return MOE_MX_OK;
}

int linear_status(cudaStream_t s)
{
    cudaError_t ce = cudaStreamSynchronize(s);
    if (ce != cudaSuccess)
        return cuda_fail(ce, "cudaStreamSynchronize");
    uint32_t word = 0;
    if ((ce = cudaMemcpyFromSymbol(&word, g_linear_err, sizeof(word))) != cudaSuccess)
        return cuda_fail(ce, "cudaMemcpyFromSymbol(error word)");
    if (word == 0)
        return MOE_MX_OK;
    const uint32_t zero = 0;
    cudaMemcpyToSymbol(g_linear_err, &zero, sizeof(zero));
    return fail(MOE_MX_ERR_TIMEOUT, "a device-side wait gave up (error word 0x%x)", word);
}

} // namespace moe_mx
