// permute.cu -- token rows to the grouped (sorted by expert) layout and back: dispatch, the
// weighted combine and its gradient.  Pair p = t*k + j of token t sits at grouped row pos[p]
// (outside [0, rows): no row, e.g. a pair of another shard's expert).  Token-major throughout, so a
// token's own row is read or written once and every grouped row once; no atomics.
#include "kernels.cuh"
#include "ptx.cuh"
#include "routed.cuh"
#include "vec.cuh"

namespace moe_mx {

namespace {

constexpr int kMaxSlots = 32;
// Slots whose rows are in flight together.  Measured (bf16): combine of 16384 x 4096, top-8: 2 rows 198 us,
// 4 rows 175, 8 rows 186 (fewer CTAs fit an SM); combine_backward of 8192 x 7168, top-8: 4 rows 325 us,
// 8 rows 314 (dout is read once for all).
constexpr int kCombineRows = 4, kBackwardRows = 8;

// Grouped rows of n slots of token t from j0; -1: none.
template <int n> __device__ __forceinline__ void slot_rows(const PermuteArgs &a, int t, int j0, int (&row)[n])
{
#pragma unroll
    for (int j = 0; j < n; ++j) {
        row[j] = -1;
        if (j0 + j < a.k) {
            const int r = a.pos[(size_t)t * a.k + j0 + j];
            row[j] = r >= 0 && r < a.rows ? r : -1;
        }
    }
}

// One thread per (token, vector of V elements): x is read once, each grouped row written once, and
// that traffic bounds it (177 us, 6.0 TB/s, at 8192 x 7168, top-8, mostly writes).
template <typename T, int V>
__global__ void __launch_bounds__(256) dispatch_kernel(const PermuteArgs a)
{
    grid_dep_wait();
    grid_dep_launch();
    const int t = blockIdx.x, c = (blockIdx.y * blockDim.x + threadIdx.x) * V;
    if (c >= a.H)
        return;
    Raw<T, V> v;
    v.load(static_cast<const T *>(a.tok) + (size_t)t * a.H + c);
    for (int j0 = 0; j0 < a.k; j0 += kBackwardRows) {
        int row[kBackwardRows];
        slot_rows(a, t, j0, row);
#pragma unroll
        for (int j = 0; j < kBackwardRows; ++j)
            if (row[j] >= 0)
                *reinterpret_cast<Raw<T, V> *>(static_cast<T *>(a.grouped_out) + (size_t)row[j] * a.H + c) = v;
    }
}

// out[t] = sum_j w[t,j] y[pos[t,j]], j ascending, in float32; one rounding at the end.  One thread per
// (token, vector), four rows' loads in flight: bound by y's bytes, read at 6.9 TB/s (16384 x 4096, top-8).
template <typename T, typename TO, int V>
__global__ void __launch_bounds__(256) combine_rows_kernel(const PermuteArgs a)
{
    grid_dep_wait();
    grid_dep_launch();
    const int t = blockIdx.x, c = (blockIdx.y * blockDim.x + threadIdx.x) * V;
    if (c >= a.H)
        return;
    float acc[V];
#pragma unroll
    for (int i = 0; i < V; ++i)
        acc[i] = 0.f;
    for (int j0 = 0; j0 < a.k; j0 += kCombineRows) {
        int row[kCombineRows];
        Raw<T, V> v[kCombineRows];
        slot_rows(a, t, j0, row);
#pragma unroll
        for (int j = 0; j < kCombineRows; ++j)
            if (row[j] >= 0)
                v[j].load(static_cast<const T *>(a.grouped) + (size_t)row[j] * a.H + c);
#pragma unroll
        for (int j = 0; j < kCombineRows; ++j)
            if (row[j] >= 0) {
                const float w = a.w ? a.w[(size_t)t * a.k + j0 + j] : 1.f;
                float f[V];
                v[j].get(f);
#pragma unroll
                for (int i = 0; i < V; ++i)
                    acc[i] = fmaf(w, f[i], acc[i]);
            }
    }
    Raw<TO, V>::put(static_cast<TO *>(a.tok_out) + (size_t)t * a.H + c, acc);
}

// One CTA per token: dy[pos] = w dout (one rounding), dw = <dout, y[pos]> (float32, a fixed order),
// and the gradient through w = softmax over the token's k chosen logits:
// dlogits[id_j] += w_j (dw_j - sum_i w_i dw_i), every other logit 0.  dout is read once for eight slots,
// whose rows are in flight together and whose dot products meet in one reduction.  Bound by its bytes:
// 6.4 TB/s at 8192 x 7168, top-8.
template <typename T, typename TO, int V>
__global__ void __launch_bounds__(256) combine_backward_kernel(const PermuteArgs a)
{
    grid_dep_wait();
    grid_dep_launch();
    __shared__ float s_part[8][kBackwardRows], s_dw[kMaxSlots], s_w[kMaxSlots];
    __shared__ int s_id[kMaxSlots];
    const int t = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    const bool dots = a.dw || a.dlogits;
    for (int j = threadIdx.x; j < a.k; j += blockDim.x) {
        s_w[j] = a.w[(size_t)t * a.k + j];
        s_id[j] = a.dlogits ? a.ids[(size_t)t * a.k + j] : -1;
    }
    __syncthreads();
    for (int j0 = 0; j0 < a.k; j0 += kBackwardRows) {
        int row[kBackwardRows];
        slot_rows(a, t, j0, row);
        float dot[kBackwardRows] = {};
        for (int c = threadIdx.x * V; c < a.H; c += blockDim.x * V) {
            Raw<TO, V> d;
            Raw<T, V> y[kBackwardRows];
            float f[V], g[V];
            d.load(static_cast<const TO *>(a.tok) + (size_t)t * a.H + c);
            if (dots) {
#pragma unroll
                for (int j = 0; j < kBackwardRows; ++j)
                    if (row[j] >= 0)
                        y[j].load(static_cast<const T *>(a.grouped) + (size_t)row[j] * a.H + c);
            }
            d.get(f);
            if (a.grouped_out) {
#pragma unroll
                for (int j = 0; j < kBackwardRows; ++j)
                    if (row[j] >= 0) {
                        const float w = s_w[j0 + j];
#pragma unroll
                        for (int i = 0; i < V; ++i)
                            g[i] = w * f[i];
                        Raw<T, V>::put(static_cast<T *>(a.grouped_out) + (size_t)row[j] * a.H + c, g);
                    }
            }
            if (dots) {
#pragma unroll
                for (int j = 0; j < kBackwardRows; ++j)
                    if (row[j] >= 0) {
                        y[j].get(g);
#pragma unroll
                        for (int i = 0; i < V; ++i)
                            dot[j] = fmaf(f[i], g[i], dot[j]);
                    }
            }
        }
        if (!dots)
            continue;
#pragma unroll
        for (int j = 0; j < kBackwardRows; ++j) {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
                dot[j] += __shfl_xor_sync(0xFFFFFFFFu, dot[j], o);
            if (lane == 0)
                s_part[warp][j] = dot[j];
        }
        __syncthreads();
        if (threadIdx.x < kBackwardRows && j0 + threadIdx.x < a.k) {
            float d = 0.f;
            for (int i = 0; i < nw; ++i)
                d += s_part[i][threadIdx.x];
            s_dw[j0 + threadIdx.x] = d;
            if (a.dw)
                a.dw[(size_t)t * a.k + j0 + threadIdx.x] = d;
        }
        __syncthreads();
    }
    if (!a.dlogits)
        return;
    float sum = 0.f;
    for (int j = 0; j < a.k; ++j)
        sum = fmaf(s_w[j], s_dw[j], sum);
    for (int e = threadIdx.x; e < a.E; e += blockDim.x) {
        float g = 0.f;
        for (int j = 0; j < a.k; ++j)
            if (s_id[j] == e)
                g += s_w[j] * (s_dw[j] - sum);
        a.dlogits[(size_t)t * a.E + e] = g;
    }
}

// Threads of a CTA and CTAs per token row for `n` vectors.
dim3 row_grid(int T, int n, int *threads)
{
    const int ny = (n + 127) / 128; // at most 128 threads: 2 to 10 % faster than 256 on long rows
    *threads = ((n + ny - 1) / ny + 31) / 32 * 32;
    return dim3(T, ny);
}

template <typename F> void by_type(int type, F f)
{
    if (type == kTypeF32)
        f(float());
    else if (type == kTypeF16)
        f(__half());
    else
        f(__nv_bfloat16());
}

} // namespace

// Rows are read and written in vectors of 8 elements when every row starts on 16 bytes.  All are
// programmatic dependents: each waits for what precedes it in the stream before its first access.
void launch_dispatch(const PermuteArgs &a, cudaStream_t s)
{
    by_type(a.type, [&](auto x) {
        using T = decltype(x);
        int threads;
        const bool vec = a.H % 8 == 0;
        const dim3 g = row_grid(a.T, vec ? a.H / 8 : a.H, &threads);
        launch_kernel(vec ? dispatch_kernel<T, 8> : dispatch_kernel<T, 1>, g, dim3(threads), 0, s, true, a);
    });
}

void launch_combine_rows(const PermuteArgs &a, cudaStream_t s)
{
    by_type(a.type, [&](auto x) {
        by_type(a.io_type, [&](auto y) {
            using T = decltype(x);
            using TO = decltype(y);
            int threads;
            const bool vec = a.H % 8 == 0;
            const dim3 g = row_grid(a.T, vec ? a.H / 8 : a.H, &threads);
            launch_kernel(vec ? combine_rows_kernel<T, TO, 8> : combine_rows_kernel<T, TO, 1>, g, dim3(threads), 0, s,
                          true, a);
        });
    });
}

void launch_combine_backward(const PermuteArgs &a, cudaStream_t s)
{
    by_type(a.type, [&](auto x) {
        by_type(a.io_type, [&](auto y) {
            using T = decltype(x);
            using TO = decltype(y);
            int threads; // equal rounds over the row
            const bool vec = a.H % 8 == 0;
            row_grid(a.T, vec ? a.H / 8 : a.H, &threads);
            launch_kernel(vec ? combine_backward_kernel<T, TO, 8> : combine_backward_kernel<T, TO, 1>, dim3(a.T),
                          dim3(threads), 0, s, true, a);
        });
    });
}

} // namespace moe_mx
