// permute.cu -- token rows to the grouped (sorted by expert) layout and back: dispatch, the
// weighted combine and its gradient.  Pair p = t*k + j of token t sits at grouped row pos[p]
// (outside [0, rows): no row, e.g. a pair of another shard's expert).  Token-major throughout, so a
// token's own row is read or written once and every grouped row once; no atomics.
#include "routed.cuh"
#include "vec.cuh"

namespace moe_mx {

namespace {

// One thread per (token, vector of V elements).
template <typename T, int V>
__global__ void __launch_bounds__(256) dispatch_kernel(const PermuteArgs a)
{
    const int t = blockIdx.x, c = (blockIdx.y * blockDim.x + threadIdx.x) * V;
    if (c >= a.H)
        return;
    Raw<T, V> v;
    v.load(static_cast<const T *>(a.tok) + (size_t)t * a.H + c);
    for (int j = 0; j < a.k; ++j) {
        const int r = __ldg(a.pos + (size_t)t * a.k + j);
        if (r >= 0 && r < a.rows)
            *reinterpret_cast<Raw<T, V> *>(static_cast<T *>(a.grouped_out) + (size_t)r * a.H + c) = v;
    }
}

// out[t] = sum_j w[t,j] y[pos[t,j]], j ascending, in float32; one rounding at the end.
template <typename T, typename TO, int V>
__global__ void __launch_bounds__(256) combine_rows_kernel(const PermuteArgs a)
{
    const int t = blockIdx.x, c = (blockIdx.y * blockDim.x + threadIdx.x) * V;
    if (c >= a.H)
        return;
    float acc[V];
#pragma unroll
    for (int i = 0; i < V; ++i)
        acc[i] = 0.f;
    for (int j = 0; j < a.k; ++j) {
        const int r = __ldg(a.pos + (size_t)t * a.k + j);
        if (r < 0 || r >= a.rows)
            continue;
        const float w = a.w ? __ldg(a.w + (size_t)t * a.k + j) : 1.f;
        Raw<T, V> v;
        float f[V];
        v.load(static_cast<const T *>(a.grouped) + (size_t)r * a.H + c);
        v.get(f);
#pragma unroll
        for (int i = 0; i < V; ++i)
            acc[i] = fmaf(w, f[i], acc[i]);
    }
    Raw<TO, V>::put(static_cast<TO *>(a.tok_out) + (size_t)t * a.H + c, acc);
}

constexpr int kMaxSlots = 32;

// One CTA per token: dy[pos] = w dout (one rounding), dw = <dout, y[pos]> (float32, a fixed order),
// and the gradient through w = softmax over the token's k chosen logits:
// dlogits[id_j] += w_j (dw_j - sum_i w_i dw_i), every other logit 0.
template <typename T, typename TO, int V>
__global__ void __launch_bounds__(256) combine_backward_kernel(const PermuteArgs a)
{
    __shared__ float s_part[8], s_dw[kMaxSlots], s_w[kMaxSlots];
    __shared__ int s_id[kMaxSlots];
    const int t = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    const bool dots = a.dw || a.dlogits;
    for (int j = 0; j < a.k; ++j) {
        const size_t p = (size_t)t * a.k + j;
        const int r = __ldg(a.pos + p);
        const float w = __ldg(a.w + p);
        float dot = 0.f;
        if (r >= 0 && r < a.rows) {
            for (int c = threadIdx.x * V; c < a.H; c += blockDim.x * V) {
                Raw<TO, V> d;
                float f[V], g[V];
                d.load(static_cast<const TO *>(a.tok) + (size_t)t * a.H + c);
                d.get(f);
                if (dots) {
                    Raw<T, V> y;
                    y.load(static_cast<const T *>(a.grouped) + (size_t)r * a.H + c);
                    y.get(g);
#pragma unroll
                    for (int i = 0; i < V; ++i)
                        dot = fmaf(f[i], g[i], dot);
                }
                if (a.grouped_out) {
#pragma unroll
                    for (int i = 0; i < V; ++i)
                        g[i] = w * f[i];
                    Raw<T, V>::put(static_cast<T *>(a.grouped_out) + (size_t)r * a.H + c, g);
                }
            }
        }
        if (!dots)
            continue;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            dot += __shfl_xor_sync(0xFFFFFFFFu, dot, o);
        if (lane == 0)
            s_part[warp] = dot;
        __syncthreads();
        if (threadIdx.x == 0) {
            float d = 0.f;
            for (int i = 0; i < nw; ++i)
                d += s_part[i];
            s_dw[j] = d;
            s_w[j] = w;
            if (a.dlogits)
                s_id[j] = __ldg(a.ids + p);
            if (a.dw)
                a.dw[p] = d;
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
    const int ny = (n + 255) / 256;
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

// Rows are read and written in vectors of 8 elements when every row starts on 16 bytes.
void launch_dispatch(const PermuteArgs &a, cudaStream_t s)
{
    by_type(a.type, [&](auto x) {
        using T = decltype(x);
        int threads;
        if (a.H % 8 == 0) {
            const dim3 g = row_grid(a.T, a.H / 8, &threads);
            dispatch_kernel<T, 8><<<g, threads, 0, s>>>(a);
        } else {
            const dim3 g = row_grid(a.T, a.H, &threads);
            dispatch_kernel<T, 1><<<g, threads, 0, s>>>(a);
        }
    });
}

void launch_combine_rows(const PermuteArgs &a, cudaStream_t s)
{
    by_type(a.type, [&](auto x) {
        by_type(a.io_type, [&](auto y) {
            using T = decltype(x);
            using TO = decltype(y);
            int threads;
            if (a.H % 8 == 0) {
                const dim3 g = row_grid(a.T, a.H / 8, &threads);
                combine_rows_kernel<T, TO, 8><<<g, threads, 0, s>>>(a);
            } else {
                const dim3 g = row_grid(a.T, a.H, &threads);
                combine_rows_kernel<T, TO, 1><<<g, threads, 0, s>>>(a);
            }
        });
    });
}

void launch_combine_backward(const PermuteArgs &a, cudaStream_t s)
{
    by_type(a.type, [&](auto x) {
        by_type(a.io_type, [&](auto y) {
            using T = decltype(x);
            using TO = decltype(y);
            if (a.H % 8 == 0)
                combine_backward_kernel<T, TO, 8><<<a.T, 256, 0, s>>>(a);
            else
                combine_backward_kernel<T, TO, 1><<<a.T, 256, 0, s>>>(a);
        });
    });
}

} // namespace moe_mx
