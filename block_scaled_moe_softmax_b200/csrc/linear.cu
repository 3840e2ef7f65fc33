// linear.cu -- out = act(x w^T + bias) + residual and its gradient, dense or over the segments of
// the grouped layout (segment e: rows pad_offsets[e] .. + counts[e], a multiple of 128 apart, with
// weights w[e] and bias[e]; the rows behind counts[e] are neither read into a result nor written).
//
//   z = x w^T + b          dz = dout * act'(z)
//   out = act(z) + res     dx = dz w      dw = dz^T x      db = sum over rows of dz
//
// dz is rounded once to the operands' type, which the products take (db sums it before that).
#include "../../include/moe_mx.h"
#include "host.cuh"
#include "routed.cuh"
#include "vec.cuh"

namespace moe_mx {

namespace {

// ---------------------------------------------------------------- activations
__device__ __forceinline__ float sigmoid(float v) { return 1.f / (1.f + __expf(-v)); }

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

// The segment holding row `r0` (a multiple of 64): its expert, and the end of its valid rows.
__device__ __forceinline__ bool find_segment(const Segments &s, int64_t r0, int &e, int64_t &end)
{
    if (s.E == 0) {
        e = 0;
        end = s.M;
        return r0 < s.M;
    }
    int lo = 0, hi = s.E; // the last e with pad_offsets[e] <= r0
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (__ldg(s.pad_offsets + mid) <= r0)
            lo = mid;
        else
            hi = mid;
    }
    e = lo;
    const int64_t first = __ldg(s.pad_offsets + e);
    end = min(s.M, first + __ldg(s.counts + e));
    return r0 >= first && r0 < end;
}

// ---------------------------------------------------------------- matrix product
struct Gemm {
    // D[m, n] = sum_k A[m, k] B[n, k]; element (i, k) of an operand at i * s0 + k * s1
    const void *a, *b;
    int64_t as0, as1, bs0, bs1;
    int64_t b_expert; // elements from one expert's B to the next's (rows segmented)
    int64_t d_expert; // elements from one expert's D to the next's (k segmented)
    Segments seg;
    int64_t M;
    int N;
    int64_t K;
    int seg_k; // segments run over k (dw) instead of the rows
    // epilogue
    const float *bias;
    const void *residual;
    void *out, *preact;
    int act, n_out; // columns of out (N / 2 for swiglu: gate columns n and up columns n + n_out)
};

constexpr int kT = 64, kTk = 16;

template <typename T, typename TO> __device__ __forceinline__ void finish(const Gemm &g, int e, int64_t m, int n,
                                                                          float z, float up)
{
    const float *bias = g.bias ? g.bias + (size_t)e * g.N : nullptr;
    const bool gated = g.act == kActSwiglu;
    if (bias) {
        z += bias[n];
        if (gated)
            up += bias[n + g.n_out];
    }
    if (g.preact) {
        static_cast<T *>(g.preact)[m * g.N + n] = from_f32<T>(z);
        if (gated)
            static_cast<T *>(g.preact)[m * g.N + n + g.n_out] = from_f32<T>(up);
    }
    float v = gated ? z * sigmoid(z) * up : act_fwd(z, g.act);
    const size_t o = (size_t)e * (g.seg_k ? g.d_expert : 0) + (size_t)m * g.n_out + n;
    if (g.residual)
        v += to_f32<TO>(static_cast<const TO *>(g.residual)[o]);
    static_cast<TO *>(g.out)[o] = from_f32<TO>(v);
}

// 64 x 64 tile of D, 16 of k at a time, 4 x 4 outputs a thread.
template <typename T, typename TO> __global__ void __launch_bounds__(256) gemm_kernel(const Gemm g)
{
    __shared__ float sa[kTk][kT + 1], sb[kTk][kT + 1], su[kTk][kT + 1];
    const bool gated = g.act == kActSwiglu;
    const int64_t m0 = (int64_t)blockIdx.x * kT;
    const int n0 = blockIdx.y * kT;
    int e = 0;
    int64_t m_end = g.M, k0 = 0, k_end = g.K;
    if (g.seg_k) {
        e = blockIdx.z;
        if (g.seg.E) {
            k0 = __ldg(g.seg.pad_offsets + e);
            k_end = min(g.seg.M, k0 + __ldg(g.seg.counts + e));
        }
    } else if (!find_segment(g.seg, m0, e, m_end)) {
        return;
    }
    const T *a = static_cast<const T *>(g.a);
    const T *b = static_cast<const T *>(g.b) + (g.seg_k ? 0 : (size_t)e * g.b_expert);
    const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
    float acc[4][4] = {}, up[4][4] = {};
    for (int64_t k = k0; k < k_end; k += kTk) {
        for (int i = threadIdx.x; i < kT * kTk; i += 256) {
            // consecutive threads along the operand's unit stride
            const int ak = g.as1 == 1 ? i % kTk : i / kT, am = g.as1 == 1 ? i / kTk : i % kT;
            const int bk = g.bs1 == 1 ? i % kTk : i / kT, bn = g.bs1 == 1 ? i / kTk : i % kT;
            const bool ka = k + ak < k_end, kb = k + bk < k_end, nb = n0 + bn < g.n_out;
            sa[ak][am] = ka && m0 + am < m_end ? to_f32<T>(a[(m0 + am) * g.as0 + (k + ak) * g.as1]) : 0.f;
            sb[bk][bn] = kb && nb ? to_f32<T>(b[(n0 + bn) * g.bs0 + (k + bk) * g.bs1]) : 0.f;
            if (gated)
                su[bk][bn] = kb && nb ? to_f32<T>(b[(n0 + bn + g.n_out) * g.bs0 + (k + bk) * g.bs1]) : 0.f;
        }
        __syncthreads();
        for (int kk = 0; kk < kTk; ++kk)
            for (int i = 0; i < 4; ++i)
                for (int j = 0; j < 4; ++j) {
                    acc[i][j] = fmaf(sa[kk][ty * 4 + i], sb[kk][tx * 4 + j], acc[i][j]);
                    if (gated)
                        up[i][j] = fmaf(sa[kk][ty * 4 + i], su[kk][tx * 4 + j], up[i][j]);
                }
        __syncthreads();
    }
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) {
            const int64_t m = m0 + ty * 4 + i;
            const int n = n0 + tx * 4 + j;
            if (m < m_end && n < g.n_out)
                finish<T, TO>(g, e, m, n, acc[i][j], up[i][j]);
        }
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

template <typename F> void by_half(int type, F f)
{
    if (type == kTypeF16)
        f(__half());
    else
        f(__nv_bfloat16());
}

void launch_gemm(const Gemm &g, int type, int out_type, cudaStream_t s)
{
    const dim3 grid((unsigned)((g.M + kT - 1) / kT), (g.n_out + kT - 1) / kT,
                    g.seg_k && g.seg.E ? g.seg.E : 1);
    by_half(type, [&](auto x) {
        using T = decltype(x);
        if (out_type == kTypeF32)
            gemm_kernel<T, float><<<grid, 256, 0, s>>>(g);
        else
            gemm_kernel<T, T><<<grid, 256, 0, s>>>(g);
    });
}

// ---------------------------------------------------------------- dz and the bias gradient
struct DzArgs {
    const void *dout, *preact;
    void *dz;     // [M, ldz] or nullptr
    float *part;  // [ceil(M / 128)][N] column sums of each 128-row block, or nullptr
    Segments seg;
    int N, n_out, ldz, act;
};

// One CTA: 128 rows x 64 columns of dout (8 lanes x 8 columns, 32 row lanes x 4 rows).  The column
// sums of a block are added in a fixed order.
template <typename T, typename TO, int V> __global__ void __launch_bounds__(256) dz_kernel(const DzArgs a)
{
    __shared__ float red[32][65];
    const int64_t m0 = (int64_t)blockIdx.x * 128;
    int e;
    int64_t end;
    const bool any = find_segment(a.seg, m0, e, end);
    if (!any)
        return; // a block of padding, or past the last segment
    const bool gated = a.act == kActSwiglu;
    const int cl = threadIdx.x % 8, rl = threadIdx.x / 8;
    float sum[2][8] = {};
    for (int i = 0; i < 4; ++i) {
        const int64_t m = m0 + i * 32 + rl;
        if (m >= end)
            continue;
        for (int v = 0; v < 8; v += V) {
            const int n = blockIdx.y * 64 + cl * 8 + v;
            if (n >= a.n_out)
                break;
            Raw<TO, V> rd;
            Raw<T, V> rz;
            float d[V], z[V], u[V], dz[V], du[V];
            rd.load(static_cast<const TO *>(a.dout) + m * a.n_out + n);
            rd.get(d);
            if (a.act != kActNone) {
                rz.load(static_cast<const T *>(a.preact) + m * a.N + n);
                rz.get(z);
            }
            if (gated) {
                rz.load(static_cast<const T *>(a.preact) + m * a.N + n + a.n_out);
                rz.get(u);
            }
#pragma unroll
            for (int q = 0; q < V; ++q) {
                if (gated) {
                    const float sg = sigmoid(z[q]);
                    dz[q] = d[q] * u[q] * (sg * (1.f + z[q] * (1.f - sg)));
                    du[q] = d[q] * z[q] * sg;
                    sum[1][v + q] += du[q];
                } else {
                    dz[q] = a.act == kActNone ? d[q] : d[q] * act_grad(z[q], a.act);
                }
                sum[0][v + q] += dz[q];
            }
            if (a.dz) {
                T *o = static_cast<T *>(a.dz) + m * a.ldz + n;
                Raw<T, V>::put(o, dz);
                if (gated)
                    Raw<T, V>::put(o + a.n_out, du);
            }
        }
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

// dbias[e][n]: the sum of the segment's row blocks, in order.
__global__ void __launch_bounds__(256) dbias_kernel(const float *part, Segments seg, int N, float *dbias)
{
    const int n = blockIdx.x * blockDim.x + threadIdx.x, e = blockIdx.y;
    if (n >= N)
        return;
    int64_t b0 = 0, rows = seg.M;
    if (seg.E) {
        const int64_t first = __ldg(seg.pad_offsets + e);
        b0 = first / 128;
        rows = min((int64_t)__ldg(seg.counts + e), seg.M - first);
    }
    float t = 0.f;
    for (int64_t b = 0; b * 128 < rows; ++b)
        t += part[(b0 + b) * N + n];
    dbias[(size_t)e * N + n] = t;
}

int ldz_of(int N) { return (int)round_up(N, 8); }

bool dz_is_dout(int act, int type, int dout_type, int N) { return act == kActNone && type == dout_type && N % 8 == 0; }

} // namespace

int64_t linear_workspace(int, int64_t, int, int, int, int, int) { return 0; }

int64_t linear_backward_workspace(int, int64_t M, int N, int, int act, int type, int dout_type)
{
    int64_t b = round_up((M + 127) / 128 * N * 4, 256);
    if (!dz_is_dout(act, type, dout_type, N))
        b += round_up(M * ldz_of(N) * 2, 256);
    return b;
}

int launch_linear(const LinearArgs &a, cudaStream_t s)
{
    Gemm g{};
    g.a = a.x, g.as0 = a.K, g.as1 = 1;
    g.b = a.w, g.bs0 = a.K, g.bs1 = 1, g.b_expert = (int64_t)a.N * a.K;
    g.seg = Segments{a.counts, a.pad_offsets, a.E, a.M};
    g.M = a.M, g.N = a.N, g.K = a.K, g.n_out = a.No();
    g.bias = a.bias, g.residual = a.residual, g.out = a.out, g.preact = a.preact, g.act = a.act;
    launch_gemm(g, a.type, a.out_type, s);
    return MOE_MX_OK;
}

int launch_linear_backward(const LinearBackwardArgs &a, cudaStream_t s)
{
    const Segments seg{a.counts, a.pad_offsets, a.E, a.M};
    const bool direct = dz_is_dout(a.act, a.type, a.dout_type, a.N);
    float *part = static_cast<float *>(a.ws);
    DzArgs d{};
    d.dout = a.dout, d.preact = a.preact, d.seg = seg;
    d.N = a.N, d.n_out = a.No(), d.ldz = ldz_of(a.N), d.act = a.act;
    d.part = a.dbias ? part : nullptr;
    if (!direct && (a.dx || a.dw))
        d.dz = static_cast<char *>(a.ws) + round_up((a.M + 127) / 128 * a.N * 4, 256);
    if (a.M > 0 && (d.part || d.dz)) {
        const dim3 grid((unsigned)((a.M + 127) / 128), (d.n_out + 63) / 64);
        by_half(a.type, [&](auto x) {
            using T = decltype(x);
            auto go = [&](auto y) {
                using TO = decltype(y);
                if (d.n_out % 8 == 0)
                    dz_kernel<T, TO, 8><<<grid, 256, 0, s>>>(d);
                else
                    dz_kernel<T, TO, 1><<<grid, 256, 0, s>>>(d);
            };
            if (a.dout_type == kTypeF32)
                go(float());
            else
                go(T());
        });
    }
    if (a.dbias) {
        const dim3 grid((a.N + 255) / 256, a.E ? a.E : 1);
        dbias_kernel<<<grid, 256, 0, s>>>(part, seg, a.N, a.dbias);
    }
    const void *dz = direct ? a.dout : d.dz;
    const int ldz = direct ? a.N : d.ldz;
    if (a.dx && a.M > 0) {
        Gemm g{};
        g.a = dz, g.as0 = ldz, g.as1 = 1;
        g.b = a.w, g.bs0 = 1, g.bs1 = a.K, g.b_expert = (int64_t)a.N * a.K;
        g.seg = seg, g.M = a.M, g.N = g.n_out = a.K, g.K = a.N, g.out = a.dx;
        launch_gemm(g, a.type, a.type, s);
    }
    if (a.dw) {
        Gemm g{};
        g.a = dz, g.as0 = 1, g.as1 = ldz;
        g.b = a.x, g.bs0 = 1, g.bs1 = a.K;
        g.seg = seg, g.seg_k = 1, g.d_expert = (int64_t)a.N * a.K;
        g.M = a.N, g.N = g.n_out = a.K, g.K = a.M, g.out = a.dw;
        launch_gemm(g, a.type, a.type, s);
    }
    return MOE_MX_OK;
}

} // namespace moe_mx
