// api_routed.cu -- entry points of the routed operators (declared in include/moe_mx.h): dispatch,
// combine and its gradient, linear and its gradient.  Argument checks, the device of the call, and
// the launchers of permute.cu and linear.cu.
#include <cuda_runtime.h>

#include "../../include/moe_mx.h"
#include "host.cuh"
#include "routed.cuh"

using namespace moe_mx;

namespace {

constexpr int kMaxSlotsApi = 32;      // top_k
constexpr int kMaxExpertsApi = 1024;
constexpr int kMaxDim = 1 << 20;      // hidden, N, K

bool type_ok(int t) { return t == MOE_MX_TYPE_BF16 || t == MOE_MX_TYPE_F32 || t == MOE_MX_TYPE_F16; }

// The device of a call: the one that holds its first tensor, which is checked like the others.
int device_of(const void *p, const char *name, int *dev)
{
    cudaPointerAttributes at;
    if (!p || cudaPointerGetAttributes(&at, p) != cudaSuccess ||
        (at.type != cudaMemoryTypeDevice && at.type != cudaMemoryTypeManaged)) {
        cudaGetLastError();
        return fail(MOE_MX_ERR_INVALID_ARG, "%s must be a device pointer", name);
    }
    if (reinterpret_cast<uintptr_t>(p) % 16 != 0)
        return fail(MOE_MX_ERR_INVALID_ARG, "%s must be 16-byte aligned", name);
    *dev = at.device;
    return MOE_MX_OK;
}

int launched(const char *what)
{
    const cudaError_t ce = cudaGetLastError();
    return ce == cudaSuccess ? MOE_MX_OK : cuda_fail(ce, what);
}

int check_permute(int T, int H, int k, int64_t rows, int type)
{
    if (T < 0)
        return fail(MOE_MX_ERR_INVALID_ARG, "num_tokens=%d must be >= 0", T);
    if (H < 1 || H > kMaxDim)
        return fail(MOE_MX_ERR_INVALID_ARG, "hidden=%d must be in [1, %d]", H, kMaxDim);
    if (k < 1 || k > kMaxSlotsApi)
        return fail(MOE_MX_ERR_INVALID_ARG, "top_k=%d must be in [1, %d]", k, kMaxSlotsApi);
    if (rows < 0 || rows > INT32_MAX)
        return fail(MOE_MX_ERR_INVALID_ARG, "rows=%lld must be in [0, 2^31)", (long long)rows);
    if (!type_ok(type))
        return fail(MOE_MX_ERR_INVALID_ARG, "dtype=%d is not MOE_MX_TYPE_*", type);
    return MOE_MX_OK;
}

// Byte ranges [p, p + n) and [q, q + m) overlap.
bool overlap(const void *p, size_t n, const void *q, size_t m)
{
    const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
    return p && q && n && m && a < b + m && b < a + n;
}

struct Range {
    const void *p;
    size_t n;
};

// One of outs overlaps another of them or one of ins.
template <int O, int I> bool clash(const Range (&outs)[O], const Range (&ins)[I])
{
    for (int i = 0; i < O; ++i) {
        for (const Range &r : ins)
            if (overlap(outs[i].p, outs[i].n, r.p, r.n))
                return true;
        for (int j = 0; j < i; ++j)
            if (overlap(outs[i].p, outs[i].n, outs[j].p, outs[j].n))
                return true;
    }
    return false;
}

struct LinearSizes {
    int64_t rows;
    int E, N, K, act;
    size_t slots() const { return E ? (size_t)E : 1; }
    int No() const { return act == MOE_MX_LINEAR_SWIGLU ? N / 2 : N; }
};

int check_linear(const LinearSizes &z, int type, int io_type, const char *io_name)
{
    if (z.E < 0 || z.E > kMaxExpertsApi)
        return fail(MOE_MX_ERR_INVALID_ARG, "num_experts=%d must be in [0, %d]", z.E, kMaxExpertsApi);
    if (z.rows < 0 || z.rows > INT32_MAX - 1024)
        return fail(MOE_MX_ERR_INVALID_ARG, "rows=%lld must be in [0, 2^31 - 1024)", (long long)z.rows);
    if (z.N < 1 || z.N > kMaxDim || z.K < 1 || z.K > kMaxDim)
        return fail(MOE_MX_ERR_INVALID_ARG, "N=%d, K=%d must be in [1, %d]", z.N, z.K, kMaxDim);
    if (type != MOE_MX_TYPE_BF16 && type != MOE_MX_TYPE_F16)
        return fail(MOE_MX_ERR_INVALID_ARG, "dtype=%d is not MOE_MX_TYPE_BF16 or MOE_MX_TYPE_F16", type);
    if (io_type != type && io_type != MOE_MX_TYPE_F32)
        return fail(MOE_MX_ERR_INVALID_ARG, "%s=%d is neither dtype nor MOE_MX_TYPE_F32", io_name, io_type);
    if (z.act < MOE_MX_LINEAR_NONE || z.act > MOE_MX_LINEAR_SWIGLU)
        return fail(MOE_MX_ERR_INVALID_ARG, "activation=%d is not MOE_MX_LINEAR_*", z.act);
    if (z.act == MOE_MX_LINEAR_SWIGLU && z.N % 2)
        return fail(MOE_MX_ERR_INVALID_ARG, "N=%d must be even for MOE_MX_LINEAR_SWIGLU", z.N);
    return MOE_MX_OK;
}

int check_routing(const int32_t *counts, const int32_t *pad_offsets, int E, int dev)
{
    if (E == 0) {
        if (counts || pad_offsets)
            return fail(MOE_MX_ERR_INVALID_ARG, "counts and pad_offsets must be NULL when num_experts is 0");
        return MOE_MX_OK;
    }
    int rc = check_ptr(counts, dev, "counts");
    return rc ? rc : check_ptr(pad_offsets, dev, "pad_offsets");
}

int check_workspace(void *ws, int64_t given, int64_t need, int dev)
{
    if (need == 0)
        return MOE_MX_OK;
    if (given < need)
        return fail(MOE_MX_ERR_INVALID_ARG, "workspace_bytes=%lld: this call needs %lld", (long long)given,
                    (long long)need);
    return check_ptr(ws, dev, "workspace");
}

int check_device(int device)
{
    int ndev = 0;
    const cudaError_t ce = cudaGetDeviceCount(&ndev);
    if (ce != cudaSuccess)
        return cuda_fail(ce, "cudaGetDeviceCount");
    if (device < 0 || device >= ndev)
        return fail(MOE_MX_ERR_INVALID_ARG, "device %d out of range (%d devices)", device, ndev);
    return MOE_MX_OK;
}

} // namespace

extern "C" {

int moe_mx_dispatch(const void *x, int num_tokens, int hidden, int top_k, const int32_t *pos_of_pair, int64_t rows,
                    int dtype, void *grouped, void *stream)
{
    clear_error();
    int rc = check_permute(num_tokens, hidden, top_k, rows, dtype);
    if (rc || num_tokens == 0 || rows == 0)
        return rc;
    int dev;
    if ((rc = device_of(x, "x", &dev)) ||
        (rc = check_ptr(pos_of_pair, dev, "pos_of_pair")) || (rc = check_ptr(grouped, dev, "grouped")))
        return rc;
    const size_t T = num_tokens, row = (size_t)hidden * type_bytes(dtype);
    const Range outs[] = {{grouped, rows * row}}, ins[] = {{x, T * row}, {pos_of_pair, T * top_k * 4}};
    if (clash(outs, ins))
        return fail(MOE_MX_ERR_INVALID_ARG, "grouped must not overlap x or pos_of_pair");
    const DeviceGuard guard(dev);
    PermuteArgs a{};
    a.T = num_tokens, a.H = hidden, a.k = top_k, a.rows = rows, a.pos = pos_of_pair, a.type = dtype;
    a.tok = x, a.grouped_out = grouped;
    launch_dispatch(a, static_cast<cudaStream_t>(stream));
    return launched("dispatch launch");
}

int moe_mx_combine(const void *grouped, int64_t rows, int num_tokens, int hidden, int top_k,
                   const int32_t *pos_of_pair, const float *topk_w, int dtype, int out_dtype, void *out, void *stream)
{
    clear_error();
    int rc = check_permute(num_tokens, hidden, top_k, rows, dtype);
    if (rc)
        return rc;
    if (!type_ok(out_dtype))
        return fail(MOE_MX_ERR_INVALID_ARG, "out_dtype=%d is not MOE_MX_TYPE_*", out_dtype);
    if (num_tokens == 0)
        return MOE_MX_OK;
    int dev;
    if ((rc = device_of(out, "out", &dev)) ||
        (rows && (rc = check_ptr(grouped, dev, "grouped"))) || (rc = check_ptr(pos_of_pair, dev, "pos_of_pair")) ||
        (topk_w && (rc = check_ptr(topk_w, dev, "topk_w"))))
        return rc;
    const size_t T = num_tokens, pairs = T * top_k * 4;
    const Range outs[] = {{out, T * hidden * type_bytes(out_dtype)}},
                ins[] = {{grouped, (size_t)rows * hidden * type_bytes(dtype)}, {pos_of_pair, pairs}, {topk_w, pairs}};
    if (clash(outs, ins))
        return fail(MOE_MX_ERR_INVALID_ARG, "out must not overlap grouped, pos_of_pair or topk_w");
    const DeviceGuard guard(dev);
    PermuteArgs a{};
    a.T = num_tokens, a.H = hidden, a.k = top_k, a.rows = rows, a.pos = pos_of_pair, a.w = topk_w;
    a.type = dtype, a.io_type = out_dtype, a.grouped = grouped, a.tok_out = out;
    launch_combine_rows(a, static_cast<cudaStream_t>(stream));
    return launched("combine launch");
}

int moe_mx_combine_backward(const void *dout, const void *grouped, int64_t rows, int num_tokens, int hidden, int top_k,
                            const int32_t *pos_of_pair, const float *topk_w, const int32_t *topk_ids, int num_experts,
                            int dtype, int dout_dtype, void *dgrouped, float *dtopk_w, float *dlogits, void *stream)
{
    clear_error();
    int rc = check_permute(num_tokens, hidden, top_k, rows, dtype);
    if (rc)
        return rc;
    if (!type_ok(dout_dtype))
        return fail(MOE_MX_ERR_INVALID_ARG, "dout_dtype=%d is not MOE_MX_TYPE_*", dout_dtype);
    if (dlogits && (num_experts < 1 || num_experts > kMaxExpertsApi))
        return fail(MOE_MX_ERR_INVALID_ARG, "num_experts=%d must be in [1, %d] when dlogits is given", num_experts,
                    kMaxExpertsApi);
    if (!dgrouped && !dtopk_w && !dlogits)
        return fail(MOE_MX_ERR_INVALID_ARG, "none of dgrouped, dtopk_w and dlogits is given");
    if (num_tokens == 0)
        return MOE_MX_OK;
    int dev;
    if ((rc = device_of(dout, "dout", &dev)) ||
        (rc = check_ptr(pos_of_pair, dev, "pos_of_pair")) || (rc = check_ptr(topk_w, dev, "topk_w")) ||
        (dgrouped && rows && (rc = check_ptr(dgrouped, dev, "dgrouped"))) ||
        ((dtopk_w || dlogits) && rows && (rc = check_ptr(grouped, dev, "grouped"))) ||
        (dtopk_w && (rc = check_ptr(dtopk_w, dev, "dtopk_w"))) ||
        (dlogits && ((rc = check_ptr(dlogits, dev, "dlogits")) || (rc = check_ptr(topk_ids, dev, "topk_ids")))))
        return rc;
    const bool dots = dtopk_w || dlogits;
    const size_t T = num_tokens, pairs = T * top_k * 4, g_bytes = (size_t)rows * hidden * type_bytes(dtype);
    const Range outs[] = {{dgrouped, g_bytes}, {dtopk_w, pairs}, {dlogits, T * num_experts * 4}},
                ins[] = {{dout, T * hidden * type_bytes(dout_dtype)}, {dots ? grouped : nullptr, g_bytes},
                         {pos_of_pair, pairs}, {dtopk_w == topk_w ? nullptr : topk_w, pairs}, {dlogits ? topk_ids : nullptr, pairs}};
    if (clash(outs, ins))
        return fail(MOE_MX_ERR_INVALID_ARG, "dgrouped, dtopk_w and dlogits must not overlap each other, dout, grouped "
                                            "or the routing (dtopk_w may be topk_w itself)");
    const DeviceGuard guard(dev);
    PermuteArgs a{};
    a.T = num_tokens, a.H = hidden, a.k = top_k, a.rows = rows, a.pos = pos_of_pair, a.w = topk_w, a.ids = topk_ids;
    a.E = num_experts, a.type = dtype, a.io_type = dout_dtype, a.tok = dout, a.grouped = grouped;
    a.grouped_out = dgrouped, a.dw = dtopk_w, a.dlogits = dlogits;
    launch_combine_backward(a, static_cast<cudaStream_t>(stream));
    return launched("combine_backward launch");
}

int64_t moe_mx_linear_workspace(int num_experts, int64_t rows, int N, int K, int dtype, int activation, int out_dtype)
{
    clear_error();
    const LinearSizes z{rows, num_experts, N, K, activation};
    if (int rc = check_linear(z, dtype, out_dtype, "out_dtype"))
        return rc;
    return linear_workspace(num_experts, rows, N, K, activation, dtype, out_dtype);
}

int64_t moe_mx_linear_backward_workspace(int num_experts, int64_t rows, int N, int K, int dtype, int activation,
                                         int dout_dtype)
{
    clear_error();
    const LinearSizes z{rows, num_experts, N, K, activation};
    if (int rc = check_linear(z, dtype, dout_dtype, "dout_dtype"))
        return rc;
    return linear_backward_workspace(num_experts, rows, N, K, activation, dtype, dout_dtype);
}

int moe_mx_debug_linear_plan(int which, int num_experts, int64_t rows, int N, int K, int dtype, int activation,
                             int io_dtype, int32_t *plan)
{
    clear_error();
    const LinearSizes z{rows, num_experts, N, K, activation};
    if (int rc = check_linear(z, dtype, io_dtype, which ? "dout_dtype" : "out_dtype"))
        return rc;
    if (which < 0 || which > 2)
        return fail(MOE_MX_ERR_INVALID_ARG, "which=%d must be in [0, 2]", which);
    if (!plan)
        return fail(MOE_MX_ERR_INVALID_ARG, "plan is NULL");
    linear_plan(which, num_experts, rows, N, K, activation, dtype, io_dtype, plan);
    return MOE_MX_OK;
}

int moe_mx_linear(const void *x, const void *w, const float *bias, const void *residual, const int32_t *counts,
                  const int32_t *pad_offsets, int num_experts, int64_t rows, int N, int K, int dtype, int activation,
                  int out_dtype, void *out, void *preact, void *workspace, int64_t workspace_bytes, void *stream)
{
    clear_error();
    const LinearSizes z{rows, num_experts, N, K, activation};
    int rc = check_linear(z, dtype, out_dtype, "out_dtype");
    if (rc || rows == 0)
        return rc;
    int dev;
    const int64_t need = linear_workspace(num_experts, rows, N, K, activation, dtype, out_dtype);
    if ((rc = device_of(x, "x", &dev)) || (rc = check_ptr(w, dev, "w")) ||
        (rc = check_ptr(out, dev, "out")) || (bias && (rc = check_ptr(bias, dev, "bias"))) ||
        (residual && (rc = check_ptr(residual, dev, "residual"))) ||
        (preact && (rc = check_ptr(preact, dev, "preact"))) ||
        (rc = check_routing(counts, pad_offsets, num_experts, dev)) ||
        (rc = check_workspace(workspace, workspace_bytes, need, dev)))
        return rc;
    const size_t ob = (size_t)rows * z.No() * type_bytes(out_dtype);
    const Range outs[] = {{out, ob}, {preact, (size_t)rows * N * 2}, {workspace, (size_t)need}},
                ins[] = {{x, (size_t)rows * K * 2}, {w, z.slots() * N * K * 2}, {bias, z.slots() * N * 4},
                         {residual == out ? nullptr : residual, ob}, {counts, (size_t)num_experts * 4},
                         {pad_offsets, ((size_t)num_experts + 1) * 4}};
    if (clash(outs, ins))
        return fail(MOE_MX_ERR_INVALID_ARG, "out, preact and workspace must not overlap each other, x, w, bias, residual "
                                            "(out may be residual itself) or the routing");
    const DeviceGuard guard(dev);
    LinearArgs a{};
    a.M = rows, a.N = N, a.K = K, a.E = num_experts, a.type = dtype, a.out_type = out_dtype, a.act = activation;
    a.x = x, a.w = w, a.bias = bias, a.residual = residual, a.counts = counts, a.pad_offsets = pad_offsets;
    a.out = out, a.preact = preact, a.ws = workspace;
    if ((rc = launch_linear(a, static_cast<cudaStream_t>(stream))))
        return rc;
    return launched("linear launch");
}

int moe_mx_linear_status(int device, void *stream)
{
    clear_error();
    if (int rc = check_device(device))
        return rc;
    const DeviceGuard guard(device);
    return linear_status(static_cast<cudaStream_t>(stream));
}

int moe_mx_debug_linear_watchdog(int device, int timeout_us, void *stream)
{
    clear_error();
    if (timeout_us < 1 || timeout_us > 10000000)
        return fail(MOE_MX_ERR_INVALID_ARG, "timeout_us=%d must be in [1, 1e7]", timeout_us);
    if (int rc = check_device(device))
        return rc;
    const DeviceGuard guard(device);
    if (int rc = linear_watchdog((unsigned long long)timeout_us * 1000ull, static_cast<cudaStream_t>(stream)))
        return rc;
    return launched("watchdog launch");
}

int moe_mx_linear_backward(const void *dout, const void *x, const void *w, const void *preact, const int32_t *counts,
                           const int32_t *pad_offsets, int num_experts, int64_t rows, int N, int K, int dtype,
                           int activation, int dout_dtype, void *dx, void *dw, float *dbias, void *workspace,
                           int64_t workspace_bytes, void *stream)
{
    clear_error();
    const LinearSizes z{rows, num_experts, N, K, activation};
    int rc = check_linear(z, dtype, dout_dtype, "dout_dtype");
    if (rc)
        return rc;
    if (!dx && !dw && !dbias)
        return fail(MOE_MX_ERR_INVALID_ARG, "none of dx, dw and dbias is given");
    if (activation != MOE_MX_LINEAR_NONE && !preact && rows > 0)
        return fail(MOE_MX_ERR_INVALID_ARG, "preact must be given for an activation");
    int dev;
    const int64_t need = linear_backward_workspace(num_experts, rows, N, K, activation, dtype, dout_dtype);
    const bool some = rows > 0; // with no rows only the zero gradients dw and dbias are written
    if (some && ((rc = device_of(dout, "dout", &dev))))
        return rc;
    if (!some) {
        if (!dw && !dbias)
            return MOE_MX_OK;
        if ((rc = device_of(dw ? dw : (void *)dbias, dw ? "dw" : "dbias", &dev)))
            return rc;
    }
    if ((some && dw && (rc = check_ptr(x, dev, "x"))) || (some && dx && (rc = check_ptr(w, dev, "w"))) ||
        (some && activation != MOE_MX_LINEAR_NONE && (rc = check_ptr(preact, dev, "preact"))) ||
        (some && dx && (rc = check_ptr(dx, dev, "dx"))) || (dw && (rc = check_ptr(dw, dev, "dw"))) ||
        (dbias && (rc = check_ptr(dbias, dev, "dbias"))) ||
        (rc = check_routing(counts, pad_offsets, num_experts, dev)) ||
        (rc = check_workspace(workspace, workspace_bytes, need, dev)))
        return rc;
    const size_t xb = (size_t)rows * K * 2, wb = z.slots() * N * K * 2;
    const Range outs[] = {{dx, xb}, {dw, wb}, {dbias, z.slots() * N * 4}, {workspace, (size_t)need}},
                ins[] = {{dout, (size_t)rows * z.No() * type_bytes(dout_dtype)}, {x, xb}, {w, wb},
                         {preact, (size_t)rows * N * 2}, {counts, (size_t)num_experts * 4},
                         {pad_offsets, ((size_t)num_experts + 1) * 4}};
    if (clash(outs, ins))
        return fail(MOE_MX_ERR_INVALID_ARG, "dx, dw, dbias and workspace must not overlap each other, dout, x, w, preact "
                                            "or the routing");
    const DeviceGuard guard(dev);
    LinearBackwardArgs a{};
    a.M = rows, a.N = N, a.K = K, a.E = num_experts, a.type = dtype, a.dout_type = dout_dtype, a.act = activation;
    a.dout = dout, a.x = x, a.w = w, a.preact = preact, a.counts = counts, a.pad_offsets = pad_offsets;
    a.dx = dx, a.dw = dw, a.dbias = dbias, a.ws = workspace;
    if ((rc = launch_linear_backward(a, static_cast<cudaStream_t>(stream))))
        return rc;
    return launched("linear_backward launch");
}

} // extern "C"
