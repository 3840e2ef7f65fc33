// routed.cuh -- argument structs and launchers of the routed operators (permute.cu, linear.cu),
// called by their entry points in api_routed.cu.  Internal to libmoe_mx.so.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace moe_mx {

// Element types, numbered as MOE_MX_TYPE_*.
enum { kTypeBf16 = 0, kTypeF32 = 1, kTypeF16 = 2 };
inline int type_bytes(int t) { return t == kTypeF32 ? 4 : 2; }

struct PermuteArgs {
    int T, H, k;
    int64_t rows;         // rows of the grouped buffers; a pair's row outside [0, rows) is left out
    const int32_t *pos;   // [T*k]
    const float *w;       // [T, k] or nullptr (combine: weights of 1)
    const int32_t *ids;   // [T, k], combine_backward with dlogits
    int E;                // columns of dlogits
    int type, io_type;    // grouped rows' type; the token rows' type
    const void *tok;      // token rows read: x (dispatch), dout (combine_backward)
    void *tok_out;        // token rows written: out (combine)
    const void *grouped;  // y
    void *grouped_out;    // dispatch's output, dy
    float *dw, *dlogits;
};
void launch_dispatch(const PermuteArgs &a, cudaStream_t s);
void launch_combine_rows(const PermuteArgs &a, cudaStream_t s);
void launch_combine_backward(const PermuteArgs &a, cudaStream_t s);

enum { kActNone = 0, kActSilu = 1, kActGelu = 2, kActSwiglu = 3 };

// out[M, No] = act(x w^T + bias) + residual over dense rows (E = 0) or the segments of the grouped
// layout (segment e: rows pad_offsets[e] .. + counts[e], weights w + e * N * K).
struct LinearArgs {
    int64_t M;            // rows of x and out
    int N, K, E;
    int type, out_type, act;
    const void *x, *w;
    const float *bias;
    const void *residual;
    const int32_t *counts, *pad_offsets;
    void *out, *preact;
    void *ws;
    int No() const { return act == kActSwiglu ? N / 2 : N; }
};
struct LinearBackwardArgs {
    int64_t M;
    int N, K, E;
    int type, dout_type, act;
    const void *dout, *x, *w, *preact;
    const int32_t *counts, *pad_offsets;
    void *dx, *dw;
    float *dbias;
    void *ws;
    int No() const { return act == kActSwiglu ? N / 2 : N; }
};
int64_t linear_workspace(int E, int64_t M, int N, int K, int act, int type, int out_type);
int64_t linear_backward_workspace(int E, int64_t M, int N, int K, int act, int type, int dout_type);
// How linear (0), its dx (1) or dw (2) runs: columns of a tile (0: the few-row kernel), tokens of one (0: a tile
// has 256 rows), splits of k, and whether chains are summed in registers.
void linear_plan(int which, int E, int64_t M, int N, int K, int act, int type, int io_type, int *o);
// MOE_MX_OK or a negative status (text recorded).
int launch_linear(const LinearArgs &a, cudaStream_t s);
int launch_linear_backward(const LinearBackwardArgs &a, cudaStream_t s);
// Synchronises s; MOE_MX_ERR_TIMEOUT if a wait of the current device's products gave up.
int linear_status(cudaStream_t s);
// One kernel whose wait runs out after timeout_ns, recorded as a product's would be.
int linear_watchdog(unsigned long long timeout_ns, cudaStream_t s);

} // namespace moe_mx
