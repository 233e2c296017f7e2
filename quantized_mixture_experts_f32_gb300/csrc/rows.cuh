// rows.cuh -- the 8-bit path's row operators: what their kernels and the C ABI share.
#pragma once
#include "kv4.cuh"

namespace qmoe {

enum : int { ROWS_E4M3 = 3 };                 // beside KV4_F32, KV4_F16, KV4_BF16
constexpr int FP8_BLOCK = 128;                // elements of a row, and rows of W, that share a scale

// y = h / sqrt(mean(h^2) + eps) * w with h = x + res; norm 0: y = x
struct NormArgs {
    const void* x;
    const void* res;                          // or null
    void* sum;                                // or null
    const float* w;                           // or null
    void* y;
    float* scale;                             // of 8-bit rows
    int64_t x_stride, res_stride, y_stride;   // elements between rows; sum's is res_stride
    int x_t, res_t, y_t;
    int rows, dim;
    float eps;
    int norm;
};
cudaError_t launch_rmsnorm_rows(const NormArgs& a, int num_sms, cudaStream_t st);

struct LinearArgs {
    const uint8_t* x;                         // [T][K]
    const float* xs;                          // [T][ceil(K/128)]
    const uint8_t* w;                         // [N][K]
    const float* ws;                          // [ceil(N/128)][ceil(K/128)]
    const float* bias;                        // or null
    const void* res;                          // or null
    void* out;
    int64_t res_stride, out_stride;
    int T, K, N, act, out_t;
    int* status;
    unsigned long long stall_ns;              // test hook: scales of one CTA of a pair come this late
};
enum : int { ACT_NONE = 0, ACT_RELU = 1, ACT_SILU = 2, ACT_GELU = 3 };
struct LinearChoice {
    int tile;                                 // features of a pair of CTAs' tile, 0: mma.sync
    int parts;                                // pairs that share a tile's k
};
LinearChoice linear_fp8_choice(int T, int K, int N, int num_sms);
// Where a product runs, and which kernels this context has set up: each with its first call, as
// there are many, and most contexts use few or none.
struct LinearRun {
    int num_sms;
    cudaStream_t st;
    uint64_t* ready;
};
cudaError_t launch_linear_fp8(const LinearArgs& a, const LinearRun& run);

// Rotary positions on the heads of rows, and the append of K and V rows behind them.
struct RopeArgs {
    const float* table;                       // [n_pos][2][rot/2]: cosines, sines
    int n_pos, rot, interleaved;
    int t, n_tokens, hd;                      // t: the rows' type
    const int32_t* pos;
    const void* q;
    void* q_out;
    int64_t q_stride, q_out_stride;
    int nq;                                   // heads of a q row, 0: none
    const float *q_norm, *k_norm;             // or null
    float eps;
    int* status;
    // the append's: nkv 0 for none
    int nkv;
    const void* k;
    const void* v;
    int64_t k_stride, v_stride;
    const int64_t* slots;
    float* k_hat;
    float* v_hat;
    Kv4Cache c;
    int page, page_log2, n_pages;
    float2 minus_zero;                        // launch_rope sets it
};
cudaError_t launch_rope(const RopeArgs& a, cudaStream_t st);

struct RopeFreq {                             // angle of each pair at position 1
    double f[128];
};
cudaError_t launch_rope_rows_table(const RopeFreq& f, int half, int n_pos, double mscale, float* table, cudaStream_t st);

}  // namespace qmoe
