// linear_fp8.cu -- out = act(x W^T + bias) + residual over E4M3 codes with block scales.
//
//   z[t][n] = sum_b xs[t][b] ws[n/128][b] sum_{k in block b} x[t][k] W[n][k]
#include "kv4_row.cuh"
#include "ptx_sync.cuh"
#include "rows.cuh"

namespace qmoe {

namespace {

constexpr int LN_TOKENS = 8;     // tokens a warp takes at once

__device__ __forceinline__ float activate(float z, int act) {
    if (act == ACT_RELU) return z < 0.f ? 0.f : z;            // NaN stays
    if (act == ACT_SILU) return z / (1.f + __expf(-z));
    if (act == ACT_GELU) return 0.5f * z * (1.f + erff(z * 0.70710678118654752f));
    return z;
}

__device__ __forceinline__ float row_load(const void* p, size_t at, int t) {
    if (t == KV4_F32) return static_cast<const float*>(p)[at];
    if (t == KV4_F16) return __half2float(static_cast<const __half*>(p)[at]);
    return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[at]);
}

__device__ __forceinline__ void row_store(void* p, size_t at, int t, float v) {
    if (t == KV4_F32) static_cast<float*>(p)[at] = v;
    else if (t == KV4_F16) static_cast<__half*>(p)[at] = __float2half_rn(v);
    else static_cast<__nv_bfloat16*>(p)[at] = __float2bfloat16_rn(v);
}

// one feature a warp, a lane 16 elements of K at a time
__global__ void __launch_bounds__(256) linear_fp8_kernel(const LinearArgs a) {
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int n = (int)(blockIdx.x * 8 + (threadIdx.x >> 5));
    if (n >= a.N) return;
    const int kb = (a.K + FP8_BLOCK - 1) / FP8_BLOCK;
    const float* ws = a.ws + (size_t)(n / FP8_BLOCK) * kb;
    for (int t0 = (int)blockIdx.y * LN_TOKENS; t0 < a.T; t0 += (int)gridDim.y * LN_TOKENS) {
        float z[LN_TOKENS] = {};
        for (int k = lane * 16; k < a.K; k += 512) {
            const uint4 w = *reinterpret_cast<const uint4*>(a.w + (size_t)n * a.K + k);
            const uint32_t wi[4] = {w.x, w.y, w.z, w.w};
            const float sw = ws[k / FP8_BLOCK];
#pragma unroll
            for (int t = 0; t < LN_TOKENS; ++t) {
                if (t0 + t >= a.T) break;
                const uint4 x = *reinterpret_cast<const uint4*>(a.x + (size_t)(t0 + t) * a.K + k);
                const uint32_t xi[4] = {x.x, x.y, x.z, x.w};
                float s = 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float2 p = e4m3x2_f2((wi[i / 2] >> (16 * (i & 1))) & 0xffffu), q = e4m3x2_f2((xi[i / 2] >> (16 * (i & 1))) & 0xffffu);
                    s = fmaf(p.x, q.x, fmaf(p.y, q.y, s));
                }
                z[t] = fmaf(s, sw * a.xs[(size_t)(t0 + t) * kb + k / FP8_BLOCK], z[t]);
            }
        }
#pragma unroll
        for (int t = 0; t < LN_TOKENS; ++t) {
            float v = group_sum<32>(z[t]);
            if (lane || t0 + t >= a.T) continue;
            if (a.bias) v += a.bias[n];
            v = activate(v, a.act);
            if (a.res) v += row_load(a.res, (size_t)(t0 + t) * a.res_stride + n, a.out_t);
            row_store(a.out, (size_t)(t0 + t) * a.out_stride + n, a.out_t, v);
        }
    }
}

}  // namespace

cudaError_t linear_fp8_prepare() { return cudaSuccess; }

cudaError_t launch_linear_fp8(const LinearArgs& a, int num_sms, cudaStream_t st) {
    (void)num_sms;
    const int turns = (a.T + LN_TOKENS - 1) / LN_TOKENS;
    return launch_pdl(linear_fp8_kernel, dim3((unsigned)((a.N + 7) / 8), (unsigned)(turns < 65535 ? turns : 65535)), dim3(256),
                      0, st, a);
}

}  // namespace qmoe
