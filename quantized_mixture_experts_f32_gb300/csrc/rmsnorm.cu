// rmsnorm.cu -- h = x + residual, y = h / sqrt(mean(h^2) + eps) * weight, and rows into
// 8 bits: E4M3 codes with one fp32 scale per 128 elements, with the norm or without.
#include "kv4_row.cuh"
#include "ptx_sync.cuh"
#include "rows.cuh"

namespace qmoe {

namespace {

// eight values under a scale as E4M3 codes; the quotients are correctly rounded
__device__ __forceinline__ uint2 rows_e4m3x8(const float (&v)[8], float s) {
    float q[8];
    if (s >= 0x1p-90f && s <= 0x1p90f) {
        const float r = __frcp_rn(s);
#pragma unroll
        for (int i = 0; i < 8; ++i) q[i] = kv4_quotient(v[i], s, r);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) q[i] = s > 0.f || v[i] != v[i] ? v[i] / s : 0.f;
    }
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] = __nv_cvt_float2_to_fp8x2(make_float2(q[2 * i], q[2 * i + 1]), __NV_SATFINITE, __NV_E4M3);
    return make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
}

// eight elements as they lie in memory
template <int F32>
struct Raw8 {
    uint4 u[F32 + 1];
    __device__ __forceinline__ void load(const void* p, int64_t at) {
        const uint4* s = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p) + at * (F32 ? 4 : 2));
#pragma unroll
        for (int i = 0; i <= F32; ++i) u[i] = s[i];
    }
    __device__ __forceinline__ void widen(int t, float (&v)[8]) const { kv4_floats8(u, t, v); }
};

// Bound by HBM where rows are many and have up to 4096 elements: 16384 rows of 2048, BF16 added to an
// F32 residual, 8 bits out, take 55.5 us, 6.66 TB/s of 6.7; of 4096, BF16 all through, 78 us, 6.9.
// A row in registers is read once; loads that began one by one behind branches on types and ends
// took 80 us.  Rows of 4112 and more take eight chunks a thread (128 registers, up to 96 bytes spilled):
// 7168 elements, BF16 with a BF16 residual, 161 us, 5.8 TB/s, in 8 bits 197 us, 4.2; F32 in 8 bits 316 us, 4.85.
//
// A row by tpr threads (a multiple of 32), CH chunks of eight elements each, rows_cta rows a
// CTA.  X, RES: whether x, the residual are F32; RES -1: no residual; NORM 0: quantise.
// All of a thread's loads are on their way before the first is used.
template <int CH, int X, int RES, int NORM>
__global__ void __launch_bounds__(512) rmsnorm_kernel(const NormArgs a, int tpr, int rows_cta) {
    __shared__ float part[16];
    pdl_wait();
    pdl_launch_dependents();
    const int r = rows_cta > 1 ? (int)threadIdx.x / tpr : 0, lane = (int)threadIdx.x - r * tpr, chunks = a.dim >> 3;
    const int64_t row0 = (int64_t)blockIdx.x * rows_cta + r;
    const bool in = row0 < a.rows;
    const int64_t row = in ? row0 : 0;                        // lanes without work load and write nothing
    Raw8<X> rx[CH];
    Raw8<RES == 1> rr[RES >= 0 ? CH : 1];
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        const int c = i * tpr + lane, at = c < chunks ? 8 * c : 0;
        rx[i].load(a.x, row * a.x_stride + at);
        if (RES >= 0) rr[i].load(a.res, row * a.res_stride + at);
    }
    float h[CH][8];
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        const int c = i * tpr + lane;
        rx[i].widen(X ? KV4_F32 : a.x_t, h[i]);
        if (RES >= 0) {
            float g[8];
            rr[i].widen(RES == 1 ? KV4_F32 : a.res_t, g);
#pragma unroll
            for (int j = 0; j < 8; ++j) h[i][j] += g[j];
            if (a.sum && in && c < chunks) kv4_store8(a.sum, row * a.res_stride + 8 * c, RES == 1 ? KV4_F32 : a.res_t, h[i]);
        }
        if (c >= chunks) {
#pragma unroll
            for (int j = 0; j < 8; ++j) h[i][j] = 0.f;
        }
        if (NORM) {
#pragma unroll
            for (int j = 0; j < 8; ++j) ss = fmaf(h[i][j], h[i][j], ss);
        }
    }
    float inv = 1.f;
    if (NORM) {
        ss = group_sum<32>(ss);
        if (tpr > 32) {
            if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = ss;
            __syncthreads();
            const int warps = tpr >> 5, w = (int)threadIdx.x & 31;
            ss = group_sum<32>(w < warps ? part[r * warps + w] : 0.f);
        }
        inv = __frsqrt_rn(ss / (float)a.dim + a.eps);
    }
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        const int c = i * tpr + lane;
        const bool live = in && c < chunks;
        if (NORM) {
#pragma unroll
            for (int j = 0; j < 8; ++j) h[i][j] *= inv;
            if (a.w) {
                const float4* w4 = reinterpret_cast<const float4*>(a.w + (c < chunks ? 8 * c : 0));
                const float4 p = __ldg(w4), q = __ldg(w4 + 1);
                const float w[8] = {p.x, p.y, p.z, p.w, q.x, q.y, q.z, q.w};
#pragma unroll
                for (int j = 0; j < 8; ++j) h[i][j] *= w[j];
            }
        }
        if (a.y_t != ROWS_E4M3) {
            if (live) kv4_store8(a.y, row * a.y_stride + 8 * c, a.y_t, h[i]);
            continue;
        }
        float m = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(h[i][j]));
#pragma unroll
        for (int o = 1; o < 16; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));   // 16 lanes: a block
        if (live) {
            const float s = m / 448.f;
            *reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.y) + row * a.dim + 8 * c) = rows_e4m3x8(h[i], s);
            if ((c & 15) == 0) a.scale[row * ((a.dim + FP8_BLOCK - 1) / FP8_BLOCK) + (c >> 4)] = s;
        }
        __syncwarp();
    }
}

using NormKernel = void (*)(NormArgs, int, int);

template <int CH, int X>
NormKernel rmsnorm_of(const NormArgs& a) {
    return !a.norm               ? rmsnorm_kernel<CH, X, -1, 0>
           : !a.res              ? rmsnorm_kernel<CH, X, -1, 1>
           : a.res_t == KV4_F32  ? rmsnorm_kernel<CH, X, 1, 1>
                                 : rmsnorm_kernel<CH, X, 0, 1>;
}
template <int CH>
NormKernel rmsnorm_of(const NormArgs& a) {
    return a.x_t == KV4_F32 ? rmsnorm_of<CH, 1>(a) : rmsnorm_of<CH, 0>(a);
}

}  // namespace

cudaError_t launch_rmsnorm_rows(const NormArgs& a, int num_sms, cudaStream_t st) {
    const int chunks = a.dim / 8;
    const int want = a.rows > 4 * num_sms ? 128 : 256;       // threads of a row
    int ch = 1;
    while (ch < 8 && (chunks + ch - 1) / ch > want) ch *= 2;
    const int tpr = ((chunks + ch - 1) / ch + 31) / 32 * 32;
    const int rows_cta = tpr < 128 ? 128 / tpr : 1;
    const dim3 grid((unsigned)((a.rows + (int64_t)rows_cta - 1) / rows_cta)), block(tpr * rows_cta);
    const NormKernel k = ch == 1 ? rmsnorm_of<1>(a) : ch == 2 ? rmsnorm_of<2>(a) : ch == 4 ? rmsnorm_of<4>(a) : rmsnorm_of<8>(a);
    return launch_pdl(k, grid, block, 0, st, a, tpr, rows_cta);
}

}  // namespace qmoe
