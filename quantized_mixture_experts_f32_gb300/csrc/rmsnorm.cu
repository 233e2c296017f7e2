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

// A row by tpr threads (a multiple of 32), CH chunks of eight elements each, rows_cta
// rows a CTA at a time.
template <int CH, int NORM>
__global__ void __launch_bounds__(1024) rmsnorm_kernel(const NormArgs a, int tpr, int rows_cta) {
    __shared__ float part[2][32];
    pdl_wait();
    pdl_launch_dependents();
    const int r = (int)threadIdx.x / tpr, lane = (int)threadIdx.x - r * tpr, chunks = a.dim >> 3;
    const int warps = tpr >> 5, warp0 = r * warps;
    int turn = 0;
    for (int64_t base = (int64_t)blockIdx.x * rows_cta; base < a.rows; base += (int64_t)gridDim.x * rows_cta) {
        const int64_t row = base + r;
        float h[CH][8];
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            const int c = i * tpr + lane;
            const bool live = row < a.rows && c < chunks;
#pragma unroll
            for (int j = 0; j < 8; ++j) h[i][j] = 0.f;
            if (!live) continue;
            rows_load8(a.x, row * a.x_stride + 8 * c, a.x_t, h[i]);
            if (NORM && a.res) {
                float g[8];
                const size_t at = row * a.res_stride + 8 * c;
                rows_load8(a.res, at, a.res_t, g);
#pragma unroll
                for (int j = 0; j < 8; ++j) h[i][j] += g[j];
                if (a.sum) kv4_store8(a.sum, at, a.res_t, h[i]);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) ss = fmaf(h[i][j], h[i][j], ss);
        }
        float inv = 1.f;
        if (NORM) {
            ss = group_sum<32>(ss);
            if (warps > 1) {
                if ((threadIdx.x & 31) == 0) part[turn][threadIdx.x >> 5] = ss;
                __syncthreads();
                ss = 0.f;
                for (int w = 0; w < warps; ++w) ss += part[turn][warp0 + w];
                turn ^= 1;
            }
            inv = __frsqrt_rn(ss / (float)a.dim + a.eps);
        }
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            const int c = i * tpr + lane;
            const bool live = row < a.rows && c < chunks;
            float m = 0.f;
            if (NORM && live) {
                float w[8] = {1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f};
                if (a.w) rows_load8(a.w, 8 * c, KV4_F32, w);
#pragma unroll
                for (int j = 0; j < 8; ++j) h[i][j] = h[i][j] * inv * w[j];
            }
            if (a.y_t != ROWS_E4M3) {
                if (live) kv4_store8(a.y, row * a.y_stride + 8 * c, a.y_t, h[i]);
                continue;
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(h[i][j]));
#pragma unroll
            for (int o = 1; o < 16; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));   // 16 lanes: a block
            if (!live) continue;
            const float s = m / 448.f;
            *reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.y) + row * a.dim + 8 * c) = rows_e4m3x8(h[i], s);
            if ((c & 15) == 0) a.scale[row * ((a.dim + FP8_BLOCK - 1) / FP8_BLOCK) + (c >> 4)] = s;
        }
    }
}

template <int CH>
cudaError_t launch_ch(const NormArgs& a, int grid, int tpr, int rows_cta, cudaStream_t st) {
    return a.norm ? launch_pdl(rmsnorm_kernel<CH, 1>, dim3(grid), dim3(tpr * rows_cta), 0, st, a, tpr, rows_cta)
                  : launch_pdl(rmsnorm_kernel<CH, 0>, dim3(grid), dim3(tpr * rows_cta), 0, st, a, tpr, rows_cta);
}

}  // namespace

cudaError_t launch_rmsnorm_rows(const NormArgs& a, int num_sms, cudaStream_t st) {
    const int chunks = a.dim / 8;
    int ch = 1;
    while (ch < 8 && (chunks + ch - 1) / ch > 256) ch *= 2;
    const int tpr = ((chunks + ch - 1) / ch + 31) / 32 * 32;
    const int rows_cta = tpr < 256 ? 256 / tpr : 1;
    const int64_t need = (a.rows + (int64_t)rows_cta - 1) / rows_cta, cap = (int64_t)num_sms * (2048 / (tpr * rows_cta));
    const int grid = (int)(need < cap ? need : cap);
    switch (ch) {
        case 1: return launch_ch<1>(a, grid, tpr, rows_cta, st);
        case 2: return launch_ch<2>(a, grid, tpr, rows_cta, st);
        case 4: return launch_ch<4>(a, grid, tpr, rows_cta, st);
        default: return launch_ch<8>(a, grid, tpr, rows_cta, st);
    }
}

}  // namespace qmoe
