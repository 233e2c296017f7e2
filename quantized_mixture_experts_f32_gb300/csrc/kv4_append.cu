// kv4_append.cu -- new K and V rows quantised to NVFP4 into their cache slots.
//
// Per 16 elements of a head, every decision in fp32: s = e4m3_rn(bmax / (6 g)),
// d = e4m3(s) g, code = e2m1_rn(x / d) (ties to the even code, saturating); zero
// where d = 0.  g is the kv head's global scale.
//
// Bound by the rows read and the values written back once the quotients are cheap.  A
// lane takes eight elements of a row (16 or 32 bytes), so that rows, codes and values
// move in whole sectors; the two lanes of a block share its maximum by a shuffle.
#include "kv4.cuh"
#include "kv4_row.cuh"
#include "ptx_sync.cuh"

namespace qmoe {

namespace {

constexpr int AP_THREADS = 256;

// v / d, correctly rounded, from r = 1 / d rounded: two of Markstein's corrections
// (Computation of elementary functions on the IBM RISC System/6000 processor, 1990).
// q = v r is within two units in the last place, the first correction brings it within
// one, and from there q + r (v - q d), the remainder being exact, rounds as v / d does.
// Exact while the remainder is a normal number; where |v| is too small for that, v / d
// is far below the first code's border.
__device__ __forceinline__ float quotient(float v, float d, float r) {
    const float q = v * r, p = fmaf(fmaf(-q, d, v), r, q);
    return copysignf(fmaf(fmaf(-p, d, v), r, p), v);          // the corrections lose the sign of -0
}

// The eight elements from c of row t (live: there are any; a block's lanes are live together).
template <int F32>
__device__ __forceinline__ void append_lane(const Kv4AppendArgs& a, int t, int c, bool live, int row, int hd_log2) {
    const bool isv = blockIdx.y != 0;
    const int h = live ? c >> hd_log2 : 0, e = c - (h << hd_log2);   // kv head, element in it
    const int64_t slot = live ? a.slots[t] : -1;
    float v[8];
    {
        uint4 u[F32 ? 2 : 1];
        const uint4* x = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(isv ? a.v : a.k) +
                                                        ((size_t)t * (isv ? a.v_stride : a.k_stride) + c) * (F32 ? 4 : 2));
#pragma unroll
        for (int i = 0; i < (F32 ? 2 : 1); ++i) u[i] = live ? x[i] : make_uint4(0, 0, 0, 0);
        kv4_floats8(u, a.dtype, v);
    }
    const float g = (isv ? a.c.vg : a.c.kg)[h];
    float bmax = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) bmax = fmaxf(bmax, fabsf(v[j]));
    bmax = fmaxf(bmax, __shfl_xor_sync(0xffffffffu, bmax, 1));
    // (448 for infinity over a 6 g that is infinite too: a scale is never NaN)
    const uint32_t s = g > 0.f ? __nv_cvt_float_to_fp8(fminf(bmax / (6.0f * g), 448.f), __NV_SATFINITE, __NV_E4M3) : 0u;
    const float sf = e4m3_f(s), d = sf * g;
    uint32_t code = 0u;
    if (d >= 0x1p-90f && d <= 0x1p90f && bmax <= d * 0x1p30f) {
        const float r = __frcp_rn(d);
#pragma unroll
        for (int j = 0; j < 8; j += 2)
            code |= (uint32_t)__nv_cvt_float2_to_fp4x2(make_float2(quotient(v[j], d, r), quotient(v[j + 1], d, r)), __NV_E2M1,
                                                       cudaRoundNearest) << (4 * j);
    } else if (d > 0.f) {
#pragma unroll
        for (int j = 0; j < 8; j += 2)
            code |= (uint32_t)__nv_cvt_float2_to_fp4x2(make_float2(v[j] / d, v[j + 1] / d), __NV_E2M1, cudaRoundNearest) << (4 * j);
    }
    float* hat = isv ? a.v_hat : a.k_hat;
    if (hat && live) {
        float4* o = reinterpret_cast<float4*>(hat + (size_t)t * row + c);
        __half2 w[4];
        kv4_widen8(code, w);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const float2 x = __half22float2(w[2 * j]), y = __half22float2(w[2 * j + 1]);
            o[j] = make_float4(x.x * sf * g, x.y * sf * g, y.x * sf * g, y.y * sf * g);
        }
    }
    if (slot < 0) return;
    const int64_t pg = slot >> a.s.page_log2;
    if (pg >= a.s.n_pages) {
        atomicExch(a.status, ST_DEVICE_CHECK);
        return;
    }
    const size_t at = ((size_t)pg * a.s.nkv + h) * a.s.page + (size_t)(slot & (a.s.page - 1));
    *reinterpret_cast<uint32_t*>((isv ? a.c.vc : a.c.kc) + at * (a.s.hd / 2) + e / 2) = code;
    if ((e & 15) == 0) (isv ? a.c.vs : a.c.ks)[at * (a.s.hd / 16) + e / 16] = (uint8_t)s;
}

// blockIdx.y: 0 = K, 1 = V.  A CTA takes rows_cta whole rows where they fit its
// threads, else one row in turns, so that indices stay 32 bits wide.  16384 F32 rows of
// four heads of 128 take 24.7 us, 5.8 TB/s of rows, codes and values (75% of the issue
// slots, 61% of the warps); four elements a lane and the compiler's division took 37 us,
// bound by instructions.  64 BF16 rows take 1.8 us, latency alone.
template <int F32>
__global__ void __launch_bounds__(AP_THREADS) kv4_append_kernel(const Kv4AppendArgs a, int lanes_row, int rows_cta,
                                                                int hd_log2) {
    pdl_wait();
    pdl_launch_dependents();
    const int r = rows_cta > 1 ? (int)threadIdx.x / lanes_row : 0;
    const int t = (int)blockIdx.x * rows_cta + r;             // row
    for (int lane0 = (int)threadIdx.x - r * lanes_row; lane0 - (int)(threadIdx.x & 31) < lanes_row; lane0 += AP_THREADS)
        append_lane<F32>(a, t, lane0 * 8, r < rows_cta && t < a.n_tokens && lane0 < lanes_row, lanes_row * 8, hd_log2);
}

}  // namespace

cudaError_t launch_kv4_append(const Kv4AppendArgs& a, cudaStream_t st) {
    const int lanes_row = a.s.nkv * a.s.hd / 8;
    const int rows_cta = lanes_row < AP_THREADS ? AP_THREADS / lanes_row : 1;
    const int hd_log2 = a.s.hd == 64 ? 6 : a.s.hd == 128 ? 7 : 8;
    const dim3 grid((unsigned)((a.n_tokens + rows_cta - 1) / rows_cta), 2);
    return a.dtype == KV4_F32
               ? launch_pdl(kv4_append_kernel<1>, grid, dim3(AP_THREADS), 0, st, a, lanes_row, rows_cta, hd_log2)
               : launch_pdl(kv4_append_kernel<0>, grid, dim3(AP_THREADS), 0, st, a, lanes_row, rows_cta, hd_log2);
}

}  // namespace qmoe
