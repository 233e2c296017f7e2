// kv4_append.cu -- new K and V rows quantised to NVFP4 into their cache slots.
//
// Per 16 elements of a head, every decision in fp32: s = e4m3_rn(bmax / (6 g)),
// d = e4m3(s) g, code = e2m1_rn(x / d) (ties to the even code, saturating); zero
// where d = 0.  g is the kv head's global scale.
//
// Bound by the rows read and the values written back.  A lane takes 16 bytes of a
// row (four F32 or eight 16-bit elements), so that rows, codes and values move in
// whole lines; the lanes of a block share its maximum by shuffles.
#include "kv4.cuh"
#include "kv4_row.cuh"
#include "ptx_sync.cuh"

namespace qmoe {

namespace {

constexpr int AP_THREADS = 256;

// E elements a lane; blockIdx.y: 0 = K, 1 = V; a warp's lanes are in one row or the next
template <int E>
__global__ void __launch_bounds__(AP_THREADS) kv4_append_kernel(const Kv4AppendArgs a, int lanes_row) {
    constexpr int LB = 16 / E;                                // lanes of a block
    pdl_wait();
    pdl_launch_dependents();
    const bool isv = blockIdx.y != 0;
    const size_t i = (size_t)blockIdx.x * AP_THREADS + threadIdx.x;
    const int t = (int)(i / lanes_row), c = (int)(i - (size_t)t * lanes_row) * E;   // row, element in it
    const bool live = t < a.n_tokens;                         // whole blocks: their lanes are live together
    const int h = live ? c / a.s.hd : 0, e = c - h * a.s.hd;  // kv head, element in it
    float v[E];
    {
        uint4 u = make_uint4(0, 0, 0, 0);
        if (live)
            u = *reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(isv ? a.v : a.k) +
                                                ((size_t)t * (isv ? a.v_stride : a.k_stride) + c) * (16 / E));
        if constexpr (E == 4) {
            v[0] = __uint_as_float(u.x);
            v[1] = __uint_as_float(u.y);
            v[2] = __uint_as_float(u.z);
            v[3] = __uint_as_float(u.w);
        } else {
            const uint4 one[1] = {u};
            kv4_floats8(one, a.dtype, v);
        }
    }
    const float g = (isv ? a.c.vg : a.c.kg)[h];
    float bmax = 0.f;
#pragma unroll
    for (int j = 0; j < E; ++j) bmax = fmaxf(bmax, fabsf(v[j]));
#pragma unroll
    for (int o = LB / 2; o; o >>= 1) bmax = fmaxf(bmax, __shfl_xor_sync(0xffffffffu, bmax, o));
    const uint32_t s = g > 0.f ? __nv_cvt_float_to_fp8(bmax / (6.0f * g), __NV_SATFINITE, __NV_E4M3) : 0u;
    const float sf = e4m3_f(s), d = sf * g;
    uint32_t code = 0u;                                       // E of them
    if (d > 0.f) {
#pragma unroll
        for (int j = 0; j < E; j += 2)
            code |= (uint32_t)__nv_cvt_float2_to_fp4x2(make_float2(v[j] / d, v[j + 1] / d), __NV_E2M1, cudaRoundNearest) << (4 * j);
    }
    float* hat = isv ? a.v_hat : a.k_hat;
    if (hat && live) {
        float4* o = reinterpret_cast<float4*>(hat + (size_t)t * lanes_row * E + c);
#pragma unroll
        for (int j = 0; j < E; j += 4) {
            const float2 x = e2m1x2_f2(code >> (4 * j)), y = e2m1x2_f2(code >> (4 * j + 8));
            o[j / 4] = make_float4(x.x * sf * g, x.y * sf * g, y.x * sf * g, y.y * sf * g);
        }
    }
    if constexpr (E == 4) code |= __shfl_xor_sync(0xffffffffu, code, 1) << 16;     // in the even lanes
    if (!live || (E == 4 && (threadIdx.x & 1))) return;
    const int64_t slot = a.slots[t];
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

}  // namespace

cudaError_t launch_kv4_append(const Kv4AppendArgs& a, cudaStream_t st) {
    const int per = a.dtype == KV4_F32 ? 4 : 8, lanes_row = a.s.nkv * a.s.hd / per;
    const size_t lanes = (size_t)a.n_tokens * lanes_row;
    const dim3 grid((unsigned)((lanes + AP_THREADS - 1) / AP_THREADS), 2);
    return per == 4 ? launch_pdl(kv4_append_kernel<4>, grid, dim3(AP_THREADS), 0, st, a, lanes_row)
                    : launch_pdl(kv4_append_kernel<8>, grid, dim3(AP_THREADS), 0, st, a, lanes_row);
}

}  // namespace qmoe
