// kv4_append.cu -- new K and V rows quantised to NVFP4 into their cache slots.
//
// Per 16 elements of a head, every decision in fp32: s = e4m3_rn(bmax / (6 g)),
// d = e4m3(s) g, code = e2m1_rn(x / d) (ties to the even code, saturating); zero
// where d = 0.  g is the kv head's global scale.
#include "kv4.cuh"
#include "ptx_sync.cuh"

namespace qmoe {

namespace {

constexpr int AP_THREADS = 256;

// one thread per 16-element block; blockIdx.y: 0 = K, 1 = V
__global__ void __launch_bounds__(AP_THREADS) kv4_append_kernel(const Kv4AppendArgs a) {
    pdl_wait();
    const bool isv = blockIdx.y != 0;
    const int nb = a.s.nkv * a.s.hd / 16;                     // blocks of a row
    const size_t i = (size_t)blockIdx.x * AP_THREADS + threadIdx.x;
    if (i >= (size_t)a.n_tokens * nb) return;
    const int t = (int)(i / nb), b = (int)(i - (size_t)t * nb);
    const int h = b * 16 / a.s.hd, e = b * 16 - h * a.s.hd;   // kv head, element in it
    const void* x = isv ? a.v : a.k;
    const size_t row = (size_t)t * (isv ? a.v_stride : a.k_stride) + (size_t)b * 16;
    const float g = (isv ? a.c.vg : a.c.kg)[h];
    float v[16], bmax = 0.f;
#pragma unroll
    for (int j = 0; j < 16; ++j) {
        v[j] = kv4_load(x, row + j, a.dtype);
        bmax = fmaxf(bmax, fabsf(v[j]));
    }
    const uint32_t s = g > 0.f ? __nv_cvt_float_to_fp8(bmax / (6.0f * g), __NV_SATFINITE, __NV_E4M3) : 0u;
    const float sf = e4m3_f(s), d = sf * g;
    uint32_t out[2] = {0u, 0u};
    if (d > 0.f) {
#pragma unroll
        for (int j = 0; j < 16; ++j) out[j >> 3] |= kv4_e2m1_code(v[j] / d) << (4 * (j & 7));
    }
    float* hat = isv ? a.v_hat : a.k_hat;
    if (hat) {
        float* o = hat + (size_t)t * nb * 16 + (size_t)b * 16;
#pragma unroll
        for (int j = 0; j < 16; j += 2) {
            const float2 c = e2m1x2_f2(out[j >> 3] >> (4 * (j & 7)));
            o[j] = c.x * sf * g;
            o[j + 1] = c.y * sf * g;
        }
    }
    const int64_t slot = a.slots[t];
    if (slot < 0) return;
    const int64_t pg = slot / a.s.page;
    if (pg >= a.s.n_pages) {
        atomicExch(a.status, ST_DEVICE_CHECK);
        return;
    }
    const size_t at = ((size_t)pg * a.s.nkv + h) * a.s.page + (size_t)(slot - pg * a.s.page);
    *reinterpret_cast<uint2*>((isv ? a.c.vc : a.c.kc) + at * (a.s.hd / 2) + e / 2) = make_uint2(out[0], out[1]);
    (isv ? a.c.vs : a.c.ks)[at * (a.s.hd / 16) + e / 16] = (uint8_t)s;
}

}  // namespace

cudaError_t launch_kv4_append(const Kv4AppendArgs& a, cudaStream_t st) {
    const size_t blocks = (size_t)a.n_tokens * (a.s.nkv * a.s.hd / 16);
    return launch_pdl(kv4_append_kernel, dim3((unsigned)((blocks + AP_THREADS - 1) / AP_THREADS), 2),
                      dim3(AP_THREADS), 0, st, a);
}

}  // namespace qmoe
