// kv4_row.cuh -- arithmetic the cache's attention kernels share: widening codes,
// splitting fp32 values into fp16 terms, rows of any type.
#pragma once
#include "kv4.cuh"

namespace qmoe {

// A row's weights are held as 2^(z - m + P_UP) and its m follows the running maximum
// once that is P_SLACK ahead: at most 2^14 in fp16, and the low parts of all but
// vanishing weights stay normal.
constexpr float KV4_P_UP = 6.f;
constexpr float KV4_P_SLACK = 8.f;

__device__ __forceinline__ float kv4_ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint32_t kv4_u(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }
__device__ __forceinline__ uint32_t kv4_pack(float x, float y) { return kv4_u(__floats2half2_rn(x, y)); }

// x = hi + lo to 22 bits, as fp16 pairs
__device__ __forceinline__ void kv4_split(float x, float y, uint32_t& hi, uint32_t& lo) {
    const __half2 h = __floats2half2_rn(x, y);
    hi = kv4_u(h);
    lo = kv4_pack(x - __low2float(h), y - __high2float(h));
}

// For a row whose largest magnitude is `big`, the e for which 2^-e brings it to [1, 2):
// -126 .. 126, so that 2^-e is a normal number (a row below 2^-126 is a multiple of
// 2^-149, and 2^126 of it exact in two fp16 terms; a 16-bit row's in one); 0 for zero,
// infinity and NaN.
__device__ __forceinline__ int kv4_exponent(float big) {
    const int e = (int)(__float_as_uint(big) >> 23) - 127;
    return e == -127 && big == 0.f || e > 127 ? 0 : min(max(e, -126), 126);
}
__device__ __forceinline__ float kv4_pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }   // |e| < 127

// What brings a row's product with K's codes to its scores in powers of two, in size:
// scale * log2(e) * global * 2^e for a row that was scaled by 2^-e.  The factors' own
// powers of two are set apart (f in 2^-46 .. 2^5, or 0) and put in with the row's as one
// exponent, so that nothing leaves fp32's range on the way where the result is in it.
struct Kv4Factor {
    float f;
    int e;
};
__device__ __forceinline__ Kv4Factor kv4_factor(float scale, float global) {
    scale = fabsf(scale);
    global = fabsf(global);
    const int es = kv4_exponent(scale), eg = kv4_exponent(global);
    const float f = scale * kv4_pow2(-es) * (1.4426950408889634f * (global * kv4_pow2(-eg)));
    return {f, f == 0.f ? -1024 : es + eg};
}
// Not 0, so that a masked -inf stays -inf (1e-38 q.k is 0 to any other score), and finite,
// so that a q.k of 0 stays 0.
__device__ __forceinline__ float kv4_factor_of(const Kv4Factor& x, int e) {
    const int bits = (int)__float_as_uint(x.f), all = x.e + e, to = (bits >> 23) + all;
    return to < 1 ? 1e-38f : to > 254 ? 3.4e38f : __uint_as_float((uint32_t)(bits + all * (1 << 23)));
}
// The argument of a weight's exponential is q.k fac - m in one rounding, m itself rounded
// to fp32.  Whether scores may be so large, past 2^21, that m's rounding is no small part
// of it (|q.k| < 2^13 head_dim, q scaled): then q.k fac is rounded as m is first.
template <int HD>
__device__ __forceinline__ bool kv4_far(float fac) {
    return fac > 0x1p8f / HD;
}
// whether that product is negative
__device__ __forceinline__ bool kv4_negative(float scale, float global) {
    return (int)(__float_as_uint(scale) ^ __float_as_uint(global)) < 0;
}

// Eight E2M1 codes -> four half2, bytes in order.  One conversion a byte: naming the
// bytes of w in PTX lets the conversion pick its byte, where extracting them first
// cost an instruction more on the same (half-rate) pipe.
__device__ __forceinline__ void kv4_widen8(uint32_t w, __half2 (&h)[4]) {
    uint32_t r[4];
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\tcvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\tcvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
        : "r"(w));
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = *reinterpret_cast<__half2*>(&r[i]);
}

// two E4M3 codes (bytes 0 and 1 of x) -> half2
__device__ __forceinline__ __half2 kv4_scale2(uint32_t x) {
    return __half2(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(x), __NV_E4M3));
}
// the low bytes of two words, as bytes 0 and 1
__device__ __forceinline__ uint32_t kv4_bytes(uint32_t lo, uint32_t hi) { return __byte_perm(lo, hi, 0x0040); }

// Eight elements each of two positions -> bytes that hold one element of both: the
// even elements, the odd elements.
__device__ __forceinline__ void kv4_pair(uint32_t a, uint32_t b, uint32_t& even, uint32_t& odd) {
    constexpr uint32_t lo4 = 0x0f0f0f0fu;
    even = (a & lo4) | ((b << 4) & ~lo4);
    odd = ((a >> 4) & lo4) | (b & ~lo4);
}

// two neighbouring elements of a row of type t, at element `at` (even)
__device__ __forceinline__ float2 kv4_load2(const void* p, size_t at, int t) {
    if (t == KV4_F32) return *reinterpret_cast<const float2*>(static_cast<const float*>(p) + at);
    uint32_t b = *reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(p) + at);
    if (t == KV4_F16) return __half22float2(*reinterpret_cast<__half2*>(&b));
    return make_float2(__uint_as_float(b << 16), __uint_as_float(b & 0xffff0000u));
}

__device__ __forceinline__ void kv4_store2(void* p, size_t at, int t, float x, float y) {
    if (t == KV4_F32) *reinterpret_cast<float2*>(static_cast<float*>(p) + at) = make_float2(x, y);
    else if (t == KV4_F16) *reinterpret_cast<__half2*>(static_cast<__half*>(p) + at) = __floats2half2_rn(x, y);
    else *reinterpret_cast<__nv_bfloat162*>(static_cast<__nv_bfloat16*>(p) + at) = __floats2bfloat162_rn(x, y);
}

// eight elements as they were loaded: F32 from two words of 16 bytes, else one
template <int N>
__device__ __forceinline__ void kv4_floats8(const uint4 (&u)[N], int t, float (&v)[8]) {
    const uint32_t w[4] = {u[0].x, u[0].y, u[0].z, u[0].w}, w2[4] = {u[N - 1].x, u[N - 1].y, u[N - 1].z, u[N - 1].w};
    if constexpr (N == 2) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[i] = __uint_as_float(w[i]);
            v[4 + i] = __uint_as_float(w2[i]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t x = w[i];
            const float2 f = t == KV4_F16 ? __half22float2(*reinterpret_cast<__half2*>(&x))
                                          : make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u));
            v[2 * i] = f.x;
            v[2 * i + 1] = f.y;
        }
    }
}

// two values as F16 or BF16
__device__ __forceinline__ uint32_t kv4_pack16(float x, float y, int t) {
    if (t == KV4_F16) return kv4_pack(x, y);
    const __nv_bfloat162 b = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&b);
}

// eight elements at a multiple of eight
__device__ __forceinline__ void kv4_store8(void* p, size_t at, int t, const float* v) {
    if (t == KV4_F32) {
        float4* f = reinterpret_cast<float4*>(static_cast<float*>(p) + at);
        f[0] = make_float4(v[0], v[1], v[2], v[3]);
        f[1] = make_float4(v[4], v[5], v[6], v[7]);
        return;
    }
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = kv4_pack16(v[2 * i], v[2 * i + 1], t);
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + at) = make_uint4(w[0], w[1], w[2], w[3]);
}

}  // namespace qmoe
