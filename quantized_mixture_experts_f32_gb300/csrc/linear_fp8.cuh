// linear_fp8.cuh -- what the kernels of qmoe_linear_fp8 share.
#pragma once
#include "kv4_row.cuh"
#include "ptx_sync.cuh"
#include "rows.cuh"
#include "umma.cuh"

namespace qmoe {

// prefill_umma.cu: tensor maps over E4M3 codes [rows][cols] (boxes of 128 columns) and over
// rows of any type (boxes of 128 bytes), both with the 128-byte swizzle
bool tensor_map_codes(CUtensorMap* m, const void* base, uint64_t cols, uint64_t rows, uint32_t box_rows);
bool tensor_map_rows(CUtensorMap* m, const void* base, int t, uint64_t cols, uint64_t rows, uint64_t stride, uint32_t box_rows);

// linear_fp8_pair.cu
// tiles of 128 or 256 features; of 128, a tile's k may be shared by 2 to 4 pairs, each at least a
// group of four blocks
cudaError_t launch_linear_pair(const LinearArgs& a, int tile, int parts, const LinearRun& run);

// linear_fp8_few.cu: a CTA takes 16 features of a group of tokens
constexpr int LF_ROWS = 16;
inline int linear_few_group(int tokens) { return tokens <= 8 ? 8 : tokens <= 32 ? 16 : 32; }
cudaError_t launch_linear_few(const LinearArgs& a, int num_sms, cudaStream_t st);

// (x, y) += (a sx, b sy), two roundings in one instruction
__device__ __forceinline__ void fma2(float2& acc, uint32_t a, uint32_t b, float sx, float sy) {
    asm("{\n\t.reg .b64 d, v, s;\n\tmov.b64 d, {%0, %1};\n\tmov.b64 v, {%2, %3};\n\tmov.b64 s, {%4, %5};\n\t"
        "fma.rn.f32x2 d, v, s, d;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "+f"(acc.x), "+f"(acc.y)
        : "r"(a), "r"(b), "f"(sx), "f"(sy));
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    fma2(c, __float_as_uint(a.x), __float_as_uint(a.y), b.x, b.y);
    return c;
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

__device__ __forceinline__ float relu(float z) {                                             // NaN stays
    float y;
    asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(y) : "f"(z));
    return y;
}
// z / (1 + exp(-z)); where the sum is infinite its reciprocal is 0
__device__ __forceinline__ float silu(float z) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + __expf(-z)));
    return z * r;
}
// z Phi(z) = max(z, 0) - m erfc(m / sqrt 2) / 2, m = |z|, erfc as 2^-q(m) with q a polynomial without a
// constant, fitted to log2 erfc for the least largest error of the result over |z|, m up to 6, where the
// second term is 6e-9 and stays.  The fit alone is off by 1.3e-8 |z| and by 3.5e-8 at most; in fp32, with
// the exponential's error and the result rounded, 8.5e-8 |z| was the most found (2e-7 |z| is promised).
// Two results at a time: 9 instructions each, where a form with a quotient (1.5e-7 |z|) took 20.
__device__ __forceinline__ float2 gelu(float2 z) {
    const float2 m = make_float2(fminf(fabsf(z.x), 6.f), fminf(fabsf(z.y), 6.f));
    float2 p = both(-2.8349129e-06f);
    p = fma2(p, m, both(3.93776900e-05f));
    p = fma2(p, m, both(-1.86180245e-04f));
    p = fma2(p, m, both(-1.36936374e-04f));
    p = fma2(p, m, both(7.06342002e-03f));
    p = fma2(p, m, both(-5.24961799e-02f));
    p = fma2(p, m, both(-4.59208190e-01f));
    p = fma2(p, m, both(-1.15110517f));
    p = make_float2(p.x * m.x, p.y * m.y);
    const float2 e = make_float2(kv4_ex2(p.x), kv4_ex2(p.y));
    return fma2(make_float2(-0.5f * m.x, -0.5f * m.y), e, make_float2(relu(z.x), relu(z.y)));
}

template <int N>
__device__ __forceinline__ void activate(float (&v)[N], int act) {
    if (act == ACT_RELU) {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = relu(v[i]);
    } else if (act == ACT_SILU) {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = silu(v[i]);
    } else if (act == ACT_GELU) {
#pragma unroll
        for (int i = 0; i < N; i += 2) {
            const float2 y = gelu(make_float2(v[i], v[i + 1 < N ? i + 1 : i]));
            v[i] = y.x;
            if (i + 1 < N) v[i + 1] = y.y;
        }
    }
}

// one element of a row
template <int T>
struct RowType {
    using type = float;
    static __device__ __forceinline__ float load(float v) { return v; }
    static __device__ __forceinline__ float store(float v) { return v; }
};
template <>
struct RowType<KV4_F16> {
    using type = __half;
    static __device__ __forceinline__ float load(__half v) { return __half2float(v); }
    static __device__ __forceinline__ __half store(float v) { return __float2half_rn(v); }
};
template <>
struct RowType<KV4_BF16> {
    using type = __nv_bfloat16;
    static __device__ __forceinline__ float load(__nv_bfloat16 v) { return __bfloat162float(v); }
    static __device__ __forceinline__ __nv_bfloat16 store(float v) { return __float2bfloat16_rn(v); }
};

// token t's feature n: residual added, stored
template <int T>
__device__ __forceinline__ void put_one(const LinearArgs& a, int t, int n, float v) {
    using R = RowType<T>;
    using type = typename R::type;
    if (a.res) v += R::load(static_cast<const type*>(a.res)[(size_t)t * a.res_stride + n]);
    static_cast<type*>(a.out)[(size_t)t * a.out_stride + n] = R::store(v);
}
__device__ __forceinline__ void put_one(const LinearArgs& a, int t, int n, float v) {
    if (a.out_t == KV4_F32) put_one<KV4_F32>(a, t, n, v);
    else if (a.out_t == KV4_F16) put_one<KV4_F16>(a, t, n, v);
    else put_one<KV4_BF16>(a, t, n, v);
}

// element i of 16 bytes of a row of type T, and 16 bytes of elements
template <int T>
__device__ __forceinline__ float row_element(const uint32_t (&w)[4], int i) {
    if (T == KV4_F32) return __uint_as_float(w[i & 3]);
    uint32_t x = w[i / 2];
    if (T == KV4_BF16) return __uint_as_float(i & 1 ? x & 0xffff0000u : x << 16);
    const __half2 h = *reinterpret_cast<__half2*>(&x);
    return i & 1 ? __high2float(h) : __low2float(h);
}
template <int T, int N>
__device__ __forceinline__ void row_pack(const float (&v)[N], uint32_t (&w)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (T == KV4_F32) w[i] = __float_as_uint(v[i]);
        else w[i] = kv4_pack16(v[2 * i], v[2 * i + 1], T);
    }
}

// 16 columns of this thread's TMEM lane; tmem_arrived() before they are used
__device__ __forceinline__ void tmem_fetch16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_arrived(uint32_t (&r)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])::"memory");
}

// The warps that issue products and copies run their loops as a whole, so that descriptors
// and addresses stay in uniform registers; only the instructions are one lane's (`one`).
__device__ __forceinline__ uint32_t elected() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p;
}
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __shfl_sync(0xffffffffu, v, 0); }   // known to be
// a whole warp's bounded wait
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity));
}

// An arrival that orders no memory: for columns of TMEM, whose reads tcgen05.wait::ld has ended.
// (One that releases waits for the thread's loads in flight.)
__device__ __forceinline__ void arrive_relaxed(uint64_t* bar) {
    asm volatile("mbarrier.arrive.relaxed.cta.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// (aligned: the whole warp at once, whatever one of its lanes did before)
__device__ __forceinline__ void cluster_sync() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_addr(const void* p, uint32_t rank) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
    return a;
}

}  // namespace qmoe
