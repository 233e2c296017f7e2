// rope.cu -- rotary positions on rows of heads, alone (qmoe_rope) and on the way into the
// paged 4-bit cache (qmoe_kv4_append_rope), and the table of their cosines and sines.
//
// Pair j of a head at position p turns by p f_j: (a, b) -> (a c - b s, b c + a s).  K's rows
// decide 4-bit codes, so every step rounds to fp32 once, as the definition says, and a
// head's mean square is carried in two fp32 words: its inverse root is then the same
// fp32 number as from 64 bits.
#include "kv4_row.cuh"
#include "ptx_sync.cuh"
#include "rows.cuh"

namespace qmoe {

namespace {

constexpr int RO_THREADS = 256;

// pairs of fp32 numbers in one instruction, each rounded as by itself
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 r;
    asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmul.rn.f32x2 z, x, y;\n\t"
        "mov.b64 {%0, %1}, z;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 r;
    asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tadd.rn.f32x2 z, x, y;\n\t"
        "mov.b64 {%0, %1}, z;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}
__device__ __forceinline__ float2 sub2(float2 a, float2 b) {
    float2 r;
    asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tsub.rn.f32x2 z, x, y;\n\t"
        "mov.b64 {%0, %1}, z;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}
__device__ __forceinline__ float2 sqr_add2(float2 a, float2 c) {       // a a + c, one rounding
    float2 r;
    asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tfma.rn.f32x2 z, x, x, y;\n\t"
        "mov.b64 {%0, %1}, z;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(c.x), "f"(c.y));
    return r;
}
// a b by itself, as a b + zero with a zero of -0, which changes nothing.  The assembler was
// found to fuse a product of pairs with a sum of pairs, rounding directions or not; it
// cannot where the zero is an argument.
__device__ __forceinline__ float2 product2(float2 a, float2 b, float2 zero) {
    float2 r;
    asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
        "fma.rn.f32x2 z, x, y, z;\n\tmov.b64 {%0, %1}, z;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(zero.x), "f"(zero.y));
    return r;
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// sum over the `lanes` lanes of a head (a power of two)
__device__ __forceinline__ float head_sum(float x, int lanes) {
    for (int o = lanes >> 1; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// 1 / sqrt(mean of the head's squares + eps), rounded to fp32; the head's lanes hold 16
// elements each.  The squares are added to a power of two above their sum (which a first
// pass bounds): every partial sum is then a multiple of that number's last place, so the
// difference of two is exact, what a rounding lost is one more fused operation, and the
// lanes' sums add up without loss.  Where the sum is so far from 1 that this leaves fp32's
// range, once more from elements scaled by k.
__device__ __forceinline__ float head_rms(const float2 (&v)[8], int lanes, float eps) {
    const float inv = 1.0f / (float)(16 * lanes);            // exact: a power of two
    float k = 1.f, h, l;
    while (true) {
        float2 f[8], s = both(0.f);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            f[i] = mul2(v[i], both(k));
            s = sqr_add2(f[i], s);
        }
        const float rough = head_sum(s.x + s.y, lanes);
        const float top = __uint_as_float((__float_as_uint(rough) & 0x7f800000u) + 0x01000000u);   // 2 to 4 times rough
        float2 c = both(0.f);
        s = both(top);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float2 t = sqr_add2(f[i], s);
            c = add2(c, sqr_add2(f[i], sub2(s, t)));
            s = t;
        }
        h = head_sum(__fadd_rn(__fsub_rn(s.x, top), __fsub_rn(s.y, top)), lanes) * inv;
        l = head_sum(__fadd_rn(c.x, c.y), lanes) * inv;
        // h + eps, and what that rounding lost
        const float p = eps * k * k, t = __fadd_rn(h, p), z = __fsub_rn(t, h);
        l = __fadd_rn(l, __fadd_rn(__fsub_rn(h, __fsub_rn(t, z)), __fsub_rn(p, z)));
        h = t;
        const bool far = k == 1.f && !(rough < 1e30f && (rough > 1e-30f || rough == 0.f) && h > 1e-30f);
        if (!__any_sync(0xffffffffu, far)) break;
        k = !far ? k : rough < 1.f ? 0x1p70f : 0x1p-70f;
    }
    const float y = rsqrtf(h);
    // one step of Newton's iteration on 1 - (h + l) y^2, y^2 in two words
    const float q = __fmul_rn(y, y), ql = __fmaf_rn(y, y, -q);
    float e = __fmaf_rn(-h, q, 1.0f);
    e = __fsub_rn(e, __fmaf_rn(h, ql, __fmul_rn(l, q)));
    return (fabsf(e) < 1e-3f ? __fmaf_rn(y, __fmul_rn(e, __fmaf_rn(0.375f, e, 0.5f)), y) : y) * k;
}

// the words of eight elements at p, as pairs of floats
template <int F32>
__device__ __forceinline__ void widen(const uint4 (&u)[F32 + 1], int t, float2* v) {
    float f[8];
    kv4_floats8(u, t, f);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = make_float2(f[2 * i], f[2 * i + 1]);
}

// Sixteen elements of a head at ea and eb, eight each, as a lane holds them.
template <int F32>
struct RopeUnit {
    uint4 a[F32 + 1], b[F32 + 1];
    __device__ __forceinline__ void load(const void* row, size_t at, int ea, int eb, bool live) {
        const uint8_t* p = static_cast<const uint8_t*>(row) + at * (F32 ? 4 : 2);
#pragma unroll
        for (int i = 0; i <= F32; ++i) {
            a[i] = live ? *reinterpret_cast<const uint4*>(p + ea * (F32 ? 4 : 2) + 16 * i) : make_uint4(0, 0, 0, 0);
            b[i] = live ? *reinterpret_cast<const uint4*>(p + eb * (F32 ? 4 : 2) + 16 * i) : make_uint4(0, 0, 0, 0);
        }
    }
};

// v: the pairs at ea, then those at eb
__device__ __forceinline__ void normalise(float2 (&v)[8], float r, const float* w, int ea, int eb) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float4 g = __ldg(reinterpret_cast<const float4*>(w + (i < 2 ? ea : eb)) + (i & 1));
        v[2 * i] = mul2(mul2(v[2 * i], both(r)), make_float2(g.x, g.y));
        v[2 * i + 1] = mul2(mul2(v[2 * i + 1], both(r)), make_float2(g.z, g.w));
    }
}

// cosines and sines of eight pairs: in halves the pairs lie at ea and eb, else beside each other
__device__ __forceinline__ void turn(float2 (&v)[8], const float4 (&c4)[2], const float4 (&s4)[2], bool apart, float2 zero) {
    const float2 c[4] = {{c4[0].x, c4[0].y}, {c4[0].z, c4[0].w}, {c4[1].x, c4[1].y}, {c4[1].z, c4[1].w}};
    const float2 s[4] = {{s4[0].x, s4[0].y}, {s4[0].z, s4[0].w}, {s4[1].x, s4[1].y}, {s4[1].z, s4[1].w}};
    if (apart) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 p = sub2(product2(v[i], c[i], zero), product2(v[4 + i], s[i], zero));
            v[4 + i] = add2(product2(v[4 + i], c[i], zero), product2(v[i], s[i], zero));
            v[i] = p;
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float ci = i & 1 ? c[i / 2].y : c[i / 2].x, si = i & 1 ? s[i / 2].y : s[i / 2].x;
        const float p = __fsub_rn(__fmul_rn(v[i].x, ci), __fmul_rn(v[i].y, si));
        v[i].y = __fadd_rn(__fmul_rn(v[i].y, ci), __fmul_rn(v[i].x, si));
        v[i].x = p;
    }
}

__device__ __forceinline__ void store8(void* p, size_t at, int t, const float2* v) {
    const float f[8] = {v[0].x, v[0].y, v[1].x, v[1].y, v[2].x, v[2].y, v[3].x, v[3].y};
    kv4_store8(p, at, t, f);
}

// A K or V unit into its slot.  In halves a 16-element block is shared with the lane beside.
__device__ __forceinline__ void append_unit(const RopeArgs& a, const float2 (&v)[8], bool isv, bool live, int t, int h, int ea,
                                            int eb, bool apart, int64_t slot, float g, int hd_log2) {
    float mx = 0.f, my = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        mx = fmaxf(mx, fmaxf(fabsf(v[i].x), fabsf(v[i].y)));
        my = fmaxf(my, fmaxf(fabsf(v[4 + i].x), fabsf(v[4 + i].y)));
    }
    const float ox = __shfl_xor_sync(0xffffffffu, mx, 1), oy = __shfl_xor_sync(0xffffffffu, my, 1);
    if (!live) return;
    mx = fmaxf(mx, apart ? ox : my);
    my = apart ? fmaxf(my, oy) : mx;
    uint32_t sx, sy;
    float fx, fy;
    const float x[8] = {v[0].x, v[0].y, v[1].x, v[1].y, v[2].x, v[2].y, v[3].x, v[3].y};
    const float y[8] = {v[4].x, v[4].y, v[5].x, v[5].y, v[6].x, v[6].y, v[7].x, v[7].y};
    const uint32_t cx = kv4_encode8(x, mx, g, sx, fx), cy = kv4_encode8(y, my, g, sy, fy);
    float* hat = isv ? a.v_hat : a.k_hat;
    if (hat) {
        hat += ((size_t)t * a.nkv + h) << hd_log2;
        kv4_store_values8(hat + ea, cx, fx, g);
        kv4_store_values8(hat + eb, cy, fy, g);
    }
    if (slot < 0) return;
    const int64_t pg = slot >> a.page_log2;
    if (pg >= a.n_pages) {
        atomicExch(a.status, ST_DEVICE_CHECK);
        return;
    }
    const size_t at = ((size_t)pg * a.nkv + h) * a.page + (size_t)(slot & (a.page - 1));
    uint8_t* codes = (isv ? a.c.vc : a.c.kc) + (at << (hd_log2 - 1));
    uint8_t* scales = (isv ? a.c.vs : a.c.ks) + (at << (hd_log2 - 4));
    *reinterpret_cast<uint32_t*>(codes + ea / 2) = cx;
    *reinterpret_cast<uint32_t*>(codes + eb / 2) = cy;
    if ((ea & 15) == 0) scales[ea / 16] = (uint8_t)sx;
    if (apart && (eb & 15) == 0) scales[eb / 16] = (uint8_t)sy;
}

// A lane has the same unit of two heads, so that table and norm are read once: q heads
// nq/2 apart, or a K head and its V head.  A unit of the part that turns is eight pairs,
// so in halves its elements lie rot/2 apart; all other units are 16 neighbours.
template <int F32, int NORM, int APPEND>
__device__ __forceinline__ void rope_lane(const RopeArgs& a, int t, int lane, bool live, int hd_log2) {
    const int lph_log2 = hd_log2 - 4, hp = lane >> lph_log2, u = lane - (hp << lph_log2), nq2 = (a.nq + 1) >> 1;
    const bool isq = !APPEND || hp < nq2;
    const int h0 = isq ? hp : hp - nq2, h1 = isq ? hp + nq2 : h0;
    const bool turns = u < (a.rot >> 4), apart = turns && !a.interleaved;
    const int ea = apart ? 8 * u : 16 * u, eb = apart ? (a.rot >> 1) + 8 * u : 16 * u + 8;
    const int pos = live ? __ldg(a.pos + t) : -1;
    const bool two = live && (!isq || h1 < a.nq);
    RopeUnit<F32> r0, r1;
    {
        const size_t q0 = (size_t)t * a.q_stride, k0 = (size_t)t * a.k_stride, v0 = (size_t)t * a.v_stride;
        r0.load(isq ? a.q : a.k, (isq ? q0 : k0) + ((size_t)h0 << hd_log2), ea, eb, live);
        r1.load(isq ? a.q : a.v, (isq ? q0 : v0) + ((size_t)h1 << hd_log2), isq ? ea : 16 * u, isq ? eb : 16 * u + 8, two);
    }
    const bool kv = APPEND && !isq && live;
    const int64_t slot = kv ? __ldg(a.slots + t) : -1;
    const float kg = kv ? __ldg(a.c.kg + h0) : 0.f, vg = kv ? __ldg(a.c.vg + h0) : 0.f;
    const bool seen = pos >= 0 && pos < a.n_pos;
    if (pos >= a.n_pos) atomicExch(a.status, ST_DEVICE_CHECK);
    float4 c[2] = {}, s[2] = {};
    if (seen && turns) {
        const float4* p = reinterpret_cast<const float4*>(a.table + (size_t)pos * a.rot + 8 * u);
        const float4* p2 = reinterpret_cast<const float4*>(a.table + (size_t)pos * a.rot + (a.rot >> 1) + 8 * u);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            c[i] = __ldg(p + i);
            s[i] = __ldg(p2 + i);
        }
    }
    const float* norm = isq ? a.q_norm : a.k_norm;
    float2 v[8];
    widen<F32>(r0.a, a.t, v);
    widen<F32>(r0.b, a.t, v + 4);
    if (NORM) {
        const float r = head_rms(v, 1 << lph_log2, a.eps);
        if (norm) normalise(v, r, norm, ea, eb);
    }
    if (turns) turn(v, c, s, apart, a.minus_zero);
    if (isq && seen) {
        const size_t at = (size_t)t * a.q_out_stride + ((size_t)h0 << hd_log2);
        store8(a.q_out, at + ea, a.t, v);
        store8(a.q_out, at + eb, a.t, v + 4);
    }
    if (APPEND && __any_sync(0xffffffffu, !isq))
        append_unit(a, v, false, !isq && seen, t, h0, ea, eb, apart, slot, kg, hd_log2);
    widen<F32>(r1.a, a.t, v);
    widen<F32>(r1.b, a.t, v + 4);
    if (!APPEND || __any_sync(0xffffffffu, isq)) {
        if (NORM) {
            const float r = head_rms(v, 1 << lph_log2, a.eps);
            if (norm && isq) normalise(v, r, norm, ea, eb);
        }
        if (isq && turns) turn(v, c, s, apart, a.minus_zero);
        if (isq && seen && two) {
            const size_t at = (size_t)t * a.q_out_stride + ((size_t)h1 << hd_log2);
            store8(a.q_out, at + ea, a.t, v);
            store8(a.q_out, at + eb, a.t, v + 4);
        }
    }
    if (APPEND && __any_sync(0xffffffffu, !isq))
        append_unit(a, v, true, !isq && seen, t, h0, 16 * u, 16 * u + 8, false, slot, vg, hd_log2);
}

// A CTA takes rows_cta whole rows where they fit its threads, else one row in turns.
template <int F32, int NORM, int APPEND>
__global__ void __launch_bounds__(512) rope_kernel(RopeArgs a, int lanes_row, int rows_cta, int hd_log2) {
    pdl_wait();
    pdl_launch_dependents();
    const int r = rows_cta > 1 ? (int)threadIdx.x / lanes_row : 0;
    const int t = (int)blockIdx.x * rows_cta + r;
    for (int lane = (int)threadIdx.x - r * lanes_row; lane - (int)(threadIdx.x & 31) < lanes_row; lane += (int)blockDim.x)
        rope_lane<F32, NORM, APPEND>(a, t, lane, r < rows_cta && t < a.n_tokens && lane < lanes_row, hd_log2);
}

// angles in 64 bits: a product and the range reduction lose 2^-53 of positions' worth
__global__ void rope_table_kernel(const __grid_constant__ RopeFreq f, int half, int n_pos, double mscale, float* table) {
    pdl_wait();
    pdl_launch_dependents();
    const int64_t n = (int64_t)half * n_pos;
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += (int64_t)gridDim.x * blockDim.x) {
        const int p = (int)(i / half), j = (int)(i - (int64_t)p * half);
        double s, c;
        sincos((double)p * f.f[j], &s, &c);
        float* row = table + (size_t)p * 2 * half + j;
        row[0] = (float)(c * mscale);
        row[half] = (float)(s * mscale);
    }
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a, cudaStream_t st) {
    const int hd_log2 = a.hd == 64 ? 6 : a.hd == 128 ? 7 : 8;
    const int lanes_row = ((a.nq + 1) / 2 + a.nkv) << (hd_log2 - 4);
    // whole rows where two or more fit, else a row by as many threads as it has lanes
    const int rows_cta = lanes_row <= RO_THREADS / 2 ? RO_THREADS / lanes_row : 1;
    const int threads = rows_cta > 1 ? RO_THREADS : lanes_row < 512 ? (lanes_row + 31) / 32 * 32 : RO_THREADS;
    const dim3 grid((unsigned)((a.n_tokens + rows_cta - 1) / rows_cta));
    const int which = (a.t == KV4_F32 ? 4 : 0) + (a.q_norm || a.k_norm ? 2 : 0) + (a.nkv ? 1 : 0);
    void (*const kernels[8])(RopeArgs, int, int, int) = {rope_kernel<0, 0, 0>, rope_kernel<0, 0, 1>, rope_kernel<0, 1, 0>,
                                                         rope_kernel<0, 1, 1>, rope_kernel<1, 0, 0>, rope_kernel<1, 0, 1>,
                                                         rope_kernel<1, 1, 0>, rope_kernel<1, 1, 1>};
    RopeArgs b = a;
    b.minus_zero = make_float2(-0.f, -0.f);
    return launch_pdl(kernels[which], grid, dim3(threads), 0, st, b, lanes_row, rows_cta, hd_log2);
}

cudaError_t launch_rope_rows_table(const RopeFreq& f, int half, int n_pos, double mscale, float* table, cudaStream_t st) {
    const int64_t blocks = ((int64_t)half * n_pos + 255) / 256;
    return launch_pdl(rope_table_kernel, dim3((unsigned)(blocks < 65536 ? blocks : 65536)), dim3(256), 0, st, f, half,
                      n_pos, mscale, table);
}

}  // namespace qmoe
