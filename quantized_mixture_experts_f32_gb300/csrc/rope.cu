// rope.cu -- rotary positions on rows of heads, alone (qmoe_rope) and on the way into the
// paged 4-bit cache (qmoe_kv4_append_rope), and the table of their cosines and sines.
//
// Pair j of a head at position p turns by p f_j: (a, b) -> (a c - b s, b c + a s).  K's rows
// decide 4-bit codes, so every step rounds to fp32 once, as the definition says, and a
// head's mean square is carried in two fp32 words: its inverse root is then the same
// fp32 number as from 64 bits, but where that lies so near to the border between two
// that some 2^-45 decide (one head in a million; 64 bits for these alone took 64 tokens'
// append from 3.05 to 3.45 us).
//
// qmoe_rope is bound by HBM: 8191 rows of 40 heads of 128, F16, 28.5 us, 5.9 TB/s.  The
// append (16384 rows, 32 q and 4 kv heads of 128, BF16, both norms: 75 us, 5.1 TB/s) is bound
// by issue, 57%, with half of the warps that fit (64 registers): the exact mean square is
// two passes over the head, and codes take a corrected quotient.  CTAs of 128 and 256
// threads took 80 and 85 us; rows loaded ahead of the ones in work 81 to 97.
#include "kv4_row.cuh"
#include "ptx_sync.cuh"
#include "rows.cuh"

namespace qmoe {

namespace {

constexpr int RO_THREADS = 64;

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

// sum over the LANES lanes of a head
template <int LANES>
__device__ __forceinline__ float head_sum(float x) {
#pragma unroll
    for (int o = LANES / 2; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// The mean of a head's squares, times k^2, plus p, in two words.  The squares are added to a
// power of two above their sum (which a first pass bounds): every partial sum is then a
// multiple of that number's last place, so the difference of two is exact, what a
// rounding lost is one more fused operation, and the lanes' sums add up without loss.
template <int LANES>
__device__ __forceinline__ float2 mean_square(const float2 (&f)[8], float p, float& rough) {
    constexpr float inv = 1.0f / (float)(16 * LANES);        // exact: a power of two
    float2 s = mul2(f[0], f[0]);
#pragma unroll
    for (int i = 1; i < 8; ++i) s = sqr_add2(f[i], s);
    rough = head_sum<LANES>(s.x + s.y);
    const float top = __uint_as_float((__float_as_uint(rough) & 0x7f800000u) + 0x01000000u);   // 2 to 4 times rough
    float2 c = both(0.f);
    s = both(top);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float2 t = sqr_add2(f[i], s), lost = sqr_add2(f[i], sub2(s, t));
        c = i ? add2(c, lost) : lost;
        s = t;
    }
    const float h = head_sum<LANES>(__fadd_rn(__fsub_rn(s.x, top), __fsub_rn(s.y, top))) * inv;
    const float l = head_sum<LANES>(__fadd_rn(c.x, c.y)) * inv;
    // h + p, and what that rounding lost
    const float t = __fadd_rn(h, p), z = __fsub_rn(t, h);
    return make_float2(t, __fadd_rn(l, __fadd_rn(__fsub_rn(h, __fsub_rn(t, z)), __fsub_rn(p, z))));
}

// 1 / sqrt(mean of the head's squares + eps), rounded to fp32; the head's lanes hold 16
// elements each.  Once more from elements scaled by k where the squares or the root's leave fp32's range,
// or mean and eps are so small that what they lose below it counts.
template <int LANES>
__device__ __forceinline__ float head_rms(const float2 (&v)[8], float eps) {
    float rough, k = 1.f;
    float2 m = mean_square<LANES>(v, eps, rough);
    const bool far = !(rough < 1e30f && m.x > 1e-20f && m.x < 1e30f);
    if (__any_sync(0xffffffffu, far)) {
        k = !far ? 1.f : m.x < 1.f ? 0x1p70f : 0x1p-70f;
        float2 f[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = make_float2(v[i].x * k, v[i].y * k);
        m = mean_square<LANES>(f, eps * k * k, rough);
    }
    const float y = rsqrtf(m.x);
    // one step of Newton's iteration on 1 - (h + l) y^2, y^2 in two words
    const float q = __fmul_rn(y, y), ql = __fmaf_rn(y, y, -q);
    float e = __fmaf_rn(-m.x, q, 1.0f);
    e = __fsub_rn(e, __fmaf_rn(m.x, ql, __fmul_rn(m.y, q)));
    return (fabsf(e) < 1e-3f ? __fmaf_rn(y, __fmul_rn(e, __fmaf_rn(0.375f, e, 0.5f)), y) : y) * k;
}

// Sixteen elements of a head at ea and eb, eight each, as a lane holds them.
template <int T>
struct RopeUnit {
    static constexpr int N = T == KV4_F32 ? 2 : 1, BYTES = T == KV4_F32 ? 4 : 2;
    uint4 a[N], b[N];
    __device__ __forceinline__ void load(const void* row, size_t at, int ea, int eb) {
        const uint8_t* p = static_cast<const uint8_t*>(row) + at * BYTES;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            a[i] = *reinterpret_cast<const uint4*>(p + ea * BYTES + 16 * i);
            b[i] = *reinterpret_cast<const uint4*>(p + eb * BYTES + 16 * i);
        }
    }
    __device__ __forceinline__ void widen(float2 (&v)[8]) const {
        float f[8];
        kv4_floats8(a, T, f);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = make_float2(f[2 * i], f[2 * i + 1]);
        kv4_floats8(b, T, f);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[4 + i] = make_float2(f[2 * i], f[2 * i + 1]);
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
__device__ __forceinline__ void turn(float2 (&v)[8], const float* cos8, const float* sin8, bool apart, float2 zero) {
    float2 c[4], s[4];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float4 c4 = __ldg(reinterpret_cast<const float4*>(cos8) + i), s4 = __ldg(reinterpret_cast<const float4*>(sin8) + i);
        c[2 * i] = make_float2(c4.x, c4.y);
        c[2 * i + 1] = make_float2(c4.z, c4.w);
        s[2 * i] = make_float2(s4.x, s4.y);
        s[2 * i + 1] = make_float2(s4.z, s4.w);
    }
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

template <int T>
__device__ __forceinline__ void store_unit(void* p, size_t at, int ea, int eb, const float2 (&v)[8]) {
    const float x[8] = {v[0].x, v[0].y, v[1].x, v[1].y, v[2].x, v[2].y, v[3].x, v[3].y};
    const float y[8] = {v[4].x, v[4].y, v[5].x, v[5].y, v[6].x, v[6].y, v[7].x, v[7].y};
    kv4_store8(p, at + ea, T, x);
    kv4_store8(p, at + eb, T, y);
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

// Where a lane's unit lies in a head.  A unit of the part that turns is eight pairs, so in
// halves its elements lie rot/2 apart; all other units are 16 neighbours.
struct RopePlace {
    bool turns, apart;
    int ea, eb;
    __device__ __forceinline__ RopePlace(const RopeArgs& a, int u) {
        turns = u < (a.rot >> 4);
        apart = turns && !a.interleaved;
        ea = apart ? 8 * u : 16 * u;
        eb = apart ? (a.rot >> 1) + 8 * u : 16 * u + 8;
    }
};

// a unit's norm and turn at its row's table entries
template <int LANES, int NORM>
__device__ __forceinline__ void rope_unit(const RopeArgs& a, float2 (&v)[8], const RopePlace& w, const float* norm, const float* cs) {
    if (NORM) {
        const float r = head_rms<LANES>(v, a.eps);
        if (norm) normalise(v, r, norm, w.ea, w.eb);
    }
    if (w.turns) turn(v, cs, cs + (a.rot >> 1), w.apart, a.minus_zero);
}

// The same unit of two q heads, nq/2 apart, so that a lane has two rows' loads in flight.
// Lanes without work load the first row's and write nothing.
template <int T, int HD, int NORM>
__device__ __forceinline__ void rope_q(const RopeArgs& a, int t, int lane, bool live) {
    constexpr int LANES = HD / 16;
    t = live ? t : 0;
    lane = live ? lane : 0;
    const int h0 = lane / LANES, u = lane % LANES, nq2 = (a.nq + 1) >> 1;
    const bool two = h0 + nq2 < a.nq;
    const int h1 = two ? h0 + nq2 : h0;
    const RopePlace w(a, u);
    const int pos = __ldg(a.pos + t);
    RopeUnit<T> r0, r1;
    r0.load(a.q, (size_t)t * a.q_stride + h0 * HD, w.ea, w.eb);
    r1.load(a.q, (size_t)t * a.q_stride + h1 * HD, w.ea, w.eb);
    const bool seen = live && pos >= 0 && pos < a.n_pos;
    if (live && pos >= a.n_pos) atomicExch(a.status, ST_DEVICE_CHECK);
    const float* cs = a.table + (size_t)(seen ? pos : 0) * a.rot + (w.turns ? 8 * u : 0);
    float2 v[8];
    r0.widen(v);
    rope_unit<LANES, NORM>(a, v, w, a.q_norm, cs);
    if (seen) store_unit<T>(a.q_out, (size_t)t * a.q_out_stride + h0 * HD, w.ea, w.eb, v);
    r1.widen(v);
    rope_unit<LANES, NORM>(a, v, w, a.q_norm, cs);
    if (seen && two) store_unit<T>(a.q_out, (size_t)t * a.q_out_stride + h1 * HD, w.ea, w.eb, v);
}

// A unit of a K head and of its V head.
template <int T, int HD, int NORM>
__device__ __forceinline__ void rope_kv(const RopeArgs& a, int t, int lane, bool live) {
    constexpr int LANES = HD / 16, hd_log2 = HD == 64 ? 6 : HD == 128 ? 7 : 8;
    t = live ? t : 0;
    lane = live ? lane : 0;
    const int h = lane / LANES, u = lane % LANES;
    const RopePlace w(a, u);
    const int pos = __ldg(a.pos + t);
    RopeUnit<T> rk, rv;
    rk.load(a.k, (size_t)t * a.k_stride + h * HD, w.ea, w.eb);
    rv.load(a.v, (size_t)t * a.v_stride + h * HD, 16 * u, 16 * u + 8);
    const int64_t slot = __ldg(a.slots + t);
    const float kg = __ldg(a.c.kg + h), vg = __ldg(a.c.vg + h);
    const bool seen = live && pos >= 0 && pos < a.n_pos;
    if (live && pos >= a.n_pos) atomicExch(a.status, ST_DEVICE_CHECK);
    const float* cs = a.table + (size_t)(seen ? pos : 0) * a.rot + (w.turns ? 8 * u : 0);
    float2 v[8];
    rk.widen(v);
    rope_unit<LANES, NORM>(a, v, w, a.k_norm, cs);
    append_unit(a, v, false, seen, t, h, w.ea, w.eb, w.apart, slot, kg, hd_log2);
    rv.widen(v);
    append_unit(a, v, true, seen, t, h, 16 * u, 16 * u + 8, false, slot, vg, hd_log2);
}

// How a kind's rows are dealt to CTAs: rows_cta whole rows where they fit a CTA's threads,
// else `parts` CTAs a row.
struct RopeDeal {
    int lanes_row, rows_cta, parts, ctas;
};

// The CTAs of K and V rows first, which take longer; q's and theirs are apart, and small, so
// that little waits for a CTA's slowest warp.
template <int T, int HD, int NORM, int APPEND>
__global__ void __launch_bounds__(RO_THREADS, 16) rope_kernel(const RopeArgs a, const RopeDeal dq, const RopeDeal dkv) {
    pdl_wait();
    pdl_launch_dependents();
    const bool kv = APPEND && (int)blockIdx.x < dkv.ctas;
    const RopeDeal d = kv ? dkv : dq;
    const int cta = kv ? (int)blockIdx.x : (int)blockIdx.x - (APPEND ? dkv.ctas : 0);
    int t, lane = (int)threadIdx.x;
    bool live = true;
    if (d.parts > 1) {
        t = cta / d.parts;
        lane += (cta - t * d.parts) * RO_THREADS;
    } else {
        const int r = lane / d.lanes_row;
        t = cta * d.rows_cta + r;
        lane -= r * d.lanes_row;
        live = r < d.rows_cta;
    }
    live = live && t < a.n_tokens && lane < d.lanes_row;
    if (kv) rope_kv<T, HD, NORM>(a, t, lane, live);
    else rope_q<T, HD, NORM>(a, t, lane, live);
}

RopeDeal deal(int lanes_row, int n_tokens) {
    if (!lanes_row) return {0, 1, 1, 0};
    if (lanes_row > RO_THREADS) {
        const int parts = (lanes_row + RO_THREADS - 1) / RO_THREADS;
        return {lanes_row, 1, parts, n_tokens * parts};
    }
    const int rows_cta = RO_THREADS / lanes_row;
    return {lanes_row, rows_cta, 1, (n_tokens + rows_cta - 1) / rows_cta};
}

using RopeKernel = void (*)(RopeArgs, RopeDeal, RopeDeal);

template <int T, int HD>
RopeKernel rope_kernel_of(bool norm, bool append) {
    return norm ? append ? rope_kernel<T, HD, 1, 1> : rope_kernel<T, HD, 1, 0>
                : append ? rope_kernel<T, HD, 0, 1> : rope_kernel<T, HD, 0, 0>;
}
template <int T>
RopeKernel rope_kernel_of(int hd, bool norm, bool append) {
    return hd == 64    ? rope_kernel_of<T, 64>(norm, append)
           : hd == 128 ? rope_kernel_of<T, 128>(norm, append)
                       : rope_kernel_of<T, 256>(norm, append);
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
    const RopeDeal dq = deal((a.nq + 1) / 2 * (a.hd / 16), a.n_tokens), dkv = deal(a.nkv * (a.hd / 16), a.n_tokens);
    const bool norm = a.q_norm || a.k_norm, append = a.nkv > 0;
    const RopeKernel kernel = a.t == KV4_F32   ? rope_kernel_of<KV4_F32>(a.hd, norm, append)
                              : a.t == KV4_F16 ? rope_kernel_of<KV4_F16>(a.hd, norm, append)
                                               : rope_kernel_of<KV4_BF16>(a.hd, norm, append);
    RopeArgs b = a;
    b.minus_zero = make_float2(-0.f, -0.f);
    return launch_pdl(kernel, dim3((unsigned)(dq.ctas + dkv.ctas)), dim3(RO_THREADS), 0, st, b, dq, dkv);
}

cudaError_t launch_rope_rows_table(const RopeFreq& f, int half, int n_pos, double mscale, float* table, cudaStream_t st) {
    const int64_t blocks = ((int64_t)half * n_pos + 255) / 256;
    return launch_pdl(rope_table_kernel, dim3((unsigned)(blocks < 65536 ? blocks : 65536)), dim3(256), 0, st, f, half,
                      n_pos, mscale, table);
}

}  // namespace qmoe
