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

// s + p, and what its rounding lost added to c
__device__ __forceinline__ void add_kept(float& s, float& c, float p) {
    const float t = __fadd_rn(s, p), z = __fsub_rn(t, s);
    c = __fadd_rn(c, __fadd_rn(__fsub_rn(s, __fsub_rn(t, z)), __fsub_rn(p, z)));
    s = t;
}

// 1 / sqrt(mean of the head's squares + eps), rounded to fp32; the head's `lanes` lanes (a
// power of two) hold 16 elements each.  Where the mean is so far from 1 that squares or
// the root's correction leave fp32's range, once more from elements scaled by k.
__device__ __forceinline__ float head_rms(const float (&a)[8], const float (&b)[8], int lanes, float eps) {
    const float inv = 1.0f / (float)(16 * lanes);            // exact: a power of two
    float k = 1.f, h, l;
    while (true) {
        float s = 0.f, c = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float f = __fmul_rn(i < 8 ? a[i & 7] : b[i & 7], k), p = __fmul_rn(f, f);
            c = __fadd_rn(c, __fmaf_rn(f, f, -p));
            add_kept(s, c, p);
        }
        for (int o = lanes >> 1; o; o >>= 1) {
            const float s2 = __shfl_xor_sync(0xffffffffu, s, o), c2 = __shfl_xor_sync(0xffffffffu, c, o);
            c = __fadd_rn(c, c2);
            add_kept(s, c, s2);                               // the loss is exact, so both lanes get the same
        }
        h = s * inv;
        l = c * inv;
        add_kept(h, l, eps * k * k);
        const bool far = k == 1.f && !(h > 1e-30f && h < 1e30f);
        if (!__any_sync(0xffffffffu, far)) break;
        k = !far ? k : h <= 1e-30f ? 0x1p70f : 0x1p-70f;
    }
    const float y = rsqrtf(h);
    // one step of Newton's iteration on 1 - (h + l) y^2, y^2 in two words
    const float q = __fmul_rn(y, y), ql = __fmaf_rn(y, y, -q);
    float e = __fmaf_rn(-h, q, 1.0f);
    e = __fsub_rn(e, __fmaf_rn(h, ql, __fmul_rn(l, q)));
    return (fabsf(e) < 1e-3f ? __fmaf_rn(y, __fmul_rn(e, __fmaf_rn(0.375f, e, 0.5f)), y) : y) * k;
}

// A lane has 16 elements of a head: eight from ea and eight from eb.  A unit of the part
// that turns is eight pairs, so in the half layout its elements lie rot/2 apart; all
// other units are 16 neighbours.
template <int APPEND>
__device__ __forceinline__ void rope_lane(const RopeArgs& a, int t, int lane, bool live, int hd_log2) {
    const int lph_log2 = hd_log2 - 4, head = lane >> lph_log2, u = lane - (head << lph_log2);
    const bool isq = !APPEND || head < a.nq, isk = APPEND && !isq && head < a.nq + a.nkv;
    const int h = isq ? head : isk ? head - a.nq : head - a.nq - a.nkv;      // head in its rows
    const int pos = live ? a.pos[t] : -1;
    if (live && pos >= a.n_pos) atomicExch(a.status, ST_DEVICE_CHECK);
    live = live && pos >= 0 && pos < a.n_pos;
    const bool turns = (isq || isk) && u < (a.rot >> 4);
    const bool apart = turns && !a.interleaved;
    const int ea = apart ? 8 * u : 16 * u, eb = apart ? (a.rot >> 1) + 8 * u : 16 * u + 8;
    float x[8] = {}, y[8] = {};
    if (live) {
        const void* row = isq ? a.q : isk ? a.k : a.v;
        const size_t at = (size_t)t * (isq ? a.q_stride : isk ? a.k_stride : a.v_stride) + ((size_t)h << hd_log2);
        rows_load8(row, at + ea, a.t, x);
        rows_load8(row, at + eb, a.t, y);
    }
    float4 cs[4];
    if (live && turns) {
        const float4* p = reinterpret_cast<const float4*>(a.table + (size_t)pos * a.rot + 16 * u);
#pragma unroll
        for (int i = 0; i < 4; ++i) cs[i] = __ldg(p + i);
    }
    const float* norm = isq ? a.q_norm : isk ? a.k_norm : nullptr;
    if (a.q_norm || a.k_norm) {                               // the same for the whole grid
        const float r = head_rms(x, y, 1 << lph_log2, a.eps);
        if (norm && live) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float4 wa = __ldg(reinterpret_cast<const float4*>(norm + ea) + i);
                const float4 wb = __ldg(reinterpret_cast<const float4*>(norm + eb) + i);
                const float va[4] = {wa.x, wa.y, wa.z, wa.w}, vb[4] = {wb.x, wb.y, wb.z, wb.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    x[4 * i + j] = __fmul_rn(__fmul_rn(x[4 * i + j], r), va[j]);
                    y[4 * i + j] = __fmul_rn(__fmul_rn(y[4 * i + j], r), vb[j]);
                }
            }
        }
    }
    if (live && turns) {
        const float c[8] = {cs[0].x, cs[0].z, cs[1].x, cs[1].z, cs[2].x, cs[2].z, cs[3].x, cs[3].z};
        const float s[8] = {cs[0].y, cs[0].w, cs[1].y, cs[1].w, cs[2].y, cs[2].w, cs[3].y, cs[3].w};
        auto turn = [](float& p, float& q, float c, float s) {
            const float p2 = __fsub_rn(__fmul_rn(p, c), __fmul_rn(q, s));
            q = __fadd_rn(__fmul_rn(q, c), __fmul_rn(p, s));
            p = p2;
        };
        if (apart) {
#pragma unroll
            for (int i = 0; i < 8; ++i) turn(x[i], y[i], c[i], s[i]);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                turn(x[2 * i], x[2 * i + 1], c[i], s[i]);
                turn(y[2 * i], y[2 * i + 1], c[4 + i], s[4 + i]);
            }
        }
    }
    if (isq) {
        if (live) {
            const size_t at = (size_t)t * a.q_out_stride + ((size_t)h << hd_log2);
            kv4_store8(a.q_out, at + ea, a.t, x);
            kv4_store8(a.q_out, at + eb, a.t, y);
        }
    }
    if constexpr (APPEND) {
        // the largest of each 16-element block: a lane's own, or of the eight elements beside
        float mx = 0.f, my = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            mx = fmaxf(mx, fabsf(x[i]));
            my = fmaxf(my, fabsf(y[i]));
        }
        const float ox = __shfl_xor_sync(0xffffffffu, mx, 1), oy = __shfl_xor_sync(0xffffffffu, my, 1);
        if (isq || !live) return;
        if (apart) {
            mx = fmaxf(mx, ox);
            my = fmaxf(my, oy);
        } else {
            mx = my = fmaxf(mx, my);
        }
        const float g = (isk ? a.c.kg : a.c.vg)[h];
        uint32_t sx, sy;
        float fx, fy;
        const uint32_t cx = kv4_encode8(x, mx, g, sx, fx), cy = kv4_encode8(y, my, g, sy, fy);
        float* hat = isk ? a.k_hat : a.v_hat;
        if (hat) {
            hat += ((size_t)t * a.nkv + h) << hd_log2;
            kv4_store_values8(hat + ea, cx, fx, g);
            kv4_store_values8(hat + eb, cy, fy, g);
        }
        const int64_t slot = a.slots[t];
        if (slot < 0) return;
        const int64_t pg = slot >> a.page_log2;
        if (pg >= a.n_pages) {
            atomicExch(a.status, ST_DEVICE_CHECK);
            return;
        }
        const size_t at = ((size_t)pg * a.nkv + h) * a.page + (size_t)(slot & (a.page - 1));
        uint8_t* codes = (isk ? a.c.kc : a.c.vc) + (at << (hd_log2 - 1));
        uint8_t* scales = (isk ? a.c.ks : a.c.vs) + (at << (hd_log2 - 4));
        *reinterpret_cast<uint32_t*>(codes + ea / 2) = cx;
        *reinterpret_cast<uint32_t*>(codes + eb / 2) = cy;
        if ((ea & 15) == 0) scales[ea / 16] = (uint8_t)sx;
        if (apart && (eb & 15) == 0) scales[eb / 16] = (uint8_t)sy;
    }
}

// A CTA takes rows_cta whole rows where they fit its threads, else one row in turns.
template <int APPEND>
__global__ void __launch_bounds__(RO_THREADS) rope_kernel(const RopeArgs a, int lanes_row, int rows_cta, int hd_log2) {
    pdl_wait();
    pdl_launch_dependents();
    const int r = rows_cta > 1 ? (int)threadIdx.x / lanes_row : 0;
    const int t = (int)blockIdx.x * rows_cta + r;
    for (int lane = (int)threadIdx.x - r * lanes_row; lane - (int)(threadIdx.x & 31) < lanes_row; lane += RO_THREADS)
        rope_lane<APPEND>(a, t, lane, r < rows_cta && t < a.n_tokens && lane < lanes_row, hd_log2);
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
        reinterpret_cast<float2*>(table)[i] = make_float2((float)(c * mscale), (float)(s * mscale));
    }
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a, cudaStream_t st) {
    const int hd_log2 = a.hd == 64 ? 6 : a.hd == 128 ? 7 : 8;
    const int lanes_row = (a.nq + 2 * a.nkv) << (hd_log2 - 4);
    const int rows_cta = lanes_row < RO_THREADS ? RO_THREADS / lanes_row : 1;
    const dim3 grid((unsigned)((a.n_tokens + rows_cta - 1) / rows_cta));
    return a.nkv ? launch_pdl(rope_kernel<1>, grid, dim3(RO_THREADS), 0, st, a, lanes_row, rows_cta, hd_log2)
                 : launch_pdl(rope_kernel<0>, grid, dim3(RO_THREADS), 0, st, a, lanes_row, rows_cta, hd_log2);
}

cudaError_t launch_rope_rows_table(const RopeFreq& f, int half, int n_pos, double mscale, float* table, cudaStream_t st) {
    const int64_t blocks = ((int64_t)half * n_pos + 255) / 256;
    return launch_pdl(rope_table_kernel, dim3((unsigned)(blocks < 65536 ? blocks : 65536)), dim3(256), 0, st, f, half,
                      n_pos, mscale, table);
}

}  // namespace qmoe
