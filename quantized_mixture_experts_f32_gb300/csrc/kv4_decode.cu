// kv4_decode.cu -- attention over the paged 4-bit cache for sequences that bring a
// few tokens: decoding, draft tokens.  Bound by the cache's bytes (144 a position and
// kv head at head_dim 128), then by the instructions that widen them.
//
// Row = (token, q head of the kv head's group), eight rows to an item.  With
// z_p = q.k_p * scale * log2(e) the pass keeps a running maximum m, l = sum 2^(z-m)
// and o = sum 2^(z-m) v_p; parts of an item's positions are joined by
// m = max m_i, l = sum l_i 2^(m_i-m), o likewise.
//
// Both products are mma.sync m16n8k16 (fp16 in, fp32 out).  K and V are exact in
// fp16 (2 x 4 significant bits), and the eight rows leave half of the 16-row operand
// free: it takes the low parts, q = hi + lo and p = hi + lo (22 bits), so F32 rows
// keep their precision for the price of 16-bit ones.  tcgen05 would want the widened
// K and V in shared memory, 4x the bytes the cache has, for 128 rows of which eight
// exist; here a thread widens what it has loaded straight into operand registers.
// Each row of q is first scaled by the power of two of its largest element, so any
// fp32 or bf16 range fits fp16.
//
// The order of head elements in q.k and of positions in p.v is free: K and Q elements
// are dealt to the four lanes of a column in contiguous runs (16-byte loads), and
// columns to positions so that V's loads meet every bank once.
#include <math.h>

#include "kv4.cuh"
#include "kv4_row.cuh"
#include "ptx_sync.cuh"

namespace qmoe {

namespace {

constexpr int DW = 8;                    // warps of a CTA
constexpr int DT = 32 * DW;
constexpr int TP = 32;                   // positions a warp takes at a time
constexpr int UNIT = TP * DW;            // positions a CTA takes at a time
constexpr int STAGES = 2;                // stages per warp: one in use, one being copied

template <int HD>
struct DGeo {
    static constexpr int ROWB = HD / 2, SB = HD / 16;          // bytes of codes and scales of a position
    static constexpr int KC = 0, VC = TP * ROWB, KS = 2 * TP * ROWB, VS = KS + TP * SB;
    static constexpr int STAGE = VS + TP * SB;
    static constexpr int RING = DW * STAGES * STAGE;
    static constexpr int OLD = HD + 16;                        // row of the join buffer: 4 floats of padding a quarter
    static constexpr int QF = HD * 32;                         // q fragments
    static constexpr int PART = 8 * HD + 16;                   // floats of an item's part: o, m, l
    static constexpr size_t smem(int n_seqs) { return (size_t)RING + QF + 8 * ((size_t)n_seqs + 1); }
    static_assert(DW * 8 * OLD * 4 <= RING, "the join buffer reuses the ring");
};

__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// column c of eight <-> position of eight: 0 4 1 5 2 6 3 7
__device__ __forceinline__ int pos_of_col(int c) { return (c >> 1) + 4 * (c & 1); }
__device__ __forceinline__ int col_of_pos(int p) { return 2 * (p & 3) + (p >> 2); }

// One stage: 32 positions of one kv head, 16 at a time; row: index of the first of the
// 16 positions in the cache (negative: not copied).  K rows lie in column order.
template <int HD>
__device__ __forceinline__ void copy_stage(uint8_t* st, const Kv4Cache& c, const int64_t (&row)[2], int lane) {
    using G = DGeo<HD>;
    constexpr int CH = HD / 32;                        // 16-byte chunks of a position's codes
    constexpr int PP = 32 / CH;                        // positions a warp's 32 chunks cover
#pragma unroll
    for (int sub = 0; sub < 2; ++sub) {
        if (row[sub] < 0) continue;
        const uint8_t* kc = c.kc + (size_t)row[sub] * G::ROWB + lane * 16;
        const uint8_t* vc = c.vc + (size_t)row[sub] * G::ROWB + lane * 16;
#pragma unroll
        for (int it = 0; it < 16 / PP; ++it) {
            const int p = it * PP + lane / CH, ch = lane % CH;
            const int kr = sub * 16 + (p & 8) + col_of_pos(p & 7), vr = sub * 16 + p;
            const int kch = HD == 256 ? ch ^ (4 * (kr & 1)) : ch;
            const int vch = HD == 256 ? ch ^ (2 * (p & 3)) : HD == 128 ? ch ^ (p & 2) : ch;
            cp_async_cg16(st + G::KC + kr * G::ROWB + kch * 16, kc + it * 512);
            cp_async_cg16(st + G::VC + vr * G::ROWB + vch * 16, vc + it * 512);
        }
        // 16 positions' scales are SB chunks: K's by the lanes from 0, V's by those behind
        if (lane < 2 * G::SB) {
            const int v = lane / G::SB, ch = lane % G::SB;
            cp_async_cg16(st + (v ? G::VS : G::KS) + (sub * G::SB + ch) * 16,
                          (v ? c.vs : c.ks) + (size_t)row[sub] * G::SB + (size_t)ch * 16);
        }
    }
}

// CTA c of g takes the units [w c / g, w (c+1) / g) of w; g <= w, so each has one at least
__device__ __forceinline__ long long unit_begin(long long w, int c, int g) { return w * c / g; }
__device__ __forceinline__ int cta_of_unit(long long w, long long x, int g) { return (int)(((x + 1) * g - 1) / w); }

template <int HD>
__global__ void __launch_bounds__(DT, HD == 256 ? 1 : 2)
    kv4_decode_kernel(const Kv4AttnArgs a, int few_rows, float* __restrict__ parts, unsigned* __restrict__ arrive) {
    using G = DGeo<HD>;
    extern __shared__ __align__(16) uint8_t sm[];
    uint8_t* ring = sm;
    uint32_t* qf = reinterpret_cast<uint32_t*>(sm + G::RING);                       // [HD/16][32 lanes][4]
    long long* pre = reinterpret_cast<long long*>(sm + G::RING + G::QF);            // [n_seqs+1]
    __shared__ long long wsum[DW];
    __shared__ float fac_s[8], m_s[DW][8], l_s[DW][8];
    __shared__ int last_s;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int r = lane >> 2, j = lane & 3;             // row (and K column), quarter of a row
    const int group = a.s.nq / a.s.nkv;
    pdl_wait();
    pdl_launch_dependents();

    // units of every sequence, as prefix sums
    {
        const int per = (a.n_seqs + DT - 1) / DT, s0 = min(tid * per, a.n_seqs), s1 = min(s0 + per, a.n_seqs);
        long long run = 0;
        for (int s = s0; s < s1; ++s) {
            Kv4Seq q;
            if (!kv4_seq(a, s, q) && blockIdx.x == 0) atomicExch(a.status, ST_DEVICE_CHECK);
            pre[s] = run;
            if (q.n * group <= few_rows) run += (long long)a.s.nkv * ((q.n * group + 7) / 8) * (q.len ? (q.len + UNIT - 1) / UNIT : 1);
        }
        long long inc = run;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const long long o = __shfl_up_sync(0xffffffffu, inc, d);
            if (lane >= d) inc += o;
        }
        if (lane == 31) wsum[warp] = inc;
        __syncthreads();
        long long base = inc - run;
        for (int w = 0; w < warp; ++w) base += wsum[w];
        for (int s = s0; s < s1; ++s) pre[s] += base;
        if (tid == DT - 1) pre[a.n_seqs] = base + run;
    }
    __syncthreads();
    const long long W = pre[a.n_seqs];
    const int Gn = (int)min((long long)gridDim.x, W), me = blockIdx.x;
    if (me >= Gn) return;
    const long long u_end = unit_begin(W, me + 1, Gn);

    for (long long u = unit_begin(W, me, Gn); u < u_end;) {
        // the item that unit u belongs to: sequence, kv head, eight rows
        int s = 0;
        for (int hi = a.n_seqs; hi - s > 1;) {
            const int mid = (s + hi) >> 1;
            if (pre[mid] <= u) s = mid;
            else hi = mid;
        }
        Kv4Seq q;
        kv4_seq(a, s, q);
        const int tiles = q.len ? (q.len + UNIT - 1) / UNIT : 1;
        const int rts = (q.n * group + 7) / 8;
        const long long off = u - pre[s];
        const int item = (int)(off / tiles), t0 = (int)(off - (long long)item * tiles);
        const int g = item / rts, row0 = (item - g * rts) * 8;
        const int t1 = (int)min((long long)tiles, t0 + (u_end - u));
        const int rows = min(8, q.n * group - row0);
        const int32_t* table = a.table + (size_t)s * a.s.width;
        const float kg = a.c.kg[g], vg = a.c.vg[g];

        // page ids of 16 of the warp's turns: lane 2 i + half
        uint8_t* myring = ring + warp * STAGES * G::STAGE;
        int pid, pid_t;
        auto load_pages = [&](int t) {
            const int pos = (t + (lane >> 1)) * UNIT + warp * TP + 16 * (lane & 1);
            pid_t = t;
            pid = t + (lane >> 1) < t1 && pos < q.len ? table[pos / a.s.page] : -1;
        };
        // starts the copies of turn t; returns which of its two halves hold positions
        auto issue = [&](int t) {
            if (t - pid_t >= 16) load_pages(t);
            const int pos = t * UNIT + warp * TP;
            int64_t row[2];
            int use = 0;
#pragma unroll
            for (int sub = 0; sub < 2; ++sub) {
                const int pg = __shfl_sync(0xffffffffu, pid, 2 * (t - pid_t) + sub);
                row[sub] = -1;
                if (pos + 16 * sub < q.len) {
                    if (pg >= 0 && pg < a.s.n_pages) {
                        row[sub] = ((int64_t)pg * a.s.nkv + g) * a.s.page + ((pos + 16 * sub) & (a.s.page - 1));
                        use |= 1 << sub;
                    } else if (lane == 0) {
                        atomicExch(a.status, ST_DEVICE_CHECK);
                    }
                }
            }
            copy_stage<HD>(myring + (t & 1) * G::STAGE, a.c, row, lane);
            cp_commit();
            return use;
        };
        load_pages(t0);
        int use = issue(t0);

        // q: warp w takes row w, scaled to [1, 2) by a power of two, as two fp16 terms
        {
            const int tok = (row0 + warp) / group, h = g * group + (row0 + warp) - tok * group;
            float2 v[HD / 64];
            float big = 0.f;
#pragma unroll
            for (int i = 0; i < HD / 64; ++i) {
                v[i] = warp < rows ? kv4_load2(a.q, (size_t)(q.q0 + tok) * a.q_stride + (size_t)h * HD + 2 * lane + 64 * i, a.q_t)
                                   : make_float2(0.f, 0.f);
                big = fmaxf(big, fmaxf(fabsf(v[i].x), fabsf(v[i].y)));
            }
#pragma unroll
            for (int o = 16; o; o >>= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, o));
            const int e = kv4_exponent(big);
            if (lane == 0) fac_s[warp] = ldexpf(a.scale * 1.4426950408889634f * kg, e);
#pragma unroll
            for (int i = 0; i < HD / 64; ++i) {
                const int d = 2 * lane + 64 * i;
                const int jj = HD == 256 ? (d >> 5) & 3 : d / (HD / 4);
                const int wd = HD == 256 ? (d & 31) + 32 * (d >> 7) : d & (HD / 4 - 1);
                uint32_t* f = qf + ((wd >> 2) * 32 + warp * 4 + jj) * 4 + (wd & 2);
                kv4_split(ldexpf(v[i].x, -e), ldexpf(v[i].y, -e), f[0], f[1]);
            }
        }
        __syncthreads();

        const float fac = fac_s[r];
        const int lim = r < rows ? q.len - q.n + (row0 + r) / group + 1 : 0;   // positions this row sees
        const int lim_min = q.len - q.n + row0 / group + 1;
        float m = -INFINITY, l = 0.f;
        float o[HD / 8][4];
#pragma unroll
        for (int t = 0; t < HD / 8; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[t][i] = 0.f;

        for (int t = t0; t < t1; ++t) {
            const int cur = use;
            if (t + 1 < t1) {
                use = issue(t + 1);
                cp_wait<1>();
            } else {
                cp_wait<0>();
            }
            __syncwarp();
            if (cur) {
                const uint8_t* st = myring + (t & 1) * G::STAGE;
                const int pos = t * UNIT + warp * TP;
                // S: columns = positions, four tiles of eight
                float z[4][4];
#pragma unroll
                for (int n = 0; n < 4; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) z[n][i] = 0.f;
#pragma unroll
                for (int hh = 0; hh < (HD == 256 ? 2 : 1); ++hh) {       // 256: the two halves of a row in turn
                    constexpr int KW = HD == 64 ? 2 : 4;                 // words of codes a lane has of a row
                    uint32_t kw[4][4];
                    __half2 ks[4];                                       // their one or two scales
#pragma unroll
                    for (int n = 0; n < 4; ++n) {
                        const int row = n * 8 + r, p = n * 8 + pos_of_col(r);
                        if (HD == 64) {
                            const uint2 x = *reinterpret_cast<const uint2*>(st + G::KC + row * G::ROWB + j * 8);
                            kw[n][0] = x.x;
                            kw[n][1] = x.y;
                            ks[n] = kv4_scale2(st[G::KS + p * G::SB + j]);
                        } else {
                            const int ch = HD == 256 ? (j + 4 * hh) ^ (4 * (r & 1)) : j;
                            const uint4 x = *reinterpret_cast<const uint4*>(st + G::KC + row * G::ROWB + ch * 16);
                            kw[n][0] = x.x;
                            kw[n][1] = x.y;
                            kw[n][2] = x.z;
                            kw[n][3] = x.w;
                            ks[n] = kv4_scale2(*reinterpret_cast<const uint16_t*>(st + G::KS + p * G::SB + 8 * hh + 2 * j));
                        }
                    }
#pragma unroll
                    for (int w = 0; w < KW; ++w) {                       // a word is two steps of the product
                        const uint4* qp = reinterpret_cast<const uint4*>(qf) + (hh * 2 * KW + 2 * w) * 32 + lane;
                        const uint4 qa = qp[0], qb = qp[32];
                        const uint32_t fa[4] = {qa.x, qa.y, qa.z, qa.w}, fb[4] = {qb.x, qb.y, qb.z, qb.w};
#pragma unroll
                        for (int n = 0; n < 4; ++n) {
                            const __half2 sc = w & 2 ? __high2half2(ks[n]) : __low2half2(ks[n]);
                            __half2 k[4];
                            kv4_widen8(kw[n][w], k);
                            mma_f16(z[n], fa, kv4_u(__hmul2(k[0], sc)), kv4_u(__hmul2(k[1], sc)));
                            mma_f16(z[n], fb, kv4_u(__hmul2(k[2], sc)), kv4_u(__hmul2(k[3], sc)));
                        }
                    }
                }
                // z of this lane's row: hi + lo, columns 2 j and 2 j + 1 of each tile
                const bool edge = cur != 3 || pos + TP > lim_min;
                float mx = -INFINITY;
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    z[n][0] = (z[n][0] + z[n][2]) * fac;
                    z[n][1] = (z[n][1] + z[n][3]) * fac;
                    if (edge) {
                        const int p = pos + n * 8 + j;
                        const bool in = (cur >> (n >> 1)) & 1;
                        if (!in || p >= lim) z[n][0] = -INFINITY;
                        if (!in || p + 4 >= lim) z[n][1] = -INFINITY;
                    }
                    mx = fmaxf(mx, fmaxf(z[n][0], z[n][1]));
                }
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                if (__any_sync(0xffffffffu, mx > m + KV4_P_SLACK)) {
                    const float mn = fmaxf(m, mx);
                    const float c = m == -INFINITY ? 0.f : kv4_ex2(m - mn);
                    l *= c;
#pragma unroll
                    for (int t2 = 0; t2 < HD / 8; ++t2)
#pragma unroll
                        for (int i = 0; i < 4; ++i) o[t2][i] *= c;
                    m = mn;
                }
                const float base = m == -INFINITY ? 0.f : m - KV4_P_UP;
                uint32_t pf[2][4];
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    const float p0 = kv4_ex2(z[n][0] - base), p1 = kv4_ex2(z[n][1] - base);
                    l += p0 + p1;
                    kv4_split(p0, p1, pf[n >> 1][2 * (n & 1)], pf[n >> 1][2 * (n & 1) + 1]);
                }
                // o += p v, 16 positions at a time; column r holds the HD/8 elements from r * HD/8
#pragma unroll
                for (int sub = 0; sub < 2; ++sub) {
                    constexpr int VW = HD / 64;                          // words of codes a lane has of a position
                    uint32_t vw[4][4], vs[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int p = 4 * i + j;
                        const uint8_t* vr = st + G::VC + (sub * 16 + p) * G::ROWB;
                        const uint8_t* sr = st + G::VS + (sub * 16 + p) * G::SB;
                        if (HD == 64) {
                            vw[i][0] = *reinterpret_cast<const uint32_t*>(vr + r * 4);
                            vs[i] = sr[r >> 1];
                        } else if (HD == 128) {
                            const uint2 x = *reinterpret_cast<const uint2*>(vr + ((r >> 1) ^ (p & 2)) * 16 + (r & 1) * 8);
                            vw[i][0] = x.x;
                            vw[i][1] = x.y;
                            vs[i] = sr[r];
                        } else {
                            const uint4 x = *reinterpret_cast<const uint4*>(vr + (r ^ (2 * (p & 3))) * 16);
                            vw[i][0] = x.x;
                            vw[i][1] = x.y;
                            vw[i][2] = x.z;
                            vw[i][3] = x.w;
                            vs[i] = *reinterpret_cast<const uint16_t*>(sr + 2 * r);
                        }
                        // behind the last position the bytes may decode to NaN, which weight 0 would keep
                        if (edge && (!((cur >> sub) & 1) || pos + sub * 16 + p >= q.len)) vs[i] = 0;
                    }
#pragma unroll
                    for (int w = 0; w < VW; ++w) {
                        const int sh = HD == 256 ? 8 * (w >> 1) : 0;
                        const __half2 sa = kv4_scale2(kv4_bytes(vs[0] >> sh, vs[1] >> sh));
                        const __half2 sb = kv4_scale2(kv4_bytes(vs[2] >> sh, vs[3] >> sh));
                        uint32_t pa[2], pb[2];                           // even elements, odd elements
                        kv4_pair(vw[0][w], vw[1][w], pa[0], pa[1]);
                        kv4_pair(vw[2][w], vw[3][w], pb[0], pb[1]);
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            __half2 va[4], vb[4];
                            kv4_widen8(pa[e], va);
                            kv4_widen8(pb[e], vb);
#pragma unroll
                            for (int b = 0; b < 4; ++b)
                                mma_f16(o[8 * w + 2 * b + e], pf[sub], kv4_u(__hmul2(va[b], sa)), kv4_u(__hmul2(vb[b], sb)));
                        }
                    }
                }
            }
            __syncwarp();
        }

        // join the warps
        l += __shfl_xor_sync(0xffffffffu, l, 1);
        l += __shfl_xor_sync(0xffffffffu, l, 2);
        __syncthreads();                               // every warp is done with its ring and q
        float* ob = reinterpret_cast<float*>(ring);    // [warp][row][OLD]
        {
            float* w = ob + (warp * 8 + r) * G::OLD + j * (HD / 4 + 4);
#pragma unroll
            for (int t = 0; t < HD / 8; t += 4) {
                *reinterpret_cast<float4*>(w + t) = make_float4(o[t][0] + o[t][2], o[t + 1][0] + o[t + 1][2],
                                                                o[t + 2][0] + o[t + 2][2], o[t + 3][0] + o[t + 3][2]);
                *reinterpret_cast<float4*>(w + HD / 8 + t) =
                    make_float4(o[t][1] + o[t][3], o[t + 1][1] + o[t + 1][3], o[t + 2][1] + o[t + 2][3],
                                o[t + 3][1] + o[t + 3][3]);
            }
            if (j == 0) {
                m_s[warp][r] = m;
                l_s[warp][r] = l;
            }
        }
        __syncthreads();
        // warp -> row, lane -> HD/32 elements
        constexpr int PT = HD / 32;
        const int d0 = lane * PT;
        float2 acc[PT / 2];
        float mj = -INFINITY, lj = 0.f;
#pragma unroll
        for (int w = 0; w < DW; ++w) mj = fmaxf(mj, m_s[w][warp]);
#pragma unroll
        for (int i = 0; i < PT / 2; ++i) acc[i] = make_float2(0.f, 0.f);
        auto add = [&](float mw, float lw, const float* x, bool shared) {
            const float c = lw == 0.f ? 0.f : kv4_ex2(mw - mj);
            lj += lw * c;
#pragma unroll
            for (int i = 0; i < PT / 2; ++i) {
                const float2 y = shared ? reinterpret_cast<const float2*>(x)[i] : __ldcg(reinterpret_cast<const float2*>(x) + i);
                acc[i].x += y.x * c;
                acc[i].y += y.y * c;
            }
        };
#pragma unroll
        for (int w = 0; w < DW; ++w)
            add(m_s[w][warp], l_s[w][warp], ob + (w * 8 + warp) * G::OLD + d0 + 4 * (d0 / (HD / 4)), true);
        bool write = true;
        if (t0 != 0 || t1 != tiles) {
            // a part of the item: its CTAs leave their parts in the workspace, the last one joins them
            const long long i0 = u - t0, i1 = i0 + tiles;
            const int c0 = cta_of_unit(W, i0, Gn), c1 = cta_of_unit(W, i1 - 1, Gn);
            float* part = parts + (size_t)(2 * me + (me == c0)) * G::PART;
#pragma unroll
            for (int i = 0; i < PT / 2; ++i) reinterpret_cast<float2*>(part + warp * HD + d0)[i] = acc[i];
            if (lane == 0) {
                part[8 * HD + warp] = mj;
                part[8 * HD + 8 + warp] = lj;
            }
            __threadfence();
            __syncthreads();
            if (tid == 0) last_s = atomicAdd(arrive + c0, 1u) == (unsigned)(c1 - c0);
            __syncthreads();
            write = last_s;
            if (write) {
                __threadfence();
                if (tid == 0) arrive[c0] = 0u;
                const int ns = c1 - c0 + 1;
                auto part_of = [&](int i) { return parts + (size_t)(2 * (c0 + i) + (i == 0)) * G::PART; };
                mj = -INFINITY;
                for (int i = lane; i < ns; i += 32) mj = fmaxf(mj, __ldcg(part_of(i) + 8 * HD + warp));
#pragma unroll
                for (int x = 16; x; x >>= 1) mj = fmaxf(mj, __shfl_xor_sync(0xffffffffu, mj, x));
                lj = 0.f;
#pragma unroll
                for (int i = 0; i < PT / 2; ++i) acc[i] = make_float2(0.f, 0.f);
#pragma unroll 8
                for (int i = 0; i < ns; ++i) {
                    const float* p = part_of(i);
                    add(__ldcg(p + 8 * HD + warp), __ldcg(p + 8 * HD + 8 + warp), p + warp * HD + d0, false);
                }
            }
        }
        if (write && warp < rows) {
            const int tok = (row0 + warp) / group, h = g * group + (row0 + warp) - tok * group;
            const float inv = lj == 0.f ? 0.f : vg / lj;
            const size_t at = (size_t)(q.q0 + tok) * a.out_stride + (size_t)h * HD + d0;
#pragma unroll
            for (int i = 0; i < PT / 2; ++i) kv4_store2(a.out, at + 2 * i, a.out_t, acc[i].x * inv, acc[i].y * inv);
            if (a.lse && lane == 0)
                a.lse[(size_t)(q.q0 + tok) * a.s.nq + h] =
                    lj == 0.f ? -INFINITY : (mj - KV4_P_UP + log2f(lj)) * 0.6931471805599453f;
        }
        __syncthreads();                               // the join buffer and q are free again
        u += t1 - t0;
    }
}

template <int HD>
cudaError_t launch_decode(const Kv4AttnArgs& a, int few_rows, const Kv4Work& w, cudaStream_t st) {
    const cudaError_t e = cudaFuncSetAttribute(kv4_decode_kernel<HD>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               (int)DGeo<HD>::smem(4096));
    if (e != cudaSuccess) return e;
    return launch_pdl(kv4_decode_kernel<HD>, dim3(w.num_sms * (HD == 256 ? 1 : 2)), dim3(DT), DGeo<HD>::smem(a.n_seqs),
                      st, a, few_rows, w.parts, w.arrive);
}

}  // namespace

// a grid has two CTAs a multiprocessor at most, and each leaves two parts of eight rows at most
size_t kv4_decode_part_floats(int hd, int num_sms) { return (size_t)4 * num_sms * (8 * hd + 16); }

cudaError_t launch_kv4_decode(const Kv4AttnArgs& a, int few_rows, const Kv4Work& w, cudaStream_t st) {
    switch (a.s.hd) {
        case 64: return launch_decode<64>(a, few_rows, w, st);
        case 128: return launch_decode<128>(a, few_rows, w, st);
        default: return launch_decode<256>(a, few_rows, w, st);
    }
}

// Rows (new tokens x heads of the group) up to which a sequence is the decode kernel's.
constexpr int FEW_ROWS = 32;

int kv4_arrive_words(int num_sms) { return 2 * num_sms; }

size_t kv4_part_floats(int hd, int num_sms) {
    const size_t x = kv4_decode_part_floats(hd, num_sms), y = kv4_extend_part_floats(hd, num_sms);
    return x > y ? x : y;
}

cudaError_t launch_kv4_attention(const Kv4AttnArgs& a, const Kv4Work& w, cudaStream_t st) {
    const cudaError_t e = launch_kv4_decode(a, FEW_ROWS, w, st);
    if (e != cudaSuccess || (long long)a.max_new * (a.s.nq / a.s.nkv) <= FEW_ROWS) return e;
    return launch_kv4_extend(a, FEW_ROWS, w, st);
}

}  // namespace qmoe
