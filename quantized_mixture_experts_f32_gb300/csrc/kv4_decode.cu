// kv4_decode.cu -- attention over the paged 4-bit cache for sequences that bring a
// few tokens: decoding, draft tokens.  Bound by the cache's bytes (144 a position and
// kv head at head_dim 128), then by the instructions that widen them.
//
// Row = (token, q head of the kv head's group), 8 NR rows to an item.  With
// z_p = q.k_p * scale * log2(e) the pass keeps a running maximum m, l = sum 2^(z-m)
// and o = sum 2^(z-m) v_p; parts of an item's positions are joined by
// m = max m_i, l = sum l_i 2^(m_i-m), o likewise.
//
// Both products are mma.sync m16n8k16 (fp16 in, fp32 out) with the cache as the
// 16-row operand and the rows as the eight columns: S^T = K Q^T, O^T += V^T P^T.  K and
// V are exact in fp16 (2 x 4 significant bits).  F32 rows enter as hi + lo (TERMS = 2,
// 22 bits), two products into one accumulator, and so do their weights.  16-bit rows enter
// as one term, and their weights too: 2^-11 of each at most, no more than the half step
// that F16 results are off by themselves, where a second term would double the products of V;
// l sums the weights as they are before that rounding.  (4 sequences of 131072 positions,
// F16: 2.9e-4 from 64 bits, of which the result's own rounding is 2.1e-4.)  tcgen05 would
// want the widened K and V in shared memory, 4x the bytes the cache has, for 128 rows of
// which eight exist; here a thread widens what it has loaded straight into operand
// registers.  Each row of q is first scaled by the power of two of its largest element, so
// any fp32 or bf16 range fits fp16.
//
// The order of head elements in q.k and of positions in p.v is free: K and Q elements
// are dealt to the four lanes of a position in contiguous runs (16-byte loads), and
// operand rows to positions so that V's loads meet every bank once.
//
// All positions of all items are dealt out evenly to two CTAs a multiprocessor, whatever
// sequence they belong to.  Measured (32 q heads, 4 kv heads of 128, one token each): 4
// sequences of 131072 positions, F16, 66.7 us, 4.5 TB/s: no pipe is full (issue 61%, ALU
// 50% with the widening, tensor 23%, memory two thirds), and four warps a scheduler, all
// that 122 registers leave room for, do not cover each other's waits; 64 of 100-8192,
// BF16, 28.7 us, 2.4 TB/s, with a start and an end of about 9 us; 1 of 4096, F32, 11.4 us,
// of which the positions are 2: lengths and shares take 1.8, the first bytes 1.8, the join 3.5.
#include <limits.h>
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
constexpr int LEAD = 2;                  // what starting and joining an item costs, in units of positions

template <int HD, int TERMS, int NR>
struct DGeo {
    static constexpr int ROWS = 8 * NR;
    static constexpr int ROWB = HD / 2, SB = HD / 16;          // bytes of codes and scales of a position
    static constexpr int KC = 0, VC = TP * ROWB, KS = 2 * TP * ROWB, VS = KS + TP * SB;
    static constexpr int STAGE = VS + TP * SB;
    static constexpr int RING = DW * STAGES * STAGE;
    static constexpr int QF = HD * 16 * TERMS * NR;            // q fragments of an item
    static constexpr int PART = ROWS * (HD + 2);               // floats of an item's part: o, m, l
    static constexpr size_t smem(int n_seqs) { return (size_t)RING + 2 * QF + 8 * ((size_t)n_seqs + 1); }
    static_assert(8 * HD * 4 <= STAGE, "a warp's eight rows of o take a stage of its ring");
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

// transposes an 8 x 8 matrix of halves held as (row lane/4, columns 2 (lane%4), +1)
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// keeps a rarely taken branch a branch, where selects would run every time
__device__ __forceinline__ void apart() { asm volatile(""); }

// operand row c of eight <-> position of eight: 0 4 1 5 2 6 3 7
__device__ __forceinline__ int pos_of_row(int c) { return (c >> 1) + 4 * (c & 1); }
__device__ __forceinline__ int row_of_pos(int p) { return 2 * (p & 3) + (p >> 2); }

// where the float4 idx of a row of o lies in the join buffer, so that writing (lanes: a run of the
// elements of rows 2 j, 2 j + 1) meets every bank once
template <int HD>
__device__ __forceinline__ int join_at(int idx, int row) {
    const int j = (row >> 1) & 3;
    return idx ^ (HD == 64 ? (j & 1) | ((j & 2) << 1) : HD == 128 ? j : j | (((idx >> 3) & 1) << 2));
}

// What a CTA does next: a part of an item, all of it where t0 = 0 and t1 = tiles.
struct Segment {
    long long next;          // first unit behind it
    int s, g, row0, rows;    // sequence, kv head, first row, rows
    int q0, n, len;
    int t0, t1, tiles;       // its units of positions
    int c0, c1;              // CTAs that share the item
};

// One stage: 32 positions of one kv head, 16 at a time; row: index of the first of the
// 16 positions in the cache (negative: not copied).  K lies in the order of operand rows.
template <int HD>
__device__ __forceinline__ void copy_stage(uint8_t* st, const Kv4Cache& c, const int64_t (&row)[2], int lane) {
    using G = DGeo<HD, 1, 1>;
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
            const int kr = sub * 16 + (p & 8) + row_of_pos(p & 7), vr = sub * 16 + p;
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

// An item counts as LEAD units that hold no positions and then its positions' units, so
// that a CTA with many short items has fewer positions.  CTA c of g takes the units
// [w c / g, w (c+1) / g) of w; g <= w, so each has one at least.
// (Divisions of 64 bits take five times as long: only where 32 do not hold w g.)
__device__ __forceinline__ long long unit_begin(long long w, int c, int g) {
    return w * g < 1ll << 32 ? (uint32_t)w * (uint32_t)c / (uint32_t)g : w * c / g;
}
__device__ __forceinline__ int cta_of_unit(long long w, long long x, int g) {
    return w * g < 1ll << 32 ? (int)((((uint32_t)x + 1) * (uint32_t)g - 1) / (uint32_t)w) : (int)(((x + 1) * g - 1) / w);
}

template <int HD, int TERMS, int NR>
__global__ void __launch_bounds__(DT, HD == 256 ? 1 : 2)
    kv4_decode_kernel(const Kv4AttnArgs a, int few_rows, unsigned* __restrict__ ext_total, float* __restrict__ parts,
                      unsigned* __restrict__ arrive) {
    using G = DGeo<HD, TERMS, NR>;
    extern __shared__ __align__(16) uint8_t sm[];
    uint8_t* ring = sm;
    uint32_t* qf2 = reinterpret_cast<uint32_t*>(sm + G::RING);                      // q fragments, two items
    long long* pre = reinterpret_cast<long long*>(sm + G::RING + 2 * G::QF);        // [n_seqs+1]
    __shared__ long long wsum[DW];
    __shared__ __align__(8) float fac_s[2][G::ROWS], m_s[DW][8], l_s[DW][8];
    __shared__ Segment seg_s[2];
    __shared__ int last_s;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int r = lane >> 2, j = lane & 3;             // operand row (position, element run); a pair of q rows
    const int group = a.s.nq / a.s.nkv;
    // Behind the prompt kernel (ext_total) nothing is waited for: it started its dependents after its own wait,
    // so what it waited for is complete, and it writes nothing that is read here.  The last CTA waits for it
    // before it ends, for the sake of what comes next; the others make room for each other.
    if (!ext_total) pdl_wait();
    else __threadfence();
    pdl_launch_dependents();
    auto leave = [&] {
        if (ext_total && blockIdx.x == gridDim.x - 1) {
            pdl_wait();
            if (tid == 0) *ext_total = 0u;
        }
    };

    // units of every sequence, as prefix sums
    {
        const int per = (a.n_seqs + DT - 1) / DT, s0 = min(tid * per, a.n_seqs), s1 = min(s0 + per, a.n_seqs);
        long long run = 0;
        bool descends = false;
        for (int s = s0; s < s1; ++s) {
            Kv4Seq q;
            if (!kv4_seq(a, s, q) && blockIdx.x == 0) atomicExch(a.status, ST_DEVICE_CHECK);
            descends |= a.cu[s + 1] < a.cu[s];
            pre[s] = run;
            if (q.n * group <= few_rows)
                run += (long long)a.s.nkv * ((q.n * group + G::ROWS - 1) / G::ROWS) *
                       (LEAD + (q.len ? (q.len + UNIT - 1) / UNIT : 1));
        }
        long long inc = run;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const long long o = __shfl_up_sync(0xffffffffu, inc, d);
            if (lane >= d) inc += o;
        }
        if (lane == 31) wsum[warp] = inc;
        if (__syncthreads_or(descends)) return leave();            // rows of several sequences; the status says so
        long long base = inc - run;
        for (int w = 0; w < warp; ++w) base += wsum[w];
        for (int s = s0; s < s1; ++s) pre[s] += base;
        if (tid == DT - 1) pre[a.n_seqs] = base + run;
    }
    __syncthreads();
    const long long W = pre[a.n_seqs];
    const int Gn = (int)min((long long)gridDim.x, W), me = blockIdx.x;
    if (me >= Gn) return leave();
    const long long u_end = unit_begin(W, me + 1, Gn);

    // the segment that starts with unit u (one thread); tiles = 0: none
    auto describe = [&](long long u, Segment& r) {
        r.tiles = 0;
        if (u >= u_end) return;
        int s = 0;
        for (int hi = a.n_seqs; hi - s > 1;) {
            const int mid = (s + hi) >> 1;
            if (pre[mid] <= u) s = mid;
            else hi = mid;
        }
        Kv4Seq q;
        kv4_seq(a, s, q);
        const int tiles = q.len ? (q.len + UNIT - 1) / UNIT : 1, vu = LEAD + tiles;
        const int rts = (q.n * group + G::ROWS - 1) / G::ROWS;
        const long long off = u - pre[s];
        const int item = off < (1ll << 31) ? (int)((uint32_t)off / (uint32_t)vu) : (int)(off / vu), v0 = (int)(off - (long long)item * vu);
        const int v1 = (int)min((long long)vu, v0 + (u_end - u));
        if (v1 <= LEAD) return;                        // the lead alone: the next CTA starts the item
        r.next = u + (v1 - v0);
        r.s = s;
        r.g = item / rts;
        r.row0 = (item - r.g * rts) * G::ROWS;
        r.rows = min(G::ROWS, q.n * group - r.row0);
        r.q0 = q.q0;
        r.n = q.n;
        r.len = q.len;
        r.t0 = max(v0 - LEAD, 0);
        r.t1 = v1 - LEAD;
        r.tiles = tiles;
        const long long i0 = u - v0;                   // the item's first unit
        r.c0 = cta_of_unit(W, i0 + LEAD, Gn);
        r.c1 = cta_of_unit(W, i0 + vu - 1, Gn);
    };

    uint8_t* myring = ring + warp * STAGES * G::STAGE;
    int stage = 0;                                     // where the copies of the next turn go
    int use = 0;                                       // which halves of that turn hold positions
    int pid = -1, pid_t = 0;                           // page ids of 16 of the warp's turns: lane 2 i + half
    // starts the copies of turn t of a segment
    auto issue = [&](const Segment& r, int t, bool fresh) {
        if (fresh || t - pid_t >= 16) {
            const int pos = (t + (lane >> 1)) * UNIT + warp * TP + 16 * (lane & 1);
            pid_t = t;
            pid = t + (lane >> 1) < r.t1 && pos < r.len ? a.table[(size_t)r.s * a.s.width + (pos >> a.s.page_log2)] : -1;
        }
        const int pos = t * UNIT + warp * TP;
        int64_t row[2];
        use = 0;
#pragma unroll
        for (int sub = 0; sub < 2; ++sub) {
            const int pg = __shfl_sync(0xffffffffu, pid, 2 * (t - pid_t) + sub);
            row[sub] = -1;
            if (pos + 16 * sub < r.len) {
                if (pg >= 0 && pg < a.s.n_pages) {
                    row[sub] = ((int64_t)pg * a.s.nkv + r.g) * a.s.page + ((pos + 16 * sub) & (a.s.page - 1));
                    use |= 1 << sub;
                } else if (lane == 0) {
                    atomicExch(a.status, ST_DEVICE_CHECK);
                }
            }
        }
        copy_stage<HD>(myring + stage * G::STAGE, a.c, row, lane);
        cp_commit();
    };
    // q: warp w takes the rows w, w + 8, scaled to [1, 2) by a power of two
    struct Rows {
        float2 v[NR][HD / 64];
    };
    auto load_q = [&](const Segment& r, Rows& x) {
#pragma unroll
        for (int nr = 0; nr < NR; ++nr) {
            const int row = nr * 8 + warp;
            const int tok = (r.row0 + row) / group, h = r.g * group + (r.row0 + row) - tok * group;
#pragma unroll
            for (int i = 0; i < HD / 64; ++i)
                x.v[nr][i] = row < r.rows ? kv4_load2(a.q, (size_t)(r.q0 + tok) * a.q_stride + (size_t)h * HD + 2 * lane + 64 * i, a.q_t)
                                          : make_float2(0.f, 0.f);
        }
    };
    auto put_q = [&](const Segment& r, int buf, const Rows& x) {
        uint32_t* qf = qf2 + buf * (G::QF / 4);
        const float kg = a.c.kg[r.g];
        const Kv4Factor factor = kv4_factor(a.scale, kg);
#pragma unroll
        for (int nr = 0; nr < NR; ++nr) {
            const int row = nr * 8 + warp;
            const float2(&v)[HD / 64] = x.v[nr];
            float big = 0.f;
#pragma unroll
            for (int i = 0; i < HD / 64; ++i) big = fmaxf(big, fmaxf(fabsf(v[i].x), fabsf(v[i].y)));
#pragma unroll
            for (int o = 16; o; o >>= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, o));
            const int e = kv4_exponent(big);
            const float un = kv4_negative(a.scale, kg) ? -kv4_pow2(-e) : kv4_pow2(-e);   // z's largest is q.k's largest then
#pragma unroll
            for (int i = 0; i < HD / 64; ++i) {
                uint32_t hi, lo;
                kv4_split(v[i].x * un, v[i].y * un, hi, lo);
                // element d -> lane jj's wd-th; fragment: step wd / 4, register (wd / 2) % 2.
                // A lane's 16 bytes: TERMS = 1 two steps, TERMS = 2 the two terms of one.
                const int d = 2 * lane + 64 * i;
                const int jj = HD == 256 ? (d >> 5) & 3 : d / (HD / 4);
                const int wd = HD == 256 ? (d & 31) + 32 * (d >> 7) : d & (HD / 4 - 1);
                const int step = wd >> 2, b = (wd >> 1) & 1, at = warp * 4 + jj;
                if (TERMS == 1) {
                    qf[((nr * (HD / 32) + (step >> 1)) * 32 + at) * 4 + (step & 1) * 2 + b] = hi;
                } else {
                    qf[((nr * (HD / 16) + step) * 32 + at) * 4 + b] = hi;
                    qf[((nr * (HD / 16) + step) * 32 + at) * 4 + 2 + b] = lo;
                }
            }
            if (lane == 0) fac_s[buf][row] = kv4_factor_of(factor, e);
        }
    };

    if (tid == 0) describe(unit_begin(W, me, Gn), seg_s[0]);
    __syncthreads();
    if (seg_s[0].tiles == 0) return leave();
    {
        Rows x;
        load_q(seg_s[0], x);                           // on its way while the first page ids are
        issue(seg_s[0], seg_s[0].t0, true);
        put_q(seg_s[0], 0, x);
    }
    __syncthreads();
    for (int cur = 0;; cur ^= 1) {
        const Segment& S = seg_s[cur];
        const uint32_t* qf = qf2 + cur * (G::QF / 4);
        const int len = S.len, rows = S.rows, row0 = S.row0, t0 = S.t0, t1 = S.t1;
        if (tid == DT - 32) describe(S.next, seg_s[cur ^ 1]);      // while the others start

        // this lane's rows: 2 j and 2 j + 1 of each eight
        float fac[NR][2], m[NR][2], l[NR][2], base[NR][2];
        int lim[NR][2];                                // positions they see
#pragma unroll
        for (int nr = 0; nr < NR; ++nr)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                const int row = nr * 8 + 2 * j + y;
                fac[nr][y] = fac_s[cur][row];
                lim[nr][y] = row < rows ? len - S.n + (row0 + row) / group + 1 : 0;
                m[nr][y] = -INFINITY;
                base[nr][y] = 0.f;
                l[nr][y] = 0.f;
            }
        bool far = false;
#pragma unroll
        for (int nr = 0; nr < NR; ++nr) far |= kv4_far<HD>(fac[nr][0]) | kv4_far<HD>(fac[nr][1]);
        far = __any_sync(0xffffffffu, far);            // z takes its factor in the branch of masks, fac is 1 then
        if (far)
#pragma unroll
            for (int nr = 0; nr < NR; ++nr) fac[nr][0] = fac[nr][1] = 1.f;
        const int lim_min = len - S.n + row0 / group + 1;
        float o[NR][HD / 16][4];
#pragma unroll
        for (int nr = 0; nr < NR; ++nr)
#pragma unroll
            for (int t = 0; t < HD / 16; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[nr][t][i] = 0.f;

        for (int t = t0; t < t1; ++t) {
            const int halves = use;
            const uint8_t* st = myring + stage * G::STAGE;
            stage ^= 1;
            if (t + 1 < t1) {
                issue(S, t + 1, false);
                cp_wait<1>();
            } else {
                cp_wait<0>();
            }
            __syncwarp();
            if (halves) {
                const int pos = t * UNIT + warp * TP;
                // S^T: two tiles of 16 positions; lane: positions r, r + 8 of each, rows 2 j, 2 j + 1
                float z[2][NR][4];
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int nr = 0; nr < NR; ++nr)
#pragma unroll
                        for (int i = 0; i < 4; ++i) z[n][nr][i] = 0.f;
#pragma unroll
                for (int hh = 0; hh < (HD == 256 ? 2 : 1); ++hh) {       // 256: the two halves of a position in turn
                    constexpr int KW = HD == 64 ? 2 : 4;                 // words of codes a lane has of a position
                    uint32_t kw[4][4];
                    __half2 ks[4];                                       // their one or two scales
#pragma unroll
                    for (int n = 0; n < 4; ++n) {
                        const int row = n * 8 + r, p = n * 8 + pos_of_row(r);
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
                        uint32_t ka[2][2][4];                            // [tile][step]: operand registers
#pragma unroll
                        for (int n = 0; n < 4; ++n) {
                            const __half2 sc = w & 2 ? __high2half2(ks[n]) : __low2half2(ks[n]);
                            __half2 k[4];
                            kv4_widen8(kw[n][w], k);
#pragma unroll
                            for (int b = 0; b < 4; ++b) ka[n >> 1][b >> 1][2 * (b & 1) + (n & 1)] = kv4_u(__hmul2(k[b], sc));
                        }
#pragma unroll
                        for (int nr = 0; nr < NR; ++nr) {
                            const uint4* qp = reinterpret_cast<const uint4*>(qf) +
                                              (nr * (HD / 32) * TERMS + (hh * KW + w) * TERMS) * 32 + lane;
                            if (TERMS == 1) {
                                const uint4 x = qp[0];
#pragma unroll
                                for (int n = 0; n < 2; ++n) {
                                    mma_f16(z[n][nr], ka[n][0], x.x, x.y);
                                    mma_f16(z[n][nr], ka[n][1], x.z, x.w);
                                }
                            } else {
                                const uint4 x = qp[0], y = qp[32];
#pragma unroll
                                for (int n = 0; n < 2; ++n) {
                                    mma_f16(z[n][nr], ka[n][0], x.z, x.w);
                                    mma_f16(z[n][nr], ka[n][0], x.x, x.y);
                                    mma_f16(z[n][nr], ka[n][1], y.z, y.w);
                                    mma_f16(z[n][nr], ka[n][1], y.x, y.y);
                                }
                            }
                        }
                    }
                }
                const bool edge = halves != 3 || pos + TP > lim_min || far;
                if (edge) {
#pragma unroll
                    for (int nr = 0; nr < NR; ++nr)
#pragma unroll
                        for (int n = 0; n < 4; ++n)
#pragma unroll
                            for (int y = 0; y < 2; ++y)
                                if (!((halves >> (n >> 1)) & 1) || pos + n * 8 + pos_of_row(r) >= lim[nr][y])
                                    z[n >> 1][nr][2 * (n & 1) + y] = -INFINITY;
                    if (far) {
#pragma unroll
                        for (int nr = 0; nr < NR; ++nr) {
                            const float2 f = *reinterpret_cast<const float2*>(fac_s[cur] + nr * 8 + 2 * j);
#pragma unroll
                            for (int n = 0; n < 4; ++n) {
                                z[n >> 1][nr][2 * (n & 1)] = __fmul_rn(z[n >> 1][nr][2 * (n & 1)], f.x);
                                z[n >> 1][nr][2 * (n & 1) + 1] = __fmul_rn(z[n >> 1][nr][2 * (n & 1) + 1], f.y);
                            }
                        }
                    }
                    apart();
                }
                // m follows a row's maximum only when some lane saw it 2^SLACK ahead
                bool ahead = false;
                float mx[NR][2];
#pragma unroll
                for (int nr = 0; nr < NR; ++nr)
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        float x = -INFINITY;
#pragma unroll
                        for (int n = 0; n < 4; ++n) {
                            x = fmaxf(x, z[n >> 1][nr][2 * (n & 1) + y]);
                        }
                        mx[nr][y] = x * fac[nr][y];
                        ahead |= mx[nr][y] > m[nr][y] + KV4_P_SLACK;
                    }
                if (__any_sync(0xffffffffu, ahead)) {
#pragma unroll
                    for (int nr = 0; nr < NR; ++nr)
#pragma unroll
                        for (int y = 0; y < 2; ++y) {
                            float x = mx[nr][y];
#pragma unroll
                            for (int d = 4; d < 32; d <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, d));
                            const float mn = fmaxf(m[nr][y], x);
                            const float c = m[nr][y] == -INFINITY ? 0.f : kv4_ex2(m[nr][y] - mn);
                            m[nr][y] = mn;
                            base[nr][y] = mn == -INFINITY ? 0.f : mn - KV4_P_UP;
                            l[nr][y] *= c;
#pragma unroll
                            for (int t2 = 0; t2 < HD / 16; ++t2) {
                                o[nr][t2][y] *= c;
                                o[nr][t2][2 + y] *= c;
                            }
                        }
                }
                // P^T as the eight-column operand: rows 2 j, 2 j + 1 of a position, transposed
                uint32_t pf[2][NR][TERMS][2];
#pragma unroll
                for (int n = 0; n < 4; ++n)
#pragma unroll
                    for (int nr = 0; nr < NR; ++nr) {
                        float p[2];
#pragma unroll
                        for (int y = 0; y < 2; ++y) {
                            const float zz = z[n >> 1][nr][2 * (n & 1) + y];
                            p[y] = kv4_ex2(fmaf(zz, fac[nr][y], -base[nr][y]));
                            l[nr][y] += p[y];
                        }
                        if (TERMS == 1) {
                            pf[n >> 1][nr][0][n & 1] = transpose8(kv4_pack(p[0], p[1]));
                        } else {
                            uint32_t hi, lo;
                            kv4_split(p[0], p[1], hi, lo);
                            pf[n >> 1][nr][0][n & 1] = transpose8(hi);
                            pf[n >> 1][nr][TERMS - 1][n & 1] = transpose8(lo);
                        }
                    }
                // O^T += V^T P^T, 16 positions at a time; operand row r holds the HD/8 elements from r * HD/8
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
                    }
                    if (edge) {
                        // behind the last position the bytes may decode to NaN, which weight 0 would keep
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (!((halves >> sub) & 1) || pos + sub * 16 + 4 * i + j >= len) vs[i] = 0;
                        apart();
                    }
#pragma unroll
                    for (int w = 0; w < VW; ++w) {
                        const int sh = HD == 256 ? 8 * (w >> 1) : 0;
                        const __half2 sa = kv4_scale2(kv4_bytes(vs[0] >> sh, vs[1] >> sh));
                        const __half2 sb = kv4_scale2(kv4_bytes(vs[2] >> sh, vs[3] >> sh));
                        uint32_t pa[2], pb[2];                           // even elements, odd elements
                        kv4_pair(vw[0][w], vw[1][w], pa[0], pa[1]);
                        kv4_pair(vw[2][w], vw[3][w], pb[0], pb[1]);
                        __half2 va[2][4], vb[2][4];
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            kv4_widen8(pa[e], va[e]);
                            kv4_widen8(pb[e], vb[e]);
                        }
#pragma unroll
                        for (int b = 0; b < 4; ++b) {                    // elements 8 w + 2 b, 8 w + 2 b + 1
                            const uint32_t av[4] = {kv4_u(__hmul2(va[0][b], sa)), kv4_u(__hmul2(va[1][b], sa)),
                                                    kv4_u(__hmul2(vb[0][b], sb)), kv4_u(__hmul2(vb[1][b], sb))};
#pragma unroll
                            for (int nr = 0; nr < NR; ++nr)
#pragma unroll
                                for (int tm = TERMS - 1; tm >= 0; --tm)
                                    mma_f16(o[nr][4 * w + b], av, pf[sub][nr][tm][0], pf[sub][nr][tm][1]);
                        }
                    }
                }
            }
            __syncwarp();
        }

        // join the warps, eight rows at a time, each warp's in the stage it used last (the other one
        // takes the next segment's first copies)
        constexpr int PT = HD / 32;                    // elements of a lane then; warp -> row
        const int d0 = lane * PT, last_stage = stage ^ 1;
        const bool whole = t0 == 0 && t1 == S.tiles;
        float* part = parts + (size_t)(2 * me + (me == S.c0)) * G::PART;
        const float vg = a.c.vg[S.g];
        float2 acc[PT / 2];
        float mj, lj;
        auto clear = [&]() {
            lj = 0.f;
#pragma unroll
            for (int i = 0; i < PT / 2; ++i) acc[i] = make_float2(0.f, 0.f);
        };
        auto write = [&](int row) {
            if (row >= rows) return;
            const int tok = (row0 + row) / group, h = S.g * group + (row0 + row) - tok * group;
            const float inv = lj == 0.f ? 0.f : vg / lj;
            const size_t at = (size_t)(S.q0 + tok) * a.out_stride + (size_t)h * HD + d0;
#pragma unroll
            for (int i = 0; i < PT / 2; ++i) kv4_store2(a.out, at + 2 * i, a.out_t, acc[i].x * inv, acc[i].y * inv);
            if (a.lse && lane == 0)
                a.lse[(size_t)(S.q0 + tok) * a.s.nq + h] =
                    lj == 0.f ? -INFINITY : (mj - KV4_P_UP + log2f(lj)) * 0.6931471805599453f;
        };
#pragma unroll
        for (int nr = 0; nr < NR; ++nr) {
            if (nr) __syncthreads();                   // the first eight rows are read
            float4* mine = reinterpret_cast<float4*>(myring + last_stage * G::STAGE);
#pragma unroll
            for (int y = 0; y < 2; ++y) {
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) l[nr][y] += __shfl_xor_sync(0xffffffffu, l[nr][y], d);
                const int row = 2 * j + y;
#pragma unroll
                for (int t = 0; t < HD / 16; t += 2)
                    mine[row * (HD / 4) + join_at<HD>(r * (HD / 32) + t / 2, row)] =
                        make_float4(o[nr][t][y], o[nr][t][2 + y], o[nr][t + 1][y], o[nr][t + 1][2 + y]);
                if (r == 0) {
                    m_s[warp][row] = m[nr][y];
                    l_s[warp][row] = l[nr][y];
                }
            }
            __syncthreads();
            if (nr == 0 && seg_s[cur ^ 1].tiles) issue(seg_s[cur ^ 1], seg_s[cur ^ 1].t0, true);
            mj = -INFINITY;
#pragma unroll
            for (int w = 0; w < DW; ++w) mj = fmaxf(mj, m_s[w][warp]);
            clear();
#pragma unroll
            for (int w = 0; w < DW; ++w) {
                const float* ob = reinterpret_cast<const float*>(ring + (w * STAGES + last_stage) * G::STAGE) + warp * HD;
                const float c = l_s[w][warp] == 0.f ? 0.f : kv4_ex2(m_s[w][warp] - mj);
                lj += l_s[w][warp] * c;
#pragma unroll
                for (int i = 0; i < PT / 2; ++i) {
                    const int d = d0 + 2 * i;
                    const float2 y = *reinterpret_cast<const float2*>(ob + 4 * join_at<HD>(d >> 2, warp) + (d & 3));
                    acc[i].x += y.x * c;
                    acc[i].y += y.y * c;
                }
            }
            const int row = nr * 8 + warp;
            if (whole) {
                write(row);
            } else {
                // a part of the item: its CTAs leave their parts in the workspace, the last one joins them
#pragma unroll
                for (int i = 0; i < PT / 2; ++i) reinterpret_cast<float2*>(part + row * HD + d0)[i] = acc[i];
                if (lane == 0) {
                    part[G::ROWS * HD + row] = mj;
                    part[G::ROWS * HD + G::ROWS + row] = lj;
                }
            }
        }
        if (seg_s[cur ^ 1].tiles) {
            Rows x;
            load_q(seg_s[cur ^ 1], x);
            put_q(seg_s[cur ^ 1], cur ^ 1, x);
        }
        if (!whole) {
            const int c0 = S.c0, c1 = S.c1;
            __syncthreads();
            if (tid == 0) {
                __threadfence();
                last_s = atomicAdd(arrive + c0, 1u) == (unsigned)(c1 - c0);
                if (last_s) {
                    arrive[c0] = 0u;
                    __threadfence();
                }
            }
            __syncthreads();
            if (last_s) {
                const int ns = c1 - c0 + 1;
                auto part_of = [&](int i) { return parts + (size_t)(2 * (c0 + i) + (i == 0)) * G::PART; };
                constexpr int AT = 8;                  // parts in flight
                for (int row = warp; row < rows; row += DW) {
                    float2 v[AT][PT / 2];
                    auto load = [&](int i0) {
#pragma unroll
                        for (int y = 0; y < AT; ++y) {
                            const float2* p = reinterpret_cast<const float2*>(part_of(min(i0 + y, ns - 1)) + row * HD + d0);
#pragma unroll
                            for (int k = 0; k < PT / 2; ++k) v[y][k] = __ldcg(p + k);
                        }
                    };
                    // m and l of 32 parts a lane each, and the first parts behind them
                    auto m_of = [&](int i) { return i < ns ? __ldcg(part_of(i) + G::ROWS * HD + row) : -INFINITY; };
                    auto l_of = [&](int i) { return i < ns ? __ldcg(part_of(i) + G::ROWS * HD + G::ROWS + row) : 0.f; };
                    float mw = m_of(lane), lw = l_of(lane);
                    load(0);
                    mj = mw;
                    for (int i = lane + 32; i < ns; i += 32) mj = fmaxf(mj, m_of(i));
#pragma unroll
                    for (int x = 16; x; x >>= 1) mj = fmaxf(mj, __shfl_xor_sync(0xffffffffu, mj, x));
                    clear();
#pragma unroll 1
                    for (int i0 = 0; i0 < ns; i0 += AT) {
                        if (i0 && i0 % 32 == 0) {
                            mw = m_of(i0 + lane);
                            lw = l_of(i0 + lane);
                        }
                        const float c = lw == 0.f ? 0.f : kv4_ex2(mw - mj);          // of part i0 / 32 * 32 + lane
                        if (i0 % 32 == 0) {
                            float sum = lw * c;
#pragma unroll
                            for (int x = 16; x; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
                            lj += sum;
                        }
#pragma unroll
                        for (int y = 0; y < AT; ++y) {
                            const float cy = __shfl_sync(0xffffffffu, c, (i0 + y) & 31);
#pragma unroll
                            for (int k = 0; k < PT / 2; ++k) {
                                // a part past the last one counts nothing (its c is 0, v the last one's)
                                acc[k].x += i0 + y < ns ? v[y][k].x * cy : 0.f;
                                acc[k].y += i0 + y < ns ? v[y][k].y * cy : 0.f;
                            }
                        }
                        if (i0 + AT < ns) load(i0 + AT);
                    }
                    write(row);
                }
            }
        }
        if (seg_s[cur ^ 1].tiles == 0) return leave();
        __syncthreads();                               // the next segment's q is there, the join is read
    }
}

template <int HD, int TERMS, int NR>
cudaError_t launch_decode(const Kv4AttnArgs& a, int few_rows, bool behind, const Kv4Work& w, cudaStream_t st) {
    using G = DGeo<HD, TERMS, NR>;
    return launch_pdl(kv4_decode_kernel<HD, TERMS, NR>, dim3(w.num_sms * (HD == 256 ? 1 : 2)), dim3(DT),
                      G::smem(a.n_seqs), st, a, few_rows, behind ? w.ext_total : nullptr, w.parts, w.arrive);
}

template <int HD, int TERMS>
cudaError_t pick_rows(const Kv4AttnArgs& a, int few_rows, bool behind, const Kv4Work& w, cudaStream_t st) {
    // Items of 16 rows read and widen the cache once where items of 8 do twice, which costs less than it seems:
    // their two items run side by side, or one finds the other's bytes in L2, in shorter code.  bf16, 4 kv heads,
    // 16 rows, us (items of 16 / 8): 1 sequence of 1000 positions 15.2 / 10.3, 65536 39 / 28, 262144 70 / 68 (head_dim
    // 256: 95 / 114); 2 of 4096 17.2 / 11.5, of 131072 65 / 65; 4 of 131072 101 / 118 (head_dim 64: 62 / 83, 256:
    // 154 / 217).  So with few sequences 8.  Beside prompts too: requests bring one token there as a rule, and
    // what is smaller fills the multiprocessors that come free more evenly (24 requests of 300-6000 positions,
    // four with up to 500 new tokens, the others with one, 82.9 / 75.1; 23 with two and one with 500, 90.4 / 83.8).
    // One rule for all types and head_dim, set at 128: at 256 it picks the slower one for one or two very long
    // sequences (95 / 114 above).
    const int group = a.s.nq / a.s.nkv;
    const bool two = (long long)a.max_new * group > 8 &&
                     (behind ? group > 8 : (long long)a.n_seqs * a.s.nkv * 16 > w.num_sms);
    return two ? launch_decode<HD, TERMS, 2>(a, few_rows, behind, w, st) : launch_decode<HD, TERMS, 1>(a, few_rows, behind, w, st);
}

}  // namespace

cudaError_t kv4_decode_prepare() {
    cudaError_t e = cudaSuccess;
    auto allow = [&](auto kernel, size_t smem) {
        if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    };
    allow(kv4_decode_kernel<64, 1, 1>, DGeo<64, 1, 1>::smem(4096));
    allow(kv4_decode_kernel<64, 1, 2>, DGeo<64, 1, 2>::smem(4096));
    allow(kv4_decode_kernel<64, 2, 1>, DGeo<64, 2, 1>::smem(4096));
    allow(kv4_decode_kernel<64, 2, 2>, DGeo<64, 2, 2>::smem(4096));
    allow(kv4_decode_kernel<128, 1, 1>, DGeo<128, 1, 1>::smem(4096));
    allow(kv4_decode_kernel<128, 1, 2>, DGeo<128, 1, 2>::smem(4096));
    allow(kv4_decode_kernel<128, 2, 1>, DGeo<128, 2, 1>::smem(4096));
    allow(kv4_decode_kernel<128, 2, 2>, DGeo<128, 2, 2>::smem(4096));
    allow(kv4_decode_kernel<256, 1, 1>, DGeo<256, 1, 1>::smem(4096));
    allow(kv4_decode_kernel<256, 1, 2>, DGeo<256, 1, 2>::smem(4096));
    allow(kv4_decode_kernel<256, 2, 1>, DGeo<256, 2, 1>::smem(4096));
    allow(kv4_decode_kernel<256, 2, 2>, DGeo<256, 2, 2>::smem(4096));
    return e;
}

// a grid has two CTAs a multiprocessor at most, and each leaves two parts of 16 rows at most
size_t kv4_decode_part_floats(int hd, int num_sms) { return (size_t)4 * num_sms * 16 * (hd + 2); }

cudaError_t launch_kv4_decode(const Kv4AttnArgs& a, int few_rows, bool behind, const Kv4Work& w, cudaStream_t st) {
    const bool two = a.q_t == KV4_F32;
    switch (a.s.hd) {
        case 64: return two ? pick_rows<64, 2>(a, few_rows, behind, w, st) : pick_rows<64, 1>(a, few_rows, behind, w, st);
        case 128: return two ? pick_rows<128, 2>(a, few_rows, behind, w, st) : pick_rows<128, 1>(a, few_rows, behind, w, st);
        default: return two ? pick_rows<256, 2>(a, few_rows, behind, w, st) : pick_rows<256, 1>(a, few_rows, behind, w, st);
    }
}

int kv4_arrive_words(int num_sms) { return 2 * num_sms; }   // a CTA of the one kernel, a part of the other

// Which kernel a sequence's rows (new tokens x heads of the group) go to.  The decode kernel
// reads and widens the cache once per 16 rows, the prompt kernel once per 256, with a dearer start
// and end.  Measured, head_dim 128, 4 kv heads, bf16, us (decode / prompt kernel): 16 sequences of
// 4096 positions, 16 rows 29.6 / 38.5, 24 rows 40.2 / 38.7, 64 rows 64 / 39; 64 of 1024, 16 rows
// 33.8 / 42.3, 24 rows 49 / 42.  With few sequences the passes of the decode kernel run side by
// side: 1 of 32768, 40 rows 36.0 / 40.2, 64 rows 39.4 / 40.4, 80 rows 45.6 / 50.2; 1 of 4096, 64
// rows 19.4 / 26.8.  There 64 is on the decode kernel's side of the border, which lies past 80 rows
// at 32768; other types and head_dim were not measured for it.
//
// The prompt kernel goes first: its CTAs do not end together, and the decode kernel's, smaller and
// more, run where it has ended (bf16, 24 requests of 300-6000 positions, four of them with up to 500
// new tokens: 75.1 us, the decode kernel first 82.1; 64 that decode and one with 500: 80.9, 85.8; 8
// that decode and 8 with 200: 83.9, 97.7).
cudaError_t launch_kv4_attention(const Kv4AttnArgs& a, const Kv4Work& w, cudaStream_t st) {
    constexpr int few_alone = 64;
    const int few = (long long)a.n_seqs * a.s.nkv * 8 <= w.num_sms ? few_alone : KV4_FEW_ROWS;
    const bool prompts = (long long)a.max_new * (a.s.nq / a.s.nkv) > few;
    if (prompts) {
        const cudaError_t e = launch_kv4_extend(a, few, w, st);
        if (e != cudaSuccess) return e;
    }
    const cudaError_t e = launch_kv4_decode(a, few, prompts, w, st);
    if (e != cudaSuccess && prompts) cudaMemsetAsync(w.ext_total, 0, sizeof(unsigned), st);   // which the kernel would have
    return e;
}

}  // namespace qmoe
