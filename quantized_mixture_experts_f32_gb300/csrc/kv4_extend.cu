// kv4_extend.cu -- attention over the paged 4-bit cache for sequences that bring many
// tokens (prompt chunks): bound by the two matrix products and the exponentials.
//
// An item is (sequence, kv head, 128 NT rows of (token, head of the group)); a CTA
// walks its visible positions in chunks of KC.  Warps have roles:
//   softmax  4 warps per 128 rows, a thread to a row (its TMEM lane): z from TMEM,
//            running maximum m and sum l, p = 2^(z - m) back into TMEM as fp16
//   K, V     4 warps each: codes from the cache, widened (exactly) to fp16 into
//            128B-swizzled K-major tiles, V transposed so that positions are K
//   MMA      one thread: S = Q K^T and O += P V^T, tcgen05, P read from TMEM
// With NT = 2 the two 128-row tiles share every widened K and V tile (the widening
// costs as many issue slots as one tile's softmax) and their softmaxes alternate
// with their products; with NT = 1 (F32 rows, head_dim 256: shared memory has no
// room for two) the chunks of one tile alternate over two S buffers.  P overlays the
// S it came from: the MMA thread issues the next S into it after the product that
// reads P, and the tensor pipe runs them in that order.
// O is rescaled only when a row's maximum rose by 2^8 since the last time.
// F32 rows: q = hi + lo and p = hi + lo, two products each (TERMS = 2).
// Few items: the chunks of an item are split over CTAs, the last one joins the parts.
#include <math.h>

#include <type_traits>

#include "kv4.cuh"
#include "kv4_row.cuh"
#include "umma.cuh"

namespace qmoe {

namespace {

template <int HD, int TERMS>
struct EGeo {
    static constexpr int NT = HD <= 128 && TERMS == 1 ? 2 : 1;       // 128-row tiles
    static constexpr int KC = HD == 256 ? 64 : 128;                  // positions of a chunk
    static constexpr int BUF = HD == 256 && TERMS == 2 ? 1 : 2;      // K and V tiles in shared memory
    static constexpr int ROWS = 128 * NT;
    static constexpr int SOFT = 128 * NT;                            // softmax threads
    static constexpr int THREADS = SOFT + 256 + 32;
    static constexpr int QT = 128 * HD * 2, KT = KC * HD * 2;        // bytes of a tile
    static constexpr int Q = 0, K = NT * TERMS * QT, V = K + BUF * KT, BARS = V + BUF * KT;
    static constexpr size_t SMEM = 1024 + BARS + 256;
    static constexpr int LPR = HD / 32;                              // 16-byte runs of a position's codes
    static constexpr int KP = KC * LPR / 128;                        // runs a K thread widens
    static constexpr int RPP = 128 / LPR;                            // rows between them
    static constexpr int PART = ROWS * (HD + 2);                     // floats of a part
};

// D[tmem] (+)= A[tmem] * B^T, issued by one thread
__device__ __forceinline__ void umma_f16_ta(uint32_t d, uint32_t a, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ void tmem_ld32(uint32_t t, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(t)
        : "memory");
}

__device__ __forceinline__ void tmem_st16(uint32_t t, const uint32_t* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(t),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// a wait whose outcome the whole warp shares: what follows is collective
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity));
}

// What a CTA works on.
struct Piece {
    int s, g, row0;          // sequence, kv head, first row
    int q0, n, len;
    int c0, c1;              // chunks
    int split, splits, item;
};

template <int HD, int TERMS>
__global__ void __launch_bounds__(EGeo<HD, TERMS>::THREADS, 1)
    kv4_extend_kernel(const Kv4AttnArgs a, int few_rows, float* __restrict__ parts, unsigned* __restrict__ arrive,
                      int num_sms) {
    using G = EGeo<HD, TERMS>;
    constexpr int NT = G::NT, KC = G::KC, BUF = G::BUF;
    extern __shared__ __align__(1024) uint8_t smraw[];
    uint8_t* sm = smraw + ((1024u - (smem_u32(smraw) & 1023u)) & 1023u);
    uint64_t* bars = reinterpret_cast<uint64_t*>(sm + G::BARS);
    uint64_t *kfull = bars, *kempty = bars + 2, *vfull = bars + 4, *vempty = bars + 6, *sfull = bars + 8,
             *pfull = bars + 10, *odone = bars + 12, *qfull = bars + 14;
    uint32_t* tslot = reinterpret_cast<uint32_t*>(bars + 15);
    __shared__ int wsum[G::THREADS / 32];
    __shared__ Piece piece_s;
    __shared__ int last_s;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int group = a.s.nq / a.s.nkv;
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(kfull + i, 128);
            mbar_init(kempty + i, 1);
            mbar_init(vfull + i, 128);
            mbar_init(vempty + i, 1);
            mbar_init(sfull + i, 1);
            mbar_init(pfull + i, 128);
            mbar_init(odone + i, 1);
        }
        mbar_init(qfull, G::SOFT);
        fence_barrier_init();
        piece_s.s = -1;
    }
    pdl_wait();
    pdl_launch_dependents();

    // the items of every sequence with more than few_rows rows; this CTA's piece of them
    {
        constexpr int T = G::THREADS;
        const int per = (a.n_seqs + T - 1) / T, s0 = min(tid * per, a.n_seqs), s1 = min(s0 + per, a.n_seqs);
        int run = 0;
        for (int s = s0; s < s1; ++s) {
            Kv4Seq q;
            kv4_seq(a, s, q);                          // out of range: no rows (the other kernel reports it)
            const int rows = q.n * group;
            if (rows > few_rows) run += a.s.nkv * ((rows + G::ROWS - 1) / G::ROWS);
        }
        int inc = run;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, inc, d);
            if (lane >= d) inc += o;
        }
        if (lane == 31) wsum[warp] = inc;
        __syncthreads();
        int base = inc - run, items = 0;
        for (int w = 0; w < T / 32; ++w) {
            if (w < warp) base += wsum[w];
            items += wsum[w];
        }
        const int splits = items ? max(1, min(num_sms / items, 32)) : 1;
        const int item = (int)blockIdx.x / splits, split = (int)blockIdx.x - item * splits;
        if (item >= base && item < base + run) {
            for (int s = s0; s < s1; ++s) {
                Kv4Seq q;
                kv4_seq(a, s, q);
                const int rows = q.n * group;
                if (rows <= few_rows) continue;
                const int qts = (rows + G::ROWS - 1) / G::ROWS, mine = a.s.nkv * qts;
                if (item < base + mine) {
                    // the last rows see the most positions: they start first
                    const int x = item - base, qt = qts - 1 - x / a.s.nkv;
                    Piece p;
                    p.s = s;
                    p.g = x % a.s.nkv;
                    p.row0 = qt * G::ROWS;
                    p.q0 = q.q0;
                    p.n = q.n;
                    p.len = q.len;
                    const int last_tok = min(p.row0 + G::ROWS, rows) - 1;
                    const int end = min(q.len, q.len - q.n + last_tok / group + 1);
                    const int nch = end > 0 ? (end + KC - 1) / KC : 0;
                    p.splits = max(1, min(splits, nch / 4));       // four chunks to a split at least
                    p.split = split;
                    p.c0 = (int)((long long)nch * split / p.splits);
                    p.c1 = (int)((long long)nch * (split + 1) / p.splits);
                    p.item = item;
                    if (split < p.splits) piece_s = p;
                    break;
                }
                base += mine;
            }
        }
        __syncthreads();
    }
    const Piece p = piece_s;
    if (p.s < 0) return;
    if (warp == 0) tmem_alloc(tslot, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tslot;
    const int32_t* table = a.table + (size_t)p.s * a.s.width;
    const int rows = min(G::ROWS, p.n * group - p.row0);
    const int nact = (rows + 127) / 128;
    bool ok = true;

    if (warp < 4 * NT) {
        // ----------------------------------------------------------------- softmax
        const int x = tid >> 7, t = tid & 127;
        const int row = p.row0 + tid, tok = row / group, h = p.g * group + row - tok * group;
        const bool live = tid < rows;
        const int lim = live ? p.len - p.n + tok + 1 : 0;
        const int lim_min = p.len - p.n + (p.row0 + (tid & ~31)) / group + 1;    // the warp's first row's
        const size_t qat = (size_t)(p.q0 + tok) * a.q_stride + (size_t)h * HD;
        float fac;
        {
            float big = 0.f;
            if (live)
                for (int d = 0; d < HD; d += 8) {
                    float v[8];
                    kv4_load8(a.q, qat + d, a.q_t, v);
#pragma unroll
                    for (int i = 0; i < 8; ++i) big = fmaxf(big, fabsf(v[i]));
                }
            const int e = kv4_exponent(big);
            fac = ldexpf(a.scale * 1.4426950408889634f * a.c.kg[p.g], e);
            const float sign = fac < 0.f ? -1.f : 1.f;             // z's largest is s's largest then
            fac = fabsf(fac);
            uint8_t* qs = sm + G::Q + x * TERMS * G::QT;
            for (int d = 0; d < HD; d += 8) {
                float v[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = 0.f;
                if (live) kv4_load8(a.q, qat + d, a.q_t, v);
                uint32_t hi[4], lo[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    kv4_split(ldexpf(v[2 * i], -e) * sign, ldexpf(v[2 * i + 1], -e) * sign, hi[i], lo[i]);
                uint8_t* at = qs + (d >> 6) * 16384 + sw128_offset(t, d & 63);
                *reinterpret_cast<uint4*>(at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                if (TERMS == 2) *reinterpret_cast<uint4*>(at + G::QT) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
            }
            fence_proxy_async();
            mbar_arrive(qfull);
        }
        float m = -INFINITY, l = 0.f;
        const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
        const uint32_t tO = tmem + lanes + 256 + x * HD;
        // which 16-position runs of a chunk have a page: one bit each
        auto pages_of = [&](int c) {
            const int pos = c * KC + 16 * lane;
            bool good = true;
            if (lane < KC / 16 && pos < p.len) {
                const int pg = table[pos / a.s.page];
                good = pg >= 0 && pg < a.s.n_pages;
                if (!good) atomicExch(a.status, ST_DEVICE_CHECK);
            }
            return __ballot_sync(0xffffffffu, good);
        };
        if (x < nact) {
            uint32_t good = p.c0 < p.c1 ? pages_of(p.c0) : 0u;
            for (int c = p.c0; c < p.c1; ++c) {
                const int i = c - p.c0;
                const int slot = NT == 2 ? x : i & 1;
                const uint32_t par = NT == 2 ? i & 1 : (i >> 1) & 1;
                const uint32_t tS = tmem + lanes + slot * 128;
                const bool edge = (c + 1) * KC > lim_min || good != 0xffffffffu;
                const uint32_t good_c = good;
                if (c + 1 < p.c1) good = pages_of(c + 1);
                if (!warp_wait(sfull + slot, par)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                auto largest = [&](auto masked) {
                    float mx = -INFINITY;
#pragma unroll
                    for (int b = 0; b < KC; b += 32) {
                        uint32_t s[32];
                        tmem_ld32(tS + b, s);
#pragma unroll
                        for (int k = 0; k < 32; ++k) {
                            const bool see = !masked || (c * KC + b + k < lim && ((good_c >> ((b + k) >> 4)) & 1));
                            if (see) mx = fmaxf(mx, __uint_as_float(s[k]));
                        }
                    }
                    return mx > -INFINITY ? mx * fac : -INFINITY;
                };
                const float mx = edge ? largest(std::true_type{}) : largest(std::false_type{});
                if (__any_sync(0xffffffffu, mx > m + KV4_P_SLACK)) {
                    const float mn = fmaxf(m, mx);
                    const float f = m == -INFINITY ? 0.f : kv4_ex2(m - mn);
                    l *= f;
                    m = mn;
                    if (i) {
                        if (NT == 1 && !warp_wait(odone + ((i - 1) & 1), ((i - 1) >> 1) & 1)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        for (int d = 0; d < HD; d += 32) {
                            uint32_t o[32];
                            tmem_ld32(tO + d, o);
#pragma unroll
                            for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
                            tmem_st16(tO + d, o);
                            tmem_st16(tO + d + 16, o + 16);
                        }
                        tmem_st_wait();
                    }
                }
                const float base = m == -INFINITY ? 0.f : m - KV4_P_UP;
                auto weights = [&](auto masked) {
                    uint32_t lo_all[TERMS == 2 ? KC / 2 : 1];
#pragma unroll
                    for (int b = 0; b < KC; b += 32) {
                        uint32_t s[32], hi[16];
                        tmem_ld32(tS + b, s);
#pragma unroll
                        for (int k = 0; k < 32; k += 2) {
                            float p0 = kv4_ex2(fmaf(__uint_as_float(s[k]), fac, -base));
                            float p1 = kv4_ex2(fmaf(__uint_as_float(s[k + 1]), fac, -base));
                            if (masked) {
                                const int at = c * KC + b + k;
                                const bool run = (good_c >> ((b + k) >> 4)) & 1;
                                if (!run || at >= lim) p0 = 0.f;
                                if (!run || at + 1 >= lim) p1 = 0.f;
                            }
                            l += p0 + p1;
                            if (TERMS == 2) kv4_split(p0, p1, hi[k / 2], lo_all[(b + k) / 2]);
                            else hi[k / 2] = kv4_pack(p0, p1);
                        }
                        tmem_st16(tS + b / 2, hi);
                    }
                    if (TERMS == 2) {                  // over columns of S that are all read by now
#pragma unroll
                        for (int b = 0; b < KC / 2; b += 16) tmem_st16(tS + KC / 2 + b, lo_all + b);
                    }
                };
                if (edge) weights(std::true_type{});
                else weights(std::false_type{});
                tmem_st_wait();
                tc_fence_before();
                mbar_arrive(pfull + slot);
            }
        }
        // O, joined with the item's other parts where it was split
        const int nc = p.c1 - p.c0;
        // S of the last chunk came after the second but last product of its slot, so the phase waited for
        // here is that barrier's current one or the one just completed
        const int lc = nc - 1;
        if (ok && x < nact && nc && !warp_wait(odone + (NT == 2 ? x : lc & 1), (NT == 2 ? lc : lc >> 1) & 1)) ok = false;
        tc_fence_after();
        bool write = ok && live;
        const float vg = a.c.vg[p.g];
        const size_t oat = (size_t)(p.q0 + tok) * a.out_stride + (size_t)h * HD;
        if (p.splits == 1) {
            const float inv = l == 0.f ? 0.f : vg / l;
            for (int d = 0; d < HD && x < nact; d += 32) {
                uint32_t o[32];
                if (nc) tmem_ld32(tO + d, o);
#pragma unroll
                for (int k = 0; k < 32; k += 8) {
                    float v[8];
#pragma unroll
                    for (int y = 0; y < 8; ++y) v[y] = nc && l != 0.f ? __uint_as_float(o[k + y]) * inv : 0.f;
                    if (write) kv4_store8(a.out, oat + d + k, a.out_t, v);
                }
            }
        } else {
            // part: O as float4 [HD/4][ROWS], then m, l [ROWS]
            float* part = parts + (size_t)blockIdx.x * G::PART;
            for (int d = 0; d < HD && x < nact; d += 32) {
                uint32_t o[32];
                tmem_ld32(tO + d, o);
#pragma unroll
                for (int k = 0; k < 32; k += 4)
                    reinterpret_cast<float4*>(part)[(size_t)((d + k) / 4) * G::ROWS + tid] =
                        make_float4(__uint_as_float(o[k]), __uint_as_float(o[k + 1]), __uint_as_float(o[k + 2]),
                                    __uint_as_float(o[k + 3]));
            }
            part[(size_t)HD * G::ROWS + tid] = m;
            part[(size_t)(HD + 1) * G::ROWS + tid] = l;
            __threadfence();
            named_bar(1, G::SOFT);
            if (tid == 0) last_s = atomicAdd(arrive + p.item, 1u) == (unsigned)(p.splits - 1);
            named_bar(1, G::SOFT);
            if (last_s) {
                __threadfence();
                if (tid == 0) arrive[p.item] = 0u;
                const float* first = parts + (size_t)((int)blockIdx.x - p.split) * G::PART;
                m = -INFINITY;
                l = 0.f;
                for (int i = 0; i < p.splits; ++i)
                    m = fmaxf(m, __ldcg(first + (size_t)i * G::PART + (size_t)HD * G::ROWS + tid));
                auto weight = [&](int i, float& li) {
                    const float* pi = first + (size_t)i * G::PART + (size_t)HD * G::ROWS + tid;
                    li = __ldcg(pi + G::ROWS);
                    return li == 0.f ? 0.f : kv4_ex2(__ldcg(pi) - m);
                };
                for (int i = 0; i < p.splits; ++i) {
                    float li;
                    const float w = weight(i, li);
                    l += li * w;
                }
                const float inv = l == 0.f ? 0.f : vg / l;
                for (int d = 0; d < HD; d += 32) {
                    float v[32];
#pragma unroll
                    for (int y = 0; y < 32; ++y) v[y] = 0.f;
                    for (int i = 0; i < p.splits; ++i) {
                        float li;
                        const float w = weight(i, li);
                        if (li == 0.f) continue;
                        const float4* pi = reinterpret_cast<const float4*>(first + (size_t)i * G::PART) +
                                           (size_t)(d / 4) * G::ROWS + tid;
#pragma unroll
                        for (int y = 0; y < 8; ++y) {
                            const float4 u = __ldcg(pi + (size_t)y * G::ROWS);
                            v[4 * y] += u.x * w;
                            v[4 * y + 1] += u.y * w;
                            v[4 * y + 2] += u.z * w;
                            v[4 * y + 3] += u.w * w;
                        }
                    }
#pragma unroll
                    for (int y = 0; y < 32; ++y) v[y] *= inv;
#pragma unroll
                    for (int y = 0; y < 32; y += 8)
                        if (write) kv4_store8(a.out, oat + d + y, a.out_t, v + y);
                }
            } else {
                write = false;
            }
        }
        if (write && a.lse)
            a.lse[(size_t)(p.q0 + tok) * a.s.nq + h] =
                l == 0.f ? -INFINITY : (m - KV4_P_UP + log2f(l)) * 0.6931471805599453f;
    } else if (warp < 4 * NT + 4) {
        // ----------------------------------------------------------------- K
        const int kt = tid - G::SOFT, jj = kt % G::LPR, r0 = kt / G::LPR;
        const int rot = G::LPR == 4 ? jj & 2 : G::LPR == 8 ? jj >> 1 : 0;   // quarter-warps store to eight banks groups
        auto page_ids = [&](int c, int (&id)[G::KP]) {
#pragma unroll
            for (int i = 0; i < G::KP; ++i) {
                const int pos = c * KC + i * G::RPP + r0;
                id[i] = c < p.c1 && pos < p.len ? table[pos / a.s.page] : -1;
            }
        };
        auto load = [&](int c, const int (&id)[G::KP], uint4 (&w)[G::KP], uint32_t (&sc)[G::KP]) {
#pragma unroll
            for (int i = 0; i < G::KP; ++i) {
                w[i] = make_uint4(0, 0, 0, 0);
                sc[i] = 0;
                if (id[i] >= 0 && id[i] < a.s.n_pages) {
                    const int pos = c * KC + i * G::RPP + r0;
                    const size_t at = ((size_t)id[i] * a.s.nkv + p.g) * a.s.page + (pos & (a.s.page - 1));
                    w[i] = __ldg(reinterpret_cast<const uint4*>(a.c.kc + at * (HD / 2) + jj * 16));
                    sc[i] = __ldg(reinterpret_cast<const uint16_t*>(a.c.ks + at * (HD / 16) + jj * 2));
                }
            }
        };
        int id[G::KP];
        uint4 w[G::KP];
        uint32_t sc[G::KP];
        page_ids(p.c0, id);
        load(p.c0, id, w, sc);
        page_ids(p.c0 + 1, id);
        for (int c = p.c0; c < p.c1; ++c) {
            uint4 wn[G::KP];
            uint32_t sn[G::KP];
            load(c + 1, id, wn, sn);
            page_ids(c + 2, id);
            const int i0 = c - p.c0, b = i0 % BUF, use = i0 / BUF;
            if (use && !mbar_wait(kempty + b, (use - 1) & 1)) {
                ok = false;
                break;
            }
            uint8_t* tile = sm + G::K + b * G::KT + (jj >> 1) * (KC * 128);
#pragma unroll
            for (int i = 0; i < G::KP; ++i) {
                const int row = i * G::RPP + r0;
                const __half2 both = kv4_scale2(sc[i]), s0 = __low2half2(both), s1 = __high2half2(both);
                uint32_t x0 = w[i].x, x1 = w[i].y, x2 = w[i].z, x3 = w[i].w;
                if (rot & 2) {
                    const uint32_t y0 = x0, y1 = x1;
                    x0 = x2;
                    x1 = x3;
                    x2 = y0;
                    x3 = y1;
                }
                if (rot & 1) {
                    const uint32_t y0 = x0;
                    x0 = x1;
                    x1 = x2;
                    x2 = x3;
                    x3 = y0;
                }
                const uint32_t xs[4] = {x0, x1, x2, x3};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int kk = (k + rot) & 3;
                    const __half2 s = kk & 2 ? s1 : s0;
                    __half2 e[4];
                    kv4_widen8(xs[k], e);
                    *reinterpret_cast<uint4*>(tile + sw128_offset(row, ((jj & 1) * 4 + kk) * 8)) =
                        make_uint4(kv4_u(__hmul2(e[0], s)), kv4_u(__hmul2(e[1], s)), kv4_u(__hmul2(e[2], s)), kv4_u(__hmul2(e[3], s)));
                }
            }
            fence_proxy_async();
            mbar_arrive(kfull + b);
#pragma unroll
            for (int i = 0; i < G::KP; ++i) {
                w[i] = wn[i];
                sc[i] = sn[i];
            }
        }
    } else if (warp < 4 * NT + 8) {
        // ----------------------------------------------------------------- V
        const int vt = tid - G::SOFT - 128, pg8 = vt & 7, dg = (vt >> 3) % (HD / 16), kb = (vt >> 3) / (HD / 16);
        const bool work = kb < KC / 64;
        const int p0 = kb * 64 + pg8 * 8;              // eight positions, sixteen elements of each
        auto page_id = [&](int c) {
            const int pos = c * KC + p0;
            return work && c < p.c1 && pos < p.len ? table[pos / a.s.page] : -1;
        };
        auto load = [&](int c, int id, uint2 (&w)[8], uint32_t (&sc)[8]) {
            const bool there = id >= 0 && id < a.s.n_pages;
            const int pos = c * KC + p0;
            const size_t at = there ? ((size_t)id * a.s.nkv + p.g) * a.s.page + (pos & (a.s.page - 1)) : 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                // behind the last position the bytes may decode to NaN, which weight 0 would keep
                w[i] = make_uint2(0, 0);
                sc[i] = 0;
                if (there && pos + i < p.len) {
                    w[i] = __ldg(reinterpret_cast<const uint2*>(a.c.vc + (at + i) * (HD / 2) + dg * 8));
                    sc[i] = __ldg(a.c.vs + (at + i) * (HD / 16) + dg);
                }
            }
        };
        uint2 w[8];
        uint32_t sc[8];
        int id = page_id(p.c0);
        load(p.c0, id, w, sc);
        id = page_id(p.c0 + 1);
        for (int c = p.c0; c < p.c1; ++c) {
            uint2 wn[8];
            uint32_t sn[8];
            load(c + 1, id, wn, sn);
            id = page_id(c + 2);
            const int i0 = c - p.c0, b = i0 % BUF, use = i0 / BUF;
            if (use && !mbar_wait(vempty + b, (use - 1) & 1)) {
                ok = false;
                break;
            }
            if (work) {
                uint8_t* tile = sm + G::V + b * G::KT + kb * (HD * 128);
                __half2 s[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) s[i] = kv4_scale2(kv4_bytes(sc[2 * i], sc[2 * i + 1]));
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    uint32_t pr[4][2];                 // bytes of one element of two positions: even, odd
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        kv4_pair(y ? w[2 * i].y : w[2 * i].x, y ? w[2 * i + 1].y : w[2 * i + 1].x, pr[i][0], pr[i][1]);
#pragma unroll
                    for (int odd = 0; odd < 2; ++odd) {
                        __half2 v[4][4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) kv4_widen8(pr[i][odd], v[i]);
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            *reinterpret_cast<uint4*>(tile + sw128_offset(dg * 16 + y * 8 + 2 * e + odd, pg8 * 8)) =
                                make_uint4(kv4_u(__hmul2(v[0][e], s[0])), kv4_u(__hmul2(v[1][e], s[1])),
                                           kv4_u(__hmul2(v[2][e], s[2])), kv4_u(__hmul2(v[3][e], s[3])));
                    }
                }
            }
            fence_proxy_async();
            mbar_arrive(vfull + b);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                w[i] = wn[i];
                sc[i] = sn[i];
            }
        }
    } else if (lane == 0) {
        // ----------------------------------------------------------------- MMA
        const int nc = p.c1 - p.c0;
        const uint32_t idS = umma_idesc_f16(128, KC), idO = umma_idesc_f16(128, HD);
        auto issue_s = [&](int x, int slot, int i) {   // S of tile x, chunk i, into the slot
            const int b = i % BUF;
#pragma unroll
            for (int tm = 0; tm < TERMS; ++tm)
#pragma unroll
                for (int ks = 0; ks < HD / 16; ++ks) {
                    const uint64_t ad = umma_sdesc(smem_u32(sm + G::Q + (x * TERMS + tm) * G::QT + (ks >> 2) * 16384)) + 2 * (ks & 3);
                    const uint64_t bd = umma_sdesc(smem_u32(sm + G::K + b * G::KT + (ks >> 2) * (KC * 128))) + 2 * (ks & 3);
                    umma_f16(tmem + slot * 128, ad, bd, idS, tm | ks);
                }
            umma_commit(sfull + slot);
        };
        auto issue_pv = [&](int x, int slot, int i) {
            const int b = i % BUF;
#pragma unroll
            for (int tm = 0; tm < TERMS; ++tm)
#pragma unroll
                for (int ks = 0; ks < KC / 16; ++ks) {
                    const uint64_t bd = umma_sdesc(smem_u32(sm + G::V + b * G::KT + (ks >> 2) * (HD * 128))) + 2 * (ks & 3);
                    umma_f16_ta(tmem + 256 + x * HD, tmem + slot * 128 + tm * (KC / 2) + ks * 8, bd, idO, (uint32_t)(i | tm | ks));
                }
            umma_commit(odone + slot);
        };
        auto wait_k = [&](int i) { return mbar_wait(kfull + i % BUF, (i / BUF) & 1); };
        ok = mbar_wait(qfull, 0);
        tc_fence_after();
        if (NT == 2) {
            if (ok && nc) ok = wait_k(0);
            tc_fence_after();
            for (int x = 0; ok && nc && x < nact; ++x) issue_s(x, x, 0);
            if (ok && nc) umma_commit(kempty);
            for (int i = 0; ok && i < nc; ++i) {
                ok = mbar_wait(vfull + i % BUF, (i / BUF) & 1);
                for (int x = 0; ok && x < nact; ++x) {
                    ok = mbar_wait(pfull + x, i & 1);
                    if (!ok) break;
                    tc_fence_after();
                    issue_pv(x, x, i);
                    if (x == nact - 1) umma_commit(vempty + i % BUF);
                    if (i + 1 < nc) {
                        if (x == 0) ok = wait_k(i + 1);
                        if (!ok) break;
                        tc_fence_after();
                        issue_s(x, x, i + 1);
                        if (x == nact - 1) umma_commit(kempty + (i + 1) % BUF);
                    }
                }
            }
        } else {
            for (int i = 0; ok && i < nc && i < 2; ++i) {
                ok = wait_k(i);
                if (!ok) break;
                tc_fence_after();
                issue_s(0, i, i);
                umma_commit(kempty + i % BUF);
            }
            for (int i = 0; ok && i < nc; ++i) {
                ok = mbar_wait(vfull + i % BUF, (i / BUF) & 1) && mbar_wait(pfull + (i & 1), (i >> 1) & 1);
                if (!ok) break;
                tc_fence_after();
                issue_pv(0, i & 1, i);
                umma_commit(vempty + i % BUF);
                if (i + 2 < nc) {
                    ok = wait_k(i + 2);
                    if (!ok) break;
                    tc_fence_after();
                    issue_s(0, i & 1, i + 2);
                    umma_commit(kempty + (i + 2) % BUF);
                }
            }
        }
    }
    if (!ok) atomicExch(a.status, ST_TIMEOUT);
    tc_fence_before();
    __syncthreads();
    if (warp == 0) tmem_dealloc(tmem, 512);
}

template <int HD, int TERMS>
cudaError_t launch_extend(const Kv4AttnArgs& a, int few_rows, const Kv4Work& w, cudaStream_t st) {
    using G = EGeo<HD, TERMS>;
    static_assert(G::SMEM <= 227 * 1024, "one CTA's shared memory");
    const cudaError_t e = cudaFuncSetAttribute(kv4_extend_kernel<HD, TERMS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               (int)G::SMEM);
    if (e != cudaSuccess) return e;
    // items: whole tiles of rows, and one that is not whole per sequence with enough rows
    const long long rows = (long long)a.n_tokens * (a.s.nq / a.s.nkv);
    const long long ragged = rows / (few_rows + 1) < a.n_seqs ? rows / (few_rows + 1) : a.n_seqs;
    long long grid = a.s.nkv * (rows / G::ROWS + ragged);
    if (grid < w.num_sms) grid = w.num_sms;
    return launch_pdl(kv4_extend_kernel<HD, TERMS>, dim3((unsigned)grid), dim3(G::THREADS), G::SMEM, st, a, few_rows,
                      w.parts, w.arrive, w.num_sms);
}

}  // namespace

// a split item's parts: at most one CTA a multiprocessor
size_t kv4_extend_part_floats(int hd, int num_sms) {
    const size_t rows = hd <= 128 ? 256 : 128;
    return (size_t)num_sms * rows * (hd + 2);
}

cudaError_t launch_kv4_extend(const Kv4AttnArgs& a, int few_rows, const Kv4Work& w, cudaStream_t st) {
    const bool two = a.q_t == KV4_F32;
    switch (a.s.hd) {
        case 64: return two ? launch_extend<64, 2>(a, few_rows, w, st) : launch_extend<64, 1>(a, few_rows, w, st);
        case 128: return two ? launch_extend<128, 2>(a, few_rows, w, st) : launch_extend<128, 1>(a, few_rows, w, st);
        default: return two ? launch_extend<256, 2>(a, few_rows, w, st) : launch_extend<256, 1>(a, few_rows, w, st);
    }
}

}  // namespace qmoe
