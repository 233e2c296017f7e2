// kv4_extend.cu -- attention over the paged 4-bit cache for sequences that bring many
// tokens (prompt chunks): bound by the two matrix products and the exponentials.
//
// An item is (sequence, kv head, 128 NT rows of (token, head of the group)); a CTA
// walks its visible positions in chunks of KC, and its softmax in steps of 64.  Its
// warps have roles:
//   softmax  4 warps per 128 rows, a thread to a row (its TMEM lane): z of a step from
//            TMEM, running maximum m and sum l, p = 2^(z - m) back into TMEM as fp16
//   K, V     3 and 4 warps: codes from the cache, widened (exactly) to fp16 into
//            128B-swizzled K-major tiles, V transposed so that positions are K
//   MMA      one thread: S = Q K^T and O += P V^T, tcgen05, P read from TMEM
// With NT = 2 two 128-row tiles share every widened K and V tile (the widening costs
// as many issue slots as one tile's softmax); with NT = 1 (F32 rows, head_dim 256)
// shared memory has no room for two.
// Every tile has two S slots of 64 columns, so the next step's S is there when a step's
// softmax ends: with one slot a step waited for its own two products, which took
// longer than its softmax.  P overlays the S it came from; the next S into the slot is
// issued after the product that reads P and runs after it.
// O is rescaled only when a row's maximum rose by 2^8 since the last time.
// F32 rows: q = hi + lo and p = hi + lo, two products each (TERMS = 2).
// Few items: the chunks of an item are split over CTAs, the last one joins the parts.
#include <math.h>

#include "kv4.cuh"
#include "kv4_row.cuh"
#include "umma.cuh"

namespace qmoe {

namespace {

constexpr int EXTEND_PARTS = 2;                                      // parts of split items, a multiprocessor
constexpr int SC = 64;                                               // positions of a softmax step

template <int HD, int TERMS>
struct EGeo {
    static constexpr int NT = HD <= 128 && TERMS == 1 ? 2 : 1;       // 128-row tiles
    static constexpr int KC = HD == 256 ? 64 : 128;                  // positions of a chunk
    static constexpr int SPC = KC / SC;                              // steps of a chunk
    static constexpr int BUF = HD == 256 && TERMS == 2 ? 1 : 2;      // K and V tiles in shared memory
    static constexpr int ROWS = 128 * NT;
    static constexpr int SOFT = 128 * NT;                            // softmax threads, then K's, V's and MMA's
    static constexpr int KTH = 96, VTH = 128, THREADS = SOFT + KTH + VTH + 32;
    static constexpr int QT = 128 * HD * 2, KT = KC * HD * 2;        // bytes of a tile
    static constexpr int Q = 0, K = NT * TERMS * QT, V = K + BUF * KT, BARS = V + BUF * KT;
    static constexpr size_t SMEM = 1024 + BARS + 256;
    static constexpr int LPR = HD / 32;                              // 16-byte runs of a position's codes
    static constexpr int RPP = KTH / LPR;                            // positions the K threads take at a time
    static constexpr int KP = (KC + RPP - 1) / RPP;
    static constexpr int PART = ROWS * (HD + 2);                     // floats of a part
    static_assert(33 * ROWS * 4 <= 2 * BUF * KT, "the weights of a join take the buffers of K and V");
};

// The MMA warp runs its loop as a whole, so that descriptors and addresses stay in
// uniform registers; only the instructions themselves are one lane's (`one`; a branch
// around them took the operands through lane registers, twice the time a product).
// Descriptors change in their low words alone (addresses in units of 16 bytes).
__device__ __forceinline__ uint32_t elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p;
}

// D[tmem] = A[shared] * B^T, or += it
template <int ADD>
__device__ __forceinline__ void mma_ss(uint32_t one, uint32_t d, uint32_t a, uint32_t b, uint32_t high, uint32_t idesc) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b64 x, y;\n\tsetp.ne.u32 p, %5, 0;\n\tsetp.ne.u32 q, %6, 0;\n\tmov.b64 x, {%1, %3};\n\tmov.b64 y, {%2, %3};\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %4, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(high), "r"(idesc), "n"(ADD), "r"(one)
        : "memory");
}

// D[tmem] (+)= A[tmem] * B^T
__device__ __forceinline__ void mma_ts(uint32_t one, uint32_t d, uint32_t a, uint32_t b, uint32_t high, uint32_t idesc, uint32_t add) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b64 y;\n\tsetp.ne.u32 p, %5, 0;\n\tsetp.ne.u32 q, %6, 0;\n\tmov.b64 y, {%2, %3};\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %4, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(high), "r"(idesc), "r"(add), "r"(one)
        : "memory");
}

// one arrival on the barrier at this shared address once the products issued so far are done
__device__ __forceinline__ void mma_commit(uint32_t one, uint32_t bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar), "r"(one)
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

// the same without the wait: the values are there after tmem_ld_wait
__device__ __forceinline__ void tmem_ld32_start(uint32_t t, uint32_t* r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(t)
        : "memory");
}
__device__ __forceinline__ void tmem_ld_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void tmem_st32(uint32_t t, const uint32_t* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
        "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(t),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
        "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
        "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}

__device__ __forceinline__ void tmem_st16(uint32_t t, const uint32_t* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(t),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

// two fp32 values at a time
__device__ __forceinline__ unsigned long long pair64(uint32_t x, uint32_t y) {
    unsigned long long d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(x), "r"(y));
    return d;
}
__device__ __forceinline__ void unpair64(unsigned long long d, float& x, float& y) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(d));
}
__device__ __forceinline__ unsigned long long fma2(unsigned long long a, unsigned long long b, unsigned long long c) {
    unsigned long long d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ unsigned long long add2(unsigned long long a, unsigned long long b) {
    unsigned long long d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
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
    int split, splits;
    int part;                // the item's first part in the workspace; its arrival counter
};

template <int HD, int TERMS>
__global__ void __launch_bounds__(EGeo<HD, TERMS>::THREADS, 1)
    kv4_extend_kernel(const Kv4AttnArgs a, int few_rows, float* __restrict__ parts, unsigned* __restrict__ arrive,
                      int num_sms, int max_parts) {
    using G = EGeo<HD, TERMS>;
    constexpr int NT = G::NT, KC = G::KC, BUF = G::BUF;
    extern __shared__ __align__(1024) uint8_t smraw[];
    uint8_t* sm = smraw + ((1024u - (smem_u32(smraw) & 1023u)) & 1023u);
    uint64_t* bars = reinterpret_cast<uint64_t*>(sm + G::BARS);
    // by buffer: kfull .. vempty; by tile and slot: sfull .. odone
    uint64_t *kfull = bars, *kempty = bars + 2, *vfull = bars + 4, *vempty = bars + 6, *sfull = bars + 8,
             *pfull = bars + 12, *odone = bars + 16, *qfull = bars + 20;
    uint32_t* tslot = reinterpret_cast<uint32_t*>(bars + 21);
    __shared__ int wsum[G::THREADS / 32];
    __shared__ Piece piece_s;
    __shared__ int last_s;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int group = a.s.nq / a.s.nkv;
    if (tid == 0) piece_s.s = -1;
    pdl_wait();
    pdl_launch_dependents();

    // the items of every sequence with more than few_rows rows, and this CTA's piece of them.  An item's
    // chunks are split where it has more than the GPU's average share of a multiprocessor.
    {
        constexpr int T = G::THREADS;
        const int per = (a.n_seqs + T - 1) / T, s0 = min(tid * per, a.n_seqs), s1 = min(s0 + per, a.n_seqs);
        struct Seq {
            Kv4Seq q;
            int rows, qts, last;               // row tiles, chunks of the last of them
        };
        auto chunks = [&](const Kv4Seq& q, int row_end) {          // that rows up to row_end see
            const int end = min(q.len, q.len - q.n + (row_end - 1) / group + 1);
            return end > 0 ? (end + KC - 1) / KC : 0;
        };
        auto seq = [&](int s, Seq& r) {
            kv4_seq(a, s, r.q);                        // out of range: no rows (the other kernel reports it)
            r.rows = r.q.n * group;
            r.qts = r.rows > few_rows ? (r.rows + G::ROWS - 1) / G::ROWS : 0;
            r.last = r.qts ? chunks(r.q, r.rows) : 0;
        };
        auto block_sum = [&](int v, int& before) {     // sum over the CTA, and over the threads before
            int inc = v;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int o = __shfl_up_sync(0xffffffffu, inc, d);
                if (lane >= d) inc += o;
            }
            __syncthreads();
            if (lane == 31) wsum[warp] = inc;
            __syncthreads();
            int all = 0;
            before = inc - v;
            for (int w = 0; w < T / 32; ++w) {
                if (w < warp) before += wsum[w];
                all += wsum[w];
            }
            return all;
        };
        // total chunks, a sequence's tiles taken as evenly spread between its first and last
        // (as far as 2^18 a sequence: it only sets the share)
        int work = 0, pieces = 0, parts_n = 0, base, part0, unused;
        bool descends = false;
        for (int s = s0; s < s1; ++s) {
            Seq r;
            seq(s, r);
            descends |= a.cu[s + 1] < a.cu[s];
            const float both = (float)r.last + (float)chunks(r.q, min(r.rows, (int)G::ROWS));
            if (r.qts) work += (int)fminf(0.5f * (float)a.s.nkv * (float)r.qts * both, 262144.f);
        }
        if (__syncthreads_or(descends)) return;        // rows of several sequences (the other kernel reports it)
        work = block_sum(work, unused);
        const int share = max(8, (int)(1.25f * (float)work / (float)num_sms) + 1);   // pieces fill one wave
        auto splits_of = [&](const Seq& r) { return min(32, max(1, (r.last + share - 1) / share)); };
        for (int s = s0; s < s1; ++s) {
            Seq r;
            seq(s, r);
            const int k = splits_of(r), items = a.s.nkv * r.qts;
            pieces += items * k;
            if (k > 1) parts_n += items * k;
        }
        const int all = block_sum(pieces, base), all_parts = block_sum(parts_n, part0);
        // not more CTAs or parts than there are: every item whole then
        const bool whole = all > (int)gridDim.x || all_parts > max_parts;
        if (whole) {
            pieces = 0;
            for (int s = s0; s < s1; ++s) {
                Seq r;
                seq(s, r);
                pieces += a.s.nkv * r.qts;
            }
            block_sum(pieces, base);
        }
        const int me = blockIdx.x;
        if (me >= base && me < base + pieces) {
            for (int s = s0; s < s1; ++s) {
                Seq r;
                seq(s, r);
                const int k = whole ? 1 : splits_of(r), mine = a.s.nkv * r.qts * k;
                if (me < base + mine) {
                    // the last rows see the most positions: they start first
                    const int at = me - base, split = at % k, item = at / k, qt = r.qts - 1 - item / a.s.nkv;
                    Piece p;
                    p.s = s;
                    p.g = item % a.s.nkv;
                    p.row0 = qt * G::ROWS;
                    p.q0 = r.q.q0;
                    p.n = r.q.n;
                    p.len = r.q.len;
                    const int nch = chunks(r.q, min(p.row0 + G::ROWS, r.rows));
                    p.splits = max(1, min(k, nch / 4));            // four chunks to a split at least
                    p.split = split;
                    p.c0 = (int)((long long)nch * split / p.splits);
                    p.c1 = (int)((long long)nch * (split + 1) / p.splits);
                    p.part = part0 + item * k;
                    if (split < p.splits) piece_s = p;
                    break;
                }
                base += mine;
                if (k > 1) part0 += mine;
            }
        }
        __syncthreads();
    }
    const Piece& p = piece_s;                          // read where it is used: registers are scarce
    if (p.s < 0) return;
    const int32_t* table = a.table + (size_t)p.s * a.s.width;
    const int rows = min(G::ROWS, p.n * group - p.row0);
    const int nact = (rows + 127) / 128;               // tiles with rows
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(kfull + i, G::KTH);
            mbar_init(kempty + i, 1);
            mbar_init(vfull + i, G::VTH);
            mbar_init(vempty + i, 1);
        }
        for (int i = 0; i < 2 * NT; ++i) {
            mbar_init(sfull + i, 1);
            mbar_init(pfull + i, 128);
            mbar_init(odone + i, 1);
        }
        mbar_init(qfull, G::SOFT);
        fence_barrier_init();
    }
    if (warp == 0) tmem_alloc(tslot, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tslot;
    bool ok = true;

    if (warp < 4 * NT) {
        // ----------------------------------------------------------------- softmax
        const int x = tid >> 7, len = p.len;
        // token of the sequence and q head of a row of the item
        auto tok_of = [&](int row) { return (p.row0 + row) / group; };
        auto head_of = [&](int row, int tok) { return p.g * group + p.row0 + row - tok * group; };
        const int lim = tid < rows ? len - p.n + tok_of(tid) + 1 : 0;
        const int lim_min = len - p.n + tok_of(tid & ~31) + 1;                   // the warp's first row's
        float fac;
        {
            // the warp's 32 rows of q, 16 bytes a lane, copied to where their fp16 terms belong (F32
            // elements fill the places of both); then each thread scales its own row to [1, 2) by a
            // power of two and splits it in place
            constexpr int LR = HD / 8, RW = 32 / LR;   // lanes of a row, rows at a time
            const float fac0 = a.scale * 1.4426950408889634f * a.c.kg[p.g];
            uint8_t* qs = sm + G::Q + x * TERMS * G::QT;
            {
                const int d = (lane % LR) * 8, sub = lane / LR;
                long long mine = -1;                   // where this thread's row starts
                if (tid < rows) {
                    const int tok = tok_of(tid), h = head_of(tid, tok);
                    mine = ((long long)(p.q0 + tok) * a.q_stride + (long long)h * HD) * (TERMS == 2 ? 4 : 2);
                }
#pragma unroll 4
                for (int r = 0; r < 32; r += RW) {
                    const long long at = __shfl_sync(0xffffffffu, mine, r + sub);
                    uint8_t* to = qs + (d >> 6) * 16384 + sw128_offset((tid & 96) + r + sub, d & 63);
#pragma unroll
                    for (int z = 0; z < TERMS; ++z) {
                        if (at >= 0) cp_async_cg16(to + z * G::QT, static_cast<const uint8_t*>(a.q) + at + d * (TERMS == 2 ? 4 : 2) + 16 * z);
                        else *reinterpret_cast<uint4*>(to + z * G::QT) = make_uint4(0, 0, 0, 0);
                    }
                }
            }
            cp_async_wait_all();
            __syncwarp();
            int exponent = 0;
            auto load_q = [&](int d, float (&v)[8]) {
                const uint8_t* at = qs + (d >> 6) * 16384 + sw128_offset(tid & 127, d & 63);
                uint4 raw[TERMS];
#pragma unroll
                for (int z = 0; z < TERMS; ++z) raw[z] = *reinterpret_cast<const uint4*>(at + z * G::QT);
                kv4_floats8(raw, a.q_t, v);
            };
            if (TERMS == 2 || a.q_t != KV4_F16) {      // fp16 rows are what they have to be
                float big[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 2
                for (int d = 0; d < HD; d += 8) {
                    float v[8];
                    load_q(d, v);
#pragma unroll
                    for (int i = 0; i < 4; ++i) big[i] = max3(big[i], fabsf(v[i]), fabsf(v[4 + i]));
                }
                exponent = kv4_exponent(fmaxf(fmaxf(big[0], big[1]), fmaxf(big[2], big[3])));
            }
            if (TERMS == 2 || a.q_t != KV4_F16 || fac0 < 0.f) {
                const Kv4Scale un = kv4_unscale(exponent);
                const float ub = fac0 < 0.f ? -un.b : un.b;        // z's largest is q.k's largest then
#pragma unroll 2
                for (int d = 0; d < HD; d += 8) {
                    float v[8];
                    load_q(d, v);
                    uint32_t hi[4], lo[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float v0 = v[2 * i] * un.a * ub, v1 = v[2 * i + 1] * un.a * ub;
                        if (TERMS == 2) kv4_split(v0, v1, hi[i], lo[i]);
                        else hi[i] = kv4_pack(v0, v1);
                    }
                    uint8_t* at = qs + (d >> 6) * 16384 + sw128_offset(tid & 127, d & 63);
                    *reinterpret_cast<uint4*>(at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                    if (TERMS == 2) *reinterpret_cast<uint4*>(at + G::QT) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                }
            }
            fac = fmaxf(ldexpf(fabsf(fac0), exponent), 1e-38f);    // not 0: -inf stays -inf, and 1e-38 q.k is 0
            fence_proxy_async();
            mbar_arrive(qfull);
        }
        float m = -INFINITY, l = 0.f;
        const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
        const uint32_t tO = tmem + lanes + 256 + x * HD;
        const int ns = (p.c1 - p.c0) * G::SPC, first = p.c0 * KC;        // steps, their first position
        // which 16-position runs of a step have a page: one lane looks each up, a step ahead (at a
        // position of the sequence in any case: a load without a condition waits for nothing)
        auto run_page = [&](int step) {
            return table[min(first + step * SC + 16 * (lane & 3), len - 1) >> a.s.page_log2];
        };
        if (x < nact && ns) {
            int pg = run_page(0);
            for (int step = 0; step < ns; ++step) {
                const int slot = step & 1, bar = 2 * x + slot, pos = first + step * SC;
                const uint32_t tS = tmem + lanes + x * 128 + slot * 64;
                const bool there = pg >= 0 && pg < a.s.n_pages;
                const uint32_t good = __ballot_sync(0xffffffffu, there || pos + 16 * (lane & 3) >= len);
                const bool edge = pos + SC > lim_min || good != 0xffffffffu;
                if (good != 0xffffffffu && lane == 0) atomicExch(a.status, ST_DEVICE_CHECK);
                pg = run_page(step + 1);
                if (!warp_wait(sfull + bar, (step >> 1) & 1)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                uint32_t z[SC];
                tmem_ld32_start(tS, z);
                tmem_ld32_start(tS + 32, z + 32);
                tmem_ld_wait();
                if (edge) {
#pragma unroll
                    for (int k = 0; k < SC; ++k)
                        if (pos + k >= lim || !((good >> (k >> 4)) & 1)) z[k] = 0xff800000u;
                    asm volatile("");                  // a branch, not selects that run every time
                }
                float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int k = 0; k < SC; k += 8)
#pragma unroll
                    for (int y = 0; y < 4; ++y)
                        mx4[y] = max3(mx4[y], __uint_as_float(z[k + 2 * y]), __uint_as_float(z[k + 2 * y + 1]));
                const float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3])) * fac;
                if (__any_sync(0xffffffffu, mx > m + KV4_P_SLACK)) {
                    const float mn = fmaxf(m, mx);
                    const float f = m == -INFINITY ? 0.f : kv4_ex2(m - mn);
                    l *= f;
                    m = mn;
                    if (step) {
                        // S of this step came after the product before the last one
                        if (!warp_wait(odone + (bar ^ 1), ((step - 1) >> 1) & 1)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
#pragma unroll 1
                        for (int d = 0; d < HD; d += 16) {         // small blocks: z stays in its registers
                            float o[16];
                            tmem_ld16(tO + d, o);
                            uint32_t u[16];
#pragma unroll
                            for (int k = 0; k < 16; ++k) u[k] = __float_as_uint(o[k] * f);
                            tmem_st16(tO + d, u);
                        }
                    }
                }
                const float base = m == -INFINITY ? 0.f : m - KV4_P_UP;
                // p over the z that made it
                const unsigned long long fac2 = pair64(__float_as_uint(fac), __float_as_uint(fac));
                const unsigned long long base2 = pair64(__float_as_uint(-base), __float_as_uint(-base));
                unsigned long long l2[2] = {0ull, 0ull};
                uint32_t hi[SC / 2], lo[TERMS == 2 ? SC / 2 : 1];
#pragma unroll
                for (int k = 0; k < SC; k += 2) {
                    float p0, p1;
                    unpair64(fma2(pair64(z[k], z[k + 1]), fac2, base2), p0, p1);
                    p0 = kv4_ex2(p0);
                    p1 = kv4_ex2(p1);
                    l2[(k >> 1) & 1] = add2(l2[(k >> 1) & 1], pair64(__float_as_uint(p0), __float_as_uint(p1)));
                    if (TERMS == 2) kv4_split(p0, p1, hi[k / 2], lo[k / 2]);
                    else hi[k / 2] = kv4_pack(p0, p1);
                    if (k % 32 == 30) tmem_st16(tS + k / 32 * 16, hi + k / 32 * 16);
                }
                if (TERMS == 2) tmem_st32(tS + 32, lo);
                {
                    float x0, x1, x2, x3;
                    unpair64(l2[0], x0, x1);
                    unpair64(l2[1], x2, x3);
                    l += (x0 + x1) + (x2 + x3);
                }
                tmem_st_wait();
                tc_fence_before();
                mbar_arrive(pfull + bar);
            }
        }
        // O, joined with the item's other parts where it was split.
        // S of the last step came after the second but last product of its slot, so the phase waited for
        // here is that barrier's current one or the one just completed
        const int nc = p.c1 - p.c0;
        if (ok && x < nact && ns && !warp_wait(odone + 2 * x + ((ns - 1) & 1), ((ns - 1) >> 1) & 1)) ok = false;
        tc_fence_after();
        const int tok = tok_of(tid), h = head_of(tid, tok);
        bool write = ok && tid < rows;
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
            float* part = parts + (size_t)(p.part + p.split) * G::PART;
            for (int d = 0; d < HD && x < nact; d += 32) {
                uint32_t o[32];
                tmem_ld32(tO + d, o);
                if (tid < rows) {
#pragma unroll
                    for (int k = 0; k < 32; k += 4)
                        reinterpret_cast<float4*>(part)[(size_t)((d + k) / 4) * G::ROWS + tid] =
                            make_float4(__uint_as_float(o[k]), __uint_as_float(o[k + 1]), __uint_as_float(o[k + 2]),
                                        __uint_as_float(o[k + 3]));
                }
            }
            part[(size_t)HD * G::ROWS + tid] = m;
            part[(size_t)(HD + 1) * G::ROWS + tid] = l;
            __threadfence();
            named_bar(1, G::SOFT);
            if (tid == 0) last_s = atomicAdd(arrive + p.part, 1u) == (unsigned)(p.splits - 1);
            named_bar(1, G::SOFT);
            write = false;                             // below
            if (last_s) {
                __threadfence();
                if (tid == 0) arrive[p.part] = 0u;
                const int splits = p.splits;
                const float* first_part = parts + (size_t)p.part * G::PART;
                // weights of the parts by row (the buffers of K and V are free: every product is done)
                float* wt = reinterpret_cast<float*>(sm + G::K);       // [splits][ROWS], 1 / sum at the end
                if (tid < rows) {
                    const float* ml = first_part + (size_t)HD * G::ROWS + tid;
                    float mj = -INFINITY, lj = 0.f;
#pragma unroll 8
                    for (int y = 0; y < splits; ++y) mj = fmaxf(mj, __ldcg(ml + (size_t)y * G::PART));
#pragma unroll 8
                    for (int y = 0; y < splits; ++y) {
                        const float li = __ldcg(ml + (size_t)y * G::PART + G::ROWS), mi = __ldcg(ml + (size_t)y * G::PART);
                        const float w = li == 0.f ? 0.f : kv4_ex2(mi - mj);
                        lj += li * w;
                        wt[y * G::ROWS + tid] = w;
                    }
                    wt[splits * G::ROWS + tid] = lj == 0.f ? 0.f : vg / lj;
                    if (ok && a.lse)
                        a.lse[(size_t)(p.q0 + tok) * a.s.nq + h] =
                            lj == 0.f ? -INFINITY : (mj - KV4_P_UP + log2f(lj)) * 0.6931471805599453f;
                }
                named_bar(1, G::SOFT);
                // eight elements of a row at a time, four of these in flight; neighbouring threads have
                // neighbouring rows, as the parts do
                const int total = rows * (HD / 8);
#pragma unroll 1
                for (int i0 = tid; i0 < total; i0 += 4 * G::SOFT) {
                    float v[4][8];
                    const float4* pi[4];
                    int row[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int i = min(i0 + k * G::SOFT, total - 1), d8 = i / rows;
                        row[k] = i - d8 * rows;
                        pi[k] = reinterpret_cast<const float4*>(first_part) + (size_t)(2 * d8) * G::ROWS + row[k];
#pragma unroll
                        for (int y = 0; y < 8; ++y) v[k][y] = 0.f;
                    }
#pragma unroll 2
                    for (int y = 0; y < splits; ++y)
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const float4 u0 = __ldcg(pi[k] + (size_t)y * (G::PART / 4));
                            const float4 u1 = __ldcg(pi[k] + (size_t)y * (G::PART / 4) + G::ROWS);
                            const float w = wt[y * G::ROWS + row[k]];
                            v[k][0] += u0.x * w;
                            v[k][1] += u0.y * w;
                            v[k][2] += u0.z * w;
                            v[k][3] += u0.w * w;
                            v[k][4] += u1.x * w;
                            v[k][5] += u1.y * w;
                            v[k][6] += u1.z * w;
                            v[k][7] += u1.w * w;
                        }
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int i = i0 + k * G::SOFT;
                        if (i >= total || !ok) break;
                        const float inv = wt[splits * G::ROWS + row[k]];
#pragma unroll
                        for (int y = 0; y < 8; ++y) v[k][y] *= inv;
                        const int tk = tok_of(row[k]), hd = head_of(row[k], tk);
                        kv4_store8(a.out, (size_t)(p.q0 + tk) * a.out_stride + (size_t)hd * HD + i / rows * 8, a.out_t, v[k]);
                    }
                }
            }
        }
        if (write && a.lse)
            a.lse[(size_t)(p.q0 + tok) * a.s.nq + h] =
                l == 0.f ? -INFINITY : (m - KV4_P_UP + log2f(l)) * 0.6931471805599453f;
    } else if (tid < G::SOFT + G::KTH) {
        // ----------------------------------------------------------------- K
        const int wt = tid - G::SOFT;
        // a thread widens KP runs of 32 elements
        const int jj = wt % G::LPR, r0 = wt / G::LPR;
        const int rot = G::LPR == 4 ? jj & 2 : G::LPR == 8 ? jj >> 1 : 0;   // a quarter-warp's stores meet every bank once
        int id[G::KP];
        uint4 kw[G::KP], kn[G::KP];
        uint32_t kscale[G::KP], kscale_n[G::KP];
        auto at_of = [&](int c, int i) { return c * KC + min(i * G::RPP + r0, KC - 1); };
        auto pages = [&](int c) {
#pragma unroll
            for (int i = 0; i < G::KP; ++i) id[i] = table[min(at_of(c, i), p.len - 1) >> a.s.page_log2];
        };
        auto load = [&](int c) {
#pragma unroll
            for (int i = 0; i < G::KP; ++i) {
                kn[i] = make_uint4(0, 0, 0, 0);
                kscale_n[i] = 0;
                const int pos = at_of(c, i);
                if (c < p.c1 && pos < p.len && id[i] >= 0 && id[i] < a.s.n_pages) {
                    const size_t at = ((size_t)id[i] * a.s.nkv + p.g) * a.s.page + (pos & (a.s.page - 1));
                    kn[i] = __ldg(reinterpret_cast<const uint4*>(a.c.kc + at * (HD / 2) + jj * 16));
                    kscale_n[i] = __ldg(reinterpret_cast<const uint16_t*>(a.c.ks + at * (HD / 16) + jj * 2));
                }
            }
        };
        auto k_store = [&](int b) {
            uint8_t* tile = sm + G::K + b * G::KT + (jj >> 1) * (KC * 128);
#pragma unroll
            for (int i = 0; i < G::KP; ++i) {
                const int row = i * G::RPP + r0;
                if (KC % G::RPP && row >= KC) break;
                const __half2 both = kv4_scale2(kscale[i]), s0 = __low2half2(both), s1 = __high2half2(both);
                uint32_t x0 = kw[i].x, x1 = kw[i].y, x2 = kw[i].z, x3 = kw[i].w;
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
        };
        if (p.c0 < p.c1) {
            pages(p.c0);
            load(p.c0);
            pages(p.c0 + 1);
        }
        for (int c = p.c0; c < p.c1; ++c) {
#pragma unroll
            for (int i = 0; i < G::KP; ++i) {
                kw[i] = kn[i];
                kscale[i] = kscale_n[i];
            }
            load(c + 1);
            pages(c + 2);
            const int i0 = c - p.c0, b = i0 % BUF, use = i0 / BUF;
            if (use && !mbar_wait(kempty + b, (use - 1) & 1)) {
                ok = false;
                break;
            }
            k_store(b);
            fence_proxy_async();
            mbar_arrive(kfull + b);
        }
    } else if (tid < G::SOFT + G::KTH + G::VTH) {
        // ----------------------------------------------------------------- V
        const int wt = tid - G::SOFT - G::KTH;         // eight positions of sixteen elements
        const int pg8 = wt & 7, dg = (wt >> 3) % (HD / 16), kb = (wt >> 3) / (HD / 16);
        const bool v_work = kb < KC / 64;
        const int p0 = kb * 64 + pg8 * 8;
        int id;
        uint2 vw[8], vn[8];
        uint32_t vscale[8], vscale_n[8];
        auto page = [&](int c) { id = table[min(c * KC + p0, p.len - 1) >> a.s.page_log2]; };
        auto load = [&](int c) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                vn[i] = make_uint2(0, 0);
                vscale_n[i] = 0;
            }
            const int pos = c * KC + p0;
            if (v_work && c < p.c1 && pos < p.len && id >= 0 && id < a.s.n_pages) {
                const size_t at = ((size_t)id * a.s.nkv + p.g) * a.s.page + (pos & (a.s.page - 1));
                const uint8_t* codes = a.c.vc + at * (HD / 2) + dg * 8;
                const uint8_t* scales = a.c.vs + at * (HD / 16) + dg;
                // behind the last position the bytes may decode to NaN, which weight 0 would keep
                const int there = p.len - pos;
                if (there >= 8) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        vn[i] = __ldg(reinterpret_cast<const uint2*>(codes + i * (HD / 2)));
                        vscale_n[i] = __ldg(scales + i * (HD / 16));
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (i < there) {
                            vn[i] = __ldg(reinterpret_cast<const uint2*>(codes + i * (HD / 2)));
                            vscale_n[i] = __ldg(scales + i * (HD / 16));
                        }
                }
            }
        };
        auto v_store = [&](int b) {
            uint8_t* tile = sm + G::V + b * G::KT + kb * (HD * 128);
            __half2 s[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) s[i] = kv4_scale2(kv4_bytes(vscale[2 * i], vscale[2 * i + 1]));
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                uint32_t pr[4][2];                     // bytes of one element of two positions: even, odd
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    kv4_pair(y ? vw[2 * i].y : vw[2 * i].x, y ? vw[2 * i + 1].y : vw[2 * i + 1].x, pr[i][0], pr[i][1]);
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
        };
        if (p.c0 < p.c1) {
            page(p.c0);
            load(p.c0);
            page(p.c0 + 1);
        }
        for (int c = p.c0; c < p.c1; ++c) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                vw[i] = vn[i];
                vscale[i] = vscale_n[i];
            }
            load(c + 1);
            page(c + 2);
            const int i0 = c - p.c0, b = i0 % BUF, use = i0 / BUF;
            if (use && !mbar_wait(vempty + b, (use - 1) & 1)) {
                ok = false;
                break;
            }
            if (v_work) v_store(b);
            fence_proxy_async();
            mbar_arrive(vfull + b);
        }
    } else {
        // ----------------------------------------------------------------- MMA
        const uint32_t one = elect_one();
        auto same = [](uint32_t v) { return __shfl_sync(0xffffffffu, v, 0); };    // known to be uniform
        const int ns = (int)same((p.c1 - p.c0) * G::SPC), tiles = (int)same(nact);
        const uint32_t tm0 = same(tmem), smem0 = same(smem_u32(sm)), bar0 = smem0 + G::BARS;
        const uint32_t high = (uint32_t)(umma_sdesc(0) >> 32);                    // of every descriptor
        const uint32_t qd = (uint32_t)umma_sdesc(smem0 + G::Q), kd = (uint32_t)umma_sdesc(smem0 + G::K),
                       vd = (uint32_t)umma_sdesc(smem0 + G::V);
        const uint32_t idS = umma_idesc_f16(128, SC), idO = umma_idesc_f16(128, HD);
        auto wait = [&](uint64_t* bar, uint32_t parity) { return warp_wait(bar, parity); };
        auto k_there = [&](int step) {
            const int i = step / G::SPC;
            const bool there = wait(kfull + i % BUF, (i / BUF) & 1);
            tc_fence_after();
            return there;
        };
        // S of a step into its slot; the last one of a chunk frees the buffer.  A product takes 32 bytes of
        // a tile's 64-wide block
        auto s_of = [&](int x, int step) {
            const int b = step / G::SPC % BUF, h = step % G::SPC;
            const uint32_t ad = qd + x * TERMS * (G::QT / 16), bd = kd + b * (G::KT / 16) + h * (SC * 8);
            const uint32_t d = tm0 + x * 128 + (step & 1) * 64;
            const uint32_t full = bar0 + 8 * (8 + 2 * x + (step & 1)), empty = bar0 + 8 * (2 + b);
            const bool last = x == tiles - 1 && h == G::SPC - 1;
#pragma unroll
            for (int tm = TERMS - 1; tm >= 0; --tm)
#pragma unroll
                for (int ks = 0; ks < HD / 16; ++ks) {
                    const uint32_t ak = ad + (tm * (G::QT / 16) + (ks >> 2) * 1024 + 2 * (ks & 3));
                    const uint32_t bk = bd + ((ks >> 2) * (KC * 8) + 2 * (ks & 3));
                    if (tm == TERMS - 1 && ks == 0) mma_ss<0>(one, d, ak, bk, high, idS);
                    else mma_ss<1>(one, d, ak, bk, high, idS);
                }
            mma_commit(one, full);
            if (last) mma_commit(one, empty);
        };
        auto pv_of = [&](int x, int step) {
            const int b = step / G::SPC % BUF, h = step % G::SPC;
            const uint32_t bd = vd + b * (G::KT / 16) + h * (HD * 8);
            const uint32_t d = tm0 + 256 + x * HD, ap = tm0 + x * 128 + (step & 1) * 64;
            const uint32_t done = bar0 + 8 * (16 + 2 * x + (step & 1)), empty = bar0 + 8 * (6 + b);
            const bool last = x == tiles - 1 && h == G::SPC - 1;
#pragma unroll
            for (int tm = TERMS - 1; tm >= 0; --tm)
#pragma unroll
                for (int ks = 0; ks < SC / 16; ++ks)
                    mma_ts(one, d, ap + (tm * (SC / 2) + ks * 8), bd + 2 * ks, high, idO, (uint32_t)(step | (tm < TERMS - 1) | ks));
            mma_commit(one, done);
            if (last) mma_commit(one, empty);
        };
        ok = wait(qfull, 0);
        tc_fence_after();
        for (int step = 0; ok && step < 2 && step < ns; ++step) {
            if (step % G::SPC == 0) ok = k_there(step);
            for (int x = 0; ok && x < tiles; ++x) s_of(x, step);
        }
        for (int step = 0; ok && step < ns; ++step) {
            const int i = step / G::SPC;
            if (step % G::SPC == 0) ok = wait(vfull + i % BUF, (i / BUF) & 1);
            for (int x = 0; ok && x < tiles; ++x) {
                ok = wait(pfull + 2 * x + (step & 1), (step >> 1) & 1);
                if (!ok) break;
                tc_fence_after();
                pv_of(x, step);
                if (step + 2 < ns) {
                    if (x == 0 && (step + 2) % G::SPC == 0) ok = k_there(step + 2);
                    if (!ok) break;
                    s_of(x, step + 2);
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
    // items: whole tiles of rows, and one that is not whole per sequence with enough rows; splitting adds
    // about two pieces a multiprocessor
    const long long rows = (long long)a.n_tokens * (a.s.nq / a.s.nkv);
    const long long ragged = rows / (few_rows + 1) < a.n_seqs ? rows / (few_rows + 1) : a.n_seqs;
    const long long grid = a.s.nkv * (rows / G::ROWS + ragged) + 2 * w.num_sms;
    return launch_pdl(kv4_extend_kernel<HD, TERMS>, dim3((unsigned)grid), dim3(G::THREADS), G::SMEM, st, a, few_rows,
                      w.parts, w.arrive, w.num_sms, EXTEND_PARTS * w.num_sms);
}

}  // namespace

cudaError_t kv4_extend_prepare() {
    cudaError_t e = cudaSuccess;
    auto allow = [&](auto kernel, size_t smem) {
        if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    };
    allow(kv4_extend_kernel<64, 1>, EGeo<64, 1>::SMEM);
    allow(kv4_extend_kernel<64, 2>, EGeo<64, 2>::SMEM);
    allow(kv4_extend_kernel<128, 1>, EGeo<128, 1>::SMEM);
    allow(kv4_extend_kernel<128, 2>, EGeo<128, 2>::SMEM);
    allow(kv4_extend_kernel<256, 1>, EGeo<256, 1>::SMEM);
    allow(kv4_extend_kernel<256, 2>, EGeo<256, 2>::SMEM);
    return e;
}

// none for calls whose every row is the decode kernel's
size_t kv4_extend_part_floats(int hd, int num_sms) {
    const size_t rows = hd <= 128 ? 256 : 128;
    return (size_t)EXTEND_PARTS * num_sms * rows * (hd + 2);
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
