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
//   MMA      one warp, one lane of which issues: S = Q K^T and O += P V^T, tcgen05, P
//            read from TMEM
// With NT = 2 two 128-row tiles share every widened K and V tile (the widening costs
// as many issue slots as one tile's softmax); with NT = 1 (F32 rows, head_dim 256)
// shared memory has no room for two.
// Every tile has two S slots of 64 columns, so the next step's S is there when a step's
// softmax ends: with one slot a step waited for its own two products, which took
// longer than its softmax.  P overlays the S it came from; the next S into the slot is
// issued after the product that reads P and runs after it.
// O is rescaled only when a row's maximum rose by 2^8 since the last time.
// F32 rows: q = hi + lo and p = hi + lo, two products each (TERMS = 2).  16-bit rows: one
// fp16 term of each, p's rounding 2^-11 of it at most, as in kv4_decode.cu.
// Few items: the chunks of an item are split over CTAs; the one that comes last keeps its
// part and joins the others' to it.
//
// Measured (32 q heads, 4 kv heads of 128): 4 sequences of 8192-16384 positions that bring
// 2048 BF16 tokens each, 1172 us, 1380 TFLOP/s of visible products; the issue slots are
// 61% taken (widening, exponentials, moves from and to TMEM) and the tensor pipe 58%: the
// softmax of a step, its two products and the widening of its positions each take most of
// the step's 900 ns.  777 F32 tokens from their first, 29.9 us: an item's start (lengths, q)
// and end take 10 of its 20 us, and 196 items are 1.3 waves.  Pieces taken in turn by CTAs
// that stay were no faster (1173 us; the short calls 2 us slower).
#include <limits.h>
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
    static constexpr int GPR = KTH / LPR / (KC / 16);                // positions of a run of 16 at a time
    static constexpr int KP = (16 + GPR - 1) / GPR;                  // times
    static constexpr int PART = ROWS * (HD + 2);                     // floats of a part
    static constexpr int SPLITS = 31;                                // of an item at most
    static_assert(ROWS * HD * 4 <= V, "O passes through the tiles of Q and K on its way out");
    static_assert((SPLITS + 1) * ROWS * 4 <= BUF * KT, "the weights of a join take the buffers of V");
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
        "{\n\t.reg .pred p, q;\n\t.reg .b64 x, y;\n\tsetp.ne.u32 p, %5, 0;\n\tsetp.ne.u32 q, %6, 0;\n\t"
        "mov.b64 x, {%1, %3};\n\tmov.b64 y, {%2, %3};\n\t"
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
                      unsigned* __restrict__ total, int num_sms, int max_parts, unsigned long long stall_ns) {
    using G = EGeo<HD, TERMS>;
    constexpr int NT = G::NT, KC = G::KC, BUF = G::BUF;
    extern __shared__ __align__(1024) uint8_t smraw[];
    uint8_t* sm = smraw + ((1024u - (smem_u32(smraw) & 1023u)) & 1023u);
    uint64_t* bars = reinterpret_cast<uint64_t*>(sm + G::BARS);
    // by buffer: kfull .. vempty; by tile and slot: sfull .. odone
    uint64_t *kfull = bars, *kempty = bars + 2, *vfull = bars + 4, *vempty = bars + 6, *sfull = bars + 8,
             *pfull = bars + 12, *odone = bars + 16, *qfull = bars + 20;
    uint32_t* tslot = reinterpret_cast<uint32_t*>(bars + 21);
    __shared__ int2 wsum[G::THREADS / 32];
    __shared__ int3 wsum3[G::THREADS / 32];
    __shared__ Piece piece_s;
    __shared__ int last_s, joined_s;
    __shared__ long long row_at[G::SOFT];              // bytes to where a row of the item is stored
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int group = a.s.nq / a.s.nkv;
    if (tid == 0) {
        piece_s.s = -1;
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
    pdl_wait();
    pdl_launch_dependents();
    // The grid is as large as the host has to fear; a CTA behind the last piece need not scan to learn that if
    // the first one has told (total: pieces + 1, or 0; the decode kernel behind this one clears it).  500 new
    // tokens beside 512 requests of one: 131 us, all scanning 151; beside 2000, 264 and 346.
    if ((int)blockIdx.x >= num_sms) {
        const unsigned t = tid == 0 ? ld_acquire_gpu(total) : 0u;
        if (__syncthreads_or(t && blockIdx.x + 1 >= t)) return;
    }

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
        // with no more sequences than threads a thread's only one is looked up once
        const bool single = per == 1;
        Seq one;
        one.qts = 0;
        bool descends = false;
        // total chunks, a sequence's tiles taken as evenly spread between its first and last, and as if all were
        // its last (as far as 2^18 a sequence: they only set the share)
        int work = 0, most = 0;
        for (int s = s0; s < s1; ++s) {
            seq(s, one);
            descends |= a.cu[s + 1] < a.cu[s];
            const float both = (float)one.last + (float)chunks(one.q, min(one.rows, (int)G::ROWS));
            if (one.qts) {
                work += (int)fminf(0.5f * (float)a.s.nkv * (float)one.qts * both, 262144.f);
                most += (int)fminf((float)a.s.nkv * (float)one.qts * (float)one.last, 262144.f);
            }
        }
        work = __reduce_add_sync(0xffffffffu, work);
        most = __reduce_add_sync(0xffffffffu, most);
        if (lane == 0) wsum[warp] = make_int2(work, most);
        if (__syncthreads_or(descends)) return;        // rows of several sequences (the other kernel reports it)
        work = most = 0;
#pragma unroll
        for (int w = 0; w < T / 32; ++w) {
            work += wsum[w].x;
            most += wsum[w].y;
        }
        // pieces that fill one wave, and no more of them than items and multiprocessors
        const int share = max(8, (int)(fmaxf(1.25f * (float)work, (float)most) / (float)num_sms) + 1);
        auto splits_of = [&](const Seq& r) { return min(G::SPLITS, max(1, (r.last + share - 1) / share)); };
        int items = 0, pieces = 0, parts_n = 0;
        for (int s = s0; s < s1; ++s) {
            if (!single) seq(s, one);
            const int k = splits_of(one), it = a.s.nkv * one.qts;
            items += it;
            pieces += it * k;
            if (k > 1) parts_n += it * k;
        }
        // sums over the CTA, and over the threads before
        int inc_i = items, inc_p = pieces, inc_n = parts_n;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int oi = __shfl_up_sync(0xffffffffu, inc_i, d), op = __shfl_up_sync(0xffffffffu, inc_p, d),
                      on = __shfl_up_sync(0xffffffffu, inc_n, d);
            if (lane >= d) {
                inc_i += oi;
                inc_p += op;
                inc_n += on;
            }
        }
        if (lane == 31) wsum3[warp] = make_int3(inc_i, inc_p, inc_n);
        __syncthreads();
        int all = 0, all_parts = 0, base_i = inc_i - items, base_p = inc_p - pieces, part0 = inc_n - parts_n;
#pragma unroll
        for (int w = 0; w < T / 32; ++w) {
            const int3 o = wsum3[w];
            all += o.y;
            all_parts += o.z;
            if (w < warp) {
                base_i += o.x;
                base_p += o.y;
                part0 += o.z;
            }
        }
        // not more CTAs or parts than there are (past the sums' limit): every item whole then
        const bool whole = all > (int)gridDim.x || all_parts > max_parts;
        const int me = blockIdx.x;
        int base = whole ? base_i : base_p;
        if (me == 0 && tid == 0 && !whole) atomicExch(total, (unsigned)all + 1u);
        if (me >= base && me < base + (whole ? items : pieces)) {
            for (int s = s0; s < s1; ++s) {
                if (!single) seq(s, one);
                const int k = whole ? 1 : splits_of(one), mine = a.s.nkv * one.qts * k;
                if (me < base + mine) {
                    // the last rows see the most positions: they start first
                    const int at = me - base, split = at % k, item = at / k, qt = one.qts - 1 - item / a.s.nkv;
                    Piece p;
                    p.s = s;
                    p.g = item % a.s.nkv;
                    p.row0 = qt * G::ROWS;
                    p.q0 = one.q.q0;
                    p.n = one.q.n;
                    p.len = one.q.len;
                    const int nch = chunks(one.q, min(p.row0 + G::ROWS, one.rows));
                    p.splits = max(1, min(k, nch / 4));            // four chunks to a split at least
                    p.split = split;
                    p.c0 = nch * split / p.splits;
                    p.c1 = nch * (split + 1) / p.splits;
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
        int lim_min = len - p.n + tok_of(tid & ~31) + 1;                         // the warp's first row's
        // where the thread's row starts: in q, and in out
        const int tok = tok_of(tid), h = head_of(tid, tok);
        float fac = 0.f;
        if (x < nact) {
            // Eight elements of a row a lane, first as they are to where their fp16 terms belong (F32 elements
            // fill the places of both), all at once; then the row's largest by shuffles, and the row scaled to
            // [1, 2) by a power of two (to what is exact below 2^-126) and split in place.
            constexpr int LR = HD / 8, RW = 32 / LR;   // lanes of a row, rows at a time
            const float kg = a.c.kg[p.g];
            // of scale * kg: z's largest is q.k's largest then
            const uint32_t sign = kv4_negative(a.scale, kg) ? 0x80008000u : 0u;
            const int d = (lane % LR) * 8, sub = lane / LR;
            const long long mine = tid < rows ? ((long long)(p.q0 + tok) * a.q_stride + (long long)h * HD) * (TERMS == 2 ? 4 : 2) : -1;
            uint8_t* qs = sm + G::Q + x * TERMS * G::QT + (d >> 6) * 16384;
            auto word = [&](int r) { return qs + sw128_offset((tid & 96) + r + sub, d & 63); };
#pragma unroll 4
            for (int r = 0; r < 32; r += RW) {
                const long long at = __shfl_sync(0xffffffffu, mine, r + sub);
#pragma unroll
                for (int z = 0; z < TERMS; ++z) {
                    if (at >= 0) cp_async_cg16(word(r) + z * G::QT, static_cast<const uint8_t*>(a.q) + at + d * (TERMS == 2 ? 4 : 2) + 16 * z);
                    else *reinterpret_cast<uint4*>(word(r) + z * G::QT) = make_uint4(0, 0, 0, 0);
                }
            }
            cp_async_wait_all();
            int exponent = 0;
            if (TERMS == 2 || a.q_t != KV4_F16 || sign) {          // fp16 rows are what they have to be
                constexpr int RB = 32 / RW < 8 ? 32 / RW : 8;      // in flight
#pragma unroll 1
                for (int r0 = 0; r0 < 32; r0 += RB * RW) {
                    float v[RB][8], big[RB];
#pragma unroll
                    for (int i = 0; i < RB; ++i) {
                        uint4 raw[TERMS];
#pragma unroll
                        for (int z = 0; z < TERMS; ++z) raw[z] = *reinterpret_cast<const uint4*>(word(r0 + i * RW) + z * G::QT);
                        kv4_floats8(raw, a.q_t, v[i]);
                        big[i] = max3(max3(fabsf(v[i][0]), fabsf(v[i][1]), fabsf(v[i][2])),
                                      max3(fabsf(v[i][3]), fabsf(v[i][4]), fabsf(v[i][5])), fmaxf(fabsf(v[i][6]), fabsf(v[i][7])));
                    }
#pragma unroll
                    for (int o = LR / 2; o > 0; o >>= 1)
#pragma unroll
                        for (int i = 0; i < RB; ++i) big[i] = fmaxf(big[i], __shfl_xor_sync(0xffffffffu, big[i], o));
#pragma unroll
                    for (int i = 0; i < RB; ++i) {
                        const int e = kv4_exponent(big[i]);
                        const float un = kv4_pow2(-e);
                        uint32_t hi[4], lo[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const float v0 = v[i][2 * k] * un, v1 = v[i][2 * k + 1] * un;
                            if (TERMS == 2) kv4_split(v0, v1, hi[k], lo[k]);
                            else hi[k] = kv4_pack(v0, v1);
                        }
                        uint8_t* at = word(r0 + i * RW);
                        *reinterpret_cast<uint4*>(at) = make_uint4(hi[0] ^ sign, hi[1] ^ sign, hi[2] ^ sign, hi[3] ^ sign);
                        if (TERMS == 2) *reinterpret_cast<uint4*>(at + G::QT) = make_uint4(lo[0] ^ sign, lo[1] ^ sign, lo[2] ^ sign, lo[3] ^ sign);
                        // the thread whose row it is keeps the exponent
                        const int back = lane - r0 - i * RW, er = __shfl_sync(0xffffffffu, e, (back * LR) & 31);
                        if (back >= 0 && back < RW) exponent = er;
                    }
                }
            }
            fac = kv4_factor_of(kv4_factor(a.scale, kg), exponent);
            float largest = fac;                       // for rows in [1, 2)
            if (TERMS == 1 && a.q_t == KV4_F16 && !sign) {
                __half2 big = __float2half2_rn(0.f);   // of what this lane has of any of the warp's rows
#pragma unroll
                for (int r = 0; r < 32; r += RW) {
                    const uint4 u = *reinterpret_cast<const uint4*>(word(r));
                    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                    for (int k = 0; k < 4; ++k) big = __hmax2(big, __habs2(*reinterpret_cast<const __half2*>(&w[k])));
                }
                largest *= kv4_pow2(kv4_exponent(fminf(fmaxf(__low2float(big), __high2float(big)), 65504.f)));
            }
            if (__any_sync(0xffffffffu, kv4_far<HD>(largest))) lim_min = INT_MIN;   // z takes fac in the branch of masks
            fence_proxy_async();
        }
        mbar_arrive(qfull);
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
                    if (lim_min == INT_MIN)
#pragma unroll
                        for (int k = 0; k < SC; ++k) z[k] = __float_as_uint(__fmul_rn(__uint_as_float(z[k]), fac));
                    asm volatile("");                  // a branch, not selects that run every time
                }
                float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int k = 0; k < SC; k += 8)
#pragma unroll
                    for (int y = 0; y < 4; ++y)
                        mx4[y] = max3(mx4[y], __uint_as_float(z[k + 2 * y]), __uint_as_float(z[k + 2 * y + 1]));
                const float f1 = lim_min == INT_MIN ? 1.f : fac;   // what z still wants
                const float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3])) * f1;
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
                const unsigned long long fac2 = pair64(__float_as_uint(f1), __float_as_uint(f1));
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
        if (ok && x < nact && ns && !warp_wait(odone + 2 * x + ((ns - 1) & 1), ((ns - 1) >> 1) & 1)) ok = false;
        tc_fence_after();
        if (!ns) named_bar(1, G::SOFT);                // q is no longer stored where O goes
        const int split = p.split, splits = p.splits;
        const float vg = a.c.vg[p.g];
        // the CTA that comes last to the end of an item keeps its part; the others leave theirs to it
        bool keeps = false;
        if (splits > 1) {
            named_bar(1, G::SOFT);
            if (tid == 0) last_s = atomicAdd(arrive + p.part, 1u) == (unsigned)(splits - 1);
            named_bar(1, G::SOFT);
            keeps = last_s;
        }
        float* part = parts + (size_t)(p.part + split) * G::PART;            // O [ROWS][HD], then m, l [ROWS]
        const bool to_part = splits > 1 && !keeps;
        // A warp's rows of O in shared memory (every S is done: the tiles of Q and K are free), as they will
        // be stored, rows in order with their 16-byte words permuted; then neighbouring lanes store
        // neighbouring words (a thread storing its own row took twice as long).
        uint8_t* mine = sm + (size_t)warp * 32 * HD * 4;
        row_at[tid] = tid >= rows || !ok ? -1
                      : to_part ? (long long)tid * HD * 4
                                : ((long long)(p.q0 + tok) * a.out_stride + (long long)h * HD) * (a.out_t == KV4_F32 ? 4 : 2);
        const int to_t = splits > 1 ? KV4_F32 : a.out_t, words = HD / (to_t == KV4_F32 ? 4 : 8);
        if (x < nact) {
            const float inv = splits > 1 ? 1.f : l == 0.f ? 0.f : vg / l;
            const bool some = ns && (splits > 1 || l != 0.f);
            uint8_t* row = mine + lane * words * 16;
#pragma unroll 1
            for (int d = 0; d < HD; d += 32) {
                uint32_t o[32];
                tmem_ld32(tO + d, o);
#pragma unroll
                for (int k = 0; k < 32; ++k) o[k] = some ? __float_as_uint(__uint_as_float(o[k]) * inv) : 0u;
                if (to_t == KV4_F32) {
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        *reinterpret_cast<uint4*>(row + ((d / 4 + k) ^ (lane & 7)) * 16) =
                            make_uint4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
                } else {
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        uint32_t u[4];
#pragma unroll
                        for (int y = 0; y < 4; ++y)
                            u[y] = kv4_pack16(__uint_as_float(o[8 * k + 2 * y]), __uint_as_float(o[8 * k + 2 * y + 1]), to_t);
                        *reinterpret_cast<uint4*>(row + ((d / 8 + k) ^ (lane & 7)) * 16) = make_uint4(u[0], u[1], u[2], u[3]);
                    }
                }
            }
            __syncwarp();
            if (!keeps) {
                uint8_t* base = to_part ? reinterpret_cast<uint8_t*>(part) : static_cast<uint8_t*>(a.out);
                const int shift = __ffs(words) - 1;
#pragma unroll 1
                for (int i0 = lane; i0 < 32 * words; i0 += 8 * 32) {
                    uint4 u[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const int i = i0 + 32 * k;
                        u[k] = *reinterpret_cast<const uint4*>(mine + (i ^ ((i >> shift) & 7)) * 16);
                    }
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const int i = i0 + 32 * k;
                        const long long at = row_at[warp * 32 + (i >> shift)];
                        if (at >= 0) *reinterpret_cast<uint4*>(base + at + 16 * (i & (words - 1))) = u[k];
                    }
                }
            }
        }
        auto log_sum = [&](float mr, float lr) {
            return lr == 0.f ? -INFINITY : (mr - KV4_P_UP + log2f(lr)) * 0.6931471805599453f;
        };
        if (splits > 1) {
            part[(size_t)HD * G::ROWS + tid] = m;
            part[(size_t)(HD + 1) * G::ROWS + tid] = l;
        }
        if (splits == 1) {
            if (ok && tid < rows && a.lse) a.lse[(size_t)(p.q0 + tok) * a.s.nq + h] = log_sum(m, l);
        } else if (to_part) {
            named_bar(1, G::SOFT);
            if (tid == 0) {
                if (stall_ns)                          // test hook, one second at most
                    for (const unsigned long long t0 = globaltimer(); globaltimer() - t0 < stall_ns;) __nanosleep(1000);
                __threadfence();
                if (atomicAdd(arrive + p.part + 1, 1u) == (unsigned)(splits - 1)) arrive[p.part] = arrive[p.part + 1] = 0u;
            }
        } else {
            // The others are past their products: their parts are there in no more time than it takes to
            // store one.  Where the wait gave up all the same, the parts that come later still count, and this
            // CTA as one of them: whoever is last clears the counters.
            if (tid == 0) {
                const bool all = grid_wait(arrive + p.part + 1, (unsigned)(splits - 1));
                __threadfence();
                if (all || atomicAdd(arrive + p.part + 1, 1u) == (unsigned)(splits - 1)) arrive[p.part] = arrive[p.part + 1] = 0u;
                joined_s = all && ok;
            }
            named_bar(1, G::SOFT);
            ok = joined_s && ok;
            const float* first_part = parts + (size_t)p.part * G::PART;
            // weights of the parts by row
            float* wt = reinterpret_cast<float*>(sm + G::V);           // [splits][ROWS], vg / sum at the end
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
                if (ok && a.lse) a.lse[(size_t)(p.q0 + tok) * a.s.nq + h] = log_sum(mj, lj);
            }
            named_bar(1, G::SOFT);
            // Eight elements of a row at a time, four of these in flight; the parts in their order, whichever of
            // them was kept, so that results do not depend on who came last.
            const int total = ok ? rows * (HD / 8) : 0;
#pragma unroll 1
            for (int i0 = tid; i0 < total; i0 += 4 * G::SOFT) {
                float v[4][8];
                const float4* pi[4];
                int row[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int i = min(i0 + k * G::SOFT, total - 1);
                    row[k] = i / (HD / 8);
                    pi[k] = reinterpret_cast<const float4*>(first_part) + 2 * i;
#pragma unroll
                    for (int y = 0; y < 8; ++y) v[k][y] = 0.f;
                }
                auto add = [&](int k, int y, const float4& u0, const float4& u1) {
                    const float f = wt[y * G::ROWS + row[k]];
                    v[k][0] += u0.x * f;
                    v[k][1] += u0.y * f;
                    v[k][2] += u0.z * f;
                    v[k][3] += u0.w * f;
                    v[k][4] += u1.x * f;
                    v[k][5] += u1.y * f;
                    v[k][6] += u1.z * f;
                    v[k][7] += u1.w * f;
                };
                auto add_parts = [&](int y0, int y1) {
#pragma unroll 2
                    for (int y = y0; y < y1; ++y)
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            add(k, y, __ldcg(pi[k] + (size_t)y * (G::PART / 4)), __ldcg(pi[k] + (size_t)y * (G::PART / 4) + 1));
                };
                add_parts(0, split);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int w = min(i0 + k * G::SOFT, total - 1) % (HD / 8) * 2, r = row[k];
                    const uint8_t* own = sm + (size_t)r * HD * 4;
                    add(k, split, *reinterpret_cast<const float4*>(own + (w ^ (r & 7)) * 16),
                        *reinterpret_cast<const float4*>(own + ((w + 1) ^ (r & 7)) * 16));
                }
                add_parts(split + 1, splits);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int i = i0 + k * G::SOFT, r = i / (HD / 8);
                    if (i >= total) break;
                    const float inv = wt[splits * G::ROWS + r];
#pragma unroll
                    for (int y = 0; y < 8; ++y) v[k][y] *= inv;
                    kv4_store8(static_cast<uint8_t*>(a.out) + row_at[r], i % (HD / 8) * 8, a.out_t, v[k]);
                }
            }
        }
    } else if (tid < G::SOFT + G::KTH) {
        // ----------------------------------------------------------------- K
        const int wt = tid - G::SOFT;
        // A thread widens 32 elements of every GPR-th position of a run of 16, which one page holds: one page id
        // and one address, the rest are constants.  Positions behind the last one are masked, whatever they hold.
        const int jj = wt % G::LPR, run = wt / G::LPR / G::GPR, sub = wt / G::LPR % G::GPR;
        const int rot = G::LPR == 4 ? jj & 2 : G::LPR == 8 ? jj >> 1 : 0;
        // (`flip`: positions of every other run change places, so that with `rot` a quarter-warp's stores meet every
        // bank once)
        const int flip = run & 1 ? G::LPR == 4 ? 1 : G::LPR == 2 ? 2 : 0 : 0;
        auto in_run = [&](int i) { return (sub + i * G::GPR) ^ flip; };
        auto there = [&](int i) { return 16 % G::GPR == 0 || i < G::KP - 1 || sub < 16 % G::GPR; };
        int id;
        uint4 kw[G::KP], kn[G::KP];
        uint32_t kscale[G::KP], kscale_n[G::KP];
        auto page = [&](int c) { id = table[min(c * KC + run * 16, p.len - 1) >> a.s.page_log2]; };
        auto load = [&](int c) {
#pragma unroll
            for (int i = 0; i < G::KP; ++i) {
                kn[i] = make_uint4(0, 0, 0, 0);
                kscale_n[i] = 0;
            }
            if (c < p.c1 && c * KC + run * 16 < p.len && id >= 0 && id < a.s.n_pages) {
                const size_t at = ((size_t)id * a.s.nkv + p.g) * a.s.page + ((c * KC + run * 16) & (a.s.page - 1));
                const uint8_t* codes = a.c.kc + at * (HD / 2) + jj * 16;
                const uint8_t* scales = a.c.ks + at * (HD / 16) + jj * 2;
#pragma unroll
                for (int i = 0; i < G::KP; ++i)
                    if (there(i)) {
                        kn[i] = __ldg(reinterpret_cast<const uint4*>(codes + in_run(i) * (HD / 2)));
                        kscale_n[i] = __ldg(reinterpret_cast<const uint16_t*>(scales + in_run(i) * (HD / 16)));
                    }
            }
        };
        auto k_store = [&](int b) {
            uint8_t* tile = sm + G::K + b * G::KT + (jj >> 1) * (KC * 128);
#pragma unroll
            for (int i = 0; i < G::KP; ++i) {
                const int row = run * 16 + in_run(i);
                if (!there(i)) break;
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
            page(p.c0);
            load(p.c0);
            page(p.c0 + 1);
        }
        for (int c = p.c0; c < p.c1; ++c) {
#pragma unroll
            for (int i = 0; i < G::KP; ++i) {
                kw[i] = kn[i];
                kscale[i] = kscale_n[i];
            }
            load(c + 1);
            page(c + 2);
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
    // items: whole tiles of rows, and one that is not whole per sequence with enough rows; splitting adds a
    // piece a multiprocessor at most
    const long long rows = (long long)a.n_tokens * (a.s.nq / a.s.nkv);
    const long long ragged = rows / (few_rows + 1) < a.n_seqs ? rows / (few_rows + 1) : a.n_seqs;
    const long long grid = a.s.nkv * (rows / G::ROWS + ragged) + w.num_sms;
    return launch_pdl(kv4_extend_kernel<HD, TERMS>, dim3((unsigned)grid), dim3(G::THREADS), G::SMEM, st, a, few_rows,
                      w.ext_parts, w.ext_arrive, w.ext_total, w.num_sms, EXTEND_PARTS * w.num_sms, w.stall_ns);
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

// none where every row is the decode kernel's
size_t kv4_extend_part_floats(int hd, int num_sms, long long max_rows) {
    if (max_rows <= KV4_FEW_ROWS) return 0;
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
