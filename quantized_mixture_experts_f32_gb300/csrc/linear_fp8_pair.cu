// linear_fp8_pair.cu -- qmoe_linear_fp8 for many tokens: pairs of CTAs on two SMs share a tile
// of 256 tokens x 256 features (tcgen05 cta_group::2, kind::f8f6f4).
//
// Each CTA brings 128 rows of x and 128 of W, half of what the tile needs from either
// side, and keeps the products of its 128 tokens: 32 KB a block of k, where a tile of
// its own would take 48 and be bound by what L2 gives.  Tokens are TMEM's lanes, so that
// a block's scale is one number a thread.  Sixteen warps scale the blocks' products into
// fp32 registers, 64 features a thread, while the next two blocks' products run; rows
// leave (and residuals come) through shared memory by TMA, a box a warp.
//
// 16384 tokens, 2048 x 5120, BF16, bias: 164.5 us back to back in a graph, 2089 TFLOP/s, 1.09 of the
// measured bf16 rate of a library product (170 to 173 us, 1.03 to 1.05, called one by one), the tensor
// pipe 44% active.  A scale for each block of 128 takes every
// product through registers, by barriers between both SMs and with the two products that
// TMEM holds at this size; products and copies without that take 114 us.
// Tiles of 128 features (four products in TMEM, 0.33 us a block of k instead of 0.52) are
// for calls with few tiles; tiles of 64 were slower than either.
// Where even these leave most SMs idle, two to four pairs in a cluster share a tile's k, and
// send their sums to one another's shared memory (256 tokens, 4096 x 2048: 14.6 us by one
// pair a tile, 11.4 by two, 10.6 by three; 16384 x 512: 45, 27, 20, 17 by four).
#include <limits.h>

#include "linear_fp8.cuh"

namespace qmoe {

namespace {

constexpr int LP_TOKENS = 256;                // of a pair's tile
constexpr int LP_COLS = 64;                   // features of a thread
constexpr int LP_STAGES_MAX = 6;
constexpr int LP_EW_MAX = 16;
constexpr int LP_GROUP = 4, LP_SLOTS = 3;     // blocks of k whose scales are staged together, such groups
constexpr int LP_SLOTS_SUM = 6;               // warps' sums that come from other pairs: 8 warps' from 1 to 3

struct PairBars {
    uint64_t full[LP_STAGES_MAX], empty[LP_STAGES_MAX], tfull[4], tempty[4], sfull[LP_SLOTS], sempty[LP_SLOTS], res[LP_EW_MAX];
    uint32_t tmem;
    int failed;
};

struct PairScales {
    float x[LP_SLOTS][LP_GROUP][128];         // of the CTA's tokens
    float w[LP_SLOTS][2][LP_GROUP];           // of the tile's two blocks of features
    __align__(16) float bias[LP_SLOTS][256];  // of the tile's features, with its first group
};

// a copy into this CTA whose bytes count on a barrier of the pair's first
__device__ __forceinline__ void tma_load_pair(uint32_t one, uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %5, 0;\n\t"
        "@q cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];\n\t}" ::
            "r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar), "r"(one)
        : "memory");
}

// D[tmem] = A * B^T over E4M3 codes (256 x 32 by N x 32), or += it; descriptors by their low words
template <int ADD>
__device__ __forceinline__ void umma_f8_pair(uint32_t one, uint32_t d, uint32_t a, uint32_t b, uint32_t high, uint32_t idesc) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b64 x, y;\n\tsetp.ne.u32 p, %5, 0;\n\tsetp.ne.u32 q, %6, 0;\n\t"
        "mov.b64 x, {%1, %3};\n\tmov.b64 y, {%2, %3};\n\t"
        "@q tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], x, y, %4, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(high), "r"(idesc), "n"(ADD), "r"(one)
        : "memory");
}

// arrive on the barrier of both CTAs once the products issued so far are done
template <int MASK>
__device__ __forceinline__ void umma_commit_mask(uint32_t one, uint32_t bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %2, 0;\n\t"
        "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}" ::"r"(bar),
        "h"((uint16_t)MASK), "r"(one)
        : "memory");
}
template <bool SPLIT>
__device__ __forceinline__ void umma_commit_pair(uint32_t one, uint32_t bar, int part) {
    if (!SPLIT || part == 0) umma_commit_mask<3>(one, bar);
    else if (part == 1) umma_commit_mask<12>(one, bar);
    else if (part == 2) umma_commit_mask<48>(one, bar);
    else umma_commit_mask<192>(one, bar);
}

__device__ __forceinline__ void arrive_cluster(uint32_t bar) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void tma_store_2d(const CUtensorMap* map, int x, int y, const void* src) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(x), "r"(y), "r"(smem_u32(src))
                 : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
__device__ __forceinline__ float4 load_shared(const float4* at) {
    float4 v;
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(smem_u32(at)) : "memory");
    return v;
}
// into another CTA of the cluster
__device__ __forceinline__ void store_cluster(uint32_t at, float2 p, float2 q) {
    asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(at), "f"(p.x), "f"(p.y), "f"(q.x), "f"(q.y) : "memory");
}
__device__ __forceinline__ void tma_stores_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }

// A variant: TILE features a pair's tile (256, or 128), OUT's type, SPLIT where 2 to 4 pairs
// of a cluster share a tile's k.  A warp's 64 features of 32 tokens lie in boxes of 32 rows
// of 128 bytes.
template <int OUT, int TILE, bool SPLIT>
struct PairTile {
    static constexpr int EW = TILE / 16, EPI = EW * 32, THREADS = EPI + 128;
    static constexpr int TB = 512 / TILE;                     // products in TMEM
    static constexpr int STAGE = 128 * 128 + TILE / 2 * 128;  // x and W rows of a block, of one CTA
    static constexpr int SIZE = OUT == KV4_F32 ? 4 : 2;
    static constexpr int BOXES = LP_COLS * SIZE / 128, BOX_COLS = 128 / SIZE;
    static constexpr int E = 16 / SIZE;                       // elements of 16 bytes
    static constexpr int BUF = 4096;                          // a warp's, for one box after the other
    static constexpr int STAGES = TILE == 256 ? 4 : SPLIT ? 5 : 6;
    static constexpr size_t SMEM = 1024 + (size_t)STAGES * STAGE + EW * BUF + (SPLIT ? LP_SLOTS_SUM * 32 * LP_COLS * 4 : 0);
};

// LATE: the test hook's kernel, where one CTA gets its scales late (a branch in the others took registers:
// 1500 tokens, 768 x 4096, BF16 12.2 -> 12.3 us).
template <int OUT, int ACT, int TILE, bool SPLIT, bool LATE = false>
__global__ void __launch_bounds__(PairTile<OUT, TILE, SPLIT>::THREADS, 1)
linear_pair_kernel(const __grid_constant__ CUtensorMap mx, const __grid_constant__ CUtensorMap mw,
                   const __grid_constant__ CUtensorMap mo, const __grid_constant__ CUtensorMap mr, const LinearArgs a, int tiles_n,
                   int tiles, int pairs) {
    using O = PairTile<OUT, TILE, SPLIT>;
    constexpr int STAGES = O::STAGES;
    extern __shared__ uint8_t dyn[];
    __shared__ PairBars bars;
    __shared__ PairScales sc;
    uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dyn) + 1023) & ~uintptr_t(1023));
    uint8_t* bufs = ring + (size_t)STAGES * O::STAGE;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = (int)blockIdx.x & 1, kb_all = (a.K + FP8_BLOCK - 1) / FP8_BLOCK;
    // a cluster's tiles, and this pair's part of k: whole groups of blocks
    const int n_parts = SPLIT ? pairs : 1, part = SPLIT ? ((int)blockIdx.x >> 1) % pairs : 0;
    const int first = ((int)blockIdx.x >> 1) / n_parts, step = ((int)gridDim.x >> 1) / n_parts;
    const int groups = (kb_all + LP_GROUP - 1) / LP_GROUP;
    const int kb0 = SPLIT ? groups * part / n_parts * LP_GROUP : 0;
    const int kb_n = SPLIT ? min(groups * (part + 1) / n_parts * LP_GROUP, kb_all) - kb0 : kb_all;
    const uint32_t lead = SPLIT ? 2 * part : 0;           // the pair's first CTA in the cluster

    if (threadIdx.x == 0) {
        for (int i = 0; i < STAGES; ++i) {
            mbar_init(&bars.full[i], 1);
            mbar_init(&bars.empty[i], 1);
        }
        for (int i = 0; i < O::TB; ++i) {
            mbar_init(&bars.tfull[i], 1);
            mbar_init(&bars.tempty[i], O::EW + (rank == 0));
        }
        for (int i = 0; i < LP_SLOTS; ++i) {
            mbar_init(&bars.sfull[i], 2);
            mbar_init(&bars.sempty[i], O::EW);
        }
        for (int i = 0; i < O::EW; ++i) mbar_init(&bars.res[i], 1);
        bars.failed = 0;
        fence_barrier_init();
    }
    pdl_wait();
    if (warp == O::EW + 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&bars.tmem)), "r"(512u)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();                                           // both have their columns and barriers
    tc_fence_after();
    pdl_launch_dependents();
    const uint32_t tmem = bars.tmem;
    volatile int* failed = &bars.failed;

    if (warp == O::EW) {
        // ---- copies
        const uint32_t one = elected(), ring0 = uniform(smem_u32(ring)), full0 = uniform(cluster_addr(&bars.full[0], lead));
        int st = 0, fresh = 1, phase = 1, left = 0;           // stage, whether never used, parity of its last emptying
        bool go = true;
        for (int tile = first; tile < tiles && go; tile += step) {
            const int t0 = tile / tiles_n * LP_TOKENS + rank * 128, n0 = tile % tiles_n * TILE + rank * (TILE / 2);
            for (int kb = 0; kb < kb_n; ++kb) {
                go = fresh || warp_wait(&bars.empty[st], phase);
                if (!go) break;
                const uint32_t to = ring0 + st * O::STAGE, bar = full0 + 8 * st;
                if (rank == 0 && one) mbar_arrive_expect_tx(&bars.full[st], 2 * O::STAGE);
                tma_load_pair(one, to, &mx, (kb0 + kb) * FP8_BLOCK, t0, bar);
                tma_load_pair(one, to + 128 * 128, &mw, (kb0 + kb) * FP8_BLOCK, n0, bar);
                ++left;
                if (++st == STAGES) {
                    st = 0;
                    fresh = 0;
                    phase ^= 1;
                }
            }
        }
        if (!go) *failed = 1;
        // before the pair ends copies in flight have landed (they count in the first CTA), and the
        // last arrivals of products, which come to both
        for (int i = left > STAGES ? left - STAGES : 0; i < left; ++i) {
            if (rank == 0) warp_wait(&bars.full[i % STAGES], (i / STAGES) & 1);
            if (go) warp_wait(&bars.empty[i % STAGES], (i / STAGES) & 1);
        }
    } else if (warp == O::EW + 1) {
        // ---- products of both
        if (rank == 0) {
            const uint32_t one = elected(), tm = uniform(tmem), ring0 = uniform(smem_u32(ring));
            const uint32_t high = (uint32_t)(umma_sdesc(0) >> 32), d0 = (uint32_t)umma_sdesc(ring0);
            const uint32_t tfull0 = uniform(smem_u32(&bars.tfull[0])), empty0 = uniform(smem_u32(&bars.empty[0]));
            constexpr uint32_t idesc = umma_idesc_f16(LP_TOKENS, TILE);  // E4M3 has F16's type number
            int st = 0, phase = 0, g = 0;
            bool go = true;
            for (int tile = first; tile < tiles && go; tile += step) {
                for (int kb = 0; kb < kb_n; ++kb, ++g) {
                    const int tb = g % O::TB;
                    go = warp_wait(&bars.full[st], phase) && (g < O::TB || warp_wait(&bars.tempty[tb], (g / O::TB - 1) & 1));
                    if (!go) break;
                    tc_fence_after();
                    const uint32_t da = d0 + st * (O::STAGE >> 4), db = da + (128 * 128 >> 4), d = tm + tb * TILE;
                    umma_f8_pair<0>(one, d, da, db, high, idesc);
                    umma_f8_pair<1>(one, d, da + 2, db + 2, high, idesc);
                    umma_f8_pair<1>(one, d, da + 4, db + 4, high, idesc);
                    umma_f8_pair<1>(one, d, da + 6, db + 6, high, idesc);
                    umma_commit_pair<SPLIT>(one, tfull0 + 8 * tb, part);
                    umma_commit_pair<SPLIT>(one, empty0 + 8 * st, part);
                    if (++st == STAGES) {
                        st = 0;
                        phase ^= 1;
                    }
                }
            }
            if (!go) {
                *failed = 1;
                if (g > 0) warp_wait(&bars.tfull[(g - 1) % O::TB], ((g - 1) / O::TB) & 1);   // products in flight
            }
        } else {
            // the second CTA's warps have read a product: one arrival tells the first
            const uint32_t e0 = cluster_addr(&bars.tempty[0], lead);
            int g = 0;
            bool go = true;
            for (int tile = first; tile < tiles && go; tile += step)
                for (int kb = 0; kb < kb_n && go; ++kb, ++g) {
                    go = warp_wait(&bars.tempty[g % O::TB], (g / O::TB) & 1);
                    if (go && lane == 0) arrive_cluster(e0 + 8 * (g % O::TB));
                }
        }
    } else if (warp >= O::EW + 2) {
        // ---- scales: two warps, 64 tokens each
        const int w2 = warp - O::EW - 2, blocks_n = (a.N + FP8_BLOCK - 1) / FP8_BLOCK;
        const bool quads = kb_all % 4 == 0 && (reinterpret_cast<uintptr_t>(a.xs) & 15) == 0;
        int gr = 0;
        if (LATE && blockIdx.x == 1)                          // one second at most
            for (const unsigned long long t0 = globaltimer(); globaltimer() - t0 < a.stall_ns;) __nanosleep(1000);
        for (int tile = first; tile < tiles && !*failed; tile += step) {
            const int t0 = tile / tiles_n * LP_TOKENS + rank * 128 + w2 * 64 + lane, nb = tile % tiles_n * TILE / 128;
            for (int kb = 0; kb < kb_n; kb += LP_GROUP, ++gr) {
                float4 v[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float* p = a.xs + (size_t)min(t0 + 32 * i, a.T - 1) * kb_all + kb0;
                    if (quads) v[i] = __ldg(reinterpret_cast<const float4*>(p + kb));
                    else
                        v[i] = make_float4(__ldg(p + kb), __ldg(p + min(kb + 1, kb_n - 1)), __ldg(p + min(kb + 2, kb_n - 1)),
                                           __ldg(p + min(kb + 3, kb_n - 1)));
                }
                float w = 0.f;
                if (w2 == 0 && lane < 2 * LP_GROUP)
                    w = __ldg(a.ws + (size_t)min(nb + lane / LP_GROUP, blocks_n - 1) * kb_all + kb0 + min(kb + lane % LP_GROUP, kb_n - 1));
                float b4[TILE / 64];
                if (kb == 0) {
#pragma unroll
                    for (int i = 0; i < TILE / 64; ++i)
                        b4[i] = a.bias && part == 0 ? __ldg(a.bias + min(tile % tiles_n * TILE + w2 * (TILE / 2) + 32 * i + lane, a.N - 1)) : 0.f;
                }
                const int slot = gr % LP_SLOTS;
                if (gr >= LP_SLOTS && !mbar_wait(&bars.sempty[slot], (gr / LP_SLOTS - 1) & 1)) *failed = 1;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int at = w2 * 64 + 32 * i + lane;
                    sc.x[slot][0][at] = v[i].x;
                    sc.x[slot][1][at] = v[i].y;
                    sc.x[slot][2][at] = v[i].z;
                    sc.x[slot][3][at] = v[i].w;
                }
                if (kb == 0) {
#pragma unroll
                    for (int i = 0; i < TILE / 64; ++i) sc.bias[slot][w2 * (TILE / 2) + 32 * i + lane] = b4[i];
                }
                if (w2 == 0 && lane < 2 * LP_GROUP) sc.w[slot][lane / LP_GROUP][lane % LP_GROUP] = w;
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars.sfull[slot]);
                if (*failed) break;
            }
        }
    } else {
        // ---- sums and results.  After a wait that ran out (ok) the warp goes on to
        // the end without waiting or writing, so that the barriers keep their counts.
        const int c0 = (warp >> 2) * LP_COLS;
        const uint32_t tcol = tmem + ((uint32_t)((warp & 3) * 32) << 16) + c0;
        uint8_t* buf = bufs + warp * O::BUF;
        // stores by TMA end on whole 16 bytes, whatever the map says: the features behind go one by one
        const int whole = a.N / O::E * O::E;
        int g = 0, gr = 0, turn = 0;                          // blocks, groups and residual boxes so far
        const int my = (warp & 3) * 32 + lane, wb = c0 / FP8_BLOCK;
        bool ok = true;
        for (int tile = first; tile < tiles; tile += step) {
            const int tw = tile / tiles_n * LP_TOKENS + rank * 128 + (warp & 3) * 32, t = tw + lane;   // the warp's rows, this one
            const int n0 = tile % tiles_n * TILE + c0;
            // the warp has something to write; the pairs of a cluster share a tile's results by warps
            const bool any = tw < a.T && n0 < a.N && warp % n_parts == part;
            if (a.res && any && ok && lane == 0) {
                tma_stores_read();
                mbar_arrive_expect_tx(&bars.res[warp], O::BUF);
                tma_load_2d(buf, &mr, n0, tw, &bars.res[warp]);
            }
            float2 acc[LP_COLS / 2];
            for (int kb = 0; kb < kb_n; ++kb, ++g) {
                const int in = kb % LP_GROUP, slot = gr % LP_SLOTS;
                if (in == 0 && ok && !mbar_wait(&bars.sfull[slot], (gr / LP_SLOTS) & 1)) {
                    *failed = 1;
                    ok = false;
                }
                if (kb == 0) {                                // sums begin with the bias
#pragma unroll
                    for (int i = 0; i < LP_COLS; i += 4) {
                        const float4 p = *reinterpret_cast<const float4*>(&sc.bias[slot][c0 + i]);
                        acc[i / 2] = make_float2(p.x, p.y);
                        acc[i / 2 + 1] = make_float2(p.z, p.w);
                    }
                }
                const float s = sc.x[slot][in][my] * sc.w[slot][wb][in];
                const int tb = g % O::TB;
                if (ok && !mbar_wait(&bars.tfull[tb], (g / O::TB) & 1)) {
                    *failed = 1;
                    ok = false;
                }
                __syncwarp();
                tc_fence_after();
                const uint32_t from = tcol + tb * TILE;
                const bool last = in == LP_GROUP - 1 || kb == kb_n - 1;
                uint32_t r[2][16];
                tmem_fetch16(from, r[0]);
#pragma unroll
                for (int c = 0; c < LP_COLS / 16; ++c) {
                    tmem_arrived(r[c & 1]);
                    if (c + 1 < LP_COLS / 16) tmem_fetch16(from + 16 * (c + 1), r[(c + 1) & 1]);
                    else {                                    // all read: the products after next may come
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) {
                            arrive_relaxed(&bars.tempty[tb]);
                            if (last) mbar_arrive(&bars.sempty[slot]);
                        }
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i) fma2(acc[8 * c + i], r[c & 1][2 * i], r[c & 1][2 * i + 1], s, s);
                }
                gr += last;
            }
            if (SPLIT) {
                // (one tile a cluster) a warp's sums go to the pair that has its results, which adds
                // the others' in their order; slots by the owner's warps, then by senders.  As pairs of
                // registers and four loads at a time: with the sums moved as quads in one batch the loop
                // above lost 0.05 us a block.  (Rows of 16 bits still spill 20 to 48 bytes here, F32
                // rows none: 256 tokens, 4096 x 2048, 10.5 and 10.15 us.)
                const int owner = warp % n_parts;
                float4* slots = reinterpret_cast<float4*>(bufs + O::EW * O::BUF) + warp / n_parts * (n_parts - 1) * (LP_COLS / 4 * 32) + lane;
                if (owner != part) {
                    const uint32_t to = cluster_addr(slots + (part - (part > owner)) * (LP_COLS / 4 * 32), 2 * owner + rank);
#pragma unroll
                    for (int i = 0; i < LP_COLS / 4; ++i) store_cluster(to + 512 * i, acc[2 * i], acc[2 * i + 1]);
                }
                __syncwarp();
                cluster_sync();
#pragma unroll 1
                for (int p = 0; p < n_parts - 1 && any; ++p) {
#pragma unroll
                    for (int i = 0; i < LP_COLS / 4; i += 4) {
                        float4 v[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j) v[j] = load_shared(slots + p * (LP_COLS / 4 * 32) + 32 * (i + j));
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            fma2(acc[2 * (i + j)], __float_as_uint(v[j].x), __float_as_uint(v[j].y), 1.f, 1.f);
                            fma2(acc[2 * (i + j) + 1], __float_as_uint(v[j].z), __float_as_uint(v[j].w), 1.f, 1.f);
                        }
                    }
                }
            }
            ok = __all_sync(0xffffffffu, ok);
            if (!any || !ok) continue;                        // the same for the whole warp
#pragma unroll
            for (int b = 0; b < O::BOXES; ++b) {
                if (a.res) {
                    if (b && lane == 0) {
                        tma_stores_read();
                        mbar_arrive_expect_tx(&bars.res[warp], O::BUF);
                        tma_load_2d(buf, &mr, n0 + b * O::BOX_COLS, tw, &bars.res[warp]);
                    }
                    if (ok && !mbar_wait(&bars.res[warp], turn & 1)) {
                        *failed = 1;
                        ok = false;
                    }
                    ++turn;
                    ok = __all_sync(0xffffffffu, ok);
                } else {
                    if (lane == 0) tma_stores_read();
                    __syncwarp();
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {                 // 16 bytes a turn
                    constexpr int E = O::E;
                    const int c = b * O::BOX_COLS + i * E;
                    float v[E];
#pragma unroll
                    for (int j = 0; j < E; ++j) v[j] = j & 1 ? acc[(c + j) / 2].y : acc[(c + j) / 2].x;
                    activate(v, ACT);
                    uint4* at = reinterpret_cast<uint4*>(buf + lane * 128 + ((i ^ (lane & 7)) << 4));
                    if (a.res) {
                        const uint4 u = *at;
                        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                        for (int j = 0; j < E; ++j) v[j] += row_element<OUT>(w, j);
                    }
                    uint32_t w[4];
                    row_pack<OUT>(v, w);
                    *at = make_uint4(w[0], w[1], w[2], w[3]);
                    if (n0 + c == whole && ok && t < a.T) {
                        using type = typename RowType<OUT>::type;
                        type* p = static_cast<type*>(a.out) + (size_t)t * a.out_stride + whole;
#pragma unroll
                        for (int j = 0; j < E - 1; ++j)
                            if (whole + j < a.N) p[j] = RowType<OUT>::store(v[j]);
                    }
                }
                fence_proxy_async();
                __syncwarp();
                if (lane == 0 && ok && n0 + b * O::BOX_COLS < whole) tma_store_2d(&mo, n0 + b * O::BOX_COLS, tw, buf);
                __syncwarp();
            }
        }
        if (lane == 0) tma_stores_read();
        __syncwarp();
    }
    if (SPLIT && warp >= O::EW) {
        __syncwarp();
        cluster_sync();                                       // where the sums meet
    }
    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 0 && *failed) atomicExch(a.status, ST_TIMEOUT);
    cluster_sync();                                           // neither works in the other's memory any more
    if (warp == O::EW + 1) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
}

template <int OUT, int ACT, int TILE, bool SPLIT>
auto pair_kernel(bool late) {
    if constexpr (OUT == KV4_F32 && ACT == ACT_NONE)
        if (late) return linear_pair_kernel<OUT, ACT, TILE, SPLIT, true>;
    return linear_pair_kernel<OUT, ACT, TILE, SPLIT>;
}

template <int OUT, int ACT, int TILE, bool SPLIT>
cudaError_t launch_out(const LinearArgs& a, int parts, const LinearRun& run) {
    using O = PairTile<OUT, TILE, SPLIT>;
    CUtensorMap mx, mw, mo, mr;
    if (!tensor_map_codes(&mx, a.x, (uint64_t)a.K, (uint64_t)a.T, 128) || !tensor_map_codes(&mw, a.w, (uint64_t)a.K, (uint64_t)a.N, TILE / 2) ||
        !tensor_map_rows(&mo, a.out, OUT, (uint64_t)(a.N < O::E ? O::E : a.N / O::E * O::E), (uint64_t)a.T, (uint64_t)a.out_stride, 32) ||
        !tensor_map_rows(&mr, a.res ? a.res : a.out, OUT, (uint64_t)a.N, (uint64_t)a.T, (uint64_t)(a.res ? a.res_stride : a.out_stride), 32))
        return cudaErrorInvalidValue;
    const int tiles_n = (a.N + TILE - 1) / TILE;
    const int64_t tiles = (int64_t)tiles_n * ((a.T + LP_TOKENS - 1) / LP_TOKENS);
    if (tiles > INT_MAX / 8) return cudaErrorInvalidValue;
    if (SPLIT != (parts > 1) || parts > 4 || (SPLIT && a.K <= FP8_BLOCK * LP_GROUP * (parts - 1))) return cudaErrorInvalidValue;
    const int pairs = SPLIT ? (int)tiles * parts : (int)(tiles < run.num_sms / 2 ? tiles : run.num_sms / 2);
    const bool late = OUT == KV4_F32 && ACT == ACT_NONE && a.stall_ns;
    const auto kernel = pair_kernel<OUT, ACT, TILE, SPLIT>(late);
    const uint64_t bit = 1ull << (((late ? 3 : OUT) * 4 + ACT) * 3 + (TILE == 256 ? 0 : SPLIT ? 1 : 2));
    if (!(*run.ready & bit)) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)O::SMEM);
        if (e != cudaSuccess) return e;
        *run.ready |= bit;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * pairs);
    cfg.blockDim = dim3(O::THREADS);
    cfg.dynamicSmemBytes = O::SMEM;
    cfg.stream = run.st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 2 * parts;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, mx, mw, mo, mr, a, tiles_n, (int)tiles, parts);
}

// A kernel an activation: 64 results' code for each is long, and is fetched past or branched
// around otherwise (16384 tokens, 2048 x 5120: none 164 us, SiLU 182, GELU 192; with one kernel for
// the three 166, 196, 203; with one for all four 191 and more).
template <int OUT, int TILE, bool SPLIT>
cudaError_t launch_act(const LinearArgs& a, int parts, const LinearRun& run) {
    return a.act == ACT_NONE   ? launch_out<OUT, ACT_NONE, TILE, SPLIT>(a, parts, run)
           : a.act == ACT_RELU ? launch_out<OUT, ACT_RELU, TILE, SPLIT>(a, parts, run)
           : a.act == ACT_SILU ? launch_out<OUT, ACT_SILU, TILE, SPLIT>(a, parts, run)
                               : launch_out<OUT, ACT_GELU, TILE, SPLIT>(a, parts, run);
}
template <int OUT>
cudaError_t launch_type(const LinearArgs& a, int tile, int parts, const LinearRun& run) {
    return tile == 256 ? launch_act<OUT, 256, false>(a, 1, run)
           : parts > 1 ? launch_act<OUT, 128, true>(a, parts, run)
                       : launch_act<OUT, 128, false>(a, 1, run);
}

}  // namespace

cudaError_t launch_linear_pair(const LinearArgs& a, int tile, int parts, const LinearRun& run) {
    return a.out_t == KV4_F32   ? launch_type<KV4_F32>(a, tile, parts, run)
           : a.out_t == KV4_F16 ? launch_type<KV4_F16>(a, tile, parts, run)
                                : launch_type<KV4_BF16>(a, tile, parts, run);
}

}  // namespace qmoe
