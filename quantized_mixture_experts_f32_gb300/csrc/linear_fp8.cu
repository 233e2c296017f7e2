// linear_fp8.cu -- out = act(x W^T + bias) + residual over E4M3 codes with block scales.
//
//   z[t][n] = sum_b xs[t][b] ws[n/128][b] sum_{k in block b} x[t][k] W[n][k]
//
// The rows of W are the 128-row operand of tcgen05 (kind::f8f6f4, E4M3), TN tokens the
// columns, so that a call of one token wastes columns of the small operand and reads W
// once.  Every block of 128 k is a product of its own in TMEM; warps of the epilogue
// scale it into fp32 registers, W's scale being one number a tile and block, while
// the next blocks' products run.  A thread has a feature and a run of tokens, so bias
// is a register and a warp's stores are neighbours.
#include <limits.h>

#include "linear_fp8.cuh"

namespace qmoe {

namespace {

constexpr int LN_M = 128;                     // features a tile
constexpr int LN_GROUP = 4, LN_SLOTS = 3;     // blocks of k whose scales are staged together, such groups
constexpr int LN_SPLIT_MAX = 8;               // CTAs of a cluster that share a tile's k blocks
constexpr int LN_STAGES_MAX = 12;

// Feature n of N tokens from t on: residual added, stored.  All residuals are read before
// the first result is written, so that their latencies overlap and out may be residual.
template <int T, int N>
__device__ __forceinline__ void put(const LinearArgs& a, int t, int n, float (&v)[N]) {
    using R = RowType<T>;
    using type = typename R::type;
    const int m = a.T - t;
    if (m <= 0) return;
    if (a.res) {
        const type* p = static_cast<const type*>(a.res) + (size_t)t * a.res_stride + n;
        type r[N];
#pragma unroll
        for (int i = 0; i < N; ++i, p += a.res_stride)
            if (i < m) r[i] = *p;
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (i < m) v[i] += R::load(r[i]);
    }
    type* p = static_cast<type*>(a.out) + (size_t)t * a.out_stride + n;
    if (m >= N) {
#pragma unroll
        for (int i = 0; i < N; ++i, p += a.out_stride) *p = R::store(v[i]);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i, p += a.out_stride)
            if (i < m) *p = R::store(v[i]);
    }
}

// Features n .. n+3 (n a multiple of four) of a token: residual added, stored.  Rows begin on
// 16 bytes, so the four lie in one word of 16 or 8 bytes.
template <int T>
__device__ __forceinline__ void put_row(const LinearArgs& a, int t, int n, float (&v)[4]) {
    using R = RowType<T>;
    using type = typename R::type;
    using word = typename R::word;
    type* out = static_cast<type*>(a.out) + (size_t)t * a.out_stride + n;
    const type* res = static_cast<const type*>(a.res) + (size_t)t * a.res_stride + n;
    if (n + 4 <= a.N) {
        if (a.res) {
            const word w = *reinterpret_cast<const word*>(res);
            const type* r = reinterpret_cast<const type*>(&w);
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] += R::load(r[j]);
        }
        word w;
        type* r = reinterpret_cast<type*>(&w);
#pragma unroll
        for (int j = 0; j < 4; ++j) r[j] = R::store(v[j]);
        *reinterpret_cast<word*>(out) = w;
        return;
    }
#pragma unroll
    for (int j = 0; j < 3; ++j)
        if (n + j < a.N) out[j] = R::store(a.res ? v[j] + R::load(res[j]) : v[j]);
}

// z + bias through the activation, and out
template <int N>
__device__ __forceinline__ void finish(const LinearArgs& a, int t, int n, float bias, float (&v)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += bias;
    activate(v, a.act);
    if (a.out_t == KV4_F32) put<KV4_F32>(a, t, n, v);
    else if (a.out_t == KV4_F16) put<KV4_F16>(a, t, n, v);
    else put<KV4_BF16>(a, t, n, v);
}

// D[tmem] = A * B^T over E4M3 codes (128 x 32 by N x 32), or += it; descriptors by their low words
template <int ADD>
__device__ __forceinline__ void umma_f8(uint32_t one, uint32_t d, uint32_t a, uint32_t b, uint32_t high, uint32_t idesc) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b64 x, y;\n\tsetp.ne.u32 p, %5, 0;\n\tsetp.ne.u32 q, %6, 0;\n\t"
        "mov.b64 x, {%1, %3};\n\tmov.b64 y, {%2, %3};\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], x, y, %4, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(high), "r"(idesc), "n"(ADD), "r"(one)
        : "memory");
}
__device__ __forceinline__ void umma_commit_one(uint32_t one, uint32_t bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar), "r"(one)
        : "memory");
}
__device__ __forceinline__ void tma_load_one(uint32_t one, uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %5, 0;\n\t"
        "@q cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];\n\t}" ::
            "r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar), "r"(one)
        : "memory");
}

__device__ __forceinline__ void st_cluster(uint32_t addr, float v) {
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

// Shapes of a variant: TN tokens a tile.
template <int TN>
struct LinearTile {
    static constexpr int EW = TN <= 32 ? 4 : 8;               // warps that scale and sum
    static constexpr int EPI = EW * 32, THREADS = EPI + 128;
    static constexpr int COLS = TN * 4 / EW;                  // tokens of a thread
    static constexpr int TB = 4;                              // products in TMEM
    static constexpr int TMEM = TN * TB;
    static constexpr int STAGE = LN_M * 128 + TN * 128;
    static constexpr int PARTS = TN * LN_M * 4;               // bytes of a tile's sums
};

struct LinearBars {
    uint64_t full[LN_STAGES_MAX], empty[LN_STAGES_MAX], tfull[4], tempty[4], sfull[LN_SLOTS], sempty[LN_SLOTS];
    uint32_t tmem;
    int failed;
};

template <int TN>
__global__ void __launch_bounds__(LinearTile<TN>::THREADS, TN <= 32 ? 2 : 1)
linear_umma_kernel(const __grid_constant__ CUtensorMap mw, const __grid_constant__ CUtensorMap mx, const LinearArgs a,
                   int stages, int split, int tiles_m, int tiles) {
    using L = LinearTile<TN>;
    extern __shared__ uint8_t dyn[];
    __shared__ LinearBars bars;
    __shared__ __align__(16) float sc[LN_SLOTS][LN_GROUP][TN];
    uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dyn) + 1023) & ~uintptr_t(1023));
    float* sums = reinterpret_cast<float*>(ring + (size_t)stages * L::STAGE);     // [TN][LN_M]
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int kb_all = (a.K + FP8_BLOCK - 1) / FP8_BLOCK;
    const int rank = split > 1 ? (int)blockIdx.x % split : 0;
    const int kb0 = (int)((int64_t)kb_all * rank / split), kb1 = (int)((int64_t)kb_all * (rank + 1) / split);
    const int first = (int)blockIdx.x / split, step = (int)gridDim.x / split;

    if (threadIdx.x == 0) {
        for (int i = 0; i < stages; ++i) {
            mbar_init(&bars.full[i], 1);
            mbar_init(&bars.empty[i], 1);
        }
        for (int i = 0; i < L::TB; ++i) {
            mbar_init(&bars.tfull[i], 1);
            mbar_init(&bars.tempty[i], L::EW);
        }
        for (int i = 0; i < LN_SLOTS; ++i) {
            mbar_init(&bars.sfull[i], 1);
            mbar_init(&bars.sempty[i], L::EW);
        }
        bars.failed = 0;
        fence_barrier_init();
    }
    if (threadIdx.x == 32) {
        prefetch_map(&mw);
        prefetch_map(&mx);
    }
    if (split > 1) cluster_arrive();                          // started
    // TMEM is taken after the kernels before have ended, and before the ones behind may
    // start: neither can wait for the other's columns
    pdl_wait();
    if (warp == L::EW + 1) tmem_alloc(&bars.tmem, L::TMEM);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    pdl_launch_dependents();
    const uint32_t tmem = bars.tmem;
    volatile int* failed = &bars.failed;

    if (warp == L::EW) {
        // ---- copies
        const uint32_t one = elected(), ring0 = uniform(smem_u32(ring)), full0 = uniform(smem_u32(&bars.full[0]));
        int st = 0, fresh = 1, phase = 1, left = 0;           // stage, whether never used, parity of its last emptying
        bool go = true;
        for (int tile = first; tile < tiles && go; tile += step) {
            const int tm = tile % tiles_m, tn = tile / tiles_m;
            for (int kb = kb0; kb < kb1; ++kb) {
                go = fresh || warp_wait(&bars.empty[st], phase);
                if (!go) break;
                const uint32_t to = ring0 + st * L::STAGE, bar = full0 + 8 * st;
                if (one) mbar_arrive_expect_tx(&bars.full[st], L::STAGE);
                tma_load_one(one, to, &mw, kb * FP8_BLOCK, tm * LN_M, bar);
                tma_load_one(one, to + LN_M * 128, &mx, kb * FP8_BLOCK, tn * TN, bar);
                ++left;
                if (++st == stages) {
                    st = 0;
                    fresh = 0;
                    phase ^= 1;
                }
            }
        }
        if (!go) {
            *failed = 1;
            // copies in flight have landed before the CTA ends
            for (int i = left > stages ? left - stages : 0; i < left; ++i) warp_wait(&bars.full[i % stages], (i / stages) & 1);
        }
    } else if (warp == L::EW + 1 || warp == L::EW + 3) {
        // ---- products: two warps take the blocks in turn, since one spends longer on a block's
        // waits and issue (470 cycles) than the tensor cores on its products (170 to 210)
        const uint32_t one = elected(), tm0 = uniform(tmem), high = (uint32_t)(umma_sdesc(0) >> 32);
        const uint32_t d0 = (uint32_t)umma_sdesc(uniform(smem_u32(ring)));
        const uint32_t tfull0 = uniform(smem_u32(&bars.tfull[0])), empty0 = uniform(smem_u32(&bars.empty[0]));
        constexpr uint32_t idesc = umma_idesc_f16(LN_M, TN);              // E4M3 has F16's type number
        const int mine = warp == L::EW + 1 ? 0 : 1, all = first < tiles ? ((tiles - 1 - first) / step + 1) * (kb1 - kb0) : 0;
        int st = mine % stages, phase = mine / stages & 1, g = mine;
        bool go = true;
        for (; g < all; g += 2) {
            const int tb = g % L::TB;
            go = warp_wait(&bars.full[st], phase) && (g < L::TB || warp_wait(&bars.tempty[tb], (g / L::TB - 1) & 1));
            if (!go) break;
            tc_fence_after();
            const uint32_t da = d0 + st * (L::STAGE >> 4), db = da + (LN_M * 128 >> 4), d = tm0 + tb * TN;
            umma_f8<0>(one, d, da, db, high, idesc);
            umma_f8<1>(one, d, da + 2, db + 2, high, idesc);
            umma_f8<1>(one, d, da + 4, db + 4, high, idesc);
            umma_f8<1>(one, d, da + 6, db + 6, high, idesc);
            umma_commit_one(one, tfull0 + 8 * tb);
            umma_commit_one(one, empty0 + 8 * st);
            for (int i = 0; i < 2; ++i)
                if (++st == stages) {
                    st = 0;
                    phase ^= 1;
                }
        }
        if (!go) {
            *failed = 1;
            if (g >= 2) warp_wait(&bars.tfull[(g - 2) % L::TB], ((g - 2) / L::TB) & 1);   // products in flight
        }
    } else if (warp == L::EW + 2) {
        // ---- scales: a token's times the block's of W, four blocks of k at a time
        constexpr int PER = TN * LN_GROUP / 32;
        int gr = 0;
        bool go = true;
        for (int tile = first; tile < tiles && go; tile += step) {
            const int t0 = (tile / tiles_m) * TN;
            const float* ws = a.ws + (size_t)(tile % tiles_m) * kb_all;
            for (int kb = kb0; kb < kb1 && go; kb += LN_GROUP, ++gr) {
                float x[PER];
                const int k = min(kb + lane % LN_GROUP, kb1 - 1);
                const float w = __ldg(ws + k);
#pragma unroll
                for (int i = 0; i < PER; ++i) x[i] = __ldg(a.xs + (size_t)min(t0 + (32 * i + lane) / LN_GROUP, a.T - 1) * kb_all + k);
                const int slot = gr % LN_SLOTS;
                go = gr < LN_SLOTS || warp_wait(&bars.sempty[slot], (gr / LN_SLOTS - 1) & 1);
#pragma unroll
                for (int i = 0; i < PER; ++i) sc[slot][lane % LN_GROUP][(32 * i + lane) / LN_GROUP] = x[i] * w;
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars.sfull[slot]);
            }
        }
        if (!go) *failed = 1;
    } else {
        // ---- sums and results.  After a wait that ran out (ok) the warp goes on to the end
        // without waiting or writing, so that the barriers keep their counts.
        const int f = (warp & 3) * 32 + lane, c0 = (warp >> 2) * L::COLS;
        const uint32_t tcol = tmem + ((uint32_t)((warp & 3) * 32) << 16) + c0;
        int g = 0, gr = 0;
        bool ok = true;
        for (int tile = first; tile < tiles; tile += step) {
            const int tm = tile % tiles_m, t0 = (tile / tiles_m) * TN;
            const int n = tm * LN_M + f;
            float2 acc[L::COLS / 2];
#pragma unroll
            for (int i = 0; i < L::COLS / 2; ++i) acc[i] = make_float2(0.f, 0.f);
            for (int kb = kb0; kb < kb1; ++kb, ++g) {
                const int in = (kb - kb0) % LN_GROUP, slot = gr % LN_SLOTS, tb = g % L::TB;
                const bool last = in == LN_GROUP - 1 || kb == kb1 - 1;
                if (ok && ((in == 0 && !mbar_wait(&bars.sfull[slot], (gr / LN_SLOTS) & 1)) ||
                           !mbar_wait(&bars.tfull[tb], (g / L::TB) & 1))) {
                    *failed = 1;
                    ok = false;
                }
                __syncwarp();
                tc_fence_after();
                const float* s = &sc[slot][in][c0];
                uint32_t r[L::COLS];
                tmem_fetch(tcol + tb * TN, r);
                tmem_arrived(r);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) arrive_relaxed(&bars.tempty[tb]);   // the product after next may come
#pragma unroll
                for (int i = 0; i < L::COLS / 4; ++i) {
                    const float4 v = *reinterpret_cast<const float4*>(s + 4 * i);
                    fma2(acc[2 * i], r[4 * i], r[4 * i + 1], v.x, v.y);
                    fma2(acc[2 * i + 1], r[4 * i + 2], r[4 * i + 3], v.z, v.w);
                }
                if (last) {
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bars.sempty[slot]);
                    ++gr;
                }
            }
            if (split > 1) {
                // to the CTA of the cluster that joins these features
                cluster_wait();                               // they have all started
                const int share = LN_M / split, to = f / share;
                const uint32_t mine = cluster_addr(sums, to) + 4 * ((rank * TN + c0) * share + f % share);
#pragma unroll
                for (int i = 0; i < L::COLS; ++i)
                    if (t0 + c0 + i < a.T) st_cluster(mine + 4 * i * share, i & 1 ? acc[i / 2].y : acc[i / 2].x);
                continue;                                     // the only tile
            }
            ok = __all_sync(0xffffffffu, ok);
            if (ok && n < a.N) {
                const float bias = a.bias ? a.bias[n] : 0.f;
#pragma unroll
                for (int c = 0; c < L::COLS; c += 8) {
                    float v[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[i] = i & 1 ? acc[(c + i) / 2].y : acc[(c + i) / 2].x;
                    finish(a, t0 + c0 + c, n, bias, v);
                }
            }
            __syncwarp();
        }
    }
    tc_fence_before();
    __syncthreads();
    // before the CTA waits for others of its cluster, so that none waits while it holds
    // columns that another's CTA needs
    if (warp == L::EW + 1) tmem_dealloc(tmem, L::TMEM);
    if (split > 1) {
        // each CTA adds its share of the features, the parts in the order of ranks
        if (warp >= L::EW) cluster_wait();
        __syncwarp();
        cluster_arrive();
        cluster_wait();
        const int tm = first % tiles_m, t0 = (first / tiles_m) * TN, share = LN_M / split, quads = share / 4;
        const int rows = min(TN, a.T - t0);
        for (int i = (int)threadIdx.x; i < rows * quads; i += L::THREADS) {
            const int t = i / quads, q = i - t * quads, n = tm * LN_M + rank * share + 4 * q;
            if (n >= a.N) continue;
            float z[4] = {};
            for (int r = 0; r < split; ++r) {
                const float4 v = *reinterpret_cast<const float4*>(sums + (r * TN + t) * share + 4 * q);
                z[0] += v.x;
                z[1] += v.y;
                z[2] += v.z;
                z[3] += v.w;
            }
            if (a.bias) {
#pragma unroll
                for (int j = 0; j < 4; ++j) z[j] += a.bias[min(n + j, a.N - 1)];
            }
            activate(z, a.act);
            if (a.out_t == KV4_F32) put_row<KV4_F32>(a, t0 + t, n, z);
            else if (a.out_t == KV4_F16) put_row<KV4_F16>(a, t0 + t, n, z);
            else put_row<KV4_BF16>(a, t0 + t, n, z);
        }
    }
    if (threadIdx.x == 0 && *failed) atomicExch(a.status, ST_TIMEOUT);
}

template <int TN>
cudaError_t prepare_one() {
    return cudaFuncSetAttribute(linear_umma_kernel<TN>, cudaFuncAttributeMaxDynamicSharedMemorySize, 212 * 1024);
}

template <int TN>
cudaError_t launch_tile(const LinearArgs& a, int split, int num_sms, cudaStream_t st) {
    using L = LinearTile<TN>;
    CUtensorMap mw, mx;
    if (!tensor_map_codes(&mw, a.w, (uint64_t)a.K, (uint64_t)a.N, LN_M) || !tensor_map_codes(&mx, a.x, (uint64_t)a.K, (uint64_t)a.T, TN))
        return cudaErrorInvalidValue;
    const int kb = (a.K + FP8_BLOCK - 1) / FP8_BLOCK, tiles_m = (a.N + LN_M - 1) / LN_M;
    const int64_t tiles = (int64_t)tiles_m * ((a.T + TN - 1) / TN);
    if (tiles > INT_MAX / LN_SPLIT_MAX) return cudaErrorInvalidValue;
    // Where every CTA has one tile, no more stages than it has blocks: what shared memory is left
    // lets the next kernel's CTAs start beside this one's.
    const int most = (int)(((TN <= 32 ? 104 : 208) * 1024 - L::PARTS) / L::STAGE);
    const int per = (kb + split - 1) / split;
    int stages = most < LN_STAGES_MAX ? most : LN_STAGES_MAX;
    if (per < stages) stages = per;
    const int cap = num_sms * (TN <= 32 ? 2 : 1);
    const int grid = split > 1 ? (int)tiles * split : (int)(tiles < cap ? tiles : cap);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(L::THREADS);
    cfg.dynamicSmemBytes = 1024 + (size_t)stages * L::STAGE + L::PARTS;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = split;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = split > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, linear_umma_kernel<TN>, mw, mx, a, stages, split, tiles_m, (int)tiles);
}

}  // namespace

cudaError_t linear_fp8_prepare() {
    cudaError_t e = prepare_one<16>();
    if (e == cudaSuccess) e = prepare_one<32>();
    if (e == cudaSuccess) e = prepare_one<64>();
    if (e == cudaSuccess) e = linear_pair_prepare();
    return e;
}

cudaError_t launch_linear_fp8(const LinearArgs& a, int num_sms, cudaStream_t st) {
    if (a.T > 256) return launch_linear_pair(a, num_sms, st);
    if (a.T <= LN_FEW) return launch_linear_few(a, st);
    const int tn = a.T <= 16 ? 16 : a.T <= 32 ? 32 : 64;
    const int kb = (a.K + FP8_BLOCK - 1) / FP8_BLOCK;
    const int64_t tiles = (int64_t)((a.N + LN_M - 1) / LN_M) * ((a.T + tn - 1) / tn);
    int split = 1;
    while (split < LN_SPLIT_MAX && 2 * split <= kb && tiles * split < num_sms) split *= 2;
    switch (tn) {
        case 16: return launch_tile<16>(a, split, num_sms, st);
        case 32: return launch_tile<32>(a, split, num_sms, st);
        default: return launch_tile<64>(a, split, num_sms, st);
    }
}

}  // namespace qmoe
