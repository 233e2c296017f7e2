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
constexpr int LN_GROUP = 4;                   // k blocks whose scales are staged together
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

// D[tmem] (+)= A * B^T over E4M3 codes (M x 32 by N x 32), issued by one thread
__device__ __forceinline__ void umma_f8(uint32_t tmem_d, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem_d),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ float ld_cluster(uint32_t saddr, int rank) {
    float v;
    asm volatile("{\n\t.reg .u32 a;\n\tmapa.shared::cluster.u32 a, %1, %2;\n\tld.shared::cluster.f32 %0, [a];\n\t}"
                 : "=f"(v)
                 : "r"(saddr), "r"(rank));
    return v;
}

// Shapes of a variant: TN tokens a tile, EW warps of the epilogue, TB products in TMEM.
template <int TN>
struct LinearTile {
    static constexpr int EW = TN <= 64 ? 4 : TN / 16;            // at most 64 columns a thread
    static constexpr int EPI = EW * 32, THREADS = EPI + 64;
    static constexpr int COLS = TN * 4 / EW;                  // columns of a thread
    static constexpr int TB = TN >= 256 ? 2 : 4;
    static constexpr int TMEM = TN * TB < 32 ? 32 : TN * TB;
    static constexpr int STAGE = LN_M * 128 + TN * 128;
};

struct LinearBars {
    uint64_t full[LN_STAGES_MAX], empty[LN_STAGES_MAX], tfull[4], tempty[4];
    uint32_t tmem;
    int failed;
};

template <int TN>
__global__ void __launch_bounds__(LinearTile<TN>::THREADS, 1)
linear_umma_kernel(const __grid_constant__ CUtensorMap mw, const __grid_constant__ CUtensorMap mx, const LinearArgs a,
                   int stages, int split, int tiles_m, int tiles) {
    using L = LinearTile<TN>;
    extern __shared__ uint8_t dyn[];
    __shared__ LinearBars bars;
    __shared__ __align__(16) float sc[2][LN_GROUP][TN + 8];
    uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dyn) + 1023) & ~uintptr_t(1023));
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
        bars.failed = 0;
        fence_barrier_init();
    }
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
        if (lane == 0) {
            int g = 0, loaded = 0;
            for (int tile = first; tile < tiles && !*failed; tile += step) {
                const int tm = tile % tiles_m, tn = tile / tiles_m;
                for (int kb = kb0; kb < kb1; ++kb, ++g) {
                    const int st = g % stages;
                    if (g >= stages && !mbar_wait(&bars.empty[st], (g / stages - 1) & 1)) {
                        *failed = 1;
                        break;
                    }
                    uint8_t* to = ring + (size_t)st * L::STAGE;
                    mbar_arrive_expect_tx(&bars.full[st], L::STAGE);
                    tma_load_2d(to, &mw, kb * FP8_BLOCK, tm * LN_M, &bars.full[st]);
                    tma_load_2d(to + LN_M * 128, &mx, kb * FP8_BLOCK, tn * TN, &bars.full[st]);
                    ++loaded;
                }
            }
            // copies in flight have landed before the CTA ends
            for (int i = loaded > stages ? loaded - stages : 0; i < loaded; ++i) mbar_wait(&bars.full[i % stages], (i / stages) & 1);
        }
    } else if (warp == L::EW + 1) {
        // ---- products
        if (lane == 0) {
            constexpr uint32_t idesc = umma_idesc_f16(LN_M, TN);          // E4M3 has F16's type number
            int g = 0;
            for (int tile = first; tile < tiles && !*failed; tile += step) {
                for (int kb = kb0; kb < kb1; ++kb, ++g) {
                    const int st = g % stages, tb = g % L::TB;
                    if (!mbar_wait(&bars.full[st], (g / stages) & 1) ||
                        (g >= L::TB && !mbar_wait(&bars.tempty[tb], (g / L::TB - 1) & 1))) {
                        *failed = 1;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t s = smem_u32(ring + (size_t)st * L::STAGE);
                    const uint64_t da = umma_sdesc(s), db = umma_sdesc(s + LN_M * 128);
#pragma unroll
                    for (int k = 0; k < 4; ++k) umma_f8(tmem + tb * TN, da + 2 * k, db + 2 * k, idesc, k > 0);
                    umma_commit(&bars.empty[st]);
                    umma_commit(&bars.tfull[tb]);
                }
            }
            if (*failed && g > 0) mbar_wait(&bars.tfull[(g - 1) % L::TB], ((g - 1) / L::TB) & 1);   // products in flight
        }
    } else {
        // ---- scales, sums and results.  After a wait that ran out (ok) the warp goes on to
        // the end without waiting or writing, so that the barriers keep their counts.
        const int e = threadIdx.x, f = (warp & 3) * 32 + lane, c0 = (warp >> 2) * L::COLS;
        const uint32_t tcol = tmem + ((uint32_t)((warp & 3) * 32) << 16) + c0;
        constexpr int PER = (TN * LN_GROUP + L::EPI - 1) / L::EPI;         // staged scales a thread
        int g = 0;
        bool ok = true;
        for (int tile = first; tile < tiles; tile += step) {
            const int tm = tile % tiles_m, t0 = (tile / tiles_m) * TN;
            const int n = tm * LN_M + f;
            const float* ws = a.ws + (size_t)tm * kb_all;
            float2 acc[L::COLS / 2];
#pragma unroll
            for (int i = 0; i < L::COLS / 2; ++i) acc[i] = make_float2(0.f, 0.f);
            float next[PER];
            auto fetch = [&](int kb) {
#pragma unroll
                for (int i = 0; i < PER; ++i) {
                    const int at = i * L::EPI + e, t = t0 + at / LN_GROUP, k = kb + at % LN_GROUP;
                    next[i] = at < TN * LN_GROUP && t < a.T && k < kb1 ? a.xs[(size_t)t * kb_all + k] * ws[k] : 0.f;
                }
            };
            fetch(kb0);
            for (int kb = kb0; kb < kb1; ++kb, ++g) {
                const int in = (kb - kb0) % LN_GROUP, half = ((kb - kb0) / LN_GROUP) & 1;
                if (in == 0) {
#pragma unroll
                    for (int i = 0; i < PER; ++i) {
                        const int at = i * L::EPI + e;
                        if (at < TN * LN_GROUP) sc[half][at % LN_GROUP][at / LN_GROUP] = next[i];
                    }
                    named_bar(1, L::EPI);
                    if (kb + LN_GROUP < kb1) fetch(kb + LN_GROUP);
                }
                const int tb = g % L::TB;
                if (ok && !mbar_wait(&bars.tfull[tb], (g / L::TB) & 1)) {
                    *failed = 1;
                    ok = false;
                }
                ok = __all_sync(0xffffffffu, ok);
                tc_fence_after();
                const float* s = &sc[half][in][c0];
                const uint32_t from = tcol + tb * TN;
                uint32_t r[2][16];
                tmem_fetch16(from, r[0]);
#pragma unroll
                for (int c = 0; c < L::COLS / 16; ++c) {
                    tmem_arrived(r[c & 1]);
                    if (c + 1 < L::COLS / 16) tmem_fetch16(from + 16 * (c + 1), r[(c + 1) & 1]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float4 v = *reinterpret_cast<const float4*>(s + 16 * c + 4 * i);
                        fma2(acc[8 * c + 2 * i], r[c & 1][4 * i], r[c & 1][4 * i + 1], v.x, v.y);
                        fma2(acc[8 * c + 2 * i + 1], r[c & 1][4 * i + 2], r[c & 1][4 * i + 3], v.z, v.w);
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars.tempty[tb]);
            }
            // the group after the last one must not overtake a reader of this tile's
            named_bar(1, L::EPI);
            if (split > 1) {
                // the ring is free: every product has been read
                float* red = reinterpret_cast<float*>(ring);
#pragma unroll
                for (int i = 0; i < L::COLS / 2; ++i) {
                    red[(c0 + 2 * i) * LN_M + f] = acc[i].x;
                    red[(c0 + 2 * i + 1) * LN_M + f] = acc[i].y;
                }
                continue;
            }
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
        // parts are added in the order of ranks; a CTA joins its share of the tile
        __syncwarp();
        cluster_sync();
        const int tm = first % tiles_m, t0 = (first / tiles_m) * TN;
        const int rows = min(TN, a.T - t0);
        const uint32_t red = smem_u32(ring);
        for (int i = rank * L::THREADS + (int)threadIdx.x; i < rows * LN_M; i += split * L::THREADS) {
            const int n = tm * LN_M + (i & (LN_M - 1)), t = t0 + i / LN_M;
            float v[LN_SPLIT_MAX];
#pragma unroll
            for (int r = 0; r < LN_SPLIT_MAX; ++r) v[r] = r < split ? ld_cluster(red + 4 * i, r) : 0.f;
            if (n >= a.N) continue;
            float z[1] = {v[0]};
#pragma unroll
            for (int r = 1; r < LN_SPLIT_MAX; ++r)
                if (r < split) z[0] += v[r];
            finish(a, t, n, a.bias ? a.bias[n] : 0.f, z);
        }
        __syncwarp();
        cluster_sync();                                       // a part stays until all have read it
    }
    if (threadIdx.x == 0 && *failed) atomicExch(a.status, ST_TIMEOUT);
}

template <int TN>
size_t ring_bytes(int stages, int split) {
    const size_t ring = (size_t)stages * LinearTile<TN>::STAGE, red = split > 1 ? (size_t)TN * LN_M * 4 : 0;
    return 1024 + (ring > red ? ring : red);
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
    const int most = (int)((TN >= 128 ? 208 : 104) * 1024 / L::STAGE);    // two CTAs share an SM where tiles are small
    const int per = (kb + split - 1) / split;
    int stages = most < LN_STAGES_MAX ? most : LN_STAGES_MAX;
    if (split > 1 && per < stages) stages = per;
    const int cap = num_sms * (TN >= 128 ? 1 : 2);
    const int grid = split > 1 ? (int)tiles * split : (int)(tiles < cap ? tiles : cap);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(L::THREADS);
    cfg.dynamicSmemBytes = ring_bytes<TN>(stages, split);
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
    if (e == cudaSuccess) e = prepare_one<128>();
    if (e == cudaSuccess) e = prepare_one<256>();
    if (e == cudaSuccess) e = linear_pair_prepare();
    return e;
}

cudaError_t launch_linear_fp8(const LinearArgs& a, int num_sms, cudaStream_t st) {
    if (a.T > 256) return launch_linear_pair(a, num_sms, st);
    const int tn = a.T <= 16 ? 16 : a.T <= 32 ? 32 : a.T <= 64 ? 64 : a.T <= 128 ? 128 : 256;
    const int kb = (a.K + FP8_BLOCK - 1) / FP8_BLOCK;
    const int64_t tiles = (int64_t)((a.N + LN_M - 1) / LN_M) * ((a.T + tn - 1) / tn);
    int split = 1;
    while (tn <= 128 && split < LN_SPLIT_MAX && 2 * split <= kb && tiles * split < num_sms) split *= 2;
    switch (tn) {
        case 16: return launch_tile<16>(a, split, num_sms, st);
        case 32: return launch_tile<32>(a, split, num_sms, st);
        case 64: return launch_tile<64>(a, split, num_sms, st);
        case 128: return launch_tile<128>(a, split, num_sms, st);
        default: return launch_tile<256>(a, split, num_sms, st);
    }
}

}  // namespace qmoe
